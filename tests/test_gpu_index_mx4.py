"""MXFP4 index keys on the GPU: the quantisers and the reader bit for bit against the oracle, and scores against the
formula in 64 bits on the values that the codes stand for.

Score tolerance, per (query, position): a score is sum_h w_h relu(sum_i q_hi k_i).  Products of codes and powers of two
are exact; 128 of them are added in fp32, which loses at most 2^-23 of the sum of magnitudes an addition (the tensor
cores may truncate), and 64 weighted heads are added with two roundings each: at most (128 + 2) 2^-23 of
sum_h |w_h| sum_i |q_hi k_i|."""
import numpy as np
import pytest
import torch

import dsa_indexed_sparse_gb300 as dsa
from oracle import dsa_oracle as O

pytestmark = pytest.mark.gpu

FORMATS = {"e4m3": dsa.DSA_E4M3, "mxfp8": dsa.DSA_MXFP8_E4M3, "mxfp4": dsa.DSA_MXFP4_E2M1}


def _vectors(g, shape, dtype=torch.float32):
    """Normal numbers, each block of 32 in a range of its own; some blocks of zeros, some of one magnitude."""
    x = torch.randn(shape, generator=g)
    b = x.unflatten(-1, (-1, 32)) if shape[-1] % 32 == 0 else x.unsqueeze(-2)
    b *= torch.exp2(torch.randint(-12, 13, b.shape[:-1], generator=g).float()).unsqueeze(-1)
    pick = torch.rand(b.shape[:-1], generator=g).unsqueeze(-1)
    b = torch.where(pick < 0.05, torch.zeros(()), torch.where(pick < 0.1, b.abs().amax(-1, keepdim=True), b))
    # multiples of an eighth of the block's power of two: many lie on a border between two codes
    step = torch.exp2(torch.floor(torch.log2(b.abs().amax(-1, keepdim=True).clamp(min=1e-30))) - 5)
    b = torch.where((pick > 0.5) & (pick < 0.8), torch.round(b / step) * step, b)
    return b.flatten(-2).to(dtype)


def _encode(x, fmt):
    """The oracle's codes and scales of x [n, D] (float32 numpy)."""
    if fmt == "mxfp4":
        return O.quantize_mx_e2m1(x)
    if fmt == "mxfp8":
        return O.quantize_mx_e4m3(x)
    pairs = [O.quantize_e4m3_row(r) for r in x]
    return np.stack([c for c, _ in pairs]), np.array([s for _, s in pairs], dtype=np.float32)


def _decode(codes, scales, fmt):
    if fmt == "mxfp4":
        return O.dequantize_mx_e2m1(codes, scales)
    if fmt == "mxfp8":
        return O.dequantize_mx_e4m3(codes, scales)
    return O.decode_e4m3(codes) * scales.astype(np.float64)[..., None]


def _buffers(fmt, rows, D, dev, fill=0):
    codes = torch.full((rows, D // 2 if fmt == "mxfp4" else D), fill, dtype=torch.uint8, device=dev)
    scale = torch.full((rows,), float(fill), device=dev) if fmt == "e4m3" else \
        torch.full((rows, D // 32), fill, dtype=torch.uint8, device=dev)
    return codes, scale


def _pool(g, B, ctx, page=64, spare=1):
    """A page table of shuffled pages of a pool with `spare` more pages than the sequences hold."""
    pages = (ctx + page - 1) // page
    n = B * pages + spare
    return torch.randperm(n, generator=g)[:B * pages].to(torch.int32).view(B, pages), n * page


# ------------------------------------------------------------------------------------------------- codes

@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T, H, D, pad", [(1, 1, 32, 0), (1, 64, 128, 0), (7, 3, 96, 32), (33, 64, 128, 64), (5, 2, 1024, 0),
                                          (3, 1, 288, 0)])
def test_query_quantize(dev, fmt, dtype, T, H, D, pad):
    g = torch.Generator().manual_seed(T * D + H)
    wide = _vectors(g, (T, H, D + pad), torch.float32).to(dtype)
    x = wide.to(dev)[..., pad:]                  # a strided view
    codes, scale = _buffers(fmt, T * H, D, dev, fill=9)
    codes, scale = codes.view(T, H, -1), (scale.view(T, H) if fmt == "e4m3" else scale.view(T, H, -1))
    dsa.index_query_quantize(x, codes, scale, dtype=FORMATS[fmt])
    dsa.check_status()
    c, s = _encode(x.float().cpu().numpy().reshape(T * H, D), fmt)
    assert np.array_equal(codes.cpu().numpy().reshape(c.shape), c)
    assert np.array_equal(scale.cpu().numpy().reshape(s.shape), s)


def test_query_quantize_short_e4m3(dev):
    """E4M3 vectors need only four values, and 8-byte strides of bf16."""
    x = torch.randn((5, 3, 20), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(dev)
    codes, scale = torch.zeros((5, 3, 20), dtype=torch.uint8, device=dev), torch.zeros((5, 3), device=dev)
    dsa.index_query_quantize(x, codes, scale)
    c, s = _encode(x.float().cpu().numpy().reshape(15, 20), "e4m3")
    assert np.array_equal(codes.cpu().numpy().reshape(15, 20), c) and np.array_equal(scale.cpu().numpy().reshape(15), s)


def test_mx4_extreme_magnitudes(dev):
    """The largest and smallest numbers of fp32, subnormal ones, and every border between two codes."""
    x = np.zeros((8, 32), dtype=np.float32)
    x[0, :4] = [3.4e38, -3.4e38, 1e38, 5e37]
    x[1, :3] = [1e-45, -1e-45, 1e-44]            # amax 2^-146: the exponent is clamped to -127
    x[2, :3] = [2.0 ** -126, 2.0 ** -125, -2.0 ** -127]
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=np.float32)
    x[3, 0], x[3, 1:8], x[3, 8:15] = 4.0, borders, -borders
    x[4, 0], x[4, 1:8], x[4, 8:15] = 4.0, np.nextafter(borders, 9), np.nextafter(borders, 0)
    x[5, :2] = [7.999, -7.5]
    x[6, :] = 1.0
    x[7, 31] = -2.0 ** -127
    t = torch.from_numpy(x).view(8, 1, 32).to(dev)
    codes, scale = torch.zeros((8, 1, 16), dtype=torch.uint8, device=dev), torch.zeros((8, 1, 1), dtype=torch.uint8, device=dev)
    dsa.index_query_quantize(t, codes, scale, dtype=dsa.DSA_MXFP4_E2M1)
    c, s = O.quantize_mx_e2m1(x)
    assert np.array_equal(codes.cpu().numpy().reshape(8, 16), c) and np.array_equal(scale.cpu().numpy().reshape(8, 1), s)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B, per, ctx, D, page", [(1, 1, 1, 32, 64), (5, 1, 300, 128, 64), (3, 77, 200, 128, 64),
                                                  (2, 9, 40, 1024, 16), (1, 3000, 3000, 64, 64)])
def test_append_mx4_and_read(dev, dtype, B, per, ctx, D, page):
    """New keys land at their rows, bit for bit, every other row stays as it was, and what is read back is the value."""
    g = torch.Generator().manual_seed(ctx + D)
    table, rows = _pool(g, B, ctx, page)
    T = B * per
    q_seq = torch.arange(B, dtype=torch.int32).repeat_interleave(per)
    q_pos = torch.cat([torch.randperm(ctx, generator=g)[:per] for _ in range(B)]).to(torch.int32)
    new = _vectors(g, (T, D)).to(dtype)
    codes, exps = _buffers("mxfp4", rows, D, dev, fill=77)
    seq = dsa.Seq(q_seq=q_seq.to(dev), q_pos=q_pos.to(dev), block_table=table.to(dev), max_ctx=ctx, cache_rows=rows, page_size=page)
    dsa.index_cache_append(seq, new.to(dev), codes, exps, dtype=dsa.DSA_MXFP4_E2M1)
    outs = {}
    for out_dtype, pad in ((torch.float32, 0), (torch.bfloat16, 8)):
        wide = torch.full((T, D + pad), float("nan"), dtype=out_dtype, device=dev)
        outs[out_dtype] = dsa.index_cache_read(seq, codes, exps, wide[:, :D], dtype=dsa.DSA_MXFP4_E2M1)
        assert bool(torch.isnan(wide[:, D:]).all())
    dsa.check_status()
    c, s = O.quantize_mx_e2m1(new.float().numpy())
    want_c, want_s = np.full((rows, D // 2), 77, np.uint8), np.full((rows, D // 32), 77, np.uint8)
    for t in range(T):
        r = O.physical_rows(table[q_seq[t]].numpy(), page, np.array([int(q_pos[t])]))[0]
        want_c[r], want_s[r] = c[t], s[t]
    assert np.array_equal(codes.cpu().numpy(), want_c) and np.array_equal(exps.cpu().numpy(), want_s)
    v = O.dequantize_mx_e2m1(c, s)               # two significant bits: exact in either type
    for o in outs.values():
        assert np.array_equal(o.float().cpu().numpy().astype(np.float64), v)


@pytest.mark.parametrize("fmt", ["e4m3", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("T, D", [(1, 128), (257, 128), (9, 96), (3, 1024)])
def test_index_read(dev, fmt, T, D):
    """Any codes and scales that a cache can hold: fp32 exactly as the product in fp32, bf16 rounded once from it."""
    g = torch.Generator().manual_seed(T + D)
    table, rows = _pool(g, 1, 300)
    codes, scale = _buffers(fmt, rows, D, dev)
    byte = torch.randint(0, 256, codes.shape, generator=g, dtype=torch.uint8)
    if fmt != "mxfp4":
        byte = torch.where((byte & 127) == 127, byte & 128, byte)       # not the NaN code
    codes.copy_(byte)
    scale.copy_(torch.rand(scale.shape, generator=g) if fmt == "e4m3" else torch.randint(0, 255, scale.shape, generator=g, dtype=torch.uint8))
    pos = torch.randint(0, 300, (T,), generator=g).to(torch.int32)
    seq = dsa.Seq(q_seq=torch.zeros(T, dtype=torch.int32, device=dev), q_pos=pos.to(dev), block_table=table.to(dev), max_ctx=300, cache_rows=rows)
    rowi = O.physical_rows(table[0].numpy(), 64, pos.numpy())
    v = _decode(codes.cpu().numpy()[rowi], scale.cpu().numpy()[rowi], fmt)
    with np.errstate(over="ignore"):
        v32 = v.astype(np.float32)               # an E4M3 code has four significant bits, an fp32 scale 24: rounded once
    a, b = (dsa.index_cache_read(seq, codes, scale, torch.empty((T, D), dtype=d, device=dev), dtype=FORMATS[fmt])
            for d in (torch.float32, torch.bfloat16))
    dsa.check_status()
    assert np.array_equal(a.cpu().numpy(), v32)
    assert torch.equal(b.cpu(), torch.from_numpy(v32).to(torch.bfloat16))
    if fmt == "e4m3":
        ones = dsa.index_cache_read(seq, codes, None, torch.empty((T, D), device=dev))
        assert np.array_equal(ones.cpu().numpy(), O.decode_e4m3(codes.cpu().numpy()[rowi]).astype(np.float32))


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("D, off, d", [(128, 0, 64), (128, 64, 64), (64, 2, 30)])
def test_append_mx4_rope(dev, layout, D, off, d):
    """The rotating writer's bytes are the plain writer's of keys rotated in fp32."""
    g = torch.Generator().manual_seed(D + off)
    T, ctx = 130, 1000
    table, rows = _pool(g, 1, ctx)
    pos = torch.randperm(ctx, generator=g)[:T].to(torch.int32).to(dev)
    seq = dsa.Seq(q_seq=torch.zeros(T, dtype=torch.int32, device=dev), q_pos=pos, block_table=table.to(dev), max_ctx=ctx, cache_rows=rows)
    new = _vectors(g, (T, D)).to(torch.bfloat16).to(dev)
    plan = dsa.Rope.make(d, layout=layout)
    a, ae = _buffers("mxfp4", rows, D, dev)
    b, be = _buffers("mxfp4", rows, D, dev)
    dsa.index_cache_append_rope(seq, plan, new, a, ae, offset=off, dtype=dsa.DSA_MXFP4_E2M1)
    turned = new.float()
    dsa.rope(plan, pos, turned[:, off:off + d], turned[:, off:off + d])
    dsa.index_cache_append(seq, turned, b, be, dtype=dsa.DSA_MXFP4_E2M1)
    dsa.check_status()
    assert torch.equal(a, b) and torch.equal(ae, be)


def test_bad_positions_are_flagged_and_skipped(dev):
    g = torch.Generator().manual_seed(4)
    table, rows = _pool(g, 2, 128)
    table[1, 1] = rows                           # a page that is not there
    q_seq = torch.tensor([0, 0, 2, 1, 1], dtype=torch.int32, device=dev)
    q_pos = torch.tensor([3, 128, 0, 70, 5], dtype=torch.int32, device=dev)
    seq = dsa.Seq(q_seq=q_seq, q_pos=q_pos, block_table=table.to(dev), max_ctx=128, cache_rows=rows)
    new = torch.randn((5, 128), generator=g)
    codes, exps = _buffers("mxfp4", rows, 128, dev, fill=5)
    dsa.index_cache_append(seq, new.to(dev), codes, exps, dtype=dsa.DSA_MXFP4_E2M1)
    with pytest.raises(dsa.DSAError, match="bad_index bad_q_pos"):
        dsa.check_status()
    good = [int(table[0, 0]) * 64 + 3, int(table[1, 0]) * 64 + 5]
    touched = (codes != 5).any(1).nonzero()[:, 0].tolist()
    assert sorted(touched) == sorted(good)
    out = torch.full((5, 128), 3.0, device=dev)
    dsa.index_cache_read(seq, codes, exps, out, dtype=dsa.DSA_MXFP4_E2M1)
    with pytest.raises(dsa.DSAError, match="bad_index bad_q_pos"):
        dsa.check_status()
    assert bool((out[1:4] == 3.0).all()) and not bool((out[0] == 3.0).all())


# ------------------------------------------------------------------------------------------------- scores

class Scores:
    """Queries and a pool of MXFP4 keys with block scales of different sizes; the formula in 64 bits."""

    def __init__(self, dev, lens, per, H=64, D=128, page=64, qps=True, seed=0, exps=(-6, 7)):
        g = torch.Generator().manual_seed(seed + sum(lens) * 31 + per)
        self.B, self.per, self.T, self.ctx, self.H, self.D, self.page, self.lens = len(lens), per, len(lens) * per, max(lens), H, D, page, lens
        self.table, self.rows = _pool(g, self.B, self.ctx, page)
        byte = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8)
        exp = lambda *s: torch.randint(127 + exps[0], 127 + exps[1], s, generator=g).to(torch.uint8)
        self.q, self.qe = byte(self.T, H, D // 2), exp(self.T, H, D // 32)
        self.k, self.ke = byte(self.rows, D // 2), exp(self.rows, D // 32)
        self.w = torch.randn((self.T, H), generator=g)
        self.q_seq = torch.arange(self.B, dtype=torch.int32).repeat_interleave(per)
        self.q_pos = torch.cat([torch.arange(n - per, n) for n in lens]).to(torch.int32)
        d = {n: getattr(self, n).to(dev) for n in ("q", "qe", "k", "ke", "w", "q_seq", "q_pos", "table")}
        self.seq = dsa.Seq(q_seq=d["q_seq"], q_pos=d["q_pos"], block_table=d["table"], max_ctx=self.ctx, cache_rows=self.rows,
                           page_size=page, q_per_seq=per if qps else 0)
        self.idx = dsa.Indexer(q=d["q"], w=d["w"], k_cache=d["k"], q_scale=d["qe"], k_scale=d["ke"], dtype=dsa.DSA_MXFP4_E2M1)
        self.ld = (self.ctx + 3) // 4 * 4
        self.dev = dev

    def run(self):
        out = torch.full((self.T, self.ld), -77.0, device=self.dev)
        dsa.indexer_scores(self.seq, self.idx, out)
        return out

    def want(self, t):
        """Scores of query t and the sums of magnitudes that bound their error."""
        n = int(self.q_pos[t]) + 1
        row = O.physical_rows(self.table[self.q_seq[t]].numpy(), self.page, np.arange(n))
        k = O.dequantize_mx_e2m1(self.k.numpy()[row], self.ke.numpy()[row])
        q = O.dequantize_mx_e2m1(self.q[t].numpy(), self.qe[t].numpy())
        w = self.w[t].numpy().astype(np.float64)
        return w @ np.maximum(q @ k.T, 0.0), np.abs(w) @ (np.abs(q) @ np.abs(k).T)

    def check(self, got, ts=None):
        got = got.cpu().numpy()
        for t in range(self.T) if ts is None else ts:
            want, mag = self.want(t)
            n = len(want)
            assert np.all(np.abs(got[t, :n] - want) <= 130 * 2.0 ** -23 * mag), (t, np.abs(got[t, :n] - want).max())
            assert np.all(got[t, n:] == -77.0)


@pytest.mark.parametrize("lens", [[1], [63], [64], [65], [127], [128], [129], [300, 1, 64, 777], [5000]])
def test_scores_single_queries(dev, lens):
    s = Scores(dev, lens, 1)
    got = s.run()
    assert "mxfp4" in dsa.last_plan() and "indexer_tc" in dsa.last_plan()
    dsa.check_status()
    s.check(got)


@pytest.mark.parametrize("lens, per", [([4], 4), ([70, 200], 4), ([130, 33, 400], 8), ([700], 6), ([900], 300), ([2000], 1)])
@pytest.mark.parametrize("qps", [True, False])
def test_scores_several_queries(dev, lens, per, qps):
    s = Scores(dev, lens, per, qps=qps)
    got = s.run()
    assert ("G=4" in dsa.last_plan()) == (qps and per % 4 == 0)
    dsa.check_status()
    s.check(got)


def test_scores_many_tiles_a_cta(dev):
    """More tiles a CTA than there are stages, accumulators and scale columns, one and four queries a group."""
    for per, qps in ((1, False), (64, True)):
        s = Scores(dev, [30000, 20011], per, qps=qps, seed=3)
        got = s.run()
        dsa.check_status()
        s.check(got, ts=[0, s.T // 2, s.T - 1])


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8", "e4m3"])
@pytest.mark.parametrize("per", [1, 4])
def test_scores_of_many_short_histories(dev, fmt, per):
    """Dozens of query groups a CTA, most of one tile, some of two to nine, in any order: query buffers, stages and
    accumulators go from warp to warp at every turn.  Five runs, all of the same bits, the first against the formula.

    Tolerance as above, with two roundings more for the weight times the query's scale and one for the key's."""
    g = torch.Generator().manual_seed(per)
    B, top, pages = 6000 // per, 1100, 256
    lens = torch.where(torch.rand(B, generator=g) < 0.7, torch.randint(per, 140, (B,), generator=g),
                       torch.randint(per, top + 1, (B,), generator=g))
    lens[0] = top
    table = torch.randint(0, pages, (B, (top + 63) // 64), generator=g).to(torch.int32)     # pages may be shared
    T, rows = B * per, pages * 64

    def codes(*n):
        c = torch.randint(0, 256, (*n, 64 if fmt == "mxfp4" else 128), generator=g).to(torch.uint8)
        return c if fmt == "mxfp4" else c & 0xF7                   # no NaN code
    scale = (lambda *n: torch.rand(n, generator=g) + 0.5) if fmt == "e4m3" else \
        (lambda *n: torch.randint(121, 134, (*n, 4), generator=g).to(torch.uint8))
    q, qs, k, ks = codes(T, 64), scale(T, 64), codes(rows), scale(rows)
    w = torch.randn((T, 64), generator=g)
    pos = (lens[:, None] - per + torch.arange(per)).flatten().to(torch.int32)
    seq = dsa.Seq(q_seq=torch.arange(B, dtype=torch.int32).repeat_interleave(per).to(dev), q_pos=pos.to(dev),
                  block_table=table.to(dev), max_ctx=top, cache_rows=rows, q_per_seq=per)
    idx = dsa.Indexer(q=q.to(dev), w=w.to(dev), k_cache=k.to(dev), q_scale=qs.to(dev), k_scale=ks.to(dev), dtype=FORMATS[fmt])
    out = [torch.full((T, (top + 3) // 4 * 4), -77.0, device=dev) for _ in range(5)]
    for o in out:
        dsa.indexer_scores(seq, idx, o)
    assert "indexer_tc" in dsa.last_plan()
    dsa.check_status()
    for o in out[1:]:
        assert torch.equal(o, out[0])
    got = out[0].cpu().numpy()
    kd = _decode(k.numpy(), ks.numpy(), fmt)
    for t in range(0, T, 3):
        n = int(pos[t]) + 1
        keys = kd[O.physical_rows(table[t // per].numpy(), 64, np.arange(n))]
        qd, wd = _decode(q[t].numpy(), qs[t].numpy(), fmt), w[t].numpy().astype(np.float64)
        want, mag = wd @ np.maximum(qd @ keys.T, 0.0), np.abs(wd) @ (np.abs(qd) @ np.abs(keys).T)
        assert np.all(np.abs(got[t, :n] - want) <= 133 * 2.0 ** -23 * mag), t
        assert np.all(got[t, n:] == -77.0)


def test_scores_of_largest_products(dev):
    """The largest dot products of either sign, which the ReLU keeps or takes to 0 whole, with weights of either sign."""
    s = Scores(dev, [130, 64], 4, seed=9)
    s.idx.q.fill_(0x77)                                            # 6
    sign = torch.randint(0, 2, (s.rows, 1), generator=torch.Generator().manual_seed(4)).to(torch.uint8)
    s.idx.k_cache.copy_((0x77 + 0x88 * sign).expand(-1, 64))       # all 6 or all -6
    s.q, s.k = s.idx.q.cpu(), s.idx.k_cache.cpu()
    got = s.run()
    dsa.check_status()
    s.check(got)


@pytest.mark.parametrize("H, D, page", [(4, 32, 64), (64, 64, 64), (64, 128, 16), (3, 256, 64)])
def test_scores_other_dims(dev, H, D, page):
    s = Scores(dev, [100, 37], 3, H=H, D=D, page=page)
    got = s.run()
    assert "generic" in dsa.last_plan()
    dsa.check_status()
    s.check(got)


def test_scores_of_far_exponents(dev):
    """Key scales of 2^90 and more against query scales of 2^-90 and less: only the sum of exponents counts."""
    s = Scores(dev, [200, 140], 4, exps=(0, 1))
    s.idx.q_scale.copy_(torch.randint(10, 38, s.idx.q_scale.shape, generator=torch.Generator().manual_seed(1)).to(torch.uint8))
    s.idx.k_scale.copy_(torch.randint(217, 245, s.idx.k_scale.shape, generator=torch.Generator().manual_seed(2)).to(torch.uint8))
    s.qe, s.ke = s.idx.q_scale.cpu(), s.idx.k_scale.cpu()
    got = s.run()
    dsa.check_status()
    s.check(got)


def test_scores_on_two_streams_are_the_same_bits(dev):
    a, b = Scores(dev, [9000, 4100], 4, seed=1), Scores(dev, [20000], 1, seed=2)
    want = a.run(), b.run()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(5):
        for s, st in ((a, streams[0]), (b, streams[1])):
            with torch.cuda.stream(st):
                got.append(s.run())
    torch.cuda.synchronize()
    dsa.check_status()
    for i, g in enumerate(got):
        assert torch.equal(g, want[i % 2])


def test_scores_bad_page_is_flagged(dev):
    s = Scores(dev, [300], 4)
    s.seq.block_table[0, 1] = -1
    got = s.run()
    with pytest.raises(dsa.DSAError, match="bad_index"):
        dsa.check_status()
    assert bool((got[:, 64:128] == -77.0).all())
    keep = got.clone()
    keep[:, 64:128] = 0
    for t in range(4):
        want, mag = s.want(t)
        want[64:128] = 0
        assert np.all(np.abs(keep[t, :len(want)].cpu().numpy() - want) <= 130 * 2.0 ** -23 * mag)


@pytest.mark.parametrize("lens, fused", [([3000] * 40, True), ([20000, 9000], False)])
def test_decode_step(dev, lens, fused):
    """The step over MXFP4 keys, in both plans: its selection is the Top-K of its scores, its attention the separate
    call's on that selection."""
    s = Scores(dev, lens, 1, seed=9)
    K, T = 256, s.T
    g = torch.Generator(device=dev).manual_seed(2)
    mla = dsa.Mla(q=torch.randn((T, 128, 576), generator=g, device=dev).to(torch.bfloat16),
                  kv_cache=torch.randn((s.rows, 576), generator=g, device=dev).to(torch.bfloat16), d_latent=512, d_rope=64,
                  softmax_scale=192 ** -0.5)
    out, lse, sel = torch.empty((T, 128, 512), dtype=torch.bfloat16, device=dev), torch.empty((T, 128), device=dev), \
        torch.empty((T, K), dtype=torch.int32, device=dev)
    ws = torch.empty(dsa.decode_workspace_size(s.seq, s.idx, mla, K), dtype=torch.uint8, device=dev)
    dsa.decode_step(s.seq, s.idx, mla, K, out, ws, lse=lse, idx_out=sel)
    assert ("fused<mxfp4>" in dsa.last_plan()) == fused
    idx = torch.empty_like(sel)
    dsa.topk(s.seq, s.run(), K, idx)
    dsa.check_status()
    assert torch.equal(sel, idx)
    o2 = torch.empty_like(out)
    dsa.sparse_mla_attn(s.seq, mla, idx, K, o2, workspace=ws)
    dsa.check_status()
    assert torch.equal(out, o2)
    if ws.numel() <= dsa.STATIC_WORKSPACE_BYTES:   # the step with the library's own scratch
        o2.fill_(7)
        dsa.decode_step_static_ws(s.seq, s.idx, mla, K, o2, idx_out=idx.fill_(-7))
        dsa.check_status()
        assert torch.equal(out, o2) and torch.equal(sel, idx)


def test_append_quantise_score_captured(dev):
    """New keys appended, queries quantised and scored, eagerly and as a replayed graph on another stream with other inputs."""
    g = torch.Generator().manual_seed(8)
    s = Scores(dev, [500, 333], 4)
    new = torch.randn((s.T, s.D), generator=g).to(dev)
    q = torch.randn((s.T, s.H, s.D), generator=g).to(torch.bfloat16).to(dev)
    out = torch.full((s.T, s.ld), -77.0, device=dev)

    def step():
        dsa.index_cache_append(s.seq, new, s.idx.k_cache, s.idx.k_scale, dtype=dsa.DSA_MXFP4_E2M1)
        dsa.index_query_quantize(q, s.idx.q, s.idx.q_scale, dtype=dsa.DSA_MXFP4_E2M1)
        dsa.indexer_scores(s.seq, s.idx, out)

    def check():
        dsa.check_status()
        s.q, s.qe, s.k, s.ke = (x.cpu() for x in (s.idx.q, s.idx.q_scale, s.idx.k_cache, s.idx.k_scale))
        c, e = O.quantize_mx_e2m1(q.float().cpu().numpy())
        assert np.array_equal(s.q.numpy(), c) and np.array_equal(s.qe.numpy(), e)
        s.check(out)

    step()
    check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        new.copy_(torch.randn(new.shape, generator=g))
        q.copy_(torch.randn(q.shape, generator=g).to(torch.bfloat16))
        graph.replay()
    side.synchronize()
    check()


def test_calls_of_no_tokens(dev):
    s = Scores(dev, [100], 1)
    none = torch.zeros(0, dtype=torch.int32, device=dev)
    seq = dsa.Seq(q_seq=none, q_pos=none, block_table=s.seq.block_table, max_ctx=100, cache_rows=s.rows)
    before = s.idx.k_cache.clone()
    dsa.index_cache_append(seq, torch.zeros((0, 128), device=dev), s.idx.k_cache, s.idx.k_scale, dtype=dsa.DSA_MXFP4_E2M1)
    dsa.index_cache_read(seq, s.idx.k_cache, s.idx.k_scale, torch.zeros((0, 128), device=dev), dtype=dsa.DSA_MXFP4_E2M1)
    dsa.index_query_quantize(torch.zeros((0, 64, 128), device=dev), torch.zeros((0, 64, 64), dtype=torch.uint8, device=dev),
                             torch.zeros((0, 64, 4), dtype=torch.uint8, device=dev), dtype=dsa.DSA_MXFP4_E2M1)
    dsa.check_status()
    assert torch.equal(before, s.idx.k_cache)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8", "e4m3"])
@pytest.mark.parametrize("shape, strides", [((1, 64, 128), (8193, 128, 1)), ((5, 1, 128), (256, 7, 1)), ((1, 1, 128), (3, 5, 1))])
def test_query_quantize_stride_of_one_token_or_head(dev, fmt, shape, strides):
    """The stride of a dimension of one is whatever the view it came from has."""
    base = torch.randn(8192 + 1024, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).to(dev)
    x = base.as_strided(shape, strides)
    n = shape[0] * shape[1]
    codes, scale = _buffers(fmt, n, 128, dev, fill=9)
    codes, scale = codes.view(*shape[:2], -1), scale.view(*shape[:2], -1) if fmt != "e4m3" else scale.view(*shape[:2])
    dsa.index_query_quantize(x, codes, scale, dtype=FORMATS[fmt])
    dsa.check_status()
    c, s = _encode(x.float().cpu().numpy().reshape(n, 128), fmt)
    assert np.array_equal(codes.cpu().numpy().reshape(c.shape), c) and np.array_equal(scale.cpu().numpy().reshape(s.shape), s)


def test_e4m3_vectors_whose_scale_would_be_zero(dev):
    """fp32 vectors so small that amax / 448 is 0 in fp32 are stored as zeros, not as the NaN of 0 / 0, by every writer."""
    edge = np.float32(1.75 * 2.0 ** -142)
    tops = [np.float32(0), np.float32(1e-45), np.float32(1e-43), edge, np.nextafter(edge, np.float32(1)), np.float32(1e-42), np.float32(1e-38)]
    x = np.zeros((len(tops), 128), np.float32)
    x[:, 3], x[:, 70], x[:, 127] = tops, -np.array(tops) / np.float32(2), np.array(tops) / np.float32(3)
    n = len(tops)
    c, s = _encode(x, "e4m3")
    assert np.all((c & 127) != 127) and np.all(s > 0) and np.all(s[:4] == 1) and s[4] < 1
    t = torch.from_numpy(x).to(dev)
    codes, scale = _buffers("e4m3", n, 128, dev, fill=9)
    dsa.index_query_quantize(t.view(n, 1, 128), codes.view(n, 1, 128), scale.view(n, 1))
    assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scale.cpu().numpy(), s)
    seq = dsa.Seq(q_seq=torch.zeros(n, dtype=torch.int32, device=dev), q_pos=torch.arange(n, dtype=torch.int32, device=dev),
                  block_table=torch.zeros((1, 1), dtype=torch.int32, device=dev), max_ctx=64, cache_rows=64)
    kc, ks = _buffers("e4m3", 64, 128, dev, fill=9)
    dsa.index_cache_append(seq, t, kc, ks)
    assert np.array_equal(kc[:n].cpu().numpy(), c) and np.array_equal(ks[:n].cpu().numpy(), s)
    kc, ks = _buffers("e4m3", 64, 128, dev, fill=9)
    dsa.index_cache_append_rope(seq, dsa.Rope.make(32), t, kc, ks, offset=80)      # dims 80 to 111: zeros
    dsa.check_status()
    kc, turned = kc[:n].cpu().numpy(), (np.arange(128) >= 80) & (np.arange(128) < 112)
    assert np.array_equal(kc[:, ~turned], c[:, ~turned]) and np.all((kc[:, turned] & 127) == 0)
    assert np.array_equal(ks[:n].cpu().numpy(), s)


@pytest.mark.parametrize("H, D, per", [(64, 128, 1), (64, 128, 4), (3, 128, 2)])
def test_keys_beyond_32_bit_offsets(dev, H, D, per):
    """Keys in the last pages of a pool whose codes and scales both pass 2^31 bytes: written, with and without rotation, read and
    scored as in a small pool, bit for bit."""
    if torch.cuda.mem_get_info()[0] < (60 << 30):
        pytest.skip("needs 36 GB and room")
    g = torch.Generator().manual_seed(H + per)
    ctx, pages = 500, 8
    far = (2 ** 29 + 64 * 64) // 64              # 2^29 rows of 64 and of 4 bytes
    byte = lambda *n: torch.randint(0, 256, n, generator=g).to(torch.uint8).to(dev)
    q, qe = byte(per, H, D // 2), torch.randint(121, 134, (per, H, D // 32), generator=g).to(torch.uint8).to(dev)
    w, new = torch.randn((per, H), generator=g).to(dev), torch.randn((ctx, D), generator=g).to(dev)
    order = torch.randperm(pages, generator=g).to(torch.int32)
    results = []
    for n in (pages, far):
        codes, exps = (torch.empty((n * 64, b), dtype=torch.uint8, device=dev) for b in (D // 2, D // 32))
        table = (order + (n - pages)).view(1, pages).to(dev)
        every = dsa.Seq(q_seq=torch.zeros(ctx, dtype=torch.int32, device=dev), q_pos=torch.arange(ctx, dtype=torch.int32, device=dev),
                        block_table=table, max_ctx=ctx, cache_rows=n * 64)
        seq = dsa.Seq(q_seq=torch.zeros(per, dtype=torch.int32, device=dev), q_pos=torch.arange(ctx - per, ctx, dtype=torch.int32, device=dev),
                      block_table=table, max_ctx=ctx, cache_rows=n * 64, q_per_seq=per)
        for rotated in (False, True):
            if rotated:
                dsa.index_cache_append_rope(every, dsa.Rope.make(64), new, codes, exps, offset=0, dtype=dsa.DSA_MXFP4_E2M1)
            else:
                dsa.index_cache_append(every, new, codes, exps, dtype=dsa.DSA_MXFP4_E2M1)
            read = dsa.index_cache_read(every, codes, exps, torch.empty((ctx, D), device=dev), dtype=dsa.DSA_MXFP4_E2M1)
            out = torch.full((per, 500), -77.0, device=dev)
            dsa.indexer_scores(seq, dsa.Indexer(q=q, w=w, k_cache=codes, q_scale=qe, k_scale=exps, dtype=dsa.DSA_MXFP4_E2M1), out)
            results.append((read, out))
        dsa.check_status()
    for near, away in zip(results[:2], results[2:]):
        assert torch.equal(near[0], away[0]) and torch.equal(near[1], away[1])
    v = O.dequantize_mx_e2m1(*O.quantize_mx_e2m1(new.cpu().numpy()))
    assert np.array_equal(results[2][0].cpu().numpy().astype(np.float64), v)
