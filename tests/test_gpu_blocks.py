"""The choice of blocks and the attention over blocks on the GPU.

The choice is compared exactly with a plain one.  The attention's tolerance against 64 bits, per output value
sum_s p_s v_s / sum_s p_s: the weights go to bf16 (2^-8 of each) and, where a query's blocks are split, the partial
outputs too (2^-8 of what they hold), the output once more (2^-8 of it); a logit is a sum of 576 products in fp32, off by
at most dl = 578 2^-23 of its sum of magnitudes (a truncating addition and the scale), a weight by 2 dl of itself (its own
logit and the normalising sum) and 2^-20 (exponential, sum)."""
import math

import numpy as np
import pytest
import torch

import dsa_indexed_sparse_gb300 as dsa

pytestmark = pytest.mark.gpu

D_ROW, D_V, SCALE = 576, 512, 192 ** -0.5


class Blocks:
    """Sequences of the lengths `lens` with `per` last tokens as queries; bf16 rows, those that hold nothing NaN."""

    def __init__(self, dev, lens, per=1, H=128, page=64, seed=0, pad=0, scale=SCALE):
        g = torch.Generator(device=dev).manual_seed(seed * 1000 + sum(lens) + per)
        self.g, self.dev, self.lens, self.H, self.page, self.scale = g, dev, lens, H, page, scale
        B, self.ctx = len(lens), max(lens)
        pages = (self.ctx + page - 1) // page
        n = B * pages + 2
        self.table = torch.randperm(n, generator=g, device=dev)[:B * pages].to(torch.int32).view(B, pages)
        self.rows = n * page
        self.wide = torch.randn((self.rows, D_ROW + pad), generator=g, device=dev).to(torch.bfloat16)
        self.cache = self.wide[:, :D_ROW]
        held = torch.zeros(self.rows, dtype=torch.bool, device=dev)
        for b, length in enumerate(lens):
            at = torch.arange(length, device=dev)
            held[self.table[b].long()[at // page] * page + at % page] = True
        self.cache[~held] = float("nan")
        self.T = B * per
        self.q = torch.randn((self.T, H, D_ROW), generator=g, device=dev).to(torch.bfloat16)
        self.q_seq = torch.arange(B, dtype=torch.int32, device=dev).repeat_interleave(per)
        self.q_pos = torch.cat([torch.arange(n - per, n) for n in lens]).to(torch.int32).to(dev)
        self.seq = dsa.Seq(q_seq=self.q_seq, q_pos=self.q_pos, block_table=self.table, max_ctx=self.ctx, cache_rows=self.rows,
                           page_size=page, q_per_seq=per)
        self.remake()

    def remake(self):
        self.mla = dsa.Mla(q=self.q, kv_cache=self.wide, d_latent=D_V, d_rope=64, softmax_scale=self.scale)

    def choose(self, N, holes=0.0, own=True, order="ascending"):
        """A random choice of each query's blocks, its own among them."""
        n = self.table.shape[1]
        last = (self.q_pos // self.page).long()
        key = torch.rand((self.T, n), generator=self.g, device=self.dev)
        if own:
            key.scatter_(1, last[:, None], -1.0)
        key.masked_fill_(torch.arange(n, device=self.dev)[None, :] > last[:, None], 2.0)
        best, idx = key.topk(min(N, n), dim=1, largest=False)
        idx = torch.where(best < 2.0, idx, n)
        if order == "ascending":
            idx = idx.sort(dim=1).values
        idx = torch.nn.functional.pad(torch.where(idx < n, idx, -1), (0, max(0, N - n)), value=-1)
        if holes:
            idx = torch.where(torch.rand((self.T, N), generator=self.g, device=self.dev) < holes, -1, idx)
        return idx.to(torch.int32).contiguous()

    def run(self, idx, workspace=True, **kw):
        out = torch.full((self.T, self.H, D_V), 7.0, dtype=torch.bfloat16, device=self.dev)
        lse = torch.full((self.T, self.H), 7.0, device=self.dev)
        ws = None
        if workspace:
            ws = torch.empty(max(16, dsa.block_mla_attn_workspace_size(self.seq, self.mla, idx.shape[1])), dtype=torch.uint8, device=self.dev)
        dsa.block_mla_attn(self.seq, self.mla, idx, out, lse=lse, workspace=ws, **kw)
        return out, lse

    def check(self, got, idx, ts=None, skip=()):
        """`got` against the formula; skip: (query, entry) pairs that count as -1."""
        out, lse = got
        inside = torch.arange(self.page, device=self.dev)
        for t in range(self.T) if ts is None else ts:
            blk = idx[t].long().clone()
            for a, e in skip:
                if a == t:
                    blk[e] = -1
            blk = blk[blk >= 0]
            if len(blk) == 0:
                assert bool((out[t] == 0).all()) and bool((lse[t] == -math.inf).all())
                continue
            pos = (blk[:, None] * self.page + inside).flatten()
            row = self.table[self.q_seq[t]].long()[blk].repeat_interleave(self.page) * self.page + inside.repeat(len(blk))
            row = row[pos <= self.q_pos[t]]
            k, q = self.cache[row].double(), self.q[t].double()
            z = q @ k.T * self.scale
            dl = 578 * 2.0 ** -23 * abs(self.scale) * (q.abs() @ k.abs().T).amax(dim=1)
            top = z.amax(dim=1, keepdim=True)
            p = (z - top).exp()
            total = p.sum(dim=1, keepdim=True)
            want, mag = p @ k[:, :D_V] / total, p @ k[:, :D_V].abs() / total
            tol = (2 * 2.0 ** -8 + 2 * dl[:, None] + 2.0 ** -20) * mag + 2.0 ** -8 * want.abs() + 1e-30
            err = (out[t].double() - want).abs()
            assert bool((err <= tol).all()), (t, float((err / tol).max()))
            w = (top + total.log())[:, 0]
            assert bool(((lse[t].double() - w).abs() <= dl + 2.0 ** -18 + w.abs() * 2.0 ** -22).all()), t


@pytest.mark.parametrize("lens, N", [([1], 1), ([63], 1), ([64], 1), ([65], 2), ([129], 1), ([200], 3), ([5000], 32), ([3000], 33),
                                     ([700, 1, 64, 321], 5), ([9000], 140), ([130], 20)])
@pytest.mark.parametrize("workspace", [True, False])
def test_single_queries(dev, lens, N, workspace):
    s = Blocks(dev, lens)
    idx = s.choose(N)
    got = s.run(idx, workspace)
    assert "attn_block" in dsa.last_plan()
    dsa.check_status()
    s.check(got, idx)


@pytest.mark.parametrize("holes, order", [(0.3, "ascending"), (0.8, "ascending"), (0.0, "any"), (0.5, "any")])
@pytest.mark.parametrize("workspace", [True, False])
def test_holes_and_order(dev, holes, order, workspace):
    s = Blocks(dev, [4000, 2500, 77, 640], per=2, seed=1)
    idx = s.choose(41, holes, own=False, order=order)
    idx[3] = -1                                  # a query that selects nothing
    idx[5, :] = -1
    idx[5, 40] = 0                               # one that selects its last entry only
    got = s.run(idx, workspace)
    dsa.check_status()
    s.check(got, idx)


def test_many_items_a_cluster(dev):
    """More queries than clusters: items follow one another in every buffer and phase, some of them empty, some of one tile."""
    s = Blocks(dev, [1500], per=400, seed=2)
    idx = s.choose(9, 0.2)
    idx[::7] = -1
    idx[3::11, 1:] = -1
    got = s.run(idx)
    dsa.check_status()
    s.check(got, idx, ts=list(range(0, 400, 9)) + list(range(0, 400, 7)) + list(range(3, 400, 44)))


def test_duplicates_count_twice(dev):
    s = Blocks(dev, [600])
    idx = torch.tensor([[2, 2, 5, 9, 9, 9]], dtype=torch.int32, device=dev)
    got = s.run(idx)
    dsa.check_status()
    s.check(got, idx)


@pytest.mark.parametrize("H", [1, 16, 64, 65, 130, 256])
def test_head_counts(dev, H):
    s = Blocks(dev, [900, 333], H=H, per=3)
    idx = s.choose(7)
    got = s.run(idx)
    dsa.check_status()
    s.check(got, idx)


@pytest.mark.parametrize("scale", [-0.05, 0.0, 1.0])
def test_scales(dev, scale):
    s = Blocks(dev, [400], scale=scale)
    idx = s.choose(6)
    got = s.run(idx)
    dsa.check_status()
    s.check(got, idx)


@pytest.mark.parametrize("workspace", [True, False])
def test_running_maximum_jumps(dev, workspace):
    """Logits that grow by a hundred and more from block to block, and fall: O has to be rescaled, and a block of far smaller
    weights must not be lost before it."""
    s = Blocks(dev, [64 * 12], per=1)
    for i, f in enumerate([0.0, 30.0, -30.0, 8.0, 60.0, 0.5, 90.0, -90.0, 85.0, 100.0, 3.0, 1.0]):
        row = s.table[0, i].long() * 64 + torch.arange(64, device=dev)
        s.cache[row] = (s.cache[row].float() + f * s.q[0, i * 7].float() / 8).to(torch.bfloat16)
    idx = torch.arange(12, dtype=torch.int32, device=dev)[None].contiguous()
    got = s.run(idx, workspace)
    dsa.check_status()
    s.check(got, idx)


def test_nan_and_infinity_of_selected_rows(dev):
    """What a selected row holds comes through: NaN as NaN; an infinite logit leaves NaN, as the formula does."""
    s = Blocks(dev, [640], per=2)
    idx = s.choose(10)
    clean = s.run(idx, workspace=False)
    s.cache[int(s.table[0, 3]) * 64 + 5, 100] = float("nan")
    for ws in (True, False):
        out, lse = s.run(idx, ws)
        assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())
    idx2 = torch.where(idx == 3, -1, idx)
    got = s.run(idx2)
    dsa.check_status()
    s.check(got, idx2)
    assert not bool(torch.isnan(clean[0]).any())


@pytest.mark.parametrize("workspace", [True, False])
def test_nan_of_a_query_head_stays_with_it(dev, workspace):
    s = Blocks(dev, [640, 200], per=1)
    idx = s.choose(9)
    s.q[0, 17, 5] = float("nan")
    s.q[1, 127, 575] = float("inf")              # logits of both signs' infinity
    out, lse = s.run(idx, workspace)
    dsa.check_status()
    assert bool(torch.isnan(out[0, 17]).all()) and bool(torch.isnan(lse[0, 17]))
    assert bool(torch.isnan(out[1, 127]).all()) and bool(torch.isnan(lse[1, 127]))
    s.q[0, 17, 5] = s.q[1, 127, 575] = 0.0
    clean = s.run(idx, workspace)
    s.check(clean, idx)
    out[0, 17], out[1, 127], lse[0, 17], lse[1, 127] = clean[0][0, 17], clean[0][1, 127], clean[1][0, 17], clean[1][1, 127]
    assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])


def test_the_same_call_gives_the_same_bits(dev):
    s = Blocks(dev, [5000, 3000, 2000], per=4, seed=12)
    idx = s.choose(31, 0.1)
    a = s.run(idx)
    for _ in range(3):
        b = s.run(idx)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    dsa.check_status()


@pytest.mark.parametrize("group", [0, 1, 2, 3])
@pytest.mark.parametrize("per, N", [(700, 9), (150, 12), (3, 16)])
def test_one_group_of_heads_behind_the_others(dev, group, per, N):
    """Blocks in any order, so that the query's own, whose rows behind the position are zeroed, lies in any tile, and maxima
    that jump for one group of 32 heads only, which then rescales O: the groups of either CTA pass a tile at different times,
    and P V has to wait for the last of them.  Five runs of the same bits."""
    s = Blocks(dev, [64 * 40 - 17], per=per, seed=20 + group)
    u = torch.randn(D_ROW, generator=s.g, device=dev)
    heads = slice(32 * group, 32 * group + 32)
    s.q[:, heads] = (u + 0.5 * s.q[:, heads].float()).to(torch.bfloat16)
    for i in range(40):                          # logits of these heads: about 5 f
        row = s.table[0, i].long() * 64 + torch.arange(64, device=dev)
        s.cache[row] = (s.cache[row].float() + float((i * 17) % 40 - 15) * u / 8).to(torch.bfloat16)
    idx = s.choose(N, 0.1, order="any")
    first = s.run(idx)
    assert "attn_block" in dsa.last_plan()
    for _ in range(4):
        again = s.run(idx)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    dsa.check_status()
    s.check(first, idx, ts=range(0, s.T, max(1, s.T // 40)))


def test_bad_blocks_and_pages_are_flagged_and_skipped(dev):
    s = Blocks(dev, [640, 300], per=1)
    idx = torch.tensor([[0, 10, 3, 9], [2, 4, 1, 5]], dtype=torch.int32, device=dev)   # 10, 5: behind the position
    keep = s.table.clone()
    s.table[0, 3] = s.rows // 64                 # a page that is not there
    got = s.run(idx)
    with pytest.raises(dsa.DSAError, match="bad_index"):
        dsa.check_status()
    s.table.copy_(keep)
    s.check(got, idx, skip=[(0, 1), (0, 2), (1, 3)])
    s.q_pos[1] = 640                             # beyond max_ctx: the query selects nothing
    out, lse = s.run(idx[:, :1].contiguous())
    with pytest.raises(dsa.DSAError, match="bad_q_pos"):
        dsa.check_status()
    assert bool((out[1] == 0).all()) and bool((lse[1] == -math.inf).all()) and not bool((out[0] == 0).all())


def test_padded_rows(dev):
    s = Blocks(dev, [500, 900], pad=8)           # 1168-byte rows
    assert s.mla.desc().row_bytes == 1168
    idx = s.choose(8)
    got = s.run(idx)
    assert "attn_block" in dsa.last_plan()
    dsa.check_status()
    s.check(got, idx)


def test_rows_beyond_32_bit_offsets(dev):
    s = Blocks(dev, [640], per=1)
    n = (5 << 30) // (64 * D_ROW * 2)
    big = torch.zeros((n * 64, D_ROW), dtype=torch.bfloat16, device=dev)
    far = n - 1 - torch.arange(10, device=dev)
    for i in range(10):
        big[far[i] * 64:(far[i] + 1) * 64] = s.cache[int(s.table[0, i]) * 64:int(s.table[0, i]) * 64 + 64]
    idx = s.choose(10)
    want = s.run(idx)
    seq = dsa.Seq(q_seq=s.q_seq, q_pos=s.q_pos, block_table=far.to(torch.int32).view(1, 10), max_ctx=640, cache_rows=n * 64)
    mla = dsa.Mla(q=s.q, kv_cache=big, d_latent=D_V, d_rope=64, softmax_scale=SCALE)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    ws = torch.empty(dsa.block_mla_attn_workspace_size(seq, mla, 10), dtype=torch.uint8, device=dev)
    dsa.block_mla_attn(seq, mla, idx, out, lse=lse, workspace=ws)
    dsa.check_status()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("fmt, page, H", [("bf16", 16, 8), ("f32", 64, 4), ("f32", 8, 2), ("e4m3", 64, 128), ("e4m3_t128", 64, 128),
                                          ("e2m1", 64, 128), ("e2m1", 32, 16)])
def test_other_caches(dev, fmt, page, H):
    """The form that writes the blocks' positions out: bit for bit dsa_sparse_mla_attn on those positions."""
    g = torch.Generator(device=dev).manual_seed(page + H)
    lens, N = [300, 77], 5
    ctx, pages = max(lens), (max(lens) + page - 1) // page
    rows = 2 * pages * page
    table = torch.randperm(2 * pages, generator=g, device=dev).to(torch.int32).view(2, pages)
    seq = dsa.Seq(q_seq=torch.tensor([0, 1], dtype=torch.int32, device=dev), q_pos=torch.tensor([299, 76], dtype=torch.int32, device=dev),
                  block_table=table, max_ctx=ctx, cache_rows=rows, page_size=page)
    dt = torch.float32 if fmt == "f32" else torch.bfloat16
    code = {"bf16": None, "f32": None, "e4m3": dsa.DSA_E4M3, "e4m3_t128": dsa.DSA_E4M3_T128, "e2m1": dsa.DSA_E2M1}[fmt]
    width = {"e4m3": 656, "e4m3_t128": 656, "e2m1": 432}.get(fmt)
    cache = torch.zeros((rows, D_ROW), dtype=dt, device=dev) if width is None else torch.zeros((rows, width), dtype=torch.uint8, device=dev)
    q = torch.randn((2, H, D_ROW), generator=g, device=dev).to(dt)
    mla = dsa.Mla(q=q, kv_cache=cache, d_latent=D_V, d_rope=64, softmax_scale=SCALE, dtype=code)
    # every row written, through the cache writer
    every = dsa.Seq(q_seq=torch.arange(2, dtype=torch.int32, device=dev).repeat_interleave(ctx),
                    q_pos=torch.arange(ctx, dtype=torch.int32, device=dev).repeat(2), block_table=table, max_ctx=ctx, cache_rows=rows, page_size=page)
    dsa.latent_cache_append(every, mla, torch.randn((2 * ctx, D_ROW), generator=g, device=dev).to(dt))
    idx = torch.tensor([[0, -1, 299 // page, 1, 2], [76 // page, 0, -1, -1, 0]], dtype=torch.int32, device=dev)
    pos = (idx.unsqueeze(-1) * page + torch.arange(page, device=dev)).masked_fill((idx < 0).unsqueeze(-1), -1).flatten(1)
    pos = torch.where(pos <= seq.q_pos[:, None], pos, -1).to(torch.int32).contiguous()
    outs = []
    for call, size, arg in ((dsa.block_mla_attn, dsa.block_mla_attn_workspace_size(seq, mla, N), None),
                            (dsa.sparse_mla_attn, dsa.sparse_mla_attn_workspace_size(seq, mla, N * page), pos)):
        out, lse = torch.empty((2, H, D_V), dtype=dt, device=dev), torch.empty((2, H), device=dev)
        ws = torch.empty(max(size, 16), dtype=torch.uint8, device=dev)
        if arg is None:
            call(seq, mla, idx, out, lse=lse, workspace=ws)
            assert "expand_blocks" in dsa.last_plan()
        else:
            call(seq, mla, arg, N * page, out, lse=lse, workspace=ws)
        dsa.check_status()
        outs.append((out, lse))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    with pytest.raises(dsa.DSAError, match="workspace"):
        dsa.block_mla_attn(seq, mla, idx, outs[0][0])
    idx[0, 3] = 300
    dsa.block_mla_attn(seq, mla, idx, outs[0][0], workspace=torch.empty(dsa.block_mla_attn_workspace_size(seq, mla, N), dtype=torch.uint8, device=dev))
    with pytest.raises(dsa.DSAError, match="bad_index"):
        dsa.check_status()


def test_two_streams_and_a_graph(dev):
    """Two calls at once with workspaces of their own, then captured together and replayed with other queries."""
    a, b = Blocks(dev, [3000, 2000, 900], per=2, seed=5), Blocks(dev, [5000], per=1, seed=6)
    ia, ib = a.choose(12), b.choose(30)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        with torch.cuda.stream(s1):
            ga = a.run(ia)
        with torch.cuda.stream(s2):
            gb = b.run(ib)
    torch.cuda.synchronize()
    dsa.check_status()
    a.check(ga, ia)
    b.check(gb, ib)
    with torch.cuda.stream(s1):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s1):
            ga = a.run(ia)
            gb = b.run(ib)
        for x in (a, b):
            x.q.copy_(torch.randn(x.q.shape, generator=x.g, device=dev).to(torch.bfloat16))
        graph.replay()
        graph.replay()
    torch.cuda.synchronize()
    dsa.check_status()
    a.check(ga, ia)
    b.check(gb, ib)


@pytest.mark.parametrize("T", [1, 200])
def test_bounded_wait_runs_out_and_the_next_call_is_clean(dev, T):
    s = Blocks(dev, [1500], per=T, seed=7)
    idx = s.choose(8)
    dsa.debug_withhold_arrival(True, 2_000_000)
    try:
        s.run(idx)
        with pytest.raises(dsa.DSAError, match="timeout"):
            dsa.check_status()
    finally:
        dsa.debug_withhold_arrival(False)
    got = s.run(idx)
    dsa.check_status()
    s.check(got, idx, ts=[0, T // 2, T - 1])


# ------------------------------------------------------------------------------------------------- the choice

def _choice(scores, q_pos, page, N, first, last):
    """The plain choice, numpy, one query after the other."""
    out = np.full((len(q_pos), N), -1, np.int32)
    for t, p in enumerate(q_pos):
        n = p // page + 1
        best = []
        for b in range(n):
            v = scores[t, b * page:min((b + 1) * page, p + 1)]
            v = v[~np.isnan(v)]
            v = v.max() + 0.0 if len(v) else -np.inf
            best.append((0 if b < first or b >= n - last else 1, -v, b))
        take = sorted(b for _, _, b in sorted(best)[:N])
        out[t, :len(take)] = take
    return out


def _scores(g, T, n, kind):
    x = torch.randn((T, n), generator=g)
    if kind == "equal":
        x = torch.round(x * 2) / 2               # many blocks share their best score
    if kind == "one":
        x = torch.zeros((T, n))
        x[:, ::3] = -0.0
    if kind == "special":
        u = torch.rand((T, n), generator=g)
        x = torch.where(u < 0.05, float("nan"), torch.where(u < 0.06, float("inf"), x))
        x[:, 64:128] = float("nan")
        x[:, 192:320] = -float("inf")
    return x


@pytest.mark.parametrize("lens, per, page, N, first, last, kind", [
    ([1], 1, 64, 1, 0, 0, "normal"), ([64], 1, 64, 1, 1, 0, "normal"), ([65], 1, 64, 1, 0, 1, "normal"),
    ([5000], 1, 64, 16, 1, 1, "normal"), ([5003], 1, 64, 16, 0, 0, "equal"), ([9001, 4000, 130], 3, 64, 20, 2, 5, "equal"),
    ([8000], 1, 64, 20, 0, 0, "one"), ([8000], 2, 64, 7, 3, 4, "one"), ([4000], 1, 64, 9, 1, 1, "special"),
    ([131072], 1, 64, 32, 1, 2, "normal"), ([131072, 100000, 70001, 3], 1, 64, 33, 1, 2, "equal"),
    ([1000], 999, 64, 6, 1, 1, "normal"), ([2000] * 9, 80, 64, 5, 0, 2, "equal"), ([40000] * 40, 1, 64, 100, 1, 1, "equal"),
    ([500], 3, 16, 7, 1, 1, "normal"), ([777], 2, 1, 50, 3, 3, "equal"), ([1000], 1, 128, 3, 0, 1, "special"),
    ([3000], 1, 64, 100, 1, 1, "normal"), ([600000], 1, 64, 600, 1, 1, "equal"), ([70000], 1, 4, 40, 1, 1, "equal")])
def test_block_topk(dev, lens, per, page, N, first, last, kind):
    g = torch.Generator().manual_seed(sum(lens) + N)
    B, ctx = len(lens), max(lens)
    q_pos = torch.cat([torch.arange(n - per, n) for n in lens]).clamp(min=0).to(torch.int32)
    T, ld = B * per, (ctx + 3) // 4 * 4
    x = _scores(g, T, ld, kind)
    behind = torch.arange(ld)[None, :] > q_pos[:, None]
    x[behind] = float("inf") if kind != "special" else float("nan")   # what is not there is never a score
    seq = dsa.Seq(q_seq=torch.arange(B, dtype=torch.int32).repeat_interleave(per).to(dev), q_pos=q_pos.to(dev),
                  block_table=torch.zeros((B, (ctx + page - 1) // page), dtype=torch.int32, device=dev), max_ctx=ctx,
                  cache_rows=page, page_size=page, q_per_seq=per)
    out = torch.full((T, N), -7, dtype=torch.int32, device=dev)
    dsa.block_topk(seq, x.to(dev), N, out, first=first, last=last)
    dsa.check_status()
    assert np.array_equal(out.cpu().numpy(), _choice(x.numpy(), q_pos.numpy(), page, N, first, last))


def test_block_topk_captured_and_on_two_streams(dev):
    g = torch.Generator().manual_seed(7)
    q_pos = torch.tensor([20000, 9000, 63, 64], dtype=torch.int32)
    seq = dsa.Seq(q_seq=torch.zeros(4, dtype=torch.int32, device=dev), q_pos=q_pos.to(dev),
                  block_table=torch.zeros((1, 313), dtype=torch.int32, device=dev), max_ctx=20001, cache_rows=64)
    xs = [torch.randn((4, 20004), generator=g).to(dev) for _ in range(2)]
    outs = [torch.full((4, 12), -7, dtype=torch.int32, device=dev) for _ in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for x, o, st in zip(xs, outs, streams):
            with torch.cuda.stream(st):
                dsa.block_topk(seq, x, 12, o, first=2, last=1)
    torch.cuda.synchronize()
    for x, o in zip(xs, outs):
        assert np.array_equal(o.cpu().numpy(), _choice(x.cpu().numpy(), q_pos.numpy(), 64, 12, 2, 1))
    with torch.cuda.stream(streams[0]):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[0]):
            for x, o in zip(xs, outs):
                dsa.block_topk(seq, x, 12, o, first=2, last=1)
        for x in xs:
            x.copy_(torch.randn(x.shape, generator=g))
        graph.replay()
    torch.cuda.synchronize()
    dsa.check_status()
    for x, o in zip(xs, outs):
        assert np.array_equal(o.cpu().numpy(), _choice(x.cpu().numpy(), q_pos.numpy(), 64, 12, 2, 1))


def test_block_topk_bad_position(dev):
    x = torch.randn((3, 400), device=dev)
    seq = dsa.Seq(q_seq=torch.zeros(3, dtype=torch.int32, device=dev), q_pos=torch.tensor([399, 400, -1], dtype=torch.int32, device=dev),
                  block_table=torch.zeros((1, 7), dtype=torch.int32, device=dev), max_ctx=400, cache_rows=64)
    out = torch.full((3, 4), -7, dtype=torch.int32, device=dev)
    dsa.block_topk(seq, x, 4, out)
    with pytest.raises(dsa.DSAError, match="bad_q_pos"):
        dsa.check_status()
    assert bool((out[1:] == -1).all()) and bool((out[0] >= 0).all())


# ------------------------------------------------------------------------------------------------- the step

@pytest.mark.parametrize("keys", ["mxfp4", "e4m3"])
@pytest.mark.parametrize("lens, per", [([3000, 1700, 50], 1), ([2000], 64)])
def test_block_decode_step(dev, keys, lens, per):
    """A serving step as a user chains it: new keys and latent rows appended, queries quantised, then the step in one call
    against its three calls; eagerly, and captured and replayed with other inputs."""
    s = Blocks(dev, lens, per=per, seed=11)
    T, N = s.T, 8
    fmt = dsa.DSA_MXFP4_E2M1 if keys == "mxfp4" else dsa.DSA_E4M3
    kb = 64 if keys == "mxfp4" else 128
    codes = torch.zeros((s.rows, kb), dtype=torch.uint8, device=dev)
    ksc = torch.zeros((s.rows, 4), dtype=torch.uint8, device=dev) if keys == "mxfp4" else torch.zeros(s.rows, device=dev)
    every = dsa.Seq(q_seq=torch.cat([torch.full((n,), b) for b, n in enumerate(lens)]).to(torch.int32).to(dev),
                    q_pos=torch.cat([torch.arange(n) for n in lens]).to(torch.int32).to(dev), block_table=s.table, max_ctx=s.ctx, cache_rows=s.rows)
    rnd = lambda *n: torch.randn(n, generator=s.g, device=dev).to(torch.bfloat16)
    dsa.index_cache_append(every, rnd(sum(lens), 128), codes, ksc, dtype=fmt)
    q_new, k_new, kv_new = rnd(T, 64, 128), rnd(T, 128), rnd(T, D_ROW)
    qc = torch.empty((T, 64, kb), dtype=torch.uint8, device=dev)
    qs = torch.empty((T, 64, 4), dtype=torch.uint8, device=dev) if keys == "mxfp4" else torch.empty((T, 64), device=dev)
    idxr = dsa.Indexer(q=qc, w=torch.randn((T, 64), generator=s.g, device=dev), k_cache=codes, q_scale=qs, k_scale=ksc, dtype=fmt)
    out, lse = torch.empty((T, 128, D_V), dtype=torch.bfloat16, device=dev), torch.empty((T, 128), device=dev)
    sel = torch.empty((T, N), dtype=torch.int32, device=dev)
    ws = torch.empty(dsa.block_decode_workspace_size(s.seq, s.mla, N), dtype=torch.uint8, device=dev)

    def step():
        dsa.index_cache_append(s.seq, k_new, codes, ksc, dtype=fmt)
        dsa.latent_cache_append(s.seq, s.mla, kv_new)
        dsa.index_query_quantize(q_new, qc, qs, dtype=fmt)
        dsa.block_decode_step(s.seq, idxr, s.mla, N, out, ws, first=1, last=2, lse=lse, block_idx_out=sel)

    def check():
        dsa.check_status()
        scores = torch.zeros((T, (s.ctx + 3) // 4 * 4), device=dev)
        dsa.indexer_scores(s.seq, idxr, scores)
        blocks = torch.empty_like(sel)
        dsa.block_topk(s.seq, scores, N, blocks, first=1, last=2)
        assert torch.equal(blocks, sel)
        assert np.array_equal(sel.cpu().numpy(), _choice(scores.cpu().numpy(), s.q_pos.cpu().numpy(), 64, N, 1, 2))
        o2, l2 = s.run(sel)
        dsa.check_status()
        assert torch.equal(out, o2) and torch.equal(lse, l2)
        s.check((out, lse), sel, ts=sorted({0, T // 2, T - 1}))

    step()
    check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        for x in (q_new, k_new, kv_new, s.q):
            x.copy_(torch.randn(x.shape, generator=s.g, device=dev).to(torch.bfloat16))
        graph.replay()
    side.synchronize()
    check()


def test_calls_of_no_queries(dev):
    s = Blocks(dev, [100])
    none = torch.zeros(0, dtype=torch.int32, device=dev)
    seq = dsa.Seq(q_seq=none, q_pos=none, block_table=s.table, max_ctx=100, cache_rows=s.rows)
    mla = dsa.Mla(q=s.q[:0], kv_cache=s.wide, d_latent=D_V, d_rope=64, softmax_scale=1.0)
    out = torch.empty((0, 128, D_V), dtype=torch.bfloat16, device=dev)
    dsa.block_mla_attn(seq, mla, torch.empty((0, 4), dtype=torch.int32, device=dev), out)
    dsa.block_topk(seq, torch.empty((0, 100), device=dev), 4, torch.empty((0, 4), dtype=torch.int32, device=dev))
    dsa.check_status()


# ------------------------------------------------------------------------------------------------- many queries, other caches

@pytest.mark.parametrize("kind", ["equal", "special", "normal"])
@pytest.mark.parametrize("ctx, page, N, first, last, threads", [(16384, 64, 33, 1, 2, 64), (40000, 64, 100, 0, 0, 128), (40000, 64, 600, 2, 5, 128),
                                                               (3000, 16, 50, 1, 1, 64), (12000, 16, 90, 3, 0, 128), (5000, 7, 200, 1, 1, 128)])
def test_block_topk_of_many_queries(dev, ctx, page, N, first, last, threads, kind):
    """A prompt chunk's launches: small CTAs, each of which reads its blocks in several turns and writes its choice in several chunks."""
    g = torch.Generator().manual_seed(ctx + N)
    B, per = 40, 8
    lens = [ctx - b * 97 % (ctx - 100) for b in range(B - 1)] + [page * N // 2]
    q_pos = torch.cat([torch.arange(n - per, n) for n in lens]).to(torch.int32)
    T, ld = B * per, (ctx + 3) // 4 * 4
    x = _scores(g, T, ld, kind)
    x[torch.arange(ld)[None, :] > q_pos[:, None]] = float("inf") if kind != "special" else float("nan")
    seq = dsa.Seq(q_seq=torch.arange(B, dtype=torch.int32).repeat_interleave(per).to(dev), q_pos=q_pos.to(dev),
                  block_table=torch.zeros((B, (ctx + page - 1) // page), dtype=torch.int32, device=dev), max_ctx=ctx,
                  cache_rows=page, page_size=page, q_per_seq=per)
    out = torch.full((T, N), -7, dtype=torch.int32, device=dev)
    dsa.block_topk(seq, x.to(dev), N, out, first=first, last=last)
    assert f"threads={threads}]" in dsa.last_plan()
    dsa.check_status()
    assert np.array_equal(out.cpu().numpy(), _choice(x.numpy(), q_pos.numpy(), page, N, first, last))


@pytest.mark.parametrize("fmt, page, H", [("e4m3", 64, 128), ("e4m3_t128", 64, 128), ("e2m1", 64, 128), ("bf16", 64, 16), ("bf16", 32, 16),
                                          ("bf16", 16, 128), ("e2m1", 32, 16)])
def test_block_decode_step_over_other_caches(dev, fmt, page, H):
    """The chained step against its three calls, over every row format and over pages of other sizes; eagerly, and captured and
    replayed with other queries."""
    g = torch.Generator(device=dev).manual_seed(page + H)
    lens, per, N = [900, 333], 2, 6
    B, T, ctx = len(lens), len(lens) * per, max(lens)
    pages = (ctx + page - 1) // page
    rows = B * pages * page
    table = torch.randperm(B * pages, generator=g, device=dev).to(torch.int32).view(B, pages)
    seq = dsa.Seq(q_seq=torch.arange(B, dtype=torch.int32, device=dev).repeat_interleave(per), block_table=table, max_ctx=ctx, cache_rows=rows,
                  q_pos=torch.cat([torch.arange(n - per, n) for n in lens]).to(torch.int32).to(dev), page_size=page, q_per_seq=per)
    every = dsa.Seq(q_seq=torch.arange(B, dtype=torch.int32, device=dev).repeat_interleave(ctx), block_table=table, max_ctx=ctx, cache_rows=rows,
                    q_pos=torch.arange(ctx, dtype=torch.int32, device=dev).repeat(B), page_size=page)
    code, width = {"bf16": (None, None), "e4m3": (dsa.DSA_E4M3, 656), "e4m3_t128": (dsa.DSA_E4M3_T128, 656), "e2m1": (dsa.DSA_E2M1, 432)}[fmt]
    cache = torch.zeros((rows, D_ROW), dtype=torch.bfloat16, device=dev) if width is None else torch.zeros((rows, width), dtype=torch.uint8, device=dev)
    rnd = lambda *n: torch.randn(n, generator=g, device=dev).to(torch.bfloat16)
    mla = dsa.Mla(q=rnd(T, H, D_ROW), kv_cache=cache, d_latent=D_V, d_rope=64, softmax_scale=SCALE, dtype=code)
    dsa.latent_cache_append(every, mla, rnd(B * ctx, D_ROW))
    codes, exps = torch.zeros((rows, 64), dtype=torch.uint8, device=dev), torch.zeros((rows, 4), dtype=torch.uint8, device=dev)
    dsa.index_cache_append(every, rnd(B * ctx, 128), codes, exps, dtype=dsa.DSA_MXFP4_E2M1)
    qc, qs = torch.empty((T, 64, 64), dtype=torch.uint8, device=dev), torch.empty((T, 64, 4), dtype=torch.uint8, device=dev)
    idx = dsa.Indexer(q=qc, w=torch.randn((T, 64), generator=g, device=dev), k_cache=codes, q_scale=qs, k_scale=exps, dtype=dsa.DSA_MXFP4_E2M1)
    q_new = rnd(T, 64, 128)
    out, lse = torch.empty((T, H, D_V), dtype=torch.bfloat16, device=dev), torch.empty((T, H), device=dev)
    sel = torch.full((T, N), -7, dtype=torch.int32, device=dev)
    ws = torch.empty(dsa.block_decode_workspace_size(seq, mla, N), dtype=torch.uint8, device=dev)

    def step():
        dsa.index_query_quantize(q_new, qc, qs, dtype=dsa.DSA_MXFP4_E2M1)
        dsa.block_decode_step(seq, idx, mla, N, out, ws, first=1, last=1, lse=lse, block_idx_out=sel)

    def check():
        dsa.check_status()
        scores = torch.zeros((T, (ctx + 3) // 4 * 4), device=dev)
        dsa.indexer_scores(seq, idx, scores)
        assert np.array_equal(sel.cpu().numpy(), _choice(scores.cpu().numpy(), seq.q_pos.cpu().numpy(), page, N, 1, 1))
        o2, l2 = torch.empty_like(out), torch.empty_like(lse)
        dsa.block_mla_attn(seq, mla, sel, o2, lse=l2, workspace=torch.empty(
            max(16, dsa.block_mla_attn_workspace_size(seq, mla, N)), dtype=torch.uint8, device=dev))
        dsa.check_status()
        assert torch.equal(out, o2) and torch.equal(lse, l2) and bool(torch.isfinite(lse).all())

    step()
    assert ("expand_blocks" in dsa.last_plan()) == ((fmt, page) != ("bf16", 64))
    check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        for x in (q_new, mla.q):
            x.copy_(torch.randn(x.shape, generator=g, device=dev).to(torch.bfloat16))
        graph.replay()
    side.synchronize()
    check()
