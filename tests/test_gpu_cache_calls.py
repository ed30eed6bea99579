"""The rotating writers and the cache reader as a program chains them: records whose tensors are not on the GPU, outputs
that feed the next call at once, long lists of tokens, streams and graphs.  Values are compared bit for bit with the same
calls made one by one, or with the oracle's rows."""
import dataclasses

import numpy as np
import pytest
import torch

import dsa_indexed_sparse_gb300 as dsa
from oracle import dsa_oracle as O
from tests import parity as P
from tests.test_gpu_e2m1 import _make, _selection

pytestmark = pytest.mark.gpu


def _cache(dev, B, ctx, row_bytes=432):
    pages = (ctx + 63) // 64
    table = torch.randperm(B * pages, generator=torch.Generator().manual_seed(B * ctx)).to(torch.int32).view(B, pages)
    rows = B * pages * 64
    return table.to(dev), rows, torch.zeros((rows, row_bytes), dtype=torch.uint8, device=dev)


def _mla(kv, dtype=dsa.DSA_E2M1):
    q = torch.zeros((1, 1, 576), dtype=torch.bfloat16, device=kv.device)
    return dsa.Mla(q=q, kv_cache=kv, d_latent=512, d_rope=64, softmax_scale=1.0, dtype=dtype)


def test_records_off_the_gpu_are_refused(dev):
    table, rows, kv = _cache(dev, 2, 100)
    seq = torch.tensor([0, 1], dtype=torch.int32, device=dev)
    pos = torch.tensor([5, 7], dtype=torch.int32, device=dev)
    plan = dsa.Rope.make(64)
    new = torch.zeros((2, 576), dtype=torch.bfloat16, device=dev)
    out = torch.zeros((2, 576), dtype=torch.bfloat16, device=dev)
    key = torch.zeros((2, 128), dtype=torch.bfloat16, device=dev)
    kc, ks = torch.zeros((rows, 128), dtype=torch.uint8, device=dev), torch.zeros(rows, device=dev)
    good = dict(q_seq=seq, q_pos=pos, block_table=table, max_ctx=100, cache_rows=rows)
    for field in ("q_seq", "q_pos", "block_table"):
        s = dsa.Seq(**{**good, field: good[field].cpu()})
        with pytest.raises(ValueError, match="CUDA device"):
            dsa.latent_cache_read(s, _mla(kv), out)
        with pytest.raises(ValueError, match="CUDA device"):
            dsa.latent_cache_append_rope(s, _mla(kv), plan, new[:, :512], new[:, 512:])
        with pytest.raises(ValueError, match="CUDA device"):
            dsa.index_cache_append_rope(s, plan, key, kc, ks)
    s = dsa.Seq(**good)
    with pytest.raises(ValueError, match="CUDA device"):
        dsa.latent_cache_read(s, _mla(kv.cpu()), out)
    with pytest.raises(ValueError, match="CUDA device"):
        dsa.index_cache_append_rope(s, plan, key, kc.cpu(), ks)
    with pytest.raises(ValueError, match="CUDA device"):
        dsa.rope(plan, pos.cpu(), new[:, 512:], new[:, 512:])
    dsa.check_status()


@pytest.mark.parametrize("T", [1, 9727, 9729, 30001])
def test_append_then_read_of_many_tokens(dev, T):
    """Every token of one long sequence written and read back at once, in a random order; the sizes around the number of
    warps that the GPU holds, and an odd one."""
    table, rows, kv = _cache(dev, 1, T)
    g = torch.Generator(device=dev).manual_seed(T)
    order = torch.randperm(T, generator=g, device=dev).to(torch.int32)
    s = dsa.Seq(q_seq=torch.zeros(T, dtype=torch.int32, device=dev), q_pos=order, block_table=table, max_ctx=T, cache_rows=rows)
    new = torch.randn((T, 576), generator=g, device=dev).to(torch.bfloat16)
    plan = dsa.Rope.make(64, layout="half")
    mla = _mla(kv)
    dsa.latent_cache_append_rope(s, mla, plan, new[:, :512], new[:, 512:])
    out = torch.full((T, 576), float("nan"), dtype=torch.bfloat16, device=dev)
    dsa.latent_cache_read(s, mla, out)
    pe = torch.empty((T, 64), dtype=torch.bfloat16, device=dev)
    dsa.rope(plan, order, new[:, 512:], pe)
    dsa.check_status()
    assert torch.equal(out[:, 512:], pe)             # the writer's rotation is the rope call's, bit for bit
    for t in {0, T // 2, T - 1}:
        row = O.e2m1_row(new[t, :512].float().cpu().numpy(), np.zeros(64))
        at = int(O.physical_rows(table[0].cpu().numpy(), 64, np.array([int(order[t])]))[0])
        assert np.array_equal(kv[at, :304].cpu().numpy(), row[:304])
    # a latent value is off by at most one unit of its block scale (codes 4 and 6 lie two units apart; beyond 6 a unit is
    # not reached: the scale is rounded by 2^-4 of itself at most), which is at most amax / 6 (1 + 2^-4); exact in bf16
    x = new[:, :512].float().view(T, 32, 16)
    amax = x.abs().amax(-1, keepdim=True)
    assert bool(((out[:, :512].float().view(T, 32, 16) - x).abs() <= 1.001 * amax / 6 * (1 + 2 ** -4)).all())


def test_reader_feeds_the_next_call_at_once(dev):
    """The reader's output rotated, appended to another cache of another format and read again, without a wait between,
    eagerly and as a replayed graph on another stream."""
    T = 700
    table, rows, kv = _cache(dev, 1, T)
    _, _, kv8 = _cache(dev, 1, T, 656)
    g = torch.Generator(device=dev).manual_seed(3)
    s = dsa.Seq(q_seq=torch.zeros(T, dtype=torch.int32, device=dev), q_pos=torch.arange(T, dtype=torch.int32, device=dev),
                block_table=table, max_ctx=T, cache_rows=rows)
    new = torch.randn((T, 576), generator=g, device=dev).to(torch.bfloat16)
    plan = dsa.Rope.make(64)
    m4, m8 = _mla(kv), _mla(kv8, dsa.DSA_E4M3)
    a, b = (torch.empty((T, 576), dtype=torch.bfloat16, device=dev) for _ in range(2))

    def run():
        dsa.latent_cache_append_rope(s, m4, plan, new[:, :512], new[:, 512:])
        dsa.latent_cache_read(s, m4, a)
        dsa.rope(plan, s.q_pos, a[:, 512:], a[:, 512:], inverse=True)
        dsa.latent_cache_append_rope(s, m8, plan, a[:, :512], a[:, 512:])
        dsa.latent_cache_read(s, m8, b)

    steps = []
    for call in (lambda: dsa.latent_cache_append_rope(s, m4, plan, new[:, :512], new[:, 512:]),
                 lambda: dsa.latent_cache_read(s, m4, a),
                 lambda: dsa.rope(plan, s.q_pos, a[:, 512:], a[:, 512:], inverse=True),
                 lambda: dsa.latent_cache_append_rope(s, m8, plan, a[:, :512], a[:, 512:]),
                 lambda: dsa.latent_cache_read(s, m8, b)):
        call()
        torch.cuda.synchronize()
    want = a.clone(), b.clone(), kv8.clone()
    # rotated and turned back: two roundings to bf16, each at most 2^-8 of the pair's length (a little more in all)
    pair = new[:, 512:].float().view(T, 32, 2).norm(dim=-1, keepdim=True)
    assert bool(((a[:, 512:].float() - new[:, 512:].float()).view(T, 32, 2).abs() <= 2.01 * 2 ** -8 * pair).all())
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for again in range(3):
        for t in (a, b, kv, kv8):
            t.zero_()
        torch.cuda.synchronize()
        if again == 0:
            run()
        else:
            with torch.cuda.stream(st):
                if again == 1:
                    graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(graph, stream=st):
                        run()
                for _ in range(3):
                    graph.replay()
        torch.cuda.synchronize()
        dsa.check_status()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1]) and torch.equal(kv8, want[2])


def test_read_query_feeds_a_decode_step_at_once(dev):
    """The attention stages its query early in a decode step: here the call before has just written it."""
    wl = _make(41, ctx=[900, 500, 800], K=128, H=1)
    r = P.Run(wl, dev)
    n = wl.T
    src = torch.from_numpy(np.random.default_rng(42).normal(0, 1, (n, 576)).astype(np.float32)).to(torch.bfloat16).to(dev)
    table, rows, kv = _cache(dev, 1, 64, 1152)
    kv = kv.view(torch.bfloat16)
    s = dsa.Seq(q_seq=torch.zeros(n, dtype=torch.int32, device=dev), q_pos=torch.arange(n, dtype=torch.int32, device=dev),
                block_table=table, max_ctx=64, cache_rows=rows)
    m = _mla(kv, dsa.DSA_BF16)
    dsa.latent_cache_append(s, m, src)
    q = r.mla.q.view(n, 576)
    ws = torch.empty(dsa.decode_workspace_size(r.seq, r.idxr, r.mla, 128), dtype=torch.uint8, device=dev)
    out = torch.empty((n, 1, 512), dtype=torch.bfloat16, device=dev)
    q.copy_(src)
    dsa.decode_step(r.seq, r.idxr, r.mla, 128, out, ws)
    torch.cuda.synchronize()
    want = out.clone()
    for _ in range(50):
        q.fill_(float("nan"))
        dsa.latent_cache_read(s, m, q)
        dsa.decode_step(r.seq, r.idxr, r.mla, 128, out, ws)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    dsa.check_status()


def test_codes_at_every_border(dev):
    """For every block scale the values half way between two codes and their bf16 neighbours on both sides, of both signs:
    the codes are the oracle's, computed from 64-bit quotients."""
    scales = [v for v in O.decode_e4m3(np.arange(127, dtype=np.uint8)) if 0 < v <= 256]
    blocks = []
    for sc in scales:
        vals = []
        for mid in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
            x = torch.tensor(mid * sc, dtype=torch.float64).to(torch.bfloat16)
            assert float(x) == mid * sc                     # at most seven significant bits
            bits = int(x.view(torch.int16))
            for b in (bits - 1, bits, bits + 1):
                v = float(torch.tensor(b, dtype=torch.int16).view(torch.bfloat16))
                vals += [v, -v]
        vals += [0.0, -0.0, 6 * sc]
        for i in range(0, len(vals), 15):
            blocks.append([6 * sc] + (vals[i:i + 15] + [0.0] * 15)[:15])   # the block's maximum: its scale is sc
    top = [1536.0] + [0.0] * 15                             # the row's maximum: a row scale of 1
    blocks += [top] * (-len(blocks) % 31)
    rows = np.array([top + sum(blocks[i:i + 31], []) for i in range(0, len(blocks), 31)], np.float32)
    T = len(rows)
    table, n, kv = _cache(dev, 1, T)
    s = dsa.Seq(q_seq=torch.zeros(T, dtype=torch.int32, device=dev), q_pos=torch.arange(T, dtype=torch.int32, device=dev),
                block_table=table, max_ctx=T, cache_rows=n)
    new = torch.cat([torch.from_numpy(rows), torch.zeros((T, 64))], dim=1).to(torch.bfloat16).to(dev)
    dsa.latent_cache_append(s, _mla(kv), new)
    dsa.check_status()
    at = O.physical_rows(table[0].cpu().numpy(), 64, np.arange(T))
    got = kv.cpu().numpy()[at]
    for t in range(T):
        want = O.e2m1_row(rows[t].astype(np.float64), np.zeros(64))
        assert np.array_equal(got[t], want), (t, np.nonzero(got[t] != want)[0][:8])


def test_rows_beyond_32_bit_offsets(dev):
    """A cache of more than 2^32 bytes whose used pages lie at both ends: the same rows, values and attention as in a
    small cache, bit for bit."""
    T, n_small = 200, 256
    rows = ((1 << 32) // 432 // 64 + 80) * 64
    big = torch.empty((rows, 432), dtype=torch.uint8, device=dev)
    small = torch.zeros((n_small, 432), dtype=torch.uint8, device=dev)
    last = rows // 64 - 1
    tables = {"small": torch.tensor([[2, 0, 3, 1]], dtype=torch.int32, device=dev),
              "big": torch.tensor([[last, 0, last - 1, last - 77]], dtype=torch.int32, device=dev)}
    g = torch.Generator(device=dev).manual_seed(9)
    new = torch.randn((T, 576), generator=g, device=dev).to(torch.bfloat16)
    q = torch.randn((5, 128, 576), generator=g, device=dev).to(torch.bfloat16)
    plan = dsa.Rope.make(64)
    pos = torch.arange(T, dtype=torch.int32, device=dev)
    idx = torch.stack([torch.randperm(150 + t, generator=g, device=dev)[:140] for t in range(5)]).to(torch.int32)
    got = {}
    for name, kv in (("small", small), ("big", big)):
        common = dict(block_table=tables[name], max_ctx=256, cache_rows=kv.shape[0])
        s = dsa.Seq(q_seq=torch.zeros(T, dtype=torch.int32, device=dev), q_pos=pos, **common)
        m = dsa.Mla(q=q, kv_cache=kv, d_latent=512, d_rope=64, softmax_scale=0.07, dtype=dsa.DSA_E2M1)
        dsa.latent_cache_append_rope(s, m, plan, new[:, :512], new[:, 512:])
        vals = torch.empty((T, 576), device=dev)
        dsa.latent_cache_read(s, m, vals)
        queries = dsa.Seq(q_seq=torch.zeros(5, dtype=torch.int32, device=dev), q_pos=pos[150:155].clone(), **common)
        out = torch.empty((5, 128, 512), dtype=torch.bfloat16, device=dev)
        lse = torch.empty((5, 128), device=dev)
        ws = torch.empty(max(16, dsa.sparse_mla_attn_workspace_size(queries, m, 140)), dtype=torch.uint8, device=dev)
        dsa.sparse_mla_attn(queries, m, idx, 140, out, lse=lse, workspace=ws)
        dsa.check_status()
        got[name] = vals, out, lse
    assert all(torch.equal(a, b) for a, b in zip(got["small"], got["big"]))
    assert torch.equal(big[last * 64:], small[2 * 64:3 * 64])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("T,d", [(1, 64), (37, 16), (1000, 32), (3001, 64), (700, 512)])
def test_one_head_is_turned_as_one_of_many(dev, T, d, layout, dtype):
    """One head's tokens (which take their cosines without the detour that many heads share) against the same values as
    one of three heads, bit for bit; forwards, backwards and in place."""
    g = torch.Generator(device=dev).manual_seed(T + d)
    x = torch.randn((T, 3, d), generator=g, device=dev).to(dtype)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device=dev, dtype=torch.int32)
    plan = dsa.Rope.make(d, layout=layout, scaling="yarn", factor=8.0, original_ctx=4096)
    for inverse in (False, True):
        many = torch.empty_like(x)
        dsa.rope(plan, pos, x, many, inverse=inverse)
        one = torch.empty((T, d), dtype=dtype, device=dev)
        dsa.rope(plan, pos, x[:, 1], one, inverse=inverse)
        assert torch.equal(one, many[:, 1])
        y = x[:, 2].clone()
        dsa.rope(plan, pos, y, y, inverse=inverse)
        assert torch.equal(y, many[:, 2])
