"""The attention over 4-bit rows where its schedule shows: several queries per cluster of CTAs one after the other, slices
of one tile, pages of any size, rows that nobody selects, waits that run out, streams.  Against the float64 oracle with
the tolerances derived in test_gpu_e2m1.py."""
import dataclasses

import numpy as np
import pytest
import torch

import dsa_indexed_sparse_gb300 as dsa
import dsa_workloads as W
from oracle import dsa_oracle as O
from tests import parity as P
from tests.test_gpu_e2m1 import _check, _make, _selection

pytestmark = pytest.mark.gpu


def _repage(wl, page, seed):
    """The same cache content in pages of another size, shuffled."""
    rng = np.random.default_rng(seed)
    need = [(int(wl.q_pos[wl.q_seq == b].max()) + page) // page for b in range(wl.B)]
    perm = rng.permutation(sum(need)).astype(np.int32)
    table = np.full((wl.B, (wl.max_ctx + page - 1) // page), -1, np.int32)
    kv = rng.integers(0, 256, (len(perm) * page, wl.kv.shape[1])).astype(np.uint8)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
        pos = np.arange(int(wl.q_pos[wl.q_seq == b].max()) + 1)
        kv[O.physical_rows(table[b], page, pos)] = wl.kv[O.physical_rows(wl.block_table[b], wl.page_size, pos)]
    # the indexer's keys are not used here, but have to be there for every row
    return dataclasses.replace(wl, kv=kv, block_table=table, page_size=page, cache_rows=len(kv),
                               k_i=np.zeros((len(kv), wl.k_i.shape[1]), wl.k_i.dtype),
                               k_i_scale=np.ones(len(kv), np.float32))


@pytest.mark.parametrize("H,T,K", [(128, 500, 1), (128, 330, 128), (64, 330, 129), (130, 130, 256), (200, 170, 257),
                                   (7, 400, 40), (128, 160, 600)])
def test_several_queries_per_cluster(dev, H, T, K):
    """Queries by the hundred, some with holes, some that select nothing at all, first, last and in a row."""
    wl = _make(H + T + K, ctx=[T + 700], q_len=T, K=K, H=H)
    empty = {0, 1, 2, 77, T - 1}
    idx = _selection(np.random.default_rng(K), wl, K, hole=0.3 if K > 1 else 0.0, empty=empty)
    out, lse, plan = P.Run(wl, dev).attn(idx)
    assert "split=1," in plan
    _check(out, lse, wl, idx, ts=sorted(empty | set(range(3, T, 41)) | {T - 2}))
    again, lse2, _ = P.Run(wl, dev).attn(idx)
    assert np.array_equal(out, again) and np.array_equal(lse, lse2)


@pytest.mark.parametrize("K", [129, 640, 2000])
def test_tiles_that_select_nothing(dev, K):
    """Selections that end early: one entry at every distance from the ends, only the first or the last one, gaps of whole
    tiles, and nothing; queries by the hundred, so that the ends differ from item to item of a cluster."""
    T = 310
    wl = _make(50 + K, ctx=[900], q_len=T, K=K)
    rng = np.random.default_rng(K)
    idx = np.full((T, K), -1, np.int32)
    for t in range(T):
        n = int(wl.q_pos[t]) + 1
        kind = t % 7
        if kind == 0:
            idx[t, :rng.integers(1, min(K, n))] = 0
            m = int((idx[t] == 0).sum())
            idx[t, :m] = rng.choice(n, m, replace=False)
        elif kind == 1:
            idx[t, K - 1] = n - 1
        elif kind == 2:
            idx[t, 0] = 0
        elif kind == 3:
            idx[t, [0, K // 2, K - 1]] = [3, 1, 2]
        elif kind == 4:
            idx[t, int(rng.integers(0, K))] = int(rng.integers(0, n))
        elif kind == 5:
            at = np.sort(rng.choice(K, min(K, 90), replace=False))
            idx[t, at] = rng.choice(n, len(at), replace=False)
    out, lse, _ = P.Run(wl, dev).attn(idx)
    _check(out, lse, wl, idx, ts=list(range(0, T, 3)))
    few = dataclasses.replace(wl, T=9, q_per_seq=0, q_seq=wl.q_seq[:9], q_pos=wl.q_pos[:9], q=wl.q[:9])
    for workspace in (True, False):                  # slices, some of them empty, and one slice
        out, lse, _ = P.Run(few, dev).attn(idx[:9], workspace=workspace)
        _check(out, lse, few, idx[:9])


def test_maxima_do_not_reach_the_next_query(dev):
    """Every third query's selection has rows with logits hundreds of powers of two above the others', late in it."""
    T, K = 240, 300
    wl = _make(21, ctx=[900], q_len=T, K=K)
    kv = wl.kv.copy()
    bits = kv[:, 304:432].copy().view("<u2")
    far = np.arange(100, 160)
    rows = O.physical_rows(wl.block_table[0], 64, far)
    lift = torch.from_numpy(O.decode_bf16(bits[rows]).astype(np.float32))
    lift[:, 0] = 900.0
    bits[rows] = W._bf16_bits(lift)
    kv[:, 304:432] = bits.view(np.uint8).reshape(wl.cache_rows, 128)
    q = torch.from_numpy(O.decode_bf16(wl.q).astype(np.float32))
    q[:, ::5, 512] = 5.0
    wl = dataclasses.replace(wl, kv=kv, q=W._bf16_bits(q))
    rng = np.random.default_rng(22)
    usual = np.setdiff1d(np.arange(600), far)
    idx = np.stack([rng.choice(usual, K, replace=False) for _ in range(T)]).astype(np.int32)
    idx[::3, 150:200] = far[:50]
    out, lse, _ = P.Run(wl, dev).attn(idx)
    _check(out, lse, wl, idx, ts=[0, 1, 2, 3, 79, 80, 81, 160, 161, 162, 237, 238, 239])


@pytest.mark.parametrize("page", [1, 48, 64, 200])
def test_page_sizes(dev, page):
    wl = _repage(_make(23, ctx=[333, 500, 64], K=150), page, page)
    idx = _selection(np.random.default_rng(24), wl, 150, hole=0.1)
    out, lse, _ = P.Run(wl, dev).attn(idx)
    _check(out, lse, wl, idx)


@pytest.mark.parametrize("workspace", [True, False])
def test_rows_that_nobody_selects_may_hold_anything(dev, workspace):
    """All bytes of every other row 0xFF (NaN scales, a NaN row scale, NaN rope), row 0 of the cache among them."""
    wl = _make(25, ctx=[400, 300], K=200)
    idx = _selection(np.random.default_rng(26), wl, 200, hole=0.4)
    kv = np.full_like(wl.kv, 0xFF)
    used = np.concatenate([O.physical_rows(wl.block_table[b], 64, np.unique(idx[t][idx[t] > 0]).astype(np.int64))
                           for t, b in enumerate(wl.q_seq)])
    used = used[used != 0]
    kv[used] = wl.kv[used]
    for t, b in enumerate(wl.q_seq):
        keep = np.isin(O.physical_rows(wl.block_table[b], 64, np.maximum(idx[t], 0).astype(np.int64)), used)
        idx[t][~keep] = -1
    wl = dataclasses.replace(wl, kv=kv)
    out, lse, _ = P.Run(wl, dev).attn(idx, workspace=workspace)
    _check(out, lse, wl, idx)


@pytest.mark.parametrize("scale", [-0.09, 0.0, 1e-30])
def test_any_softmax_scale(dev, scale):
    """Negative: the order of the logits turns round; zero: the mean of the selected rows."""
    wl = dataclasses.replace(_make(27, ctx=[600, 90], K=300), softmax_scale=scale)
    idx = _selection(np.random.default_rng(28), wl, 300, hole=0.2)
    out, lse, _ = P.Run(wl, dev).attn(idx)
    _check(out, lse, wl, idx)


def test_long_selection(dev):
    """More selected entries than the context has positions: the rest are holes."""
    wl = _make(29, ctx=[700], K=5000)
    idx = np.full((1, 5000), -1, np.int32)
    where = np.sort(np.random.default_rng(30).choice(5000, 700, replace=False))
    idx[0, where] = np.arange(700)
    for workspace in (True, False):
        out, lse, _ = P.Run(wl, dev).attn(idx, workspace=workspace)
        _check(out, lse, wl, idx)


@pytest.mark.parametrize("T", [1, 300])
def test_bounded_wait_runs_out_and_the_next_call_is_clean(dev, T):
    """A producer warp withholds its first arrival (the testing aid): the waits run out, every warp unwinds, TMEM is
    released and the status says so; the next call gives what the call before gave."""
    wl = _make(31, ctx=[800], q_len=T, K=256)
    idx = _selection(np.random.default_rng(32), wl, 256)
    r = P.Run(wl, dev)
    out, lse, plan = r.attn(idx)
    dsa.debug_withhold_arrival(True, 2_000_000)
    try:
        with pytest.raises(dsa.DSAError) as e:
            r.attn(idx)
    finally:
        dsa.debug_withhold_arrival(False)
    assert e.value.status == 5 and "timeout" in str(e.value)
    dsa.check_status()
    again, lse2, _ = r.attn(idx)
    assert np.array_equal(out, again) and np.array_equal(lse, lse2)


def test_no_queries_and_other_stream(dev):
    wl = _make(33, ctx=[300], q_len=9, K=70)
    idx = _selection(np.random.default_rng(34), wl, 70)
    want, lse, _ = P.Run(wl, dev).attn(idx)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got, lse2, _ = P.Run(wl, dev).attn(idx)
    assert np.array_equal(got, want) and np.array_equal(lse2, lse)
    r = P.Run(wl, dev)
    none = dsa.Seq(q_seq=r.seq.q_seq[:0], q_pos=r.seq.q_pos[:0], block_table=r.seq.block_table, max_ctx=wl.max_ctx,
                   cache_rows=wl.cache_rows)
    m = dataclasses.replace(r.mla, q=r.mla.q[:0])
    out = torch.empty((0, wl.H, 512), dtype=torch.bfloat16, device=dev)
    assert dsa.sparse_mla_attn(none, m, torch.empty((0, 70), dtype=torch.int32, device=dev), 70, out) is out
    dsa.check_status()


def test_output_beside_other_rows(dev):
    """An output that starts 16 bytes off a 32-byte boundary, with rows before and behind that stay as they were."""
    wl = _make(35, ctx=[400], q_len=100, K=128, H=40)
    idx = _selection(np.random.default_rng(36), wl, 128)
    want, _, _ = P.Run(wl, dev).attn(idx)
    r = P.Run(wl, dev)
    n = wl.T * wl.H * 512
    buf = torch.full((n + 1024,), 7.0, dtype=torch.bfloat16, device=dev)
    out = buf[8:8 + n].view(wl.T, wl.H, 512)
    dsa.sparse_mla_attn(r.seq, r.mla, torch.from_numpy(idx).to(dev), 128, out)
    dsa.check_status()
    assert np.array_equal(out.float().cpu().numpy(), want)
    assert bool((buf[:8] == 7).all()) and bool((buf[8 + n:] == 7).all())


def test_row_scales_of_either_sign(dev):
    """Row scales are any fp32 numbers to the reader: negative ones turn a row's latent part round, large and small ones mix."""
    wl = _make(61, ctx=[700, 500], K=300)
    kv = wl.kv.copy()
    rs = kv[:, 288:292].copy().view("<f4")[:, 0]
    rng = np.random.default_rng(62)
    rs = rs * np.where(rng.random(len(rs)) < 0.5, -1.0, 1.0).astype("<f4") * 2.0 ** rng.integers(-6, 3, len(rs)).astype("<f4")
    kv[:, 288:292] = rs.astype("<f4").view(np.uint8).reshape(-1, 4)
    wl = dataclasses.replace(wl, kv=kv)
    idx = _selection(rng, wl, 300, hole=0.1)
    for workspace in (True, False):
        out, lse, _ = P.Run(wl, dev).attn(idx, workspace=workspace)
        _check(out, lse, wl, idx)
    # Values of 2^18: what a weight in f16 loses shows beside outputs that are small because the rows with weight are 0
    # there.  P = p rs 2^(m - g) is off by half of f16's smallest step, 2^-25, where it is below 2^-14, so an output by
    # 2^(g - m) / l * sum_s 2^-25 |v_s / rs_s|.  g <= max(x) + log2 max(rs) - 7 with the maximum x (log2 units) rounded up
    # by 2^-7 of itself at most, and l >= 2^(max(x) - m): 2^-32 max(rs) 2^(|max x| / 128) sum_s |v_s / rs_s|.
    kv = kv.copy()
    big = (-np.abs(rs) * np.float32(2.0 ** 18)).astype("<f4")
    kv[:, 288:292] = big.view(np.uint8).reshape(-1, 4)
    q = torch.from_numpy(O.decode_bf16(wl.q).astype(np.float32))
    q[..., :512] *= 2.0 ** -18
    wl = dataclasses.replace(wl, kv=kv, q=W._bf16_bits(q))
    out, lse, _ = P.Run(wl, dev).attn(idx)
    for t in range(wl.T):
        sel = idx[t][idx[t] >= 0].astype(np.int64)
        o_out, o_lse = O.sparse_mla_attn_row(wl, t, idx[t])
        rows = O.physical_rows(wl.block_table[wl.q_seq[t]], wl.page_size, sel)
        v = O.latent_rows(wl, rows)
        logits = wl.softmax_scale * (O.mla_query(wl, t) @ v.T)
        p = np.exp(logits - o_lse[:, None])
        A = p @ np.abs(v[:, :512])
        r = np.abs(big[rows].astype(np.float64))
        lost = 2.0 ** -32 * r.max() * (np.abs(v[:, :512]) / r[:, None]).sum(0)
        lost = lost[None] * 2.0 ** (np.abs(logits).max(1, keepdims=True) * 1.4427 / 128)
        lse_tol = 576 * 2.0 ** -24 * abs(wl.softmax_scale) * (np.abs(O.mla_query(wl, t)) @ np.abs(v).T).max(1) + 1e-4
        tol = 1.01 * 2.0 ** -8 * (2 * A + 2 * np.abs(o_out)) + 2 * lse_tol[:, None] * A + lost
        err = np.abs(out[t] - o_out)
        assert np.all(err <= tol), (t, float((err / tol).max()))
        assert np.all(np.abs(lse[t] - o_lse) <= lse_tol)


def test_two_streams_at_once(dev):
    """Two calls with several queries per cluster and two with slices, again and again on two streams: the same bits."""
    calls = []
    for seed, T, K in ((71, 300, 200), (72, 4, 900)):
        wl = _make(seed, ctx=[1100], q_len=T, K=K)
        idx = torch.from_numpy(_selection(np.random.default_rng(seed), wl, K, hole=0.1)).to(dev)
        for copy in range(2):
            r = P.Run(wl, dev)
            out = torch.empty((T, wl.H, 512), dtype=torch.bfloat16, device=dev)
            ws = torch.empty(max(16, dsa.sparse_mla_attn_workspace_size(r.seq, r.mla, K)), dtype=torch.uint8, device=dev)
            dsa.sparse_mla_attn(r.seq, r.mla, idx, K, out, workspace=ws)
            torch.cuda.synchronize()
            calls.append((r, idx, K, out, ws, out.clone(), torch.cuda.Stream()))
    for _ in range(10):
        for r, idx, K, out, ws, want, s in calls:
            with torch.cuda.stream(s):
                out.zero_()
                for _ in range(5):
                    dsa.sparse_mla_attn(r.seq, r.mla, idx, K, out, workspace=ws)
        torch.cuda.synchronize()
        for r, idx, K, out, ws, want, s in calls:
            assert torch.equal(out, want)
    dsa.check_status()
