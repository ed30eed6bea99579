"""GPU parity of the attention over 4-bit latent rows (DSA_E2M1) against the float64 oracle, alone, in the decode step,
and in the run of calls a serving step makes: rotate the query, append the new rows, attend.

Tolerances, derived: the rows' values are exact in bf16 and fp32 sums are far below a bf16 step, so an output value is
off by the rounding of the weights P to bf16 (2^-8 of each term, so at most 2^-8 A with A = sum_s p_s |v_s|), of their sum
that normalises it (2^-8 |out|), of a slice's partial output (2^-8 of values bounded by A) and of the output itself (2^-8
|out|): 2^-8 (2 A + 2 |out|), with 1 % over it for second-order terms and 1e-5 for the fp32 sums.  The log-sum-exp is
held in fp32: a logit is off by at most 576 * 2^-24 * scale * sum |q k| (fp32 accumulation in any order), the sum of
exponentials by K * 2^-24 + 2^-20 of itself (its additions and the exponential function).
"""
import dataclasses

import numpy as np
import pytest
import torch

import dsa_indexed_sparse_gb300 as dsa
import dsa_workloads as W
from oracle import dsa_oracle as O
from tests import parity as P

pytestmark = pytest.mark.gpu


def _make(seed, **over):
    base = dict(ctx_range=(60, 700), B=3, q_len=1, K=64, mla_dtype="e2m1")
    base.update(over)
    return W.make("decode_b64" if "ctx" not in base else "decode_b1", seed=seed, **base)


def _selection(rng, wl, K, hole=0.0, empty=()):
    idx = np.full((wl.T, K), -1, np.int32)
    for t in range(wl.T):
        n = int(wl.q_pos[t]) + 1
        m = min(K, n)
        if t not in empty:
            idx[t, :m] = np.sort(rng.choice(n, m, replace=False))
            idx[t][rng.random(K) < hole] = -1
    return idx


def _check(out, lse, wl, idx, ts=None, value_slack=0.0):
    """value_slack: relative rounding of the rows' values to bf16 (0 where they are exact)."""
    for t in range(wl.T) if ts is None else ts:
        sel = idx[t][idx[t] >= 0].astype(np.int64)
        o_out, o_lse = O.sparse_mla_attn_row(wl, t, idx[t])
        if not len(sel):
            assert not out[t].any() and np.all(lse[t] == -np.inf), t
            continue
        kv = O.latent_rows(wl, O.physical_rows(wl.block_table[wl.q_seq[t]], wl.page_size, sel))
        q = O.mla_query(wl, t)
        logits = wl.softmax_scale * (q @ kv.T)
        p = np.exp(logits - o_lse[:, None])
        A = p @ np.abs(kv[:, :512])
        terms = abs(wl.softmax_scale) * (np.abs(q) @ np.abs(kv).T).max(axis=1)
        lse_tol = (576 * 2.0 ** -24 + value_slack) * terms + len(sel) * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -24 * np.abs(o_lse)
        tol = 1.01 * 2.0 ** -8 * (2 * A + 2 * np.abs(o_out)) + 1e-5 + (value_slack + 2 * lse_tol[:, None]) * A
        assert np.all(np.isfinite(out[t])), t
        err = np.abs(out[t] - o_out)
        assert np.all(err <= tol), (t, float((err / tol).max()))
        lerr = np.abs(lse[t] - o_lse)
        assert np.all(lerr <= lse_tol), (t, float(lerr.max()))


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("K", [1, 2, 47, 64, 65, 129, 300, 777, 2048])
def test_attention(dev, K, workspace):
    wl = _make(K, ctx_range=(max(1, K // 3), 1200), B=4, K=K, q_len=1)
    idx = _selection(np.random.default_rng(K), wl, K, hole=0.2 if K % 2 else 0.0, empty=(2,))
    out, lse, plan = P.Run(wl, dev).attn(idx, workspace=workspace)
    _check(out, lse, wl, idx)


@pytest.mark.parametrize("H", [1, 5, 16, 64, 127, 129, 200])
def test_attention_head_counts(dev, H):
    wl = _make(H, H=H, B=2, K=150)
    idx = _selection(np.random.default_rng(H), wl, 150, hole=0.1)
    out, lse, _ = P.Run(wl, dev).attn(idx)
    _check(out, lse, wl, idx)


def test_attention_positions_zero_and_order(dev):
    """Lengths of one, unsorted selections, the same row chosen twice."""
    wl = _make(5, ctx=[1, 2, 70], K=9)
    idx = np.full((3, 9), -1, np.int32)
    idx[0, 4] = 0
    idx[1, [0, 8]] = [1, 0]
    idx[2] = [69, 3, 3, 64, -1, 63, 0, 3, 12]
    out, lse, _ = P.Run(wl, dev).attn(idx)
    _check(out, lse, wl, idx)


def test_attention_many_queries(dev):
    """More queries than the GPU holds at once, each with its own causal extent (a prompt chunk)."""
    wl = _make(6, ctx=[500], q_len=400, K=96)
    idx = _selection(np.random.default_rng(6), wl, 96)
    out, lse, _ = P.Run(wl, dev).attn(idx)
    _check(out, lse, wl, idx, ts=list(range(0, 400, 23)) + [399])


def test_attention_padded_rows_and_any_row_scale(dev):
    """Rows 448 bytes apart; row scales that are no powers of two (values are then rounded to bf16: 2^-8 of each)."""
    wl = _make(7, B=2, K=200)
    rng = np.random.default_rng(7)
    kv = np.concatenate([wl.kv, rng.integers(0, 256, (wl.cache_rows, 16)).astype(np.uint8)], axis=1)
    padded = dataclasses.replace(wl, kv=kv, row_bytes=448)
    idx = _selection(rng, wl, 200)
    a, la, _ = P.Run(padded, dev).attn(idx)
    b, lb, _ = P.Run(wl, dev).attn(idx)
    assert np.array_equal(a, b) and np.array_equal(la, lb)
    kv = wl.kv.copy()
    kv[:, 288:292] = (rng.uniform(0.6, 1.7, wl.cache_rows).astype("<f4") * wl.kv[:, 288:292].copy().view("<f4")[:, 0]
                      ).astype("<f4").view(np.uint8).reshape(-1, 4)
    scaled = dataclasses.replace(wl, kv=kv)
    out, lse, _ = P.Run(scaled, dev).attn(idx)
    _check(out, lse, scaled, idx, value_slack=2.0 ** -8)


@pytest.mark.parametrize("code,scale,row", [(0x77, 0x7E, 2.0 ** 20), (0x11, 0x01, 2.0 ** -40), (0xFF, 0x08, 1.0)])
def test_attention_extreme_codes(dev, code, scale, row):
    """Every code, scale and row scale at an end of its range; queries scaled so that the logits stay moderate."""
    wl = _make(8, B=2, K=130)
    kv = wl.kv.copy()
    kv[:, :256] = code
    kv[::2, :128] = 0x0F & code | 0x10               # a second value, so that logits differ
    kv[:, 256:288] = scale
    kv[:, 288:292] = np.frombuffer(np.float32(row).tobytes(), np.uint8)
    big = float(np.abs(O.decode_e4m3([scale])[0] * 6 * row))
    q = torch.from_numpy(np.random.default_rng(8).normal(0, 1, wl.q.shape).astype(np.float32))
    q[..., :512] /= big * 8
    wl = dataclasses.replace(wl, kv=kv, q=W._bf16_bits(q))
    idx = _selection(np.random.default_rng(9), wl, 130)
    out, lse, _ = P.Run(wl, dev).attn(idx)
    sel = np.abs(O.sparse_mla_attn(wl, idx)[0]).max()
    assert np.isfinite(sel)
    _check(out, lse, wl, idx)


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_attention_running_max_jumps(dev, workspace, sign):
    """Rows late in a selection whose logits lie far above (or far below) the first rows': hundreds of powers of two."""
    wl = _make(10, ctx=[1500], K=1024)
    kv = wl.kv.copy()
    bits = kv[:, 304:432].copy().view("<u2")
    far = np.arange(600, 700)
    rows = O.physical_rows(wl.block_table[0], 64, far)
    lift = torch.from_numpy(O.decode_bf16(bits[rows]).astype(np.float32))
    lift[:, 0] = 900.0
    bits[rows] = W._bf16_bits(lift)
    kv[:, 304:432] = bits.view(np.uint8).reshape(wl.cache_rows, 128)
    q = torch.from_numpy(O.decode_bf16(wl.q).astype(np.float32))
    q[:, ::7, 512] = sign * 5.0                      # logits of the lifted rows move by +-325 for every seventh head
    wl = dataclasses.replace(wl, kv=kv, q=W._bf16_bits(q))
    idx = np.arange(0, 1024, dtype=np.int32)[None]
    out, lse, _ = P.Run(wl, dev).attn(idx, workspace=workspace)
    _check(out, lse, wl, idx)
    # and the other way round: the far rows first
    idx = np.roll(idx, 424, axis=1)
    out, lse, _ = P.Run(wl, dev).attn(idx, workspace=workspace)
    _check(out, lse, wl, idx)


def test_attention_flags_bad_index_and_page(dev):
    wl = _make(11, B=2, K=64)
    r = P.Run(wl, dev)
    idx = _selection(np.random.default_rng(11), wl, 64)
    idx[0, 3] = int(wl.q_pos[0]) + 1                 # beyond the query's position
    out = torch.empty((wl.T, wl.H, 512), dtype=torch.bfloat16, device=dev)
    dsa.sparse_mla_attn(r.seq, r.mla, torch.from_numpy(idx).to(dev), 64, out)
    with pytest.raises(dsa.DSAError) as e:
        dsa.check_status()
    assert e.value.status == 6 and "bad_index" in str(e.value)
    skipped = idx.copy()
    skipped[0, 3] = -1
    lse = np.stack([O.sparse_mla_attn_row(wl, t, skipped[t])[1] for t in range(wl.T)])
    _check(out.float().cpu().numpy(), lse, wl, skipped)


def test_decode_step(dev):
    for over in (dict(ctx_range=(300, 900), B=5, K=128, q_len=2), dict(ctx=[20000], K=512)):
        wl = _make(12, **over)
        r = P.Run(wl, dev)
        out, lse, sel, plan = r.decode_step()
        assert np.array_equal(sel, r.chained_indices())
        _check(out, lse, wl, sel)
        o2 = torch.empty((wl.T, wl.H, 512), dtype=torch.bfloat16, device=dev)
        dsa.decode_step_static_ws(r.seq, r.idxr, r.mla, wl.K, o2)
        dsa.check_status()
        assert np.array_equal(o2.float().cpu().numpy(), out)


def test_serving_run(dev):
    """A serving step as it would be used: index keys and latent rows of the new tokens rotated into the caches, the
    query's rope heads rotated into place, then the decode step over 4-bit rows -- captured once and replayed."""
    wl = _make(13, ctx_range=(200, 600), B=4, K=96)
    rng = np.random.default_rng(13)
    r = P.Run(wl, dev)
    plan_q, plan_i = dsa.Rope.make(64, scaling="yarn", factor=4.0, original_ctx=256), dsa.Rope.make(64, layout="half")
    new = torch.from_numpy(rng.normal(0, 1, (wl.T, 576)).astype(np.float32)).to(torch.bfloat16).to(dev)
    key = torch.from_numpy(rng.normal(0, 1, (wl.T, 128)).astype(np.float32)).to(torch.bfloat16).to(dev)
    q_pe = torch.from_numpy(rng.normal(0, 1, (wl.T, 128, 64)).astype(np.float32)).to(torch.bfloat16).to(dev)
    out = torch.empty((wl.T, 128, 512), dtype=torch.bfloat16, device=dev)
    lse = torch.empty((wl.T, 128), device=dev)
    sel = torch.empty((wl.T, 96), dtype=torch.int32, device=dev)
    ws = torch.empty(dsa.decode_workspace_size(r.seq, r.idxr, r.mla, 96), dtype=torch.uint8, device=dev)

    def step():
        dsa.index_cache_append_rope(r.seq, plan_i, key, r.idxr.k_cache, r.idxr.k_scale)
        dsa.latent_cache_append_rope(r.seq, r.mla, plan_q, new[:, :512], new[:, 512:])
        dsa.rope(plan_q, r.seq.q_pos, q_pe, r.mla.q[..., 512:])
        dsa.decode_step(r.seq, r.idxr, r.mla, 96, out, ws, lse=lse, idx_out=sel)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for again in range(2):
        if again:
            new.copy_(new.roll(1, 0)); key.copy_(key.roll(1, 0)); q_pe.copy_(q_pe.roll(1, 0))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        dsa.check_status()
        got = dataclasses.replace(wl, kv=r.mla.kv_cache.cpu().numpy(), k_i=r.idxr.k_cache.cpu().numpy(),
                                  k_i_scale=r.idxr.k_scale.cpu().numpy(),
                                  q=r.mla.q.view(torch.int16).cpu().numpy().view(np.uint16))
        rows = [int(O.physical_rows(wl.block_table[wl.q_seq[t]], 64, np.array([wl.q_pos[t]]))[0]) for t in range(wl.T)]
        for t in range(wl.T):
            assert np.array_equal(got.kv[rows[t], :304], O.e2m1_row(new[t, :512].float().cpu().numpy(), np.zeros(64))[:304])
        f, m = O.rope_frequencies(64, scaling="yarn", factor=4.0, original_ctx=256)
        want = O.rope_rotate(q_pe.double().cpu().numpy(), wl.q_pos[:, None] * f[None], "interleaved", m)
        pe = O.decode_bf16(got.q)[..., 512:]
        pair = np.repeat(np.abs(q_pe.double().cpu().numpy()).reshape(wl.T, 128, 32, 2).sum(-1), 2, axis=-1)
        assert np.all(np.abs(pe - want) <= 2.0 ** -8 * np.abs(want) + 1e-6 * pair * m)
        scores = O.indexer_scores(got)
        P.check_selection(sel.cpu().numpy(), scores, wl.q_pos, 96)
        _check(out.float().cpu().numpy(), lse.cpu().numpy(), got, sel.cpu().numpy())


def test_two_graphs_and_streams(dev):
    """Two captured calls with a workspace each, replayed on two streams at once, against the calls made one by one."""
    runs = []
    for seed in (14, 15):
        wl = _make(seed, ctx=[3000], K=1500)
        r = P.Run(wl, dev)
        idx = torch.from_numpy(_selection(np.random.default_rng(seed), wl, 1500)).to(dev)
        out = torch.empty((1, 128, 512), dtype=torch.bfloat16, device=dev)
        lse = torch.empty((1, 128), device=dev)
        ws = torch.empty(max(16, dsa.sparse_mla_attn_workspace_size(r.seq, r.mla, 1500)), dtype=torch.uint8, device=dev)
        call = lambda r=r, idx=idx, out=out, lse=lse, ws=ws: dsa.sparse_mla_attn(r.seq, r.mla, idx, 1500, out, lse=lse, workspace=ws)
        call()
        torch.cuda.synchronize()
        want = out.clone(), lse.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        runs.append((graph, out, lse, want, torch.cuda.Stream(), call))   # call keeps the inputs alive
    for _ in range(20):
        for graph, out, lse, want, s, _ in runs:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    dsa.check_status()
    for graph, out, lse, want, s, _ in runs:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
