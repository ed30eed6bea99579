"""The attention over 4-bit rows where the range of its 16-bit weights shows: far maxima, rows of very unequal scale, rows
that are all zero.  Against the float64 oracle.

Tolerances, derived from the kernel's types (all sums in fp32; n selected rows, p_s the softmax weights):
* a logit: the tensor cores' fp32 sums, of N products, are off by at most N 2^-23 of the sum of their magnitudes, whatever
  the order and whether bits are rounded or cut off (a lone product of two bf16 values is exact); then the scale,
  scale * log2 e, the sum of latent and rope part and the exponent's argument, a rounding each: 2^-22 of the logit in all;
* a weight: twice the largest logit error (its own and the shift's), 2^-20 for the exponential and three fp32 products, 2^-11
  for its rounding to f16; below f16's normal range, where the rounding is absolute, 2^-25.  The largest weight times
  row scale starts at 2^7, or 2^4 at least where the row scales of a tile differ by 2^3 at most, or has grown since, so
  the latter is at most 2^-29 max_s(p_s |rs_s|) of each row's value over its scale, rs_s being the row scale of a
  row that holds any value (0 if it holds none);
* sums over the rows: n 2^-23 of the sum of magnitudes A = sum_s p_s |v_s|;
* where the rows are taken in slices (more than 128 of them, and a workspace), a slice's output rounded to bf16: 2^-8 of it,
  of A at most when they are joined;
* the output's rounding to bf16: 2^-8 of it."""
import dataclasses

import numpy as np
import pytest
import torch

import dsa_workloads as W
from oracle import dsa_oracle as O
from tests import parity as P
from tests.test_gpu_e2m1 import _make, _selection

pytestmark = pytest.mark.gpu

LOG2E = 1.4426950408889634


def _check_tight(out, lse, wl, idx, ts=None, slices=True):
    for t in range(wl.T) if ts is None else ts:
        sel = idx[t][idx[t] >= 0].astype(np.int64)
        o_out, o_lse = O.sparse_mla_attn_row(wl, t, idx[t])
        rows = O.physical_rows(wl.block_table[wl.q_seq[t]], wl.page_size, sel)
        kv, q, n, s = O.latent_rows(wl, rows), O.mla_query(wl, t), len(sel), abs(float(wl.softmax_scale))
        rs = np.abs(wl.kv[rows, 288:292].copy().view("<f4")[:, 0].astype(np.float64))
        rs[~(wl.kv[rows, 256:288] & 0x7F).any(axis=1)] = 0.0
        logits = wl.softmax_scale * (q @ kv.T)
        lat = s * (np.abs(q[:, :512]) @ np.abs(kv[:, :512]).T).max(axis=1)
        rope = s * (np.abs(q[:, 512:]) @ np.abs(kv[:, 512:]).T).max(axis=1)
        n_rope = (q[:, 512:] != 0).sum(axis=1)
        e = 2.0 ** -23 * (512 * lat + np.maximum(n_rope - 1, 0) * rope) + 2.0 ** -22 * np.abs(logits).max(axis=1)
        p = np.exp(logits - o_lse[:, None])
        A = p @ np.abs(kv[:, :512])
        v_over = np.divide(np.abs(kv[:, :512]), rs[:, None], out=np.zeros_like(kv[:, :512]), where=rs[:, None] > 0).sum(axis=0)
        lost = 2.0 ** -29 * (p * rs).max(axis=1)[:, None] * v_over
        before = (2 * e[:, None] + 2.0 ** -20 + 2.0 ** -11 + (2.0 ** -8 if slices else 0.0) + n * 2.0 ** -23) * A + lost
        tol = 1.01 * (before + 2.0 ** -8 * (np.abs(o_out) + before))
        assert np.all(np.isfinite(out[t])), t
        err = np.abs(out[t] - o_out)
        assert np.all(err <= tol), (t, float((err / np.maximum(tol, 1e-300)).max()))
        lse_tol = e + 2.0 ** -20 + n * 2.0 ** -23 + 2.0 ** -22 * np.abs(o_lse)
        assert np.all(np.abs(lse[t] - o_lse) <= lse_tol), (t, float((np.abs(lse[t] - o_lse) / lse_tol).max()))


def _lift(wl, key, query, latent=2.0 ** -4):
    """The workload with rope dim 0 of every cache row (key: [cache_rows]) and of the queries (query: [H]) set and the
    other rope dims of the queries 0, so that a logit moves by softmax_scale * key * query exactly; query latents scaled."""
    kv = wl.kv.copy()
    bits = kv[:, 304:432].copy().view("<u2")
    bits[:, 0] = W._bf16_bits(torch.from_numpy(np.asarray(key, np.float32)))
    kv[:, 304:432] = bits.view(np.uint8).reshape(wl.cache_rows, 128)
    q = torch.from_numpy(O.decode_bf16(wl.q).astype(np.float32))
    q[..., :512] *= latent
    q[..., 512:] = 0.0
    q[..., 512] = torch.from_numpy(np.asarray(query, np.float32))
    return dataclasses.replace(wl, kv=kv, q=W._bf16_bits(q))


def _set_scales(wl, factor):
    """Row scales times factor [cache_rows]."""
    kv = wl.kv.copy()
    rs = kv[:, 288:292].copy().view("<f4")[:, 0] * np.asarray(factor, np.float32)
    kv[:, 288:292] = rs.astype("<f4").view(np.uint8).reshape(-1, 4)
    return dataclasses.replace(wl, kv=kv)


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("base", [600.0, 4100.0, 8200.0, 30000.0])
def test_far_maxima(dev, base, sign, workspace):
    """All logits of a head far from 0, by base and up to one and a half times that (log2 units) from head to head; among one
    another they differ by little."""
    wl = _make(101, ctx=[700, 650], K=300)
    per = float(wl.softmax_scale) * LOG2E * 128.0
    wl = _lift(wl, np.full(wl.cache_rows, 128.0), sign * base / per * (1 + np.arange(wl.H) % 64 / 128))
    idx = _selection(np.random.default_rng(102), wl, 300, hole=0.1)
    out, lse, _ = P.Run(wl, dev).attn(idx, workspace=workspace)
    _check_tight(out, lse, wl, idx, slices=workspace)


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("order", ["large first", "small first", "mixed"])
def test_unequal_row_scales(dev, order, workspace):
    """Row scales from 2^-30 to 2^10 of the usual ones: the larger a row's scale the smaller its weight, so that the rows
    that make the output have the smallest scales (weight times scale falls by 2^-1.5 per doubling of the scale)."""
    wl = _make(111, ctx=[700, 650], K=600)
    rng = np.random.default_rng(112)
    k = rng.integers(-30, 11, wl.cache_rows).astype(np.float64)
    wl = _set_scales(wl, 2.0 ** k)
    per = float(wl.softmax_scale) * LOG2E
    wl = _lift(wl, k, np.full(wl.H, -2.5 / per), latent=0.0)
    idx = _selection(rng, wl, 600)
    for t in range(wl.T):
        n = int((idx[t] >= 0).sum())
        if order != "mixed":
            by = k[O.physical_rows(wl.block_table[t], 64, idx[t, :n].astype(np.int64))].argsort()
            idx[t, :n] = idx[t, :n][by if order == "small first" else by[::-1]]
    out, lse, _ = P.Run(wl, dev).attn(idx, workspace=workspace)
    _check_tight(out, lse, wl, idx, slices=workspace)


@pytest.mark.parametrize("K", [1, 130, 256, 700, 2048])
@pytest.mark.parametrize("workspace", [True, False])
def test_roundings_of_the_output(dev, K, workspace):
    """Values of one sign, so that the sum of magnitudes is the output itself: nothing but the weights', the output's
    and, of rows in several slices, the parts' roundings may show."""
    wl = _make(140 + K, ctx=[2500, 2300], K=K)
    kv = wl.kv.copy()
    kv[:, :256] &= 0x77                                     # the codes' signs
    wl = _lift(dataclasses.replace(wl, kv=kv), np.zeros(wl.cache_rows), np.zeros(wl.H))
    idx = _selection(np.random.default_rng(K), wl, K)
    out, lse, plan = P.Run(wl, dev).attn(idx, workspace=workspace)
    assert ("split=1," in plan) == (K <= 128 or not workspace)
    _check_tight(out, lse, wl, idx, slices="split=1," not in plan)



@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("lift", [-20.0, 0.0, 20.0])
@pytest.mark.parametrize("size", [0, -20, -30])
def test_zero_rows(dev, size, lift, workspace):
    """All-zero latent rows as the writer stores them (row scale 1) among rows of latents around 2^size, one alone, a few and
    more than a tile of them, their logits below, beside and above the others' (log2 units): they weigh in the sum and
    have no values.  Rows that hold something in one block alone, the first or the last, are no zero rows."""
    wl = _make(121, ctx=[700, 650, 600, 520], K=500)
    wl = _set_scales(wl, np.full(wl.cache_rows, 2.0 ** size))
    key = np.zeros(wl.cache_rows)
    kv = wl.kv.copy()
    row = np.zeros(432, np.uint8)
    row[288:292] = np.frombuffer(np.float32(1.0).tobytes(), np.uint8)
    for t, where in enumerate(([250], [0, 1, 200, 499], list(range(0, 140)), list(range(256, 500)))):
        rows = O.physical_rows(wl.block_table[t], 64, np.array(where))
        rope = kv[rows, 304:].copy()
        kv[rows] = row
        kv[rows, 304:] = rope
        key[rows] = lift
        for at, block in ((150, 0), (151, 31), (152, 28), (153, 27)):
            if at not in where:
                one = O.physical_rows(wl.block_table[t], 64, np.array([at]))
                kv[one, 256:288] = 0
                kv[one, 256 + block] = 0x78
    wl = dataclasses.replace(wl, kv=kv)
    wl = _lift(wl, key, np.full(wl.H, 1.0 / (float(wl.softmax_scale) * LOG2E)), latent=2.0 ** (-4 - size))
    idx = np.tile(np.arange(500, dtype=np.int32), (wl.T, 1))
    out, lse, _ = P.Run(wl, dev).attn(idx, workspace=workspace)
    _check_tight(out, lse, wl, idx, slices=workspace)


@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("where", ["rope", "block scale", "row scale", "query latent", "query rope"])
def test_nan_that_is_selected(dev, where, workspace):
    """A NaN in a selected row makes its query's outputs and log-sum-exps NaN, one in a query's head that head's; the others
    are what they are."""
    wl = _make(131, ctx=[700, 650, 620], K=600)
    idx = _selection(np.random.default_rng(132), wl, 600, hole=0.1)
    want, want_lse, _ = P.Run(wl, dev).attn(idx, workspace=workspace)
    kv, q = wl.kv.copy(), wl.q.copy()
    bad = np.zeros((wl.T, wl.H), bool)
    if where.startswith("query"):
        q[1, 77, 5 if where == "query latent" else 520] = 0x7FC0
        bad[1, 77] = True
    else:
        pos = idx[1][idx[1] >= 0][333]
        row = O.physical_rows(wl.block_table[1], 64, np.array([pos]))[0]
        if where == "rope":
            kv[row, 304:306] = (0xC0, 0x7F)
        elif where == "block scale":
            kv[row, 270] = 0x7F
        else:
            kv[row, 288:292] = np.frombuffer(np.float32(np.nan).tobytes(), np.uint8)
        bad[1] = True
    out, lse, _ = P.Run(dataclasses.replace(wl, kv=kv, q=q), dev).attn(idx, workspace=workspace)
    assert np.isnan(lse[bad]).all() and np.isnan(out[bad]).all()
    assert np.array_equal(out[~bad], want[~bad]) and np.array_equal(lse[~bad], want_lse[~bad])


@pytest.mark.parametrize("H,T,K,workspace", [(128, 1, 1, True), (128, 3, 129, False), (16, 2, 777, False), (130, 150, 300, True),
                                             (128, 2, 2048, False), (128, 2, 2048, True), (5, 300, 200, True)])
@pytest.mark.parametrize("scales", ["powers of two", "any"])
def test_ordinary_rows_and_any_row_scale(dev, H, T, K, workspace, scales):
    """Ordinary queries and rows, with holes.  Row scales enter in fp32: one that is no power of two rounds no value."""
    wl = _make(160 + H + T + K, ctx=[T + 2200], q_len=T, K=K, H=H)
    rng = np.random.default_rng(K)
    if scales == "any":
        wl = _set_scales(wl, rng.uniform(0.6, 1.7, wl.cache_rows))
    idx = _selection(rng, wl, K, hole=0.1 if K > 1 else 0.0)
    out, lse, plan = P.Run(wl, dev).attn(idx, workspace=workspace)
    _check_tight(out, lse, wl, idx, ts=sorted({0, T // 2, T - 1}), slices="split=1," not in plan)


@pytest.mark.parametrize("scale", [float("nan"), float("inf")])
def test_softmax_scale_that_is_no_number(dev, scale):
    wl = dataclasses.replace(_make(171, ctx=[300, 200], K=150), softmax_scale=scale)
    out, lse, _ = P.Run(wl, dev).attn(_selection(np.random.default_rng(172), wl, 150))
    assert np.isnan(out).all() and np.isnan(lse).all()
