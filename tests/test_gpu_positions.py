"""GPU parity of the rotary positions, the cache writers that rotate, and the cache reader against float64.

Tolerances, derived:
* rotation: a cosine or sine is off by at most 4e-7 (the phase's conversion to fp32 half-turns, 2^-25 of a half-turn
  = 1e-7 radians, and two units of the half-turn functions, 2.4e-7), each product and the sum by 2^-24 of the terms:
  together below 6e-7 (|a| + |b|) times the magnitude; then one rounding to the output's type, half a step of it;
* latent codes and scales: exact (the decisions on bf16 values are the same in 32 and 64 bits);
* rotated index keys: an E4M3 value is off by half a step (2^-4 of it, or 2^-10 of the scale among the subnormals)
  plus what the rotation's fp32 error moves it.
"""
import numpy as np
import pytest
import torch

import dsa_indexed_sparse_gb300 as dsa
import dsa_workloads as W
from oracle import dsa_oracle as O

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _angles(plan, pos):
    """Angles [T, pairs] from the plan's 64-bit turns, modulo one turn in integers."""
    t = [int(v) % (1 << 64) for v in plan.turns.cpu().numpy().view(np.uint64)]
    return np.array([[((int(p) * v) % (1 << 64)) / 2.0 ** 64 * 2 * np.pi for v in t] for p in pos])


def _check_rotated(got, x, plan, pos, layout, inverse=False):
    x64 = x.double().cpu().numpy()
    want = O.rope_rotate(x64, _angles(plan, pos.cpu().numpy()), layout, plan.magnitude, inverse)
    g = got.double().cpu().numpy()
    n = x64.shape[-1] // 2
    a, b = (x64[..., 0::2], x64[..., 1::2]) if layout == "interleaved" else (x64[..., :n], x64[..., n:])
    mag = 6e-7 * plan.magnitude * (np.abs(a) + np.abs(b))
    mag = np.repeat(mag, 2, axis=-1) if layout == "interleaved" else np.concatenate([mag, mag], axis=-1)
    bad = np.abs(g - want) > mag + HALF_STEP[got.dtype] * (np.abs(want) + mag)
    assert not bad.any(), (int(bad.sum()), np.abs(g - want).max())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("T,H,d", [(1, 1, 2), (1, 128, 64), (3, 5, 64), (7, 128, 32), (33, 1, 64), (300, 3, 96), (5, 2, 512),
                                   (65, 64, 128), (2, 300, 6), (1500, 16, 64), (1, 7, 66)])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(dev, dtype, layout, T, H, d, inverse):
    g = torch.Generator(device=dev).manual_seed(T * H + d)
    x = torch.randn((T, H, d), generator=g, device=dev).to(TYPES[dtype])
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device=dev, dtype=torch.int32)
    plan = dsa.Rope.make(d, layout=layout, scaling="yarn", factor=16.0, original_ctx=2048)
    out = torch.full_like(x, float("nan"))
    assert dsa.rope(plan, pos, x, out, inverse=inverse) is out
    _check_rotated(out, x, plan, pos, layout, inverse)
    same = x.clone()
    dsa.rope(plan, pos, same, same, inverse=inverse)           # in place
    assert torch.equal(same, out)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rope_views(dev, layout, dtype):
    """Parts of heads, transposed and odd strides, repeated rows; what lies beside the rotated part stays."""
    g = torch.Generator(device=dev).manual_seed(7)
    T, H, d = 9, 6, 64
    dt = TYPES[dtype]
    plan = dsa.Rope.make(d, layout=layout)
    pos = torch.randint(0, 5000, (T,), generator=g, device=dev, dtype=torch.int32)
    x = torch.randn((T, H, d), generator=g, device=dev).to(dt)
    want = dsa.rope(plan, pos, x, torch.empty_like(x))
    _check_rotated(want, x, plan, pos, layout)
    for off, width, plan_name in ((512, 576, "rope_vec"), (3, 71, "rope_scalar"), (1, 576, "rope_scalar"), (0, 65, "rope_scalar")):
        buf = torch.randn((T, H, width), generator=g, device=dev).to(dt)
        keep = buf.clone()
        dsa.rope(plan, pos, x, buf[..., off:off + d])
        assert dsa.last_plan().startswith(plan_name), (off, width, dsa.last_plan())
        assert torch.equal(buf[..., off:off + d], want)
        buf[..., off:off + d] = keep[..., off:off + d]
        assert torch.equal(buf, keep)
        src = keep.clone()
        src[..., off:off + d] = x
        dsa.rope(plan, pos, src[..., off:off + d], src[..., off:off + d])   # a part of a head, in place
        assert torch.equal(src[..., off:off + d], want)
        src[..., off:off + d] = keep[..., off:off + d]
        assert torch.equal(src, keep)
    heads_first = torch.empty((H, T, d), dtype=dt, device=dev)
    dsa.rope(plan, pos, x, heads_first.transpose(0, 1))
    assert torch.equal(heads_first.transpose(0, 1), want)
    one = torch.randn((T, 1, d), generator=g, device=dev).to(dt)             # one row for every head
    got = dsa.rope(plan, pos, one.expand(T, H, d), torch.empty_like(x))
    assert torch.equal(got, dsa.rope(plan, pos, one, torch.empty_like(one)).expand(T, H, d))
    flat = dsa.rope(plan, pos, x[:, 2], torch.empty((T, d), dtype=dt, device=dev))
    assert torch.equal(flat, want[:, 2])
    empty = torch.empty((0, H, d), dtype=dt, device=dev)
    dsa.rope(plan, pos[:0], empty, empty)
    with pytest.raises(dsa.DSAError):
        dsa.rope(plan, pos, x, torch.empty((T, 1, d), dtype=dt, device=dev).expand(T, H, d))
    with pytest.raises(ValueError):
        dsa.rope(plan, pos.long(), x, x)
    with pytest.raises(ValueError):
        dsa.rope(plan, pos, x, x[..., :32])


def test_rope_extreme_positions(dev):
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789, -77], dtype=torch.int32, device=dev)
    for layout in ("interleaved", "half"):
        plan = dsa.Rope.make(64, theta=5e5, layout=layout, scaling="linear", factor=4.0)
        x = torch.randn((7, 4, 64), generator=torch.Generator(device=dev).manual_seed(1), device=dev)
        out = dsa.rope(plan, pos, x, torch.empty_like(x))
        _check_rotated(out, x, plan, pos, layout)
        assert torch.equal(out[0], x[0])


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rope_gradient(dev, layout):
    """The inverse is the gradient: against the transposed matrix, and against differences."""
    g = torch.Generator(device=dev).manual_seed(3)
    plan = dsa.Rope.make(8, layout=layout, magnitude=1.25)
    pos = torch.tensor([5, 1000], dtype=torch.int32, device=dev)
    x = torch.randn((2, 3, 8), generator=g, device=dev)
    dy = torch.randn((2, 3, 8), generator=g, device=dev)
    dx = dsa.rope(plan, pos, dy, torch.empty_like(dy), inverse=True)
    base = dsa.rope(plan, pos, x, torch.empty_like(x))
    for i in range(8):
        h = torch.zeros_like(x)
        h[..., i] = 0.5
        # the rotation is linear: the difference quotient has no truncation error, only 2^-22 of the values over h
        diff = ((dsa.rope(plan, pos, x + h, torch.empty_like(x)) - base).double() * dy.double()).sum(-1) / 0.5
        assert torch.allclose(diff, dx[..., i].double(), rtol=0, atol=1e-4)


def test_rope_streams_and_graph(dev):
    plan = dsa.Rope.make(64)
    x = torch.randn((50, 128, 64), device=dev).to(torch.bfloat16)
    pos = torch.arange(50, dtype=torch.int32, device=dev)
    want = dsa.rope(plan, pos, x, torch.empty_like(x))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = torch.empty_like(x)
    dsa.rope(plan, pos, x, a, stream=s)
    b = torch.zeros_like(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.rope(plan, pos, x, b)
    x.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want * 2)


# ----------------------------------------------------------------------------- writers and reader

FORMATS = {"f32": 2304, "bf16": 1152, "e4m3": 656, "e4m3_t128": 656, "e2m1": 432}


def _layout(seed, B=3, q_len=4, lo=200, hi=900):
    return W.make("decode_b64", seed=seed, ctx_range=(lo, hi), B=B, q_len=q_len, K=64)


def _mla(dev, fmt, cache):
    q = torch.zeros((1, 128, 576), dtype=torch.float32 if fmt == "f32" else torch.bfloat16, device=dev)
    code = {"f32": None, "bf16": None, "e4m3": dsa.DSA_E4M3, "e4m3_t128": dsa.DSA_E4M3_T128, "e2m1": dsa.DSA_E2M1}[fmt]
    if code is None:
        cache = cache.view(torch.float32 if fmt == "f32" else torch.bfloat16)
    return dsa.Mla(q=q, kv_cache=cache, d_latent=512, d_rope=64, softmax_scale=1.0, dtype=code)


def _want_latent(fmt, latent, bits):
    """The bytes of a row before its rope part."""
    if fmt == "f32":
        return np.frombuffer(latent.astype("<f4").tobytes(), dtype=np.uint8)
    if fmt == "bf16":
        return np.frombuffer(bits.astype("<u2").tobytes(), dtype=np.uint8)
    if fmt == "e2m1":
        return O.e2m1_row(latent, np.zeros(64, np.uint16))[:304]
    row = O.latent_cache_append(np.zeros((1, 1), np.int32), 64, [0], [0], np.concatenate([bits, np.zeros(64, np.uint16)])[None],
                                np.zeros((64, 656), np.uint8), fp8_rows=True, tile128=fmt == "e4m3_t128")[0]
    return row[:528]


@pytest.mark.parametrize("pad", [0, 16, 80])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("fmt", list(FORMATS))
def test_latent_append_rope(dev, fmt, layout, pad):
    wl = _layout(51 + pad)
    rng = np.random.default_rng(52)
    T, row_bytes = wl.T, FORMATS[fmt] + pad
    dt = torch.float32 if fmt == "f32" else torch.bfloat16
    x = rng.normal(0, 1, (T, 704)).astype(np.float32) * np.exp2(rng.integers(-12, 12, (T, 1))).astype(np.float32)
    x[:, 8:520] *= np.repeat(np.exp2(rng.integers(-9, 2, (T, 32))), 16, axis=1).astype(np.float32)
    x[0, 8:520] = 0.0                          # an all-zero latent part
    x[1, 24:40] = 0.0                          # an all-zero block
    x[2, 8:520] = 0.0
    x[2, 300] = 2.0 ** -130                    # a bf16 subnormal alone in its row
    buf = torch.from_numpy(x).to(dt).to(dev)
    latent, k_rope = buf[:, 8:520], buf[:, 528:592]     # strided views of one projection
    cache0 = torch.from_numpy(rng.integers(0, 256, (wl.cache_rows, row_bytes)).astype(np.uint8)).to(dev)
    cache = cache0.clone()
    plan = dsa.Rope.make(64, layout=layout, scaling="yarn", factor=8.0, original_ctx=128)
    seq = dsa.Seq(**W.device_tensors(wl, dev)["seq"])
    dsa.latent_cache_append_rope(seq, _mla(dev, fmt, cache), plan, latent, k_rope)
    assert dsa.last_plan().startswith("latent_append_rope<")
    dsa.check_status()
    rows = np.array([O.physical_rows(wl.block_table[wl.q_seq[t]], 64, np.array([wl.q_pos[t]]))[0] for t in range(T)])
    got = cache.cpu().numpy()
    lat = latent.float().cpu().numpy()
    bits = latent.to(torch.bfloat16).contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
    off = {"f32": 2048, "bf16": 1024, "e2m1": 304}.get(fmt, 528)
    for t in range(T):
        assert np.array_equal(got[rows[t], :off], _want_latent(fmt, lat[t], bits[t])), (fmt, t)
    rot = cache[torch.from_numpy(rows).to(dev), off:off + 64 * dt.itemsize].contiguous().view(dt)
    _check_rotated(rot, k_rope, plan, torch.from_numpy(wl.q_pos).to(dev), layout)
    # every other byte of the pool is untouched
    rest = np.ones(got.shape, bool)
    rest[rows, :FORMATS[fmt]] = False
    assert np.array_equal(got[rest], cache0.cpu().numpy()[rest])


def test_latent_append_e2m1_without_rotation(dev):
    wl = _layout(61, q_len=3)
    rng = np.random.default_rng(62)
    x = torch.from_numpy(rng.normal(0, 1, (wl.T, 576)).astype(np.float32)).to(torch.bfloat16)
    cache0 = rng.integers(0, 256, (wl.cache_rows, 432)).astype(np.uint8)
    cache = torch.from_numpy(cache0.copy()).to(dev)
    dsa.latent_cache_append(dsa.Seq(**W.device_tensors(wl, dev)["seq"]), _mla(dev, "e2m1", cache), x.to(dev))
    assert dsa.last_plan() == "latent_append<e2m1>"
    dsa.check_status()
    bits = x.view(torch.int16).numpy().view(np.uint16)
    for t in range(wl.T):
        row = O.physical_rows(wl.block_table[wl.q_seq[t]], 64, np.array([wl.q_pos[t]]))[0]
        cache0[row] = O.e2m1_row(x[t, :512].float().numpy(), bits[t, 512:])
    assert np.array_equal(cache.cpu().numpy(), cache0)


def test_append_small_dims(dev):
    """A bf16 cache of other dims than 512 + 64 (two pairs of rope)."""
    wl = _layout(63)
    cache = torch.zeros((wl.cache_rows, 32), dtype=torch.bfloat16, device=dev)
    q = torch.zeros((1, 4, 32), dtype=torch.bfloat16, device=dev)
    mla = dsa.Mla(q=q, kv_cache=cache, d_latent=24, d_rope=8, softmax_scale=1.0)
    new = torch.randn((wl.T, 32), device=dev).to(torch.bfloat16)
    plan = dsa.Rope.make(8, layout="half")
    seq = dsa.Seq(**W.device_tensors(wl, dev)["seq"])
    dsa.latent_cache_append_rope(seq, mla, plan, new[:, :24], new[:, 24:])
    out = dsa.latent_cache_read(seq, mla, torch.empty((wl.T, 32), dtype=torch.bfloat16, device=dev))
    dsa.check_status()
    assert torch.equal(out[:, :24], new[:, :24])
    _check_rotated(out[:, 24:], new[:, 24:], plan, seq.q_pos, "half")


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("src", ["f32", "bf16"])
@pytest.mark.parametrize("layout,D,off,d", [("half", 128, 0, 64), ("interleaved", 128, 64, 64), ("half", 96, 5, 18),
                                            ("interleaved", 1024, 1, 512), ("half", 32, 0, 32)])
def test_index_append_rope(dev, layout, D, off, d, src, mx):
    wl = _layout(71)
    rng = np.random.default_rng(72)
    T = wl.T
    x = rng.normal(0, 1, (T, D + 8)).astype(np.float32) * rng.uniform(0.01, 50, (T, 1)).astype(np.float32)
    x[1] = 0.0
    k_new = torch.from_numpy(x).to(TYPES[src]).to(dev)[:, 8:]
    kc0 = rng.integers(0, 256, (wl.cache_rows, D)).astype(np.uint8)
    ks0 = rng.integers(0, 256, (wl.cache_rows, D // 32)).astype(np.uint8) if mx else rng.normal(0, 1, wl.cache_rows).astype(np.float32)
    kc, ks = torch.from_numpy(kc0.copy()).to(dev), torch.from_numpy(ks0.copy()).to(dev)
    plan = dsa.Rope.make(d, layout=layout)
    seq = dsa.Seq(**W.device_tensors(wl, dev)["seq"])
    dsa.index_cache_append_rope(seq, plan, k_new, kc, ks, offset=off, mx=mx)
    assert dsa.last_plan().startswith("index_append_rope")
    dsa.check_status()
    rows = np.array([O.physical_rows(wl.block_table[wl.q_seq[t]], 64, np.array([wl.q_pos[t]]))[0] for t in range(T)])
    want = k_new.double().cpu().numpy().copy()
    part = want[:, off:off + d].copy()
    want[:, off:off + d] = O.rope_rotate(part, _angles(plan, wl.q_pos), layout)
    codes, scales = kc.cpu().numpy()[rows], ks.cpu().numpy()[rows]
    amax = np.abs(want).max(axis=1, keepdims=True)
    if mx:
        vals = O.dequantize_mx_e4m3(codes, scales)
        scale = np.repeat(O.decode_e8m0(scales), 32, axis=1)
        # saturation: the block's maximum may pass 448 of its scale (up to 512), where codes stop
        want_q = np.clip(want, -448 * scale, 448 * scale)
    else:
        vals, scale = O.decode_e4m3(codes) * scales[:, None].astype(np.float64), scales[:, None].astype(np.float64)
        want_q = want
        ref = np.where(amax > 0, amax / 448, 1.0)
        assert np.all(np.abs(scale / ref - 1) <= 2e-6)      # the rotated maximum is off by 1.2e-6 of itself at most
    tol = 2.0 ** -4 * np.abs(want_q) + 2.0 ** -10 * scale + 2e-6 * amax
    assert np.all(np.abs(vals - want_q) <= tol), np.abs(vals - want_q).max()
    others = np.setdiff1d(np.arange(wl.cache_rows), rows)
    assert np.array_equal(kc.cpu().numpy()[others], kc0[others]) and np.array_equal(ks.cpu().numpy()[others], ks0[others])
    # position 0 turns nothing: bit for bit the writer without a rotation
    flat = dict(W.device_tensors(wl, dev)["seq"])
    flat.update(q_seq=torch.arange(3, dtype=torch.int32, device=dev), q_pos=torch.zeros(3, dtype=torch.int32, device=dev), q_per_seq=0)
    first = k_new[:3].contiguous()
    a, b = [(torch.from_numpy(kc0.copy()).to(dev), torch.from_numpy(ks0.copy()).to(dev)) for _ in range(2)]
    dsa.index_cache_append_rope(dsa.Seq(**flat), plan, first, *a, offset=off, mx=mx)
    dsa.index_cache_append(dsa.Seq(**flat), first, *b, mx=mx)
    dsa.check_status()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("T,pad", [(1, 0), (7, 16), (300, 0)])
def test_latent_read(dev, fmt, out, T, pad):
    wl = W.make("decode_b4_long", seed=81, ctx=[300, 450], K=16, q_len=1, mla_dtype=fmt, shuffle_pages=True)
    rng = np.random.default_rng(T)
    seqs = rng.integers(0, 2, T).astype(np.int32)
    pos = np.array([rng.integers(0, wl.seq_lens[b]) for b in seqs], dtype=np.int32)
    raw = wl.kv.view(np.uint8).reshape(wl.cache_rows, -1)
    raw = np.concatenate([raw, rng.integers(0, 256, (wl.cache_rows, pad)).astype(np.uint8)], axis=1)
    d = dict(W.device_tensors(wl, dev)["seq"])
    d.update(q_seq=torch.from_numpy(seqs).to(dev), q_pos=torch.from_numpy(pos).to(dev), q_per_seq=0)
    seq = dsa.Seq(**d)
    mla = _mla(dev, fmt, torch.from_numpy(raw).to(dev))
    wide = torch.full((T, 600), float("nan"), dtype=TYPES[out], device=dev)
    got = dsa.latent_cache_read(seq, mla, wide[:, 8:584])
    assert dsa.last_plan().startswith("latent_read<")
    dsa.check_status()
    rows = [int(O.physical_rows(wl.block_table[b], 64, np.array([p]))[0]) for b, p in zip(seqs, pos)]
    want = torch.from_numpy(O.latent_rows(wl, rows))
    # fp32: one product of a code and its scale; bf16: that product rounded once more
    want = want.float().to(TYPES[out])
    assert torch.equal(got.cpu(), want)
    assert wide[:, :8].isnan().all() and wide[:, 584:].isnan().all()


def test_writers_and_reader_flag_bad_positions(dev):
    wl = _layout(91)
    base = dict(W.device_tensors(wl, dev)["seq"])
    bad = dict(base, q_pos=base["q_pos"].clone(), block_table=base["block_table"].clone())
    bad["q_pos"][2] = wl.max_ctx
    bad["q_pos"][3] = -1
    bad["block_table"][1, :] = wl.cache_rows // 64         # sequence 1: pages beyond the pool
    seq = dsa.Seq(**bad)
    plan = dsa.Rope.make(64)
    cache = torch.zeros((wl.cache_rows, 432), dtype=torch.uint8, device=dev)
    mla = _mla(dev, "e2m1", cache)
    ones = torch.ones((wl.T, 576), dtype=torch.bfloat16, device=dev)
    dsa.latent_cache_append_rope(seq, mla, plan, ones[:, :512], ones[:, 512:])
    with pytest.raises(dsa.DSAError) as e:
        dsa.check_status()
    assert e.value.status == 6 and "bad_q_pos" in str(e.value) and "bad_index" in str(e.value)
    assert int((cache != 0).any(dim=1).sum()) == wl.T - 2 - 4
    out = torch.full((wl.T, 576), 7.0, device=dev)
    dsa.latent_cache_read(seq, mla, out)
    with pytest.raises(dsa.DSAError):
        dsa.check_status()
    left = [t for t in range(wl.T) if t in (2, 3) or wl.q_seq[t] == 1]
    assert (out[left] == 7.0).all() and not (out[[t for t in range(wl.T) if t not in left], :512] == 7.0).any()
    kc = torch.zeros((wl.cache_rows, 128), dtype=torch.uint8, device=dev)
    ks = torch.zeros(wl.cache_rows, device=dev)
    dsa.index_cache_append_rope(seq, plan, ones[:, :128], kc, ks)
    with pytest.raises(dsa.DSAError):
        dsa.check_status()
    assert int((ks != 0).sum()) == wl.T - 2 - 4
    dsa.check_status()
