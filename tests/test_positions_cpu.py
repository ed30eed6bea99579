"""Rotary positions, 4-bit rows and the cache writers and reader around them, as far as they
need no GPU: the oracle's formulas by hand, the library's frequencies, and every refusal."""
import ctypes
import math

import numpy as np
import pytest
import torch

import dsa_workloads as W
from oracle import dsa_oracle as O


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__
    __graft_entry__.build()
    import dsa_indexed_sparse_gb300 as m
    return m


# ----------------------------------------------------------------------------- oracle pins

def test_e2m1_codes_by_hand():
    assert O.decode_e2m1(np.arange(16)).tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]
    assert np.array_equal(O.e2m1_encode(O.decode_e2m1(np.arange(8))), np.arange(8))
    # midpoints go to the even code, everything past 6 saturates
    assert O.e2m1_encode([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 1e9]).tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 7]
    assert O.e2m1_encode([0.2500001, 0.7499999, -5.1, -0.0]).tolist() == [1, 1, 15, 8]


def test_e2m1_row_by_hand():
    x = np.zeros(512, np.float32)
    x[0], x[1], x[15], x[16] = 6.0, -3.0, 0.5, 1.0
    codes, sc, rs = O.quantize_e2m1_row(x)
    assert rs == 2.0 ** -8                       # floor(log2 6) - 10
    # block 0: 6 * 256 / 6 = 256; block 1: 256 / 6 = 42.67 -> 44 (E4M3 steps of 4)
    assert O.decode_e4m3(sc[:2]).tolist() == [256.0, 44.0] and not sc[2:].any()
    assert codes[0] == 7 | (13 << 4)             # 6 and -3
    assert codes[7] == 1 << 4                    # 0.5 at the odd dim 15
    assert codes[8] == 7                         # 256 / 44 = 5.8 -> 6
    zero, sc0, rs0 = O.quantize_e2m1_row(np.zeros(512, np.float32))
    assert rs0 == 1.0 and not zero.any() and not sc0.any()


def test_e2m1_row_error_bound():
    """Half a step of the code plus the block scale's rounding: |x - value| <= (1 / 6 + 2^-4) of the block's maximum
    (codes reach 6 of a scale that is off by at most 2^-4 of itself; the widest half step is 1 of 6)."""
    rng = np.random.default_rng(1)
    x = (rng.normal(0, 1, 512) * np.repeat(np.exp2(rng.integers(-6, 3, 32)), 16)).astype(np.float32)
    x = torch.from_numpy(x).to(torch.bfloat16).float().numpy()
    codes, sc, rs = O.quantize_e2m1_row(x)
    v = O.decode_e2m1(np.stack([codes & 15, codes >> 4], axis=1).reshape(-1)) * np.repeat(O.decode_e4m3(sc), 16) * rs
    amax = np.repeat(np.abs(x).reshape(32, 16).max(axis=1), 16)
    assert np.all(np.abs(v - x) <= amax * (1 / 6 + 2.0 ** -4))


def test_e2m1_generator_matches_oracle():
    rng = np.random.default_rng(2)
    x = torch.from_numpy((rng.normal(0, 1, (9, 576)) * np.exp2(rng.integers(-9, 9, (9, 1)))).astype(np.float32))
    x[3, :512] = 0
    x[4, 64:80] = 0
    x = x.to(torch.bfloat16).float()
    got = W._quant_rows_e2m1(x)
    bits = W._bf16_bits(x)
    for r in range(9):
        assert np.array_equal(got[r], O.e2m1_row(x[r, :512].numpy(), bits[r, 512:])), r


def test_rotation_by_hand_and_transposed_inverse():
    quarter = np.array([[math.pi / 2, 0.0]])
    x = np.array([[1.0, 2.0, 3.0, 4.0]])
    assert np.allclose(O.rope_rotate(x, quarter), [[-2.0, 1.0, 3.0, 4.0]])
    assert np.allclose(O.rope_rotate(x, quarter, "half"), [[-3.0, 2.0, 1.0, 4.0]])
    rng = np.random.default_rng(3)
    a, y = rng.normal(0, 1, (2, 5, 8)), rng.normal(0, 1, (2, 5, 8))
    ang = rng.normal(0, 9, (2, 4))
    for layout in ("interleaved", "half"):
        u = O.rope_rotate(a, ang, layout, 1.3)
        assert np.allclose((u * y).sum(), (a * O.rope_rotate(y, ang, layout, 1.3, inverse=True)).sum())
        assert np.allclose(O.rope_rotate(O.rope_rotate(a, ang, layout), ang, layout, inverse=True), a)


# ----------------------------------------------------------------------------- the library's frequencies

@pytest.mark.parametrize("d", [2, 32, 64, 96, 512])
@pytest.mark.parametrize("scaling,more", [("none", {}), ("linear", dict(factor=8.0)), ("ntk", dict(factor=8.0)),
                                          ("yarn", dict(factor=40.0, original_ctx=4096)),
                                          ("yarn", dict(factor=4.0, original_ctx=1, beta_fast=2.0, beta_slow=2.0))])
def test_frequencies(dsa, d, scaling, more):
    if scaling == "ntk" and d == 2:
        pytest.skip("NTK scaling needs two pairs")
    plan = dsa.Rope.make(d, theta=10000.0, scaling=scaling, device="cpu", **more)
    f, m = O.rope_frequencies(d, 10000.0, scaling, **more)
    turns = plan.turns.numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64
    # both sides round pow, the quotient by 2 pi and the blend: a few steps of a double
    assert np.allclose(turns, f / (2 * math.pi) % 1.0, rtol=32 * 2.0 ** -53, atol=2.0 ** -62)
    assert plan.magnitude == pytest.approx(m, rel=2.0 ** -23)
    assert plan.d_rot == d and plan.turns.shape == (d // 2,)
    assert dsa.Rope.make(d, magnitude=0.5, device="cpu").magnitude == 0.5


def test_frequency_refusals(dsa):
    make = lambda *a, **k: dsa.Rope.make(*a, device="cpu", **k)
    for d in (0, -2, 3, 514):
        with pytest.raises(dsa.DSAError) as e:
            make(d)
        assert e.value.status == 2
    for bad in (dict(theta=1.0), dict(theta=float("nan")), dict(theta=float("inf")),
                dict(scaling="linear", factor=0.5), dict(scaling="ntk", factor=float("nan")),
                dict(scaling="yarn", factor=2.0), dict(scaling="yarn", factor=2.0, original_ctx=64, beta_slow=0.0),
                dict(scaling="yarn", factor=2.0, original_ctx=64, beta_fast=0.5)):
        with pytest.raises(dsa.DSAError) as e:
            make(64, **bad)
        assert e.value.status == 1, bad
    with pytest.raises(dsa.DSAError):
        make(2, scaling="ntk", factor=2.0)
    with pytest.raises(ValueError):
        make(64, layout="other")
    with pytest.raises(ValueError):
        make(64, scaling="other")


# ----------------------------------------------------------------------------- refusals (no CUDA call is reached)

def _descs(dsa, **over):
    s = dsa.SeqDesc(B=1, T=2, max_ctx=1000, q_per_seq=0, q_seq=16, q_pos=16, block_table=16, bt_stride=16,
                    page_size=64, cache_rows=4096)
    m = dsa.MlaDesc(**{**dict(H=128, d_latent=512, d_rope=64, dtype=dsa.DSA_E2M1, q=16, kv_cache=16, row_bytes=432,
                              softmax_scale=0.1), **over})
    return s, m


def test_rope_refusals(dsa):
    lib = dsa._lib
    ok = dict(d_rot=64, layout=0, turns=16, magnitude=1.0)

    def call(r=None, T=2, H=4, pos=16, dt=dsa.DSA_BF16, x=16, xt=256, xh=64, o=4112, ot=256, oh=64):
        rd = dsa.RopeDesc(**{**ok, **(r or {})})
        return lib.dsa_rope(ctypes.byref(rd), T, H, pos, dt, x, xt, xh, o, ot, oh, 0, None)

    assert lib.dsa_rope(None, 2, 4, 16, dsa.DSA_BF16, 16, 256, 64, 16, 256, 64, 0, None) == 1
    for r in (dict(d_rot=0), dict(d_rot=63), dict(d_rot=514)):
        assert call(r) == 2, r
    for r in (dict(layout=2), dict(turns=None), dict(turns=12)):
        assert call(r) == 1, r
    assert call(dt=dsa.DSA_E4M3) == 2
    for k in (dict(T=-1), dict(H=-1), dict(H=65536), dict(pos=None), dict(x=None), dict(o=None), dict(x=17), dict(o=4113),
              dict(pos=18), dict(xt=-1), dict(oh=-64)):
        assert call(**k) == 1, k
    # rows of out that overlap, and in place with other strides
    for k in (dict(oh=32), dict(ot=255), dict(oh=0), dict(ot=0), dict(ot=64, oh=64), dict(x=4112, xh=128, xt=512)):
        assert call(**k) == 1, k
        assert "overlap" in dsa.last_error() or "same strides" in dsa.last_error()


def test_append_rope_and_read_refusals(dsa):
    lib = dsa._lib
    s, m = _descs(dsa)
    r = dsa.RopeDesc(64, 0, 16, 1.0)
    ref = ctypes.byref

    def write(s=s, m=m, r=r, lat=16, ls=512, kr=16, rs=64, c=16):
        return lib.dsa_latent_cache_append_rope(s and ref(s), m and ref(m), r and ref(r), lat, ls, kr, rs, c, None)

    assert write(s=None) == 1 and write(m=None) == 1 and write(r=None) == 1
    assert write(r=dsa.RopeDesc(32, 0, 16, 1.0)) == 1 and "d_rope" in dsa.last_error()
    for k in (dict(lat=None), dict(kr=None), dict(c=None), dict(lat=8), dict(kr=20), dict(c=24), dict(ls=-8),
              dict(ls=513), dict(rs=66)):
        assert write(**k) == 1, k
    for over, st in ((dict(row_bytes=431), 1), (dict(row_bytes=440), 1), (dict(row_bytes=416), 1),
                     (dict(d_latent=256), 2), (dict(d_rope=32), 2), (dict(dtype=9), 2)):
        assert write(m=_descs(dsa, **over)[1]) == st, over
    # copied rows: both parts in 16-byte vectors
    assert write(m=_descs(dsa, dtype=dsa.DSA_BF16, d_latent=60, d_rope=4, row_bytes=128)[1],
                 r=dsa.RopeDesc(4, 0, 16, 1.0)) == 2
    assert write(m=_descs(dsa, dtype=dsa.DSA_BF16, d_rope=0, row_bytes=1024)[1]) == 1

    def index(D=128, off=0, src=dsa.DSA_BF16, key=dsa.DSA_E4M3, k=16, ks=128, c=16, sc=16, r=r):
        return lib.dsa_index_cache_append_rope(ref(s), ref(r), D, off, src, key, k, ks, c, sc, None)

    for k, st in ((dict(D=126), 2), (dict(D=2048), 2), (dict(D=48, key=dsa.DSA_MXFP8_E4M3), 2), (dict(key=dsa.DSA_BF16), 2),
                  (dict(src=dsa.DSA_E4M3), 2), (dict(off=-1), 1), (dict(off=65), 1), (dict(k=None), 1), (dict(c=None), 1),
                  (dict(sc=None), 1), (dict(k=8), 1), (dict(ks=130), 1), (dict(ks=-4), 1), (dict(D=32), 1)):
        assert index(**k) == st, k

    def read(m=m, c=16, dt=dsa.DSA_BF16, o=16, os_=576):
        return lib.dsa_latent_cache_read(ref(s), ref(m), c, dt, o, os_, None)

    for k, st in ((dict(dt=dsa.DSA_E2M1), 2), (dict(c=None), 1), (dict(o=None), 1), (dict(o=8), 1), (dict(os_=575), 1),
                  (dict(os_=580), 1), (dict(os_=568), 1), (dict(m=_descs(dsa, row_bytes=436)[1]), 1)):
        assert read(**k) == st, k


def test_e2m1_attention_shape_refusals(dsa):
    lib = dsa._lib
    for over, st in ((dict(d_latent=64, d_rope=16), 2), (dict(row_bytes=440), 1), (dict(row_bytes=400), 1),
                     (dict(q=8), 1), (dict(kv_cache=8), 1)):
        s, m = _descs(dsa, **over)
        assert lib.dsa_sparse_mla_attn(ctypes.byref(s), ctypes.byref(m), 16, 32, 16, None, None, 0, None) == st, over


def test_binding_refuses_tensors_off_the_gpu(dsa):
    plan = dsa.Rope.make(64, device="cpu")
    x = torch.zeros(2, 3, 64)
    with pytest.raises(ValueError, match="CUDA device"):
        dsa.rope(plan, torch.zeros(2, dtype=torch.int32), x, x)
