"""MXFP4 index keys as far as they need no GPU: the oracle's format by hand, and every refusal."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import dsa_oracle as O


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__
    __graft_entry__.build()
    import dsa_indexed_sparse_gb300 as m
    return m


def test_mx4_by_hand():
    x = np.zeros((1, 64))
    x[0, 0], x[0, 1], x[0, 31], x[0, 32] = 6.0, -3.0, 0.25, 0.01
    codes, e = O.quantize_mx_e2m1(x)
    assert e.tolist() == [[127, 127 - 7 - 2]]             # floor(log2 6) - 2 = 0; floor(log2 0.01) = -7
    assert codes[0, 0] == 7 | (13 << 4) and codes[0, 15] == 0     # 0.25 is halfway to 0.5: the even code, 0
    assert codes[0, 16] == 6 + 1 or O.decode_e2m1(codes[0, 16] & 15) * 2.0 ** -9 == 0.01171875   # 5.12 -> 6
    v = O.dequantize_mx_e2m1(codes, e)
    assert v[0, :2].tolist() == [6.0, -3.0] and v[0, 32] == 6 * 2.0 ** -9
    assert O.quantize_mx_e2m1(np.zeros((1, 32)))[1].tolist() == [[0]]


def test_mx4_error_bound():
    """A value is off by at most half a step: 2^-2 of a block's maximum below 2^x (the widest half step is 1 of at least 4),
    beyond 6 by at most 2 of 8."""
    rng = np.random.default_rng(1)
    x = rng.normal(0, 1, (50, 128)) * np.exp2(rng.integers(-20, 20, (50, 1)))
    v = O.dequantize_mx_e2m1(*O.quantize_mx_e2m1(x))
    amax = np.repeat(np.abs(x).reshape(50, 4, 32).max(-1), 32, axis=1)
    assert np.all(np.abs(v - x) <= amax / 4)


def _seq(dsa, **over):
    d = dict(B=1, T=2, max_ctx=128, q_per_seq=0, q_seq=16, q_pos=16, block_table=16, bt_stride=2, page_size=64, cache_rows=256)
    return dsa.SeqDesc(**{**d, **over})


def test_refusals(dsa):
    lib, ref = dsa._lib, ctypes.byref
    s = _seq(dsa)
    M4, M8, E, B, F = dsa.DSA_MXFP4_E2M1, dsa.DSA_MXFP8_E4M3, dsa.DSA_E4M3, dsa.DSA_BF16, dsa.DSA_F32

    def append(seq=s, D=128, src=B, k=16, c=16, e=16):
        return lib.dsa_index_cache_append_mx4(seq and ref(seq), D, src, k, c, e, None)

    for kw, st in ((dict(seq=None), 1), (dict(D=48), 2), (dict(D=0), 2), (dict(D=1056), 2), (dict(src=E), 2), (dict(k=None), 1),
                   (dict(c=None), 1), (dict(e=None), 1), (dict(k=8), 1), (dict(c=24), 1), (dict(e=4), 1),
                   (dict(seq=_seq(dsa, cache_rows=100)), 1)):
        assert append(**kw) == st, kw

    def quant(T=2, H=64, D=128, src=B, dt=M4, q=16, st=8192, sh=128, c=16, sc=16):
        return lib.dsa_index_query_quantize(T, H, D, src, dt, q, st, sh, c, sc, None)

    for kw, st in ((dict(T=-1), 1), (dict(H=-1), 1), (dict(D=48), 2), (dict(D=2048), 2), (dict(dt=E, D=6), 2), (dict(dt=B), 2),
                   (dict(dt=F), 2), (dict(dt=dsa.DSA_E2M1), 2), (dict(dt=17), 2), (dict(src=M8), 2), (dict(q=None), 1),
                   (dict(c=None), 1), (dict(sc=None), 1), (dict(q=8), 1), (dict(c=8), 1), (dict(sc=8), 1), (dict(st=-8), 1),
                   (dict(sh=4), 1), (dict(st=130), 1), (dict(dt=E, sh=2), 1), (dict(src=F, sh=2), 1),
                   (dict(T=1 << 30, H=64), 1)):
        assert quant(**kw) == st, kw

    def read(seq=s, D=128, dt=M4, c=16, sc=16, od=B, o=16, os_=128):
        return lib.dsa_index_cache_read(seq and ref(seq), D, dt, c, sc, od, o, os_, None)

    for kw, st in ((dict(seq=None), 1), (dict(D=48), 2), (dict(dt=F), 2), (dict(od=E), 2), (dict(c=None), 1), (dict(sc=None), 1),
                   (dict(dt=M8, sc=None), 1), (dict(o=None), 1), (dict(o=8), 1), (dict(os_=127), 1), (dict(os_=132), 1),
                   (dict(os_=120), 1), (dict(od=F, os_=130), 1)):
        assert read(**kw) == st, kw

    x = dsa.IndexerDesc(H_I=64, D_I=128, dtype=M4, q=16, q_scale=16, w=16, k_cache=16, k_scale=16)

    def scores(**over):
        d = dsa.IndexerDesc(**{**{n: getattr(x, n) for n, _ in x._fields_}, **over})
        return lib.dsa_indexer_scores(ref(s), ref(d), 16, 128, None)

    for over, st in ((dict(D_I=48), 2), (dict(q_scale=None), 1), (dict(k_scale=None), 1), (dict(k_scale=8), 1), (dict(dtype=7), 2),
                     (dict(dtype=dsa.DSA_E2M1), 2)):
        assert scores(**over) == st, over


def test_rope_writer_refuses_short_blocks(dsa):
    s, r = _seq(dsa), dsa.RopeDesc(32, 0, 16, 1.0)
    assert dsa._lib.dsa_index_cache_append_rope(ctypes.byref(s), ctypes.byref(r), 48, 0, dsa.DSA_BF16, dsa.DSA_MXFP4_E2M1, 16,
                                                48, 16, 16, None) == 2
    assert "multiple of 32" in dsa.last_error()


def test_binding_refuses_shapes(dsa):
    z = lambda *n, d=torch.uint8: torch.zeros(n, dtype=d)
    good = dict(q=z(2, 64, 64), w=z(2, 64, d=torch.float32), k_cache=z(256, 64), q_scale=z(2, 64, 4), k_scale=z(256, 4), dtype=dsa.DSA_MXFP4_E2M1)
    d = dsa.Indexer(**good).desc()
    assert d.D_I == 128 and d.H_I == 64
    for over in (dict(q_scale=None), dict(k_scale=z(256, 2)), dict(q_scale=z(2, 64, 4, d=torch.float32)), dict(k_cache=z(256, 128))):
        with pytest.raises(ValueError, match="MXFP4"):
            dsa.Indexer(**{**good, **over}).desc()
    seq = dsa.Seq(q_seq=z(2, d=torch.int32), q_pos=z(2, d=torch.int32), block_table=z(1, 4, d=torch.int32), max_ctx=256, cache_rows=256)
    M4 = dsa.DSA_MXFP4_E2M1
    for call in (lambda: dsa.index_cache_append(seq, z(2, 128, d=torch.bfloat16), z(255, 64), z(256, 4), dtype=M4),
                 lambda: dsa.index_cache_append(seq, z(2, 128, d=torch.bfloat16), z(256, 64), z(256, 3), dtype=M4),
                 lambda: dsa.index_cache_append(seq, z(3, 128, d=torch.bfloat16), z(256, 64), z(256, 4), dtype=M4),
                 lambda: dsa.index_cache_append(seq, z(2, 128), z(256, 64), z(256, 4), dtype=M4),
                 lambda: dsa.index_cache_append(seq, z(2, 128, d=torch.bfloat16), z(256, 64), z(256, 4), dtype=dsa.DSA_E2M1),
                 lambda: dsa.index_query_quantize(z(2, 64, 128, d=torch.bfloat16), z(2, 64, 63), z(2, 64, 4), dtype=M4),
                 lambda: dsa.index_query_quantize(z(2, 64, 128, d=torch.float16), z(2, 64, 64), z(2, 64, 4), dtype=M4),
                 lambda: dsa.index_query_quantize(z(2, 64, 128, d=torch.float32), z(2, 64, 64), z(2, 64, 4), dtype=M4),
                 lambda: dsa.index_cache_read(seq, z(256, 64), None, z(2, 128, d=torch.float32), dtype=M4),
                 lambda: dsa.index_cache_read(seq, z(256, 64), z(256, 4), z(3, 128, d=torch.float32), dtype=M4),
                 lambda: dsa.index_cache_read(seq, z(256, 64), z(256, 4), z(2, 128, d=torch.float32), dtype=M4)):   # not on a GPU
        with pytest.raises(ValueError):
            call()


def test_mx4_value_beyond_the_border_at_five():
    """0.01 = 5.12 * 2^-9 lies beyond 5, the border between 4 and 6: code 7 in the low nibble, nothing in the high one."""
    x = np.zeros((1, 32))
    x[0, 0] = 0.01
    codes, e = O.quantize_mx_e2m1(x)
    assert e.tolist() == [[118]] and codes[0].tolist() == [7] + [0] * 15
    assert O.dequantize_mx_e2m1(codes, e)[0, 0] == 6 * 2.0 ** -9
