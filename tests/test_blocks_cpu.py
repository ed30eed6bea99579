"""The choice of blocks and the attention over blocks: every refusal, without a GPU."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__
    __graft_entry__.build()
    import dsa_indexed_sparse_gb300 as m
    return m


def _seq(dsa, **over):
    d = dict(B=1, T=2, max_ctx=128, q_per_seq=0, q_seq=16, q_pos=16, block_table=16, bt_stride=2, page_size=64, cache_rows=256)
    return dsa.SeqDesc(**{**d, **over})


def _mla(dsa, **over):
    d = dict(H=128, d_latent=512, d_rope=64, dtype=dsa.DSA_BF16, q=16, kv_cache=16, row_bytes=1152, softmax_scale=1.0)
    return dsa.MlaDesc(**{**d, **over})


def test_block_topk_refusals(dsa):
    ref = ctypes.byref

    def call(s=_seq(dsa), scores=16, ld=128, n=4, first=1, last=1, out=16):
        return dsa._lib.dsa_block_topk(s and ref(s), scores, ld, n, first, last, out, None)

    for kw, st in ((dict(s=None), 1), (dict(scores=None), 1), (dict(scores=8), 1), (dict(out=None), 1), (dict(out=4), 1),
                   (dict(ld=124), 1), (dict(ld=130), 1), (dict(n=0), 2), (dict(n=65537), 2), (dict(first=-1), 1), (dict(last=-1), 1),
                   (dict(first=3, last=2), 1), (dict(first=2147483647, last=2147483647), 1), (dict(s=_seq(dsa, page_size=0)), 1),
                   (dict(s=_seq(dsa, max_ctx=32769, bt_stride=32769, page_size=1), ld=32772), 2)):
        if kw.get("ld") == 32772 and not torch.cuda.is_available():
            continue                             # refused by the launcher, behind the query of the device
        assert call(**kw) == st, kw


def test_block_attention_refusals(dsa):
    ref = ctypes.byref

    def call(s=_seq(dsa), m=_mla(dsa), idx=16, n=2, out=16, lse=None, ws=None, size=0):
        return dsa._lib.dsa_block_mla_attn(s and ref(s), m and ref(m), idx, n, out, lse, ws, size, None)

    for kw, st in ((dict(s=None), 1), (dict(m=None), 1), (dict(idx=None), 1), (dict(idx=8), 1), (dict(out=None), 1), (dict(out=8), 1),
                   (dict(lse=8), 1), (dict(ws=8, size=64), 3), (dict(n=0), 2), (dict(n=65537), 2), (dict(m=_mla(dsa, q=None)), 1),
                   (dict(m=_mla(dsa, kv_cache=8)), 1), (dict(m=_mla(dsa, row_bytes=1150)), 1), (dict(m=_mla(dsa, dtype=dsa.DSA_MXFP4_E2M1)), 2),
                   (dict(m=_mla(dsa, dtype=dsa.DSA_E2M1, row_bytes=432), n=257), 2), (dict(m=_mla(dsa, row_bytes=1156), n=257), 2)):
        assert call(**kw) == st, kw


def test_block_step_refusals(dsa):
    ref = ctypes.byref
    x = dsa.IndexerDesc(H_I=64, D_I=128, dtype=dsa.DSA_E4M3, q=16, q_scale=16, w=16, k_cache=16, k_scale=16)

    def call(s=_seq(dsa), m=_mla(dsa), n=4, first=1, last=1, out=16, sel=None, ws=16, size=1 << 30):
        return dsa._lib.dsa_block_decode_step(ref(s), ref(x), ref(m), n, first, last, out, None, sel, ws, size, None)

    for kw, st in ((dict(n=0), 2), (dict(first=4), 1), (dict(ws=None), 3), (dict(ws=8), 3), (dict(sel=8), 1), (dict(m=_mla(dsa, H=0)), 1)):
        assert call(**kw) == st, kw


def test_binding_refuses_tensors_and_shapes(dsa):
    z = lambda *n, d=torch.int32: torch.zeros(n, dtype=d)
    seq = dsa.Seq(q_seq=z(2), q_pos=z(2), block_table=z(1, 4), max_ctx=256, cache_rows=256)
    mla = dsa.Mla(q=z(2, 128, 576, d=torch.bfloat16), kv_cache=z(256, 576, d=torch.bfloat16), d_latent=512, d_rope=64, softmax_scale=1.0)
    with pytest.raises(ValueError, match="CUDA device"):
        dsa.block_topk(seq, z(2, 256, d=torch.float32), 4, z(2, 4))
    with pytest.raises(ValueError, match="CUDA device"):
        dsa.block_mla_attn(seq, mla, z(2, 4), z(2, 128, 512, d=torch.bfloat16))
    with pytest.raises(ValueError):
        dsa.block_mla_attn(seq, mla, z(2), z(2, 128, 512, d=torch.bfloat16))
