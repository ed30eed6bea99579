"""A step of no valid query behind one that is under way: a padded batch whose rows are all idle (positions -1)."""
import pytest
import torch

import dsa_indexed_sparse_gb300 as dsa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["mxfp4", "e4m3"])
@pytest.mark.parametrize("blocks", [True, False])
@pytest.mark.parametrize("per", [512, 511])
def test_idle_step_leaves_the_one_before_alone(dev, blocks, fmt, per):
    """Both steps share their workspace, whose selection the first one's attention still reads when the second begins."""
    g = torch.Generator(device=dev).manual_seed(per)
    ctx, N = 4096, 32 if blocks else 2048
    pages = ctx // 64
    rnd = lambda *n: torch.randn(n, generator=g, device=dev).to(torch.bfloat16)
    seqs = [dsa.Seq(q_seq=torch.zeros(per, dtype=torch.int32, device=dev), q_pos=pos, max_ctx=ctx, cache_rows=ctx, q_per_seq=per,
                    block_table=torch.randperm(pages, generator=g, device=dev).to(torch.int32)[None])
            for pos in (torch.arange(ctx - per, ctx, dtype=torch.int32, device=dev), torch.full((per,), -1, dtype=torch.int32, device=dev))]
    mla = dsa.Mla(q=rnd(per, 128, 576), kv_cache=rnd(ctx, 576), d_latent=512, d_rope=64, softmax_scale=0.07)
    wide = 64 if fmt == "mxfp4" else 128
    codes = lambda *n: torch.randint(0, 256, (*n, wide), generator=g, device=dev).to(torch.uint8) & (0xFF if fmt == "mxfp4" else 0xF7)
    scale = (lambda *n: torch.randint(121, 134, (*n, 4), generator=g, device=dev).to(torch.uint8)) if fmt == "mxfp4" else \
        (lambda *n: torch.rand(n, generator=g, device=dev))
    idx = dsa.Indexer(q=codes(per, 64), w=torch.randn((per, 64), generator=g, device=dev), k_cache=codes(ctx), q_scale=scale(per, 64),
                      k_scale=scale(ctx), dtype=dsa.DSA_MXFP4_E2M1 if fmt == "mxfp4" else dsa.DSA_E4M3)
    size = dsa.block_decode_workspace_size if blocks else (lambda s, m, n: dsa.decode_workspace_size(s, idx, m, n))
    ws = torch.empty(size(seqs[0], mla, N), dtype=torch.uint8, device=dev)
    outs = [torch.empty((per, 128, 512), dtype=torch.bfloat16, device=dev) for _ in range(3)]

    def step(seq, out):
        (dsa.block_decode_step if blocks else dsa.decode_step)(seq, idx, mla, N, out, ws)

    step(seqs[0], outs[0])
    dsa.check_status()
    assert "indexer_tc" in dsa.last_plan()
    step(seqs[0], outs[1])
    step(seqs[1], outs[2])
    with pytest.raises(dsa.DSAError, match="bad_q_pos"):
        dsa.check_status()
    assert torch.equal(outs[0], outs[1]) and not bool(outs[2].any())
