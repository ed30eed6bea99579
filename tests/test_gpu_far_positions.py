"""Positions up to the last one that fits 32 bits: steps, tiles and slices that end behind it."""
import pytest
import torch

import dsa_indexed_sparse_gb300 as dsa

pytestmark = pytest.mark.gpu

LAST = 2 ** 31 - 2                 # with max_ctx 2^31 - 1


def _seq(dev, table, page, rows, pos=LAST):
    return dsa.Seq(q_seq=torch.zeros(1, dtype=torch.int32, device=dev), q_pos=torch.tensor([pos], dtype=torch.int32, device=dev),
                   block_table=table, max_ctx=LAST + 1, cache_rows=rows, page_size=page)


@pytest.mark.parametrize("page", [65536, 70001, 2 ** 30 + 5])
def test_block_choice(dev, page):
    g = torch.Generator(device=dev).manual_seed(page)
    scores = torch.rand((1, 2 ** 31), generator=g, device=dev)
    scores[0, LAST + 1] = 2.0                    # behind the position
    n = LAST // page + 1
    whole = n - 1
    best = torch.cat([scores[0, :whole * page].view(whole, page).amax(1), scores[0, whole * page:LAST + 1].amax()[None]])
    N = min(10, n - 1)
    want = best.argsort(descending=True, stable=True)[:N].sort().values.to(torch.int32)
    out = torch.full((1, N), -7, dtype=torch.int32, device=dev)
    dsa.block_topk(_seq(dev, torch.zeros((1, n), dtype=torch.int32, device=dev), page, page, LAST), scores, N, out, first=0, last=0)
    dsa.check_status()
    assert torch.equal(out[0], want)


@pytest.mark.parametrize("page", [10000, 16384])
def test_block_attention_over_positions(dev, page):
    """A last page that ends behind 2^31: its positions as dsa_sparse_mla_attn takes them."""
    g = torch.Generator(device=dev).manual_seed(page)
    blk, n = LAST // page, LAST // page + 1
    table = torch.zeros((1, n), dtype=torch.int32, device=dev)
    table[0, -1] = 1
    cache = torch.randn((2 * page, 576), generator=g, device=dev).to(torch.bfloat16)
    mla = dsa.Mla(q=torch.randn((1, 16, 576), generator=g, device=dev).to(torch.bfloat16), kv_cache=cache, d_latent=512, d_rope=64,
                  softmax_scale=0.07)
    seq = _seq(dev, table, page, 2 * page)
    pos = torch.arange(page, device=dev) + blk * page
    pos = torch.where(pos <= LAST, pos, -1).to(torch.int32)[None].contiguous()
    outs = []
    for size, call in ((dsa.block_mla_attn_workspace_size(seq, mla, 1), lambda o, l, ws: dsa.block_mla_attn(
            seq, mla, torch.tensor([[blk]], dtype=torch.int32, device=dev), o, lse=l, workspace=ws)),
                       (dsa.sparse_mla_attn_workspace_size(seq, mla, page), lambda o, l, ws: dsa.sparse_mla_attn(
                           seq, mla, pos, page, o, lse=l, workspace=ws))):
        out, lse = torch.empty((1, 16, 512), dtype=torch.bfloat16, device=dev), torch.empty((1, 16), device=dev)
        call(out, lse, torch.empty(max(size, 16), dtype=torch.uint8, device=dev))
        dsa.check_status()
        outs.append((out, lse))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
