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
