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


def test_topk(dev):
    g = torch.Generator(device=dev).manual_seed(1)
    scores = torch.rand((1, 2 ** 31), generator=g, device=dev)
    scores[0, LAST + 1] = 9.0                    # behind the position
    picks = torch.randint(0, LAST, (60,), generator=g, device=dev)
    eighth = (LAST // 8) & ~3
    picks = torch.cat([picks, torch.tensor([0, LAST, LAST - 1, LAST - 3, LAST // 2, eighth, eighth - 1, 3 * eighth + 5], device=dev)]).unique()
    scores[0, picks] = 2.0 + torch.rand(len(picks), generator=g, device=dev)
    K = len(picks)
    out = torch.full((1, K), -7, dtype=torch.int32, device=dev)
    dsa.topk(_seq(dev, torch.zeros((1, 2 ** 25), dtype=torch.int32, device=dev), 64, 64), scores, K, out)
    dsa.check_status()
    assert torch.equal(out[0].long(), picks)


@pytest.mark.parametrize("fmt, H, D", [("mxfp4", 64, 128), ("e4m3", 64, 128), ("mxfp4", 1, 32)])
def test_scores(dev, fmt, H, D):
    """Keys of a few pages, used over and over: each position scores, bit for bit, as its key does in a short sequence."""
    g = torch.Generator(device=dev).manual_seed(D)
    pages = 128
    code = {"mxfp4": dsa.DSA_MXFP4_E2M1, "e4m3": dsa.DSA_E4M3}[fmt]
    byte = lambda *n: torch.randint(0, 256, n, generator=g, device=dev).to(torch.uint8)
    if fmt == "mxfp4":
        q, k = byte(1, H, D // 2), byte(pages * 64, D // 2)
        qs, ks = (torch.randint(121, 134, (*n, D // 32), generator=g, device=dev).to(torch.uint8) for n in ((1, H), (pages * 64,)))
    else:
        q, k = byte(1, H, D) & 0xF7, byte(pages * 64, D) & 0xF7
        qs, ks = torch.rand((1, H), generator=g, device=dev), torch.rand(pages * 64, generator=g, device=dev)
    idx = dsa.Indexer(q=q, w=torch.randn((1, H), generator=g, device=dev), k_cache=k, q_scale=qs, k_scale=ks, dtype=code)
    short = torch.empty((1, pages * 64), device=dev)
    dsa.indexer_scores(dsa.Seq(q_seq=torch.zeros(1, dtype=torch.int32, device=dev), max_ctx=pages * 64, cache_rows=pages * 64,
                               q_pos=torch.tensor([pages * 64 - 1], dtype=torch.int32, device=dev),
                               block_table=torch.arange(pages, dtype=torch.int32, device=dev)[None]), idx, short)
    table = torch.randint(0, pages, (1, 2 ** 25), generator=g, device=dev).to(torch.int32)
    out = torch.full((1, 2 ** 31), -77.0, device=dev)
    dsa.indexer_scores(_seq(dev, table, 64, pages * 64), idx, out)
    dsa.check_status()
    assert float(out[0, LAST + 1]) == -77.0
    out[0, LAST + 1] = short[0, int(table[0, -1]) * 64 + 63]
    per_page = short.view(pages, 64)
    for a in range(0, 2 ** 25, 2 ** 21):
        assert torch.equal(out.view(-1, 64)[a:a + 2 ** 21], per_page[table[0, a:a + 2 ** 21].long()]), a
