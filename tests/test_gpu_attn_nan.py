"""A NaN in a selected row, or in a query head, on every path of the attention over single rows: the output and the
log-sum-exp of the heads that see it are NaN, those of the others bit for bit what they were."""
import math

import pytest
import torch

import dsa_indexed_sparse_gb300 as dsa

pytestmark = pytest.mark.gpu

# cache format, heads, dims: the tensor cores' rows, then CUDA cores
PATHS = [("bf16", 128, 512, 64), ("e4m3", 128, 512, 64), ("e4m3_t128", 128, 512, 64), ("e2m1", 128, 512, 64), ("bf16", 8, 512, 64),
         ("e4m3", 3, 512, 64), ("f32", 2, 32, 16)]


class Case:
    def __init__(self, dev, fmt, H, d, r, T=3, ctx=700, page=64):
        g = torch.Generator(device=dev).manual_seed(H + d + len(fmt))
        self.dev, self.T, self.H, self.d, self.ctx = dev, T, H, d, ctx
        dt = torch.float32 if fmt == "f32" else torch.bfloat16
        pages = (ctx + page - 1) // page
        self.table = torch.randperm(pages, generator=g, device=dev).to(torch.int32)[None]
        code, width = {"e4m3": (dsa.DSA_E4M3, 656), "e4m3_t128": (dsa.DSA_E4M3_T128, 656), "e2m1": (dsa.DSA_E2M1, 432)}.get(fmt, (None, 0))
        rows = pages * page
        self.cache = torch.zeros((rows, width), dtype=torch.uint8, device=dev) if width else torch.zeros((rows, d + r), dtype=dt, device=dev)
        self.q = torch.randn((T, H, d + r), generator=g, device=dev).to(dt)
        common = dict(block_table=self.table, max_ctx=ctx, cache_rows=rows, page_size=page)
        self.seq = dsa.Seq(q_seq=torch.zeros(T, dtype=torch.int32, device=dev),
                           q_pos=torch.tensor([ctx - 1, ctx // 2, ctx - 2][:T], dtype=torch.int32, device=dev), **common)
        self.mla = dsa.Mla(q=self.q, kv_cache=self.cache, d_latent=d, d_rope=r, softmax_scale=0.07, dtype=code)
        self.rows = torch.randn((ctx, d + r), generator=g, device=dev).to(dt)
        self.every = dsa.Seq(q_seq=torch.zeros(ctx, dtype=torch.int32, device=dev), q_pos=torch.arange(ctx, dtype=torch.int32, device=dev), **common)
        self.write()
        self.dt = dt

    def write(self):
        dsa.latent_cache_append(self.every, self.mla, self.rows)

    def run(self, idx, workspace=True):
        K = idx.shape[1]
        out, lse = torch.full((self.T, self.H, self.d), 7.0, dtype=self.dt, device=self.dev), torch.full((self.T, self.H), 7.0, device=self.dev)
        size = dsa.sparse_mla_attn_workspace_size(self.seq, self.mla, K)
        ws = torch.empty(max(size, 16), dtype=torch.uint8, device=self.dev) if workspace else None
        dsa.sparse_mla_attn(self.seq, self.mla, idx, K, out, lse=lse, workspace=ws)
        dsa.check_status()
        return out, lse

    def choose(self, K):
        idx = torch.full((self.T, K), -1, dtype=torch.int32, device=self.dev)
        for t in range(self.T):
            n = int(self.seq.q_pos[t]) + 1
            take = torch.arange(max(0, n - K), n, dtype=torch.int32, device=self.dev)
            idx[t, :len(take)] = take
        return idx


@pytest.mark.parametrize("fmt, H, d, r", PATHS)
@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("where", ["rope", "latent"])
def test_nan_of_a_selected_row(dev, fmt, H, d, r, workspace, where):
    if where == "latent" and fmt not in ("bf16", "f32"):
        pytest.skip("the quantised rows' NaN: that of their rope values")
    s = Case(dev, fmt, H, d, r)
    idx = s.choose(400)
    clean = s.run(idx, workspace)
    # a row that queries 0 and 2 select in their middle, and query 1, of half as many positions, does not
    s.rows[s.ctx - 200, 3 if where == "latent" else d + 3] = float("nan")
    s.write()
    out, lse = s.run(idx, workspace)
    for t in (0, 2):
        assert bool(torch.isnan(out[t]).all()) and bool(torch.isnan(lse[t]).all())
    assert torch.equal(out[1], clean[0][1]) and torch.equal(lse[1], clean[1][1]) and bool(torch.isfinite(lse[1]).all())
    alone = torch.full((s.T, 1), -1, dtype=torch.int32, device=dev)     # the NaN row and nothing else; a query of nothing
    alone[0, 0] = s.ctx - 200
    out, lse = s.run(alone, workspace)
    assert bool(torch.isnan(out[0]).all()) and bool(torch.isnan(lse[0]).all())
    assert not bool(out[1:].any()) and bool((lse[1:] == -math.inf).all())


@pytest.mark.parametrize("fmt, H, d, r", PATHS)
@pytest.mark.parametrize("workspace", [True, False])
def test_nan_of_a_query_head(dev, fmt, H, d, r, workspace):
    s = Case(dev, fmt, H, d, r)
    idx = s.choose(400)
    clean = s.run(idx, workspace)
    s.q[1, H - 1, d + 1] = float("nan")
    out, lse = s.run(idx, workspace)
    assert bool(torch.isnan(out[1, H - 1]).all()) and bool(torch.isnan(lse[1, H - 1]))
    out[1, H - 1], lse[1, H - 1] = clean[0][1, H - 1], clean[1][1, H - 1]
    assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])


@pytest.mark.parametrize("page", [64, 32])
def test_blocks_give_the_same_for_either_form(dev, page):
    """Attention over blocks: pages that are read whole, and pages whose positions are written out."""
    s = Case(dev, "bf16", 128, 512, 64, page=page)
    s.rows[s.ctx - 200, 100] = float("nan")
    s.write()
    idx = torch.full((s.T, 4 * 64 // page), -1, dtype=torch.int32, device=dev)
    idx[0, 1], idx[1, 0], idx[2, 0] = (s.ctx - 200) // page, 1, 2
    out, lse = torch.empty((s.T, 128, 512), dtype=torch.bfloat16, device=dev), torch.empty((s.T, 128), device=dev)
    ws = torch.empty(max(16, dsa.block_mla_attn_workspace_size(s.seq, s.mla, idx.shape[1])), dtype=torch.uint8, device=dev)
    dsa.block_mla_attn(s.seq, s.mla, idx, out, lse=lse, workspace=ws)
    dsa.check_status()
    assert bool(torch.isnan(out[0]).all()) and bool(torch.isnan(lse[0]).all()) and bool(torch.isfinite(lse[1:]).all())
