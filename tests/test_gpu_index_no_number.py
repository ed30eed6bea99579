"""Index codes and scales that stand for no number, and scales far from one another: the same scores on every path.

Tolerance as in test_gpu_index_mx4: 130 2^-23 of sum_h |w_h| sum_i |q_hi k_i| (products of MXFP4 and MXFP8 codes and
powers of two are exact, 128 and fewer of them are added in fp32, then 64 and fewer weighted heads), with two roundings
more for fp32 scales."""
import numpy as np
import pytest
import torch

import dsa_indexed_sparse_gb300 as dsa
from oracle import dsa_oracle as O

pytestmark = pytest.mark.gpu

FORMATS = {"e4m3": dsa.DSA_E4M3, "mxfp8": dsa.DSA_MXFP8_E4M3, "mxfp4": dsa.DSA_MXFP4_E2M1}
# heads, dims, page size and queries a sequence: tensor cores with one query and four a group, then CUDA cores
SHAPES = [(64, 128, 64, 1), (64, 128, 64, 4), (64, 128, 16, 1), (3, 64, 64, 2)]


class Case:
    def __init__(self, dev, fmt, H, D, page, per, ctx=300, exps=((121, 134), (121, 134))):
        g = torch.Generator().manual_seed(H + D + page + per)
        self.dev, self.fmt, self.ctx, self.page, self.T = dev, fmt, ctx, page, per
        pages = (ctx + page - 1) // page
        self.table, self.rows = torch.randperm(pages + 1, generator=g)[:pages].to(torch.int32)[None], (pages + 1) * page
        width = D // 2 if fmt == "mxfp4" else D

        def codes(*n):
            c = torch.randint(0, 256, (*n, width), generator=g).to(torch.uint8)
            return c if fmt == "mxfp4" else c & 0xF7               # no NaN code

        def scale(n, lo_hi):
            if fmt == "e4m3":
                return torch.rand(n, generator=g) + 0.5
            return torch.randint(*lo_hi, (*n, D // 32), generator=g).to(torch.uint8)

        self.q, self.k, self.qs, self.ks = codes(per, H), codes(self.rows), scale((per, H), exps[0]), scale((self.rows,), exps[1])
        self.w = torch.randn((per, H), generator=g)
        self.pos = torch.arange(ctx - per, ctx, dtype=torch.int32)
        self.seq = dsa.Seq(q_seq=torch.zeros(per, dtype=torch.int32, device=dev), q_pos=self.pos.to(dev), block_table=self.table.to(dev),
                           max_ctx=ctx, cache_rows=self.rows, page_size=page, q_per_seq=per)

    def row(self, s):
        return int(self.table[0, s // self.page]) * self.page + s % self.page

    def run(self):
        idx = dsa.Indexer(q=self.q.to(self.dev), w=self.w.to(self.dev), k_cache=self.k.to(self.dev), q_scale=self.qs.to(self.dev),
                          k_scale=self.ks.to(self.dev), dtype=FORMATS[self.fmt])
        out = torch.full((self.T, (self.ctx + 3) // 4 * 4), -77.0, device=self.dev)
        dsa.indexer_scores(self.seq, idx, out)
        tc = (self.q.shape[1], self.page) == (64, 64)
        assert ("indexer_tc" if tc else "indexer_generic") in dsa.last_plan()
        dsa.check_status()
        return out.cpu().numpy()

    def values(self, codes, scale):
        codes, scale = codes.numpy(), scale.numpy()
        if self.fmt == "e4m3":
            return O.decode_e4m3(codes) * scale.astype(np.float64)[..., None]
        return (O.dequantize_mx_e2m1 if self.fmt == "mxfp4" else O.dequantize_mx_e4m3)(codes, scale)

    def check(self, got, no_key=(), no_query=()):
        """Positions no_key and queries no_query score NaN, all else as the formula says."""
        rows = [self.row(s) for s in range(self.ctx)]
        k = self.values(self.k, self.ks)[rows]
        for t in range(self.T):
            n = int(self.pos[t]) + 1
            if t in no_query:
                assert np.all(np.isnan(got[t, :n]))
                continue
            fine = np.array([s not in no_key for s in range(n)])
            q, w = self.values(self.q[t], self.qs[t]), self.w[t].numpy().astype(np.float64)
            want, mag = w @ np.maximum(q @ k[:n][fine].T, 0.0), np.abs(w) @ (np.abs(q) @ np.abs(k[:n][fine]).T)
            assert np.all(np.isnan(got[t, :n][~fine])), t
            assert np.all(np.abs(got[t, :n][fine] - want) <= 133 * 2.0 ** -23 * mag), t
            assert np.all(got[t, n:] == -77.0)


@pytest.mark.parametrize("H, D, page, per", SHAPES)
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_scale_byte_255_scores_nan(dev, fmt, H, D, page, per):
    """A block of a key whose scale byte is 255 takes the key's score with it, of a query head all of the query's."""
    c = Case(dev, fmt, H, D, page, per)
    for s in (0, 77, 290):
        c.ks[c.row(s), s % (D // 32)] = 255
    c.check(c.run(), no_key=(0, 77, 290))
    c.qs[per - 1, H - 1, D // 32 - 1] = 255
    c.check(c.run(), no_key=(0, 77, 290), no_query=(per - 1,))


@pytest.mark.parametrize("H, D, page, per", SHAPES)
@pytest.mark.parametrize("fmt", ["e4m3", "mxfp8"])
def test_nan_codes_score_nan(dev, fmt, H, D, page, per):
    c = Case(dev, fmt, H, D, page, per)
    for s in (5, 150):
        c.k[c.row(s), s % D] = 0x7F
    c.check(c.run(), no_key=(5, 150))
    c.q[0, H - 1, 3] = 0xFF
    c.check(c.run(), no_key=(5, 150), no_query=(0,))


def test_nan_of_fp32_keys_scores_nan(dev):
    g = torch.Generator().manual_seed(3)
    q, k, w = torch.randn((1, 3, 20), generator=g), torch.randn((64, 20), generator=g), torch.randn((1, 3), generator=g)
    k[9, 7] = float("nan")
    k[11, 2] = -float("inf")
    seq = dsa.Seq(q_seq=torch.zeros(1, dtype=torch.int32, device=dev), q_pos=torch.tensor([39], dtype=torch.int32, device=dev),
                  block_table=torch.zeros((1, 1), dtype=torch.int32, device=dev), max_ctx=64, cache_rows=64)
    out = torch.full((1, 64), -77.0, device=dev)
    dsa.indexer_scores(seq, dsa.Indexer(q=q.to(dev), w=w.to(dev), k_cache=k.to(dev)), out)
    dsa.check_status()
    got, z = out[0].cpu().double(), q[0].double() @ k.double().T
    want, mag = (w[0].double()[:, None] * z.clamp(min=0)).sum(0), w[0].double().abs() @ (q[0].double().abs() @ k.double().abs().T)
    assert torch.isnan(got[9]) and torch.isnan(want[9])
    assert np.array_equal(got[11].numpy(), want[11].numpy(), equal_nan=True)    # infinities of one head or of several
    plain = [s for s in range(40) if s not in (9, 11)]
    assert bool(((got - want).abs() <= 30 * 2.0 ** -23 * mag)[plain].all()) and bool((got[40:] == -77.0).all())


@pytest.mark.parametrize("exps", [((0, 8), (247, 255)), ((247, 255), (0, 8))])
@pytest.mark.parametrize("H, D, page, per", SHAPES)
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_only_the_sum_of_exponents_counts(dev, fmt, H, D, page, per, exps):
    """Scales at the two ends of their range: a vector's values alone would leave fp32."""
    c = Case(dev, fmt, H, D, page, per, exps=exps)
    c.check(c.run())
