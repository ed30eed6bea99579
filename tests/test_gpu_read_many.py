"""The cache reader where it takes two rows a warp (more rows than the GPU holds warps for), every format into both types: an
odd number of rows, and positions that are out of range beside ones that are not."""
import gc

import numpy as np
import pytest
import torch

import dsa_indexed_sparse_gb300 as dsa
import dsa_workloads as W
from oracle import dsa_oracle as O
from tests.test_gpu_positions import FORMATS, TYPES, _mla

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _leave_nothing_behind():
    """Device memory that cycles of earlier tests' tracebacks still hold is freed here, not during a test that counts it."""
    yield
    gc.collect()


@pytest.mark.parametrize("bad", [False, True])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", list(FORMATS))
def test_latent_read_of_many(dev, fmt, out, bad):
    T = torch.cuda.get_device_properties(dev).multi_processor_count * 64 + 257
    wl = W.make("decode_b4_long", seed=81, ctx=[300, 450], K=16, q_len=1, mla_dtype=fmt, shuffle_pages=True)
    rng = np.random.default_rng(T)
    seqs = rng.integers(0, 2, T).astype(np.int32)
    pos = rng.integers(0, np.asarray(wl.seq_lens)[seqs]).astype(np.int32)
    skipped = np.zeros(T, bool)
    if bad:   # the first of a pair, the second, both, and the last row, which is alone
        pos[[0, 1001, 2000, 2001, T - 1]] = [-1, wl.max_ctx, 1 << 30, -7, -(1 << 31)]
        seqs[[3000, 4001]] = [2, -1]
        skipped[[0, 1001, 2000, 2001, T - 1, 3000, 4001]] = True
    d = dict(W.device_tensors(wl, dev)["seq"])
    d.update(q_seq=torch.from_numpy(seqs).to(dev), q_pos=torch.from_numpy(pos).to(dev), q_per_seq=0)
    raw = torch.from_numpy(wl.kv.view(np.uint8).reshape(wl.cache_rows, -1)).to(dev)
    wide = torch.full((T, 600), 7.0, dtype=TYPES[out], device=dev)
    dsa.latent_cache_read(dsa.Seq(**d), _mla(dev, fmt, raw), wide[:, 8:584])
    if bad:
        # (not kept by a name: the traceback would hold this frame and its tensors until some later collection)
        with pytest.raises(dsa.DSAError, match="DSA_ERR_DEVICE_CHECK.*bad_q_pos"):
            dsa.check_status()
    else:
        dsa.check_status()
    # fp32: one product of a code and its scale; bf16: that product rounded once more
    at = [O.physical_rows(wl.block_table[b], 64, np.arange(n)) for b, n in enumerate(wl.seq_lens)]
    values = [torch.from_numpy(O.latent_rows(wl, rows)).float().to(TYPES[out]) for rows in at]
    good = torch.from_numpy(~skipped)
    want = torch.full((T, 576), 7.0, dtype=TYPES[out])
    for b in (0, 1):
        of_b = good & torch.from_numpy(seqs == b)
        want[of_b] = values[b][torch.from_numpy(pos)[of_b].long()]
    got = wide.cpu()
    assert torch.equal(got[:, 8:584], want)
    assert bool((got[:, :8] == 7).all()) and bool((got[:, 584:] == 7).all())
