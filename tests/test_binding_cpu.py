"""The Python binding where no GPU is: importing it, and what it refuses before a CUDA call."""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_on_a_torch_without_cuda():
    """A torch built without CUDA lacks the two functions that the binding takes for speed: importing it and making a
    rotation on the CPU need neither."""
    code = ("import torch\n"
            "for name in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    if hasattr(torch._C, name):\n"
            "        delattr(torch._C, name)\n"
            "import dsa_indexed_sparse_gb300 as dsa\n"
            "assert dsa.Rope.make(8, device='cpu').turns.shape == (4,)\n")
    run = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert run.returncode == 0, run.stderr


def test_index_writer_refuses_caches_of_another_kind():
    """The scales of one key format given for the other, or arrays smaller than the pool: a row would be written past its
    own.  Refused before anything else is looked at."""
    import dsa_indexed_sparse_gb300 as dsa
    rows, D = 128, 64
    seq = dsa.Seq(q_seq=torch.zeros(2, dtype=torch.int32), q_pos=torch.zeros(2, dtype=torch.int32),
                  block_table=torch.zeros((1, 2), dtype=torch.int32), max_ctx=128, cache_rows=rows)
    plan = dsa.Rope.make(32, device="cpu")
    key = torch.zeros((2, D))
    kc = torch.zeros((rows, D), dtype=torch.uint8)
    f32, mx = torch.zeros(rows), torch.zeros((rows, D // 32), dtype=torch.uint8)
    call = lambda c, s, m: dsa.index_cache_append_rope(seq, plan, key, c, s, mx=m)
    for scale, m in ((mx, False), (f32, True), (f32[:-1], False), (mx[:-1], True), (f32.double(), False)):
        with pytest.raises(ValueError, match="k_scale"):
            call(kc, scale, m)
    for cache in (kc[:-1], kc.float(), kc[:, :32].contiguous()):
        with pytest.raises(ValueError, match="k_cache"):
            call(cache, f32, False)
    for scale, m in ((f32, False), (mx, True)):          # the right ones are refused for where they are
        with pytest.raises(ValueError, match="CUDA device"):
            call(kc, scale, m)
