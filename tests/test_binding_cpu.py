"""The Python binding where no GPU is: importing it, and what it refuses before a CUDA call."""
import os
import subprocess
import sys

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
