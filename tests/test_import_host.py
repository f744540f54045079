"""Importing the package in surroundings that its calls could not run in."""
import os
import subprocess
import sys

from sparse_long_context_02_b200 import build as dsa_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _run(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return r.stdout


def test_import_where_torch_has_no_cuda_bindings():
    """A torch built without CUDA has no torch._C._cuda_*: the import, the host
    functions and the refusals of host tensors work there."""
    dsa_build.build()
    out = _run("""
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import sparse_long_context_02_b200 as dsa
f, m = dsa.rope_freqs(64, device="cpu")
assert f.numel() == 32 and m == 1.0
try:
    dsa.index_topk(torch.zeros((8, 4, 64), dtype=torch.uint8), torch.zeros((8, 64)), None, 4)
except ValueError as e:
    print(e)
""")
    assert "CUDA tensor" in out
