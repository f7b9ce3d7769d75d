"""The package imports where torch was built without CUDA, and its calls refuse with words."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_getDevice") or
             n.startswith("_cuda_getCurrentRawStream")]:
    delattr(torch._C, name)
import paged_block_sparse_vt_b200 as vt
one = torch.ones(1, dtype=torch.int32)
try:
    vt.vt_free_requests(torch.zeros((1, 2), dtype=torch.int32), one, one, one)
except vt.VtError as e:
    print("refused:", e)
"""


def test_import_and_refusal():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("refused:") and "CUDA" in r.stdout, r.stderr
