"""The binding loads, makes configurations and checks arguments on a torch that
was built without CUDA. CPU only."""
import os
import subprocess
import sys

from route_permute_grouped_gb300 import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import torch
for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, n):
        delattr(torch._C, n)
from route_permute_grouped_gb300 import ops
cfg = ops.make_adapter_config(4, 64, 64, 2, 8)
assert ops.alloc_adapter_saved(cfg, "cpu").numel() == 4 * 16 * 6
try:
    ops.adapter_plan(cfg, torch.zeros(4, dtype=torch.int32))
except ops.MoeError as e:
    print("refused:", e)
"""


def test_imports_without_cuda_in_torch():
    B.build()
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.startswith("refused:") and "CUDA device" in r.stdout, r.stderr
