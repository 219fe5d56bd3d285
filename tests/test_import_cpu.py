"""The package on a PyTorch built without CUDA: it imports, and its calls on the host work."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import linear_attention_recurrence_chunk_gb300 as kda
assert kda.kda_kv4_cache(4, 2, 32, 64, device="cpu").shape == (4, 2, 2, 17 * 64)
assert kda.kda_kv4_attention_workspace_size(3, 3, 8, 2, 128, 1, torch.bfloat16) > 0
assert kda.kda_chunk_fwd_workspace_size(1, 64, 2, 128, 128, 1, torch.bfloat16) > 0
try:
    kda.kda_kv4_gather(torch.zeros(2, 1, 4, 17 * 128, dtype=torch.uint8), torch.zeros(4, dtype=torch.int32))
except ValueError:
    print("fine")
"""


def test_imports_without_cuda_in_torch():
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr
