"""What the window cache, the decode step and the binding refuse on the host, with CPU tensors; and that the binding
loads where torch lacks its private names."""
import os
import subprocess
import sys

import pytest
import torch

from sparse_kv_cache_memoryindexer_b200 import lsa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_binding_loads_without_torchs_private_names():
    code = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from sparse_kv_cache_memoryindexer_b200 import lsa
assert lsa._current_device is torch.cuda.current_device
class S:
    cuda_stream = 1234
torch.cuda.current_stream = lambda dev: S if dev == 3 else None
assert lsa._raw_stream(3) == 1234
print("loaded")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "loaded" in r.stdout, r.stderr[-2000:]
