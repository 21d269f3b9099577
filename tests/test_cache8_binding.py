"""The 8-bit cache's Python binding on the host: what it takes of torch, and which
tensors it refuses before a pointer of theirs goes into the library."""
import os
import subprocess
import sys

import pytest
import torch

bkv = pytest.importorskip("kv_cache_compression_bkv_b200.bkv")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_imports_without_a_cuda_build_of_torch():
    """Such builds lack the private call that the current stream's handle comes from."""
    code = (
        "import torch\n"
        "if hasattr(torch._C, '_cuda_getCurrentRawStream'):\n"
        "    del torch._C._cuda_getCurrentRawStream\n"
        "from types import SimpleNamespace\n"
        "from kv_cache_compression_bkv_b200 import bkv\n"
        "torch.cuda.current_device = lambda: 3\n"
        "torch.cuda.current_stream = lambda d: SimpleNamespace(cuda_stream=1000 + d)\n"
        "assert bkv._stream(None) == 1003 and bkv._stream(7) == 7\n")
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT, timeout=300)
