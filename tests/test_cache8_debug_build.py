"""The 8-bit cache on the bounds-checked build (libbkv_debug.so): its kernels guard
the indices that come from data, and no guard fires on the cases of the other tests
(one that did would turn the device status, which every case asserts to be clean, into
BKV_ERR_DEVICE_ASSERT)."""
import glob
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "kv_cache_compression_bkv_b200", "csrc")
CASES = [
    "test_cache8_gpu.py::test_append",
    "test_cache8_gpu.py::test_attend",
    "test_cache8_gpu.py::test_attend_split_over_every_cta",
    "test_cache8_gpu.py::test_attend_many_rows",
    "test_cache8_gpu.py::test_attend_many_segments_joined",
    "test_cache8_gpu.py::test_attend_nan_in_a_new_row_reaches_the_tokens_that_see_it",
    "test_cache8_gpu.py::test_attend_few_rows_on_cuda_cores",
    "test_cache8_gpu.py::test_attend_two_row_blocks",
    "test_cache8_gpu.py::test_attend_weights_of_many_rows",
    "test_cache8_gpu.py::test_evict",
    "test_cache8_gpu.py::test_evict_in_place",
    "test_cache8_gpu.py::test_decode_loop_with_eviction",
    "test_cache8_gpu.py::test_a_loop_without_a_pause",
    "test_cache8_nan_gpu.py",
]


def test_every_kernel_file_guards_its_indices():
    """Each file of kernels has guards, with tags of their own."""
    seen = {}
    files = [f for f in glob.glob(os.path.join(CSRC, "cache8_*.cu")) if "__global__" in open(f).read()]
    assert len(files) >= 5
    for f in files:
        text = re.sub(r"//[^\n]*", "", open(f).read())
        tags = set(re.findall(r"BKV_CHECK\([^;{]*?,\s*(\d+)\)", text))
        assert tags, f
        for t in tags:
            assert seen.setdefault(t, f) == f, (t, f, seen[t])


@pytest.mark.gpu
def test_cases_on_the_debug_build():
    lib = os.path.join(ROOT, "kv_cache_compression_bkv_b200", "libbkv_debug.so")
    if not os.path.exists(lib):
        pytest.skip("libbkv_debug.so is not built")
    env = dict(os.environ, BKV_LIBRARY="debug")
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
           *[os.path.join(ROOT, "tests", c) for c in CASES]]
    r = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=1200)
    tail = "\n".join((r.stdout + r.stderr).splitlines()[-30:])
    assert r.returncode == 0, tail
    assert " passed" in r.stdout, tail
