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


S, HQ, H, D, CAP, BLOCK, T = 2, 4, 2, 64, 256, 32, 3
BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def tensors():
    """One call's tensors, on the host: no refused call looks at what they hold."""
    return dict(k8=torch.zeros(S, H, CAP, D, dtype=U8), v8=torch.zeros(S, H, CAP, D, dtype=U8),
                ks=torch.ones(S, H, CAP // BLOCK), vs=torch.ones(S, H, CAP // BLOCK),
                lens=torch.ones(S, dtype=I32), n_new=torch.ones(S, dtype=I32),
                k_new=torch.zeros(S, H, T, D, dtype=BF16), v_new=torch.zeros(S, H, T, D, dtype=BF16),
                q=torch.zeros(S, HQ, T, D, dtype=BF16), out=torch.zeros(S, HQ, T, D, dtype=BF16),
                lse=torch.zeros(S, HQ, T), w=torch.zeros(S, H, CAP),
                idx=torch.zeros(S, H, 8, dtype=I32), new_lens=torch.zeros(S, dtype=I32),
                ws=torch.zeros(1 << 20, dtype=U8))


def append(t):
    geom = bkv.geometry8_of(t["k8"], t["ks"], HQ, BF16)
    bkv.bkv_cache8_append(geom, t["k8"], t["v8"], t["ks"], t["vs"], t["lens"], t["k_new"],
                          t["v_new"], T, t["n_new"], 0)


def attend(t):
    geom = bkv.geometry8_of(t["k8"], t["ks"], HQ, BF16)
    bkv.bkv_cache8_attend(geom, t["k8"], t["v8"], t["ks"], t["vs"], t["lens"], CAP, t["q"], T,
                          t["n_new"], 0.0, t["out"], t["lse"], None, t["w"], 1.0, t["ws"], 0)


def evict(t):
    geom = bkv.geometry8_of(t["k8"], t["ks"], HQ, BF16)
    bkv.bkv_cache8_evict(geom, t["k8"], t["v8"], t["ks"], t["vs"], t["w"], t["lens"], CAP, 8, 1, 1,
                         geom, t["k8"], t["v8"], t["ks"], t["vs"], t["w"], t["idx"], t["new_lens"],
                         t["ws"], 0)


@pytest.fixture
def passed(monkeypatch):
    """The calls that get past the binding, which here end at a stand-in; the host,
    which tensors give as device -1, is the current device."""
    calls = []
    monkeypatch.setattr(bkv, "_current_device", lambda: -1, raising=False)
    for name in ("_APPEND8", "_ATTEND8", "_EVICT8"):
        monkeypatch.setattr(bkv, name, lambda *a, name=name: calls.append(name) or 0)
    return calls


@pytest.mark.parametrize("call", [append, attend, evict])
def test_takes_what_the_library_reads(call, passed):
    t = tensors()
    call(t)
    t["n_new"] = t["lse"] = t["idx"] = t["new_lens"] = None
    call(t)
    assert len(passed) == 2


@pytest.mark.parametrize("call,name,dtype", [
    (append, "lens", torch.int64), (append, "n_new", torch.int64), (append, "k_new", F32),
    (append, "v_new", torch.float16), (attend, "lens", torch.int64), (attend, "n_new", torch.int16),
    (attend, "q", F32), (attend, "out", F32), (attend, "lse", BF16), (attend, "w", BF16),
    (evict, "lens", torch.int64), (evict, "w", torch.float64), (evict, "idx", torch.int64),
    (evict, "new_lens", torch.int64)])
def test_refuses_another_type(call, name, dtype, passed):
    t = tensors()
    t[name] = t[name].to(dtype)
    with pytest.raises(TypeError, match="weights" if name == "w" else name):
        call(t)
    assert not passed


@pytest.mark.parametrize("call,name", [(append, "k_new"), (append, "v_new"), (attend, "q"),
                                       (attend, "out")])
def test_refuses_rows_in_another_order(call, name, passed):
    t = tensors()
    t[name] = t[name].transpose(1, 2).contiguous().transpose(1, 2)
    with pytest.raises(ValueError, match=name):
        call(t)
    assert not passed


def test_geometry_of_scales_that_do_not_fit():
    t = tensors()
    g = bkv.geometry8_of(t["k8"], t["ks"], HQ, BF16)
    assert (g.n_seqs, g.n_q_heads, g.n_kv_heads, g.head_dim, g.capacity, g.block) == (
        S, HQ, H, D, CAP, BLOCK)
    # 15 scales for 256 rows: a floor division gives blocks of 17, 250 // 15 ones of 16
    for codes, scales in ((t["k8"], torch.ones(S, H, 15)),
                          (t["k8"][:, :, :250].contiguous(), torch.ones(S, H, 15)),
                          (t["k8"], torch.ones(S, H, 0)), (t["k8"], torch.ones(S, 1, 8)),
                          (t["k8"], torch.ones(1, H, 8)), (t["k8"], torch.ones(S * H, 8)),
                          (t["k8"], torch.ones(S, 8, H).transpose(1, 2)),
                          (t["k8"].transpose(0, 1), torch.ones(H, S, 8))):
        with pytest.raises(ValueError):
            bkv.geometry8_of(codes, scales, HQ, BF16)
    for codes, scales in ((t["k8"].to(BF16), t["ks"]), (t["k8"], t["ks"].double())):
        with pytest.raises(TypeError):
            bkv.geometry8_of(codes, scales, HQ, BF16)


@pytest.mark.parametrize("call,name", [
    (append, "lens"), (append, "k_new"), (append, "k8"), (attend, "lens"), (attend, "q"),
    (attend, "k8"), (evict, "lens"), (evict, "k8")])
def test_refuses_another_device(call, name, passed):
    class Elsewhere(torch.Tensor):
        def get_device(self):
            return 5

    t = tensors()
    t[name] = t[name].as_subclass(Elsewhere)
    with pytest.raises(ValueError, match="the cache" if name == "k8" else name):
        call(t)
    assert not passed
