"""The 8-bit cache's entry points on the host: what they refuse before anything
is launched, the workspace sizes, and the 64-bit definitions that the GPU tests
compare with.  Every rejected call fails a host-side check, so no CUDA call is
made; the pointers are fake addresses that are never dereferenced."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import cache8_helpers as ref

bkv = pytest.importorskip("kv_cache_compression_bkv_b200.bkv")
LIB = bkv.LIB
OK, INVALID, UNSUPPORTED, WORKSPACE, CUDA = 0, 1, 2, 3, 4
GB = 1 << 30
# fake, well separated, aligned device addresses
(K8, V8, KS, VS, LENS, KN, VN, NN, Q, OUT, LSE, WIN, WOUT, WS, KD, VD, KSD, VSD, WD, IDX,
 NL) = [(i + 1) * GB for i in range(21)]


def desc(S=2, Hq=8, Hkv=2, d=128, cap=1024, block=64, dt=bkv.BKV_BF16):
    return bkv.Cache8Desc(S, Hq, Hkv, d, cap, block, dt)


BAD_DESCS = [
    (desc(S=0), INVALID), (desc(Hq=7), INVALID), (desc(Hkv=0), INVALID), (desc(d=0), INVALID),
    (desc(d=72), INVALID), (desc(d=144), UNSUPPORTED), (desc(block=8), INVALID),
    (desc(block=48), INVALID), (desc(block=0), INVALID), (desc(cap=1000), INVALID),
    (desc(cap=0), INVALID), (desc(dt=5), INVALID), (desc(S=40000), INVALID),
    (desc(S=60, cap=1 << 28), INVALID),
]


def append(d, k8=K8, v8=V8, ks=KS, vs=VS, lens=LENS, kn=KN, vn=VN, T=1, nn=None):
    return LIB.bkv_cache8_append(ctypes.byref(d) if d else None, k8, v8, ks, vs, lens, kn, vn, T,
                                 nn, None)


def attend(d, k8=K8, v8=V8, ks=KS, vs=VS, lens=LENS, max_len=1000, q=Q, T=1, nn=None, scale=0.0,
           out=OUT, lse=LSE, win=WIN, wout=WOUT, decay=1.0, ws=WS, ws_bytes=GB):
    return LIB.bkv_cache8_attend(ctypes.byref(d) if d else None, k8, v8, ks, vs, lens, max_len, q,
                                 T, nn, scale, out, lse, win, wout, decay, ws, ws_bytes, None)


def evict(d, k8=K8, v8=V8, ks=KS, vs=VS, w=WIN, lens=LENS, max_len=1000, K=256, sink=4, recent=32,
          dst=None, kd=KD, vd=VD, ksd=KSD, vsd=VSD, wd=WD, idx=IDX, nl=NL, ws=WS, ws_bytes=GB):
    dst = dst or desc(cap=256)
    return LIB.bkv_cache8_evict(ctypes.byref(d) if d else None, k8, v8, ks, vs, w, lens, max_len,
                                K, sink, recent, ctypes.byref(dst), kd, vd, ksd, vsd, wd, idx, nl,
                                ws, ws_bytes, None)


@pytest.mark.parametrize("i", range(len(BAD_DESCS)))
def test_bad_geometry(i):
    d, want = BAD_DESCS[i]
    assert append(d) == want
    assert attend(d) == want
    if d.dtype == bkv.BKV_BF16 and want == INVALID:
        assert evict(d) == want
    assert LIB.bkv_cache8_workspace_size(ctypes.byref(d), 64, 1, 64, 1) == 0


def test_row_limit():
    """Positions stay in 32 bits with room for what a kernel rounds up to."""
    most = (1 << 31) - 65536
    assert evict(desc(S=1, Hq=1, Hkv=1, cap=most + 64, block=64), max_len=most + 64) == INVALID
    d = desc(S=1, Hq=1, Hkv=1, cap=most, block=64)
    assert LIB.bkv_cache8_workspace_size(ctypes.byref(d), most, 1, 0, 0) > 0
    d = desc(S=2, Hq=1, Hkv=1, cap=most, block=64)
    assert LIB.bkv_cache8_workspace_size(ctypes.byref(d), most, 1, 0, 0) == 0


def test_null_desc():
    assert append(None) == attend(None) == evict(None) == INVALID
    assert LIB.bkv_cache8_workspace_size(None, 64, 1, 64, 1) == 0


@pytest.mark.parametrize("bad", [
    dict(k8=0), dict(v8=0), dict(ks=0), dict(vs=0), dict(lens=0), dict(kn=0), dict(vn=0),
    dict(T=0), dict(T=-1), dict(T=1025), dict(k8=K8 + 8), dict(v8=V8 + 4), dict(ks=KS + 2),
    dict(vs=VS + 1), dict(lens=LENS + 2), dict(kn=KN + 8), dict(vn=VN + 2), dict(nn=NN + 1),
    dict(v8=K8), dict(v8=K8 + 512 * 1024 - 16), dict(kn=K8), dict(vn=V8 + 16), dict(vs=KS),
    dict(ks=K8 + 64), dict(lens=KS), dict(nn=VS),
])
def test_append_refuses(bad):
    assert append(desc(), **bad) == INVALID


@pytest.mark.parametrize("bad", [
    dict(k8=0), dict(v8=0), dict(ks=0), dict(vs=0), dict(lens=0), dict(q=0), dict(out=0),
    dict(T=0), dict(T=1 << 23), dict(max_len=0), dict(max_len=1025), dict(scale=-1.0),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(decay=float("nan")),
    dict(decay=float("inf")), dict(win=WIN, wout=0), dict(q=Q + 8), dict(out=OUT + 2),
    dict(lse=LSE + 2), dict(win=WIN + 4), dict(wout=WOUT + 8), dict(nn=NN + 2),
    dict(out=Q), dict(out=K8), dict(out=V8 + 64), dict(lse=OUT), dict(wout=KS), dict(wout=K8),
    dict(win=WIN, wout=WIN + 16), dict(ws=OUT), dict(ws=K8), dict(wout=Q), dict(lse=LENS),
])
def test_attend_refuses(bad):
    assert attend(desc(), **bad) == INVALID


def test_attend_workspace():
    d = desc()
    need = LIB.bkv_cache8_workspace_size(ctypes.byref(d), 1000, 1, 0, 1)
    assert need > 0
    for bad in (dict(ws=0), dict(ws=WS + 8), dict(ws_bytes=need - 1), dict(ws_bytes=0)):
        assert attend(d, **bad) == WORKSPACE


@pytest.mark.parametrize("bad", [
    dict(k8=0), dict(v8=0), dict(ks=0), dict(vs=0), dict(w=0), dict(lens=0), dict(kd=0),
    dict(vd=0), dict(ksd=0), dict(vsd=0), dict(max_len=0), dict(max_len=1025), dict(K=0),
    dict(K=-1), dict(K=1 << 31), dict(sink=-1), dict(recent=-1), dict(sink=200, recent=57),
    dict(dst=desc(cap=192)), dict(dst=desc(S=1, cap=256)), dict(dst=desc(Hq=4, Hkv=1, cap=256)),
    dict(dst=desc(d=64, cap=256)), dict(dst=desc(cap=256, block=32)), dict(dst=desc(cap=250)),
    dict(k8=K8 + 8), dict(kd=KD + 4), dict(w=WIN + 4), dict(wd=WD + 8), dict(idx=IDX + 2),
    dict(nl=NL + 1), dict(kd=K8), dict(kd=K8, vd=V8), dict(vd=KD), dict(wd=WIN), dict(idx=WIN),
    dict(nl=IDX), dict(ws=KD), dict(ksd=KS), dict(idx=LENS),
    # in place with one of the five elsewhere, or another capacity
    dict(kd=K8, vd=V8, ksd=KS, vsd=VSD, dst=desc()),
    dict(kd=K8, vd=V8, ksd=KS, vsd=VS, dst=desc(cap=512)),
    dict(kd=K8, vd=V8, ksd=KS, vsd=VS, dst=desc(), wd=WIN + 16),
])
def test_evict_refuses(bad):
    assert evict(desc(), **bad) == INVALID


def test_evict_workspace():
    d = desc()
    need = LIB.bkv_cache8_workspace_size(ctypes.byref(d), 1000, 0, 256, 0)
    assert need > 0
    for bad in (dict(ws=0), dict(ws=WS + 8), dict(ws_bytes=0), dict(idx=0, ws_bytes=need - 1)):
        assert evict(d, **bad) == WORKSPACE


def test_workspace_size():
    d = desc()
    f = lambda *a: LIB.bkv_cache8_workspace_size(ctypes.byref(d), *a)  # noqa: E731
    for bad in ((0, 1, 1, 0), (1025, 1, 1, 0), (8, -1, 1, 0), (8, 1, -1, 0), (8, 1 << 23, 1, 0),
                (8, 1, 1 << 31, 0), (8, 0, 0, 0)):
        assert f(*bad) == 0
    assert f(1000, 1, 0, 1) >= f(1000, 1, 0, 0) > 0
    assert f(1000, 1, 512, 0) >= f(1000, 0, 512, 0) > 0


def test_injected_launch_failure():
    """With the fault injection on, valid calls report the failed launch."""
    code = (
        "import test_cache8_abi as t\n"
        "assert t.append(t.desc()) == t.CUDA\n"
        "assert t.attend(t.desc()) == t.CUDA\n"
        "assert t.evict(t.desc()) == t.CUDA\n"
        "same = dict(kd=t.K8, vd=t.V8, ksd=t.KS, vsd=t.VS, wd=t.WIN, nl=t.LENS, dst=t.desc())\n"
        "assert t.evict(t.desc(), **same) == t.CUDA\n")
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, BKV_INJECT_LAUNCH_FAILURE="1",
               PYTHONPATH=os.pathsep.join([here, os.path.dirname(here)]))
    subprocess.run([sys.executable, "-c", code], check=True, env=env, timeout=300)


def test_reference_rounding_matches_the_format():
    """The helpers' E4M3 rounding against every code, every midpoint between
    neighbours (ties to even) and torch's cast."""
    pos = ref.TABLE[:127]
    assert torch.equal(ref.round_e4m3(pos), pos)
    mid = (pos[1:] + pos[:-1]) / 2
    even = torch.where(torch.arange(126) % 2 == 0, pos[:-1], pos[1:])
    assert torch.equal(ref.round_e4m3(mid), even)
    x = torch.randn(4096, generator=torch.Generator().manual_seed(1)) * 60
    x = x.clamp(-448, 448)
    assert torch.equal(ref.round_e4m3(x.double()), x.to(torch.float8_e4m3fn).double())
    assert torch.equal(torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
                       .nan_to_num(-9), ref.TABLE.nan_to_num(-9))


def test_reference_scale():
    for a, want in ((448.0, 1.0), (448.1, 2.0), (224.0, 0.5), (224.1, 1.0), (0.0, 2.0 ** -117),
                    (1e-45, 2.0 ** -117), (3.4028234e38, 2.0 ** 120), (1.75 * 2.0 ** 127, 2.0 ** 119)):
        got = float(ref.scale_for(torch.tensor(a, dtype=torch.float64)))
        assert got == want, (a, got, want)
