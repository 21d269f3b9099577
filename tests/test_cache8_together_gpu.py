"""Calls of the 8-bit cache side by side, and at the limits of its geometry."""
import math

import pytest
import torch

import cache8_helpers as ref
from test_cache8_gpu import DT, POISON, Dev, bkv, check_clean, gen, i32, run_attend, same

pytestmark = pytest.mark.gpu


class Loop:
    """A cache with a prompt in it, and one step of a padded batch: append, attend with
    weights, evict to another buffer."""

    def __init__(self, seed, dtype, Hq, H, d, T, lens):
        S, cap, block = len(lens), 1024, 32
        g = gen(seed)
        self.dtype, self.T, self.cap = dtype, T, cap
        self.dev, self.dst = (Dev(S, Hq, H, cap, d, block, dtype) for _ in range(2))
        k, v = (torch.randn(S, H, cap, d, generator=g).to(DT[dtype]).cuda() for _ in range(2))
        self.n_new = i32([max(T - 3 * i, 1) for i in range(S)])
        bkv.bkv_cache8_append(self.dev.geom, *self.dev.bufs, i32(lens), k, v, cap, i32(lens))
        self.dev.weights.zero_()
        self.dev.weights.add_(torch.rand(S, H, cap, generator=g).cuda())
        self.lens = i32(lens) + self.n_new
        self.k, self.v = (torch.randn(S, H, T, d, generator=g).to(DT[dtype]).cuda() for _ in range(2))
        self.q = torch.randn(S, Hq, T, d, generator=g).to(DT[dtype]).cuda()
        self.out = torch.zeros_like(self.q)
        self.lse = torch.zeros(S, Hq, T, device="cuda")
        self.w = torch.zeros(S, H, cap, device="cuda")
        self.idx = torch.zeros(S, H, 300, dtype=torch.int32, device="cuda")
        self.kept = i32([0] * S)
        self.ws = [torch.empty(bkv.bkv_cache8_workspace_size(self.dev.geom, cap, *n), dtype=torch.uint8,
                               device="cuda") for n in ((T, 0, True), (0, 300, False))]
        self.stream = torch.cuda.Stream()

    def step(self, stream):
        d = self.dev
        bkv.bkv_cache8_append(d.geom, *d.bufs, self.lens, self.k, self.v, self.T, self.n_new, stream)
        bkv.bkv_cache8_attend(d.geom, *d.bufs, self.lens, self.cap, self.q, self.T, self.n_new, 0.0,
                              self.out, self.lse, d.weights, self.w, 0.5, self.ws[0], stream)
        bkv.bkv_cache8_evict(d.geom, *d.bufs, self.w, self.lens, self.cap, 300, 4, 40, self.dst.geom,
                             *self.dst.bufs, self.dst.weights, self.idx, self.kept, self.ws[1], stream)

    def results(self):
        return [t.clone() for t in (self.out, self.lse, self.w, self.idx, self.kept, self.dst.weights,
                                    *self.dev.bufs, *self.dst.bufs)]


@pytest.mark.parametrize("a,b", [
    (("bf16", 8, 2, 128, 50, [700, 133, 900]), ("bf16", 4, 2, 64, 300, [500, 700, 20])),
    (("bf16", 4, 2, 128, 128, [700, 133, 800]), ("f32", 4, 1, 96, 20, [500, 900, 20])),
    (("bf16", 8, 1, 64, 40, [700, 133, 800]), ("bf16", 4, 1, 128, 4, [500, 900, 20])),
])
def test_steps_on_two_streams(a, b):
    """Steps of every kind of kernel on two streams, many at once: the bits of the same
    steps one after another."""
    loops = [Loop(1000, *a), Loop(1001, *b)]
    want = []
    for x in loops:
        x.step(None)
        torch.cuda.synchronize()
        want.append(x.results())
        for t in (x.out, x.lse, x.w, x.idx, x.kept):
            t.zero_()
        for c in "kv":
            x.dst.codes[c].fill_(POISON)
            x.dst.scale[c].fill_(math.nan)
        x.dst.weights.fill_(math.nan)
    torch.cuda.synchronize()
    for _ in range(10):                              # a step gives the same again: the rows are there
        for x in loops:
            x.step(x.stream)
    torch.cuda.synchronize()
    check_clean()
    for x, w in zip(loops, want):
        for got, t in zip(x.results(), w):
            assert same(got, t)


@pytest.mark.parametrize("T", [1, 40])
def test_as_many_heads_as_are_allowed(T):
    """65535 caches of up to 16 rows in one call."""
    S, Hq, d, block, cap = 65535, 2, 64, 16, 16
    g = gen(1010)
    dev = Dev(S, Hq, 1, cap, d, block, "bf16")
    lens = torch.randint(0, cap + 1, (S,), generator=g)
    lens[:2], lens[-1] = torch.tensor([0, 16]), 16
    k, v = (torch.randn(S, 1, cap, d, generator=g).bfloat16() for _ in range(2))
    L = lens.int().cuda()
    bkv.bkv_cache8_append(dev.geom, *dev.bufs, L, k.cuda(), v.cuda(), cap, L)
    q = torch.randn(S, Hq, T, d, generator=g).bfloat16()
    n = torch.minimum(lens, torch.tensor(T))
    out = torch.zeros(S, Hq, T, d, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(S, 1, cap, device="cuda")
    ws = torch.empty(bkv.bkv_cache8_workspace_size(dev.geom, cap, T, 8, True), dtype=torch.uint8,
                     device="cuda")
    bkv.bkv_cache8_attend(dev.geom, *dev.bufs, L, cap, q.cuda(), T, n.int().cuda(), 0.0, out, None, None,
                          w, 1.0, ws)
    idx = torch.zeros(S, 1, 8, dtype=torch.int32, device="cuda")
    kept = torch.zeros(S, dtype=torch.int32, device="cuda")
    got_w = w.cpu()
    bkv.bkv_cache8_evict(dev.geom, *dev.bufs, w, L, cap, 8, 1, 2, dev.geom, *dev.bufs, w, idx, kept, ws)
    check_clean()
    out, idx = out.double().cpu(), idx.cpu()
    assert torch.equal(kept.cpu().long(), lens.clamp(max=8))
    # a sample of the sequences, the first and the last among them, against 64 bits
    for s in [0, 1, S - 1] + torch.randint(0, S, (400,), generator=g).tolist():
        Ls, ns = int(lens[s]), int(n[s])
        if Ls == 0:
            assert not bool(out[s].any())
            continue
        rc = ref.Cache(1, 1, cap, d, block)
        rc.append([Ls], [Ls], k[s:s + 1, :, :Ls], v[s:s + 1, :, :Ls])
        kv, vv = rc.values("k", 0, 0, Ls), rc.values("v", 0, 0, Ls)
        o, _, p = ref.attend(kv, vv, q[s, :, :ns], Ls, ns, 1 / math.sqrt(d))
        mag = (q[s, :, :ns].double().abs() @ kv.abs().T).amax() / math.sqrt(d)
        rel = 2 * (d + 4) * 2.0 ** -22 * float(mag) + 2.0 ** -19       # as derived in attend_bounds
        av = p @ vv.abs()
        tol = (rel + 2.0 ** -20 + 2.0 ** -11) * av + Ls * 448 * 2.0 ** -25 * float(rc.scale["v"].max())
        assert bool(((out[s, :, :ns] - o).abs() <= tol + ref.U_BF16 * (o.abs() + tol)).all()), s
        total = p.sum((0, 1))
        assert bool(((got_w[s, 0, :Ls].double() - total).abs() <=
                     rel * total + (2 * ns + 3) * ref.U_F32 * total + 2 * ns * 2.0 ** -126).all()), s
        m = min(Ls, 8)
        assert idx[s, 0, :m].tolist() == ref.kept_positions(got_w[s, 0], Ls, 8, 1, 2), s


@pytest.mark.parametrize("dtype,Hq,H,d", [("bf16", 5, 1, 128), ("bf16", 2, 2, 64), ("f32", 2, 1, 64)])
@pytest.mark.parametrize("L", [1, 31, 128, 129, 777])
def test_whole_prompts(dtype, Hq, H, d, L):
    """Attention of every token of what was just appended, weights included."""
    run_attend(dtype, 2, Hq, H, d, 32, L, [L, max(L // 2, 1)], [L, max(L // 2, 1)], "fresh", 1020 + L)
