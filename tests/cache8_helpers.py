"""The 8-bit cache's operators in 64 bits, from their definitions, on the CPU.

Test infrastructure: it shares no code with the library.  Codes are bytes
(OCP FP8 E4M3), values code * scale with one power-of-two scale per block.
"""
from __future__ import annotations

import math

import torch

MIN_EXP = -117
U_BF16, U_F16, U_F32, U_E4M3 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24, 2.0 ** -4


def code_table() -> torch.Tensor:
    """The 256 values of E4M3, from the format's definition."""
    out = []
    for b in range(256):
        s, e, m = b >> 7, (b >> 3) & 15, b & 7
        v = math.nan if (e == 15 and m == 7) else (m / 8 * 2.0 ** -6 if e == 0
                                                   else (1 + m / 8) * 2.0 ** (e - 7))
        out.append(-v if s else v)
    return torch.tensor(out, dtype=torch.float64)


TABLE = code_table()


def decode(codes: torch.Tensor) -> torch.Tensor:
    return TABLE[codes.view(torch.uint8).cpu().long()]


def round_e4m3(x: torch.Tensor) -> torch.Tensor:
    """The E4M3 value nearest to x (|x| <= 448), ties to even; NaN stays."""
    a = x.abs()
    _, e = torch.frexp(a)                     # a = m 2^e, 1/2 <= m < 1
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.round(x / step) * step


def scale_for(amax: torch.Tensor) -> torch.Tensor:
    """The smallest power of two >= 2^-117 with amax <= 448 scale."""
    m, e = torch.frexp(amax.double())         # 448 = 0.875 * 2^9
    k = torch.where(m <= 0.875, e - 9, e - 8)
    k = torch.where(amax == 0, torch.full_like(k, MIN_EXP), k).clamp(min=MIN_EXP)
    return torch.exp2(k.double())


def finite_amax(x: torch.Tensor) -> torch.Tensor:
    return torch.where(torch.isfinite(x), x.abs(), 0.0).amax()


class Cache:
    """Values of one sequence's cache, per (KV head): code values and scales."""

    def __init__(self, S, H, cap, d, block):
        self.block = block
        self.code = {n: torch.zeros(S, H, cap, d, dtype=torch.float64) for n in "kv"}
        self.scale = {n: torch.ones(S, H, cap // block, dtype=torch.float64) for n in "kv"}

    def values(self, n, s, h, L):
        row = torch.arange(L) // self.block
        return self.code[n][s, h, :L] * self.scale[n][s, h][row, None]

    def append(self, lens, n_new, k_new, v_new):
        B = self.block
        for n, x in (("k", k_new.double()), ("v", v_new.double())):
            for s, (L, c) in enumerate(zip(lens, n_new)):
                for b in range((L - c) // B, -(-L // B) if c else 0):
                    r0, r1 = max(b * B, L - c), min((b + 1) * B, L)
                    for h in range(x.shape[1]):
                        new = x[s, h, r0 - (L - c):r1 - (L - c)]
                        want = scale_for(finite_amax(new))
                        if r0 > b * B:
                            was = self.scale[n][s, h, b]
                            want = torch.maximum(want, was)
                            old = self.code[n][s, h, b * B:r0]
                            self.code[n][s, h, b * B:r0] = round_e4m3(old * (was / want))
                        ok = torch.where(torch.isfinite(new), new, math.nan)
                        self.code[n][s, h, r0:r1] = round_e4m3(ok / want)
                        self.scale[n][s, h, b] = want


def attend(kval, vval, q, L, n, scale):
    """One KV head: q [G, n, d] -> out [G, n, d], lse [G, n], p [G, n, L]."""
    G, T, d = q.shape
    x = scale * (q.double() @ kval.T)                      # [G, n, L]
    j = torch.arange(L)
    for t in range(T):
        x[:, t, j >= L - n + t + 1] = -math.inf
    m = x.amax(-1, keepdim=True) if L else torch.full((G, T, 1), -math.inf, dtype=torch.float64)
    e = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    l = e.sum(-1, keepdim=True)
    p = e / torch.where(l == 0, 1.0, l)
    return p @ vval, (m + torch.log(l))[..., 0], p


def kept_positions(w, L, K, sink, recent):
    """Kept positions of a head of length L, ascending."""
    if L <= K:
        return list(range(L))
    mid = range(sink, L - recent)

    def key(j):
        x = float(w[j])
        return (-x if x == x else math.inf, j)             # NaN as -infinity

    order = sorted(mid, key=key)
    return sorted(list(range(sink)) + list(range(L - recent, L)) + order[:K - sink - recent])
