"""Attention over blocks whose scales lie far apart, against 64 bits: what a token
does not see, or gives no probability, costs it no bits."""
import math

import pytest
import torch

import cache8_helpers as ref
from test_cache8_gpu import DT, Dev, bkv, check_clean, gen, i32

pytestmark = pytest.mark.gpu


def attend(dev, q, lens, n_new, T):
    """Outputs, lse and weights of one call, in 64 bits on the host."""
    S, Hq = q.shape[:2]
    H, cap = dev.codes["k"].shape[1:3]
    qd = q.cuda()
    out, lse = torch.full_like(qd, 7.0), torch.full((S, Hq, T), 7.0, device="cuda")
    w = torch.full((S, H, cap), 7.0, device="cuda")
    ws = torch.full((bkv.bkv_cache8_workspace_size(dev.geom, cap, T, 0, True),), 0xff,
                    dtype=torch.uint8, device="cuda")
    bkv.bkv_cache8_attend(dev.geom, *dev.bufs, i32(lens), cap, qd, T,
                          None if n_new is None else i32(n_new), 0.0, out, lse, None, w, 1.0, ws)
    check_clean()
    return out.double().cpu(), lse.double().cpu(), w.double().cpu()


def check(rc, dtype, q, lens, n_new, T, got, tokens=None):
    """Outputs, lse and weights of the tokens t < tokens (all of them: None).

    A token's bounds come from the keys that it sees.  A logit is a sum of d products
    in 32 bits, off by at most 2^-22 of the sum of magnitudes at each step, and three
    roundings; exp makes of it twice that, relative, in p (numerator and sum), ex2 and
    the sums over keys add 2^-19.  With bf16 the second product's operand is p times
    the V scale, in f16 with 11 bits under a reference per row that leaves the largest
    at 2^6 or above: 2^-11 relative, and half of f16's smallest step, 2^-25, against
    that 2^6, times a code of at most 448.  p itself may flush to zero below 2^-126
    of a reference that the largest p is at most 2^15 above and 2^7 below."""
    out, lse, w = got
    S, Hq, _, d = q.shape
    H = rc.code["k"].shape[1]
    G, u, sc = Hq // H, ref.U_BF16 if dtype == "bf16" else ref.U_F32, 1.0 / math.sqrt(q.shape[3])
    for s, L in enumerate(lens):
        n = T if n_new is None else n_new[s]
        for h in range(H):
            kv, vv = rc.values("k", s, h, L), rc.values("v", s, h, L)
            vs = rc.scale["v"][s, h][torch.arange(L) // rc.block]
            qh = q[s, h * G:(h + 1) * G, :n]
            o, z, p = ref.attend(kv, vv, qh, L, n, sc)
            see = torch.arange(L) <= L - n + torch.arange(n)[:, None]          # [n, L]
            mag = torch.where(see, sc * (qh.double().abs() @ kv.abs().T), 0.0)
            rel = 2 * (d + 4) * 2.0 ** -22 * mag.amax(-1, keepdim=True) + 2.0 ** -19
            av = p @ vv.abs()
            top = (p * vs).amax(-1, keepdim=True)
            far = torch.where(see, vs, 0.0).amax(-1, keepdim=True)[None]
            tol = (rel + 2.0 ** -20) * av + L * 448 * 2.0 ** -126 * 2.0 ** 15 * far
            if dtype == "bf16":
                tol = tol + 2.0 ** -11 * av + L * 448 * 2.0 ** -31 * top
            m = n if tokens is None else tokens
            got_o = out[s, h * G:(h + 1) * G, :n]
            err = (got_o - o).abs() - (tol + u * (o.abs() + tol))
            assert bool((err[:, :m] <= 0).all()), (s, h, float(err[:, :m].max()),
                                                   float((got_o - o).abs()[:, :m].max()))
            err = (lse[s, h * G:(h + 1) * G, :n] - z).abs() - (rel[..., 0] + 2.0 ** -20 +
                                                              4 * ref.U_F32 * z.abs())
            assert bool((err[:, :m] <= 0).all()), (s, h, float(err[:, :m].max()))
            if tokens is None:
                tol = (rel * p).sum((0, 1)) + (G * n + 3) * ref.U_F32 * p.sum((0, 1)) + G * n * 2.0 ** -126
                assert bool(((w[s, h, :L] - p.sum((0, 1))).abs() <= tol).all()), (s, h)


# lengths that leave a few rows to a last block inside a tile of 128 keys
KERNELS = [
    # dtype, Hq, H, d, block, T, lens: every kernel and its row blocks
    ("bf16", 4, 1, 128, 16, 1, [961, 97]),
    ("bf16", 10, 2, 64, 32, 1, [961, 97]),
    ("bf16", 8, 1, 128, 16, 2, [961, 97]),
    ("bf16", 4, 1, 128, 64, 6, [961, 65]),
    ("bf16", 4, 1, 128, 16, 8, [961, 97]),
    ("bf16", 4, 1, 64, 16, 8, [961, 97]),
    ("f32", 2, 1, 128, 16, 1, [961, 97]),
    ("f32", 4, 1, 96, 16, 5, [961, 97]),
]

MANY = [
    ("bf16", 40, 1, 128, 16, 1, [961, 97]),
    ("bf16", 2, 1, 128, 16, 40, [961, 97]),
    ("bf16", 4, 2, 64, 32, 50, [961, 97]),
    ("bf16", 2, 1, 128, 16, 100, [961, 225]),
    ("bf16", 1, 1, 64, 64, 200, [961, 321]),
    ("bf16", 2, 1, 128, 16, 200, [961, 225]),
    ("bf16", 3, 1, 64, 16, 120, [2001, 225]),
]


def cache_with_a_heavy_block(Hq, H, d, block, T, lens, dtype, r, seed, at):
    """Queries of which one block of keys, `at`, gets nearly all; its V lie 2^-r under
    the others'."""
    S, cap = len(lens), (max(lens) + block - 1) // block * block
    g = gen(seed)
    x = torch.randn(2, S, H, cap, d, generator=g)
    liked = torch.nn.functional.normalize(torch.randn(d, generator=g), dim=0)
    x[0] *= 0.05
    x[0, :, :, at * block:(at + 1) * block] += 40.0 * liked
    x[1, :, :, at * block:(at + 1) * block] *= 2.0 ** -r
    rc = ref.Cache(S, H, cap, d, block)
    rc.append([cap] * S, [cap] * S, x[0], x[1])
    dev = Dev(S, Hq, H, cap, d, block, dtype)
    dev.fill(rc, lens)
    q = (20.0 * liked + 0.2 * torch.randn(S, Hq, T, d, generator=g)).to(DT[dtype])
    return dev, rc, q


def run_heavy(i, case, r):
    dtype, Hq, H, d, block, T, lens = case
    for at in (0, 1, (lens[1] - T) // block - 1):   # first, inside a tile, towards the end
        dev, rc, q = cache_with_a_heavy_block(Hq, H, d, block, T, lens, dtype, r, 40 + i, max(at, 0))
        check(rc, dtype, q, lens, None, T, attend(dev, q, lens, None, T))


def run_hidden(i, case, r):
    """The newest block's V (K) 2^r above the others': of no concern to the tokens before it."""
    dtype, Hq, H, d, block, T, lens = case
    if T < 2:
        return
    S, cap = len(lens), (max(lens) + block - 1) // block * block
    for which in (1, 0):
        g = gen(60 + i)
        rc = ref.Cache(S, H, cap, d, block)
        x = torch.randn(2, S, H, cap, d, generator=g)
        rc.append([cap] * S, [cap] * S, x[0], x[1])
        fresh = min(block, T - 1)
        for s, L in enumerate(lens):                # the last rows of each, in a block of their own
            b0 = -(-(L - fresh) // block)
            rows, name = slice(b0 * block, L), "kv"[which]
            assert b0 * block < L
            for h in range(H):
                y = x[which, s, h, rows] * 2.0 ** r
                rc.scale[name][s, h, b0] = ref.scale_for(y.abs().amax())
                rc.code[name][s, h, rows] = ref.round_e4m3(y.double() / rc.scale[name][s, h, b0])
        dev = Dev(S, Hq, H, cap, d, block, dtype)
        dev.fill(rc, lens)
        q = torch.randn(S, Hq, T, d, generator=g).to(DT[dtype])
        # the tokens before the newest rows; the others' logits pass every bound (K)
        check(rc, dtype, q, lens, None, T, attend(dev, q, lens, None, T),
              tokens=T - fresh if which == 0 else None)


@pytest.mark.parametrize("r", [16, 20, 28, 40, 80])
@pytest.mark.parametrize("i", range(len(KERNELS)))
def test_heavy_block_of_small_v(i, r):
    run_heavy(i, KERNELS[i], r)


@pytest.mark.parametrize("r", [16, 20, 28, 40, 80, 120])
@pytest.mark.parametrize("i", range(len(KERNELS)))
def test_large_block_that_only_later_tokens_see(i, r):
    run_hidden(i, KERNELS[i], r)


@pytest.mark.parametrize("r", [16, 20, 28, 40, 80])
@pytest.mark.parametrize("i", range(len(MANY)))
def test_heavy_block_of_small_v_many_rows(i, r):
    run_heavy(20 + i, MANY[i], r)


@pytest.mark.parametrize("r", [16, 20, 28, 40, 80, 120])
@pytest.mark.parametrize("i", range(len(MANY)))
def test_large_block_that_only_later_tokens_see_many_rows(i, r):
    run_hidden(20 + i, MANY[i], r)


@pytest.mark.parametrize("i", range(len(KERNELS + MANY)))
def test_logits_of_zero_under_factors_past_the_range(i):
    """K and queries whose scales multiply past f32's range, in elements that do not
    meet: logits of zero, and the average of V."""
    dtype, Hq, H, d, block, T, lens = (KERNELS + MANY)[i]
    S, cap = len(lens), (max(lens) + block - 1) // block * block
    g = gen(100 + i)
    rc = ref.Cache(S, H, cap, d, block)
    x = torch.randn(2, S, H, cap, d, generator=g)
    x[0, ..., d // 2:] = 0.0
    x[0] *= 2.0 ** 122
    rc.append([cap] * S, [cap] * S, x[0], x[1])
    dev = Dev(S, Hq, H, cap, d, block, dtype)
    dev.fill(rc, lens)
    q = torch.randn(S, Hq, T, d, generator=g) * 2.0 ** 90
    q[..., :d // 2] = 0.0
    q = q.to(DT[dtype])
    check(rc, dtype, q, lens, None, T, attend(dev, q, lens, None, T))


@pytest.mark.parametrize("mag", [2.0e38, 1.0e-34])
@pytest.mark.parametrize("i", range(len(KERNELS + MANY)))
def test_values_at_the_ends_of_the_range(i, mag):
    """Sums of many values of which a few pass f32's range, or lie at its lower end:
    the outputs are averages, and lie within."""
    dtype, Hq, H, d, block, T, lens = (KERNELS + MANY)[i]
    S, cap = len(lens), (max(lens) + block - 1) // block * block
    g = gen(80 + i)
    rc = ref.Cache(S, H, cap, d, block)
    x = torch.randn(2, S, H, cap, d, generator=g)
    x[1] = mag * (0.5 + 0.5 * torch.rand(S, H, cap, d, generator=g))
    rc.append([cap] * S, [cap] * S, x[0], x[1])
    dev = Dev(S, Hq, H, cap, d, block, dtype)
    dev.fill(rc, lens)
    q = torch.randn(S, Hq, T, d, generator=g).to(DT[dtype])
    check(rc, dtype, q, lens, None, T, attend(dev, q, lens, None, T))
