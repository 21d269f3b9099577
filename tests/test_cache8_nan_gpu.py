"""Queries and keys that are not a number, and rows without a logit above -infinity:
what they may reach of the outputs and of the attention weights, on every kernel."""
import math

import pytest
import torch

import cache8_helpers as ref
from test_cache8_gpu import DT, Dev, bkv, check_clean, gen, i32, same

pytestmark = pytest.mark.gpu


def attend(dev, q, lens, n_new, T, w_in=None):
    """Outputs, lse and weights of one call, in 64 bits on the host."""
    S, Hq = q.shape[:2]
    H, cap = dev.codes["k"].shape[1:3]
    qd = q.cuda()
    out, lse = torch.full_like(qd, 7.0), torch.full((S, Hq, T), 7.0, device="cuda")
    w = torch.full((S, H, cap), 7.0, device="cuda")
    ws = torch.full((bkv.bkv_cache8_workspace_size(dev.geom, cap, T, 0, True),), 0xff,
                    dtype=torch.uint8, device="cuda")
    bkv.bkv_cache8_attend(dev.geom, *dev.bufs, i32(lens), cap, qd, T,
                          None if n_new is None else i32(n_new), 0.0, out, lse, w_in, w, 1.0, ws)
    check_clean()
    return out.double().cpu(), lse.double().cpu(), w.double().cpu()


CASES = [
    # dtype, Hq, H, d, block, T, lens, n_new: up to 32 rows a KV head (kept logits)
    ("f32", 4, 2, 96, 16, 5, [300, 40], None),
    ("f32", 1, 1, 128, 64, 3, [700, 3], [2, 3]),
    ("bf16", 2, 1, 64, 32, 3, [300, 40], None),
    ("bf16", 4, 1, 128, 64, 5, [700, 40], [5, 4]),
    ("bf16", 8, 2, 128, 16, 8, [133, 300], None),
    ("bf16", 8, 1, 64, 16, 4, [133, 300], None),
    # and more, where the products are formed again
    ("f32", 3, 1, 96, 16, 20, [300, 40], [20, 13]),
    ("bf16", 3, 1, 128, 64, 11, [300, 700], None),
    ("bf16", 2, 1, 64, 32, 100, [260, 900], [90, 100]),
    ("bf16", 2, 1, 128, 32, 150, [260, 900], None),
    ("bf16", 2, 1, 128, 32, 300, [300, 900], [300, 201]),
    ("bf16", 1, 1, 80, 32, 40, [100, 900], None),
]


def cache_of(dtype, Hq, H, d, block, lens, seed):
    S, cap = len(lens), (max(lens) + block - 1) // block * block
    rc = ref.Cache(S, H, cap, d, block)
    x = torch.randn(2, S, H, cap, d, generator=gen(seed))
    rc.append([cap] * S, [cap] * S, x[0], x[1])
    dev = Dev(S, Hq, H, cap, d, block, dtype)
    dev.fill(rc, lens)
    return dev, rc


@pytest.mark.parametrize("i", range(len(CASES)))
def test_nan_query_reaches_only_what_its_token_sees(i):
    """A NaN in one early token's query: its own output and lse, and the weights
    of the keys it sees; all else is the same bits as without."""
    dtype, Hq, H, d, block, T, lens, n_new = CASES[i]
    S, G = len(lens), Hq // H
    dev, _ = cache_of(dtype, Hq, H, d, block, lens, 600 + i)
    q = torch.randn(S, Hq, T, d, generator=gen(620 + i)).to(DT[dtype])
    q[..., 3] = 0.01                                 # never the largest of its row
    want = attend(dev, q, lens, n_new, T)
    hit, hit_w = torch.zeros(S, Hq, T, dtype=torch.bool), torch.zeros_like(want[2], dtype=torch.bool)
    for s, L in enumerate(lens):
        n = n_new[s] if n_new else T
        h, t = (s + 1) % Hq, min(1, n - 2)
        q[s, h, t, 3] = math.nan
        hit[s, h, t] = True
        hit_w[s, h // G, :L - n + t + 1] = True
    out, lse, w = attend(dev, q, lens, n_new, T)
    assert same(out, torch.where(hit[..., None], math.nan, want[0]))
    assert same(lse, torch.where(hit, math.nan, want[1]))
    assert bool(w[hit_w].isnan().all())
    assert same(w[~hit_w], want[2][~hit_w])


@pytest.mark.parametrize("i", range(len(CASES)))
def test_nan_key_reaches_only_the_tokens_that_see_it(i):
    """A NaN in the newest token's K row, which no other token sees: its outputs and
    lse, and the weights of that head, to all of which it adds."""
    dtype, Hq, H, d, block, T, lens, n_new = CASES[i]
    S, G = len(lens), Hq // H
    dev, rc = cache_of(dtype, Hq, H, d, block, lens, 640 + i)
    q = torch.randn(S, Hq, T, d, generator=gen(660 + i)).to(DT[dtype])
    want = attend(dev, q, lens, n_new, T)
    hit = torch.zeros(S, Hq, T, dtype=torch.bool)
    for s, L in enumerate(lens):
        n = n_new[s] if n_new else T
        dev.codes["k"][s, H - 1, L - 1, 5] = 0x7f    # the last token alone sees it
        hit[s, (H - 1) * G:, n - 1] = True
    out, lse, w = attend(dev, q, lens, n_new, T)
    assert same(out, torch.where(hit[..., None], math.nan, want[0]))
    assert same(lse, torch.where(hit, math.nan, want[1]))
    for s, L in enumerate(lens):
        assert bool(w[s, H - 1, :L].isnan().all())   # the last token sees every key
        assert same(w[s, :H - 1], want[2][s, :H - 1])


@pytest.mark.parametrize("i", range(len(CASES)))
def test_row_of_logits_below_the_range_adds_no_weight(i):
    """A token whose every logit lies below f32's range counts as one that sees
    nothing: zeros, an lse of -infinity, and nothing in the weights."""
    dtype, Hq, H, d, block, T, lens, n_new = CASES[i]
    S, G, cap = len(lens), Hq // H, (max(lens) + block - 1) // block * block
    rc = ref.Cache(S, H, cap, d, block)
    x = torch.randn(2, S, H, cap, d, generator=gen(680 + i))
    x[0, ..., 0] = -1.0e12                           # every key's first element
    rc.append([cap] * S, [cap] * S, x[0], x[1])
    dev = Dev(S, Hq, H, cap, d, block, dtype)
    dev.fill(rc, lens)
    q = torch.randn(S, Hq, T, d, generator=gen(690 + i)).to(DT[dtype])
    q[..., 0] = 0.0
    hit = torch.zeros(S, Hq, T, dtype=torch.bool)
    for s in range(S):
        n = n_new[s] if n_new else T
        h, t = (s + 1) % Hq, n - 1                   # the token that sees every key
        q[s, h, t] = 0.0
        q[s, h, t, 0] = 1.0e30                       # logits of -1e42 / sqrt(d)
        hit[s, h, t] = True
    out, lse, w = attend(dev, q, lens, n_new, T)
    assert bool((out[hit] == 0).all()) and bool((lse[hit] == -math.inf).all())
    for s, L in enumerate(lens):
        n = n_new[s] if n_new else T
        for h in range(H):
            # every other row's probabilities sum to one
            rows = int((~hit[s, h * G:(h + 1) * G, :n]).sum())
            total = float(w[s, h, :L].sum())
            assert math.isfinite(total)
            # each is off by its logits' rounding alone: twice (d + 4) 2^-22 times the
            # largest sum of magnitudes, and 2^-19, as derived in attend_bounds; the
            # large elements of K meet zeros there, and cost nothing
            mag = (q[s, h * G:(h + 1) * G, :n].double().abs()[..., 1:] @
                   rc.values("k", s, h, L)[:, 1:].abs().T).amax() / math.sqrt(d)
            tol = rows * (2 * (d + 4) * 2.0 ** -22 * float(mag) + 2.0 ** -19 + (L + G * n) * ref.U_F32)
            assert abs(total - rows) <= tol, (s, h, total, rows, tol)
