"""The 8-bit cache on a B200 against its 64-bit definitions (cache8_helpers).

Codes, scales, positions and lengths have to be equal.  Attention's tolerance
is derived per element from the inputs (see `attend_bounds`)."""
import math

import pytest
import torch

import cache8_helpers as ref

pytestmark = pytest.mark.gpu
bkv = pytest.importorskip("kv_cache_compression_bkv_b200.bkv")

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
POISON = 0x7f  # a NaN code


def gen(seed):
    return torch.Generator().manual_seed(seed)


class Dev:
    """A cache on the device with stale NaN codes and NaN scales everywhere."""

    def __init__(self, S, Hq, H, cap, d, block, dtype):
        dev = "cuda"
        self.codes = {n: torch.full((S, H, cap, d), POISON, dtype=torch.uint8, device=dev) for n in "kv"}
        self.scale = {n: torch.full((S, H, cap // block), math.nan, device=dev) for n in "kv"}
        self.geom = bkv.geometry8_of(self.codes["k"], self.scale["k"], Hq, DT[dtype])
        self.weights = torch.full((S, H, cap), math.nan, device=dev)

    @property
    def bufs(self):
        return self.codes["k"], self.codes["v"], self.scale["k"], self.scale["v"]

    def fill(self, rcache, lens):
        """Rows below each length from the reference cache."""
        for n in "kv":
            for s, L in enumerate(lens):
                code = rcache.code[n][s, :, :L].float().to(torch.float8_e4m3fn).view(torch.uint8)
                self.codes[n][s, :, :L] = code.cuda()
                nb = -(-L // rcache.block)
                self.scale[n][s, :, :nb] = rcache.scale[n][s, :, :nb].float().cuda()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def same(got, want):
    got, want = got.double().cpu(), want.double().cpu()
    return torch.equal(got.nan_to_num(-12345.0), want.nan_to_num(-12345.0))


def check_clean():
    st, where = bkv.bkv_read_device_status()
    assert st == 0, (st, where)


# ----------------------------------------------------------------- append

def check_append(dev, rc, lens):
    for n in "kv":
        for s, L in enumerate(lens):
            nb = -(-L // rc.block)
            assert same(dev.scale[n][s, :, :nb], rc.scale[n][s, :, :nb]), (n, s)
            assert same(ref.decode(dev.codes[n][s, :, :L]), rc.code[n][s, :, :L]), (n, s)
            # nothing past the length was written
            assert bool((dev.codes[n][s, :, L:] == POISON).all())
            assert bool(dev.scale[n][s, :, nb:].isnan().all())


APPENDS = [
    # dtype, S, H, d, block, T, steps of new rows per sequence
    ("bf16", 3, 2, 128, 64, 1, [[1, 1, 1]] * 70),
    ("bf16", 2, 1, 64, 16, 40, [[40, 0], [3, 17], [16, 40], [1, 1]]),
    ("f32", 2, 2, 128, 128, 300, [[300, 129], [0, 128], [56, 1]]),
    ("f32", 1, 1, 16, 16, 33, [[33], [33], [1]]),
    ("bf16", 2, 3, 96, 32, 65, [[65, 31], [31, 1], [1, 33], [2, 64]]),
    ("bf16", 1, 1, 112, 128, 128, [[128], [128], [127]]),
    ("f32", 40, 1, 32, 32, 5, [[i % 6 for i in range(40)], [5] * 40, [1] * 40]),
]


@pytest.mark.parametrize("i", range(len(APPENDS)))
def test_append(i):
    dtype, S, H, d, block, T, steps = APPENDS[i]
    cap = 3 * 128 if T > 64 else 128
    g = gen(100 + i)
    dev, rc = Dev(S, H, H, cap, d, block, dtype), ref.Cache(S, H, cap, d, block)
    lens = [0] * S
    for step, n in enumerate(steps):
        lens = [a + b for a, b in zip(lens, n)]
        # magnitudes that rise and fall, so that scales have to grow, or not
        mag = 2.0 ** (6 * torch.rand(S, H, T, 1, generator=g) * (step % 4))
        k = (torch.randn(S, H, T, d, generator=g) * mag).to(DT[dtype])
        v = (torch.randn(S, H, T, d, generator=g) / mag).to(DT[dtype])
        full = all(x == T for x in n)
        bkv.bkv_cache8_append(dev.geom, *dev.bufs, i32(lens), k.cuda(), v.cuda(), T,
                              None if full else i32(n))
        rc.append(lens, n, k, v)
        check_append(dev, rc, lens)
    check_clean()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_values_at_the_borders(dtype):
    """Zeros, borders of the scale rule, subnormals, the type's largest values
    and elements that are not finite."""
    d, block = 16, 16
    big = torch.finfo(DT[dtype]).max
    tiny = torch.finfo(DT[dtype]).tiny
    rows = [[0.0], [448.0], [450.0], [447.0, 1e-3], [224.0], [225.0], [2.0 ** 20 * 1.75], [big],
            [big, 1.0], [tiny], [tiny * 2.0 ** -3], [math.inf, 1.0], [-math.inf], [math.nan, 3.0],
            [math.nan], [-0.0, 1.0], [1.75 * 2.0 ** -109, 2.0 ** -117], [0.4375 * 2.0 ** -116]]
    for row in rows:
        x = torch.zeros(1, 1, 16, d, dtype=DT[dtype])
        x[0, 0, 3, :len(row)] = torch.tensor(row, dtype=torch.float64).to(DT[dtype])
        x[0, 0, 7, 5] = x[0, 0, 3, 0] / 3
        dev, rc = Dev(1, 1, 1, 32, d, block, dtype), ref.Cache(1, 1, 32, d, block)
        bkv.bkv_cache8_append(dev.geom, *dev.bufs, i32([16]), x.cuda(), (-x).cuda(), 16)
        rc.append([16], [16], x, -x)
        check_append(dev, rc, [16])
    check_clean()


def test_append_refuses_bad_lengths_on_the_device():
    dev = Dev(5, 1, 1, 128, 16, 16, "f32")
    x = torch.ones(5, 1, 4, 16, device="cuda")
    lens, n = [3, 129, -1, 4, 8], [4, 1, 0, 5, -1]  # each is out of range
    bkv.bkv_cache8_append(dev.geom, *dev.bufs, i32(lens), x, x, 4, i32(n))
    st, where = bkv.bkv_read_device_status()
    assert (st, where) == (6, 601)
    assert bool((dev.codes["k"] == POISON).all()) and bool((dev.codes["v"] == POISON).all())
    assert bool(dev.scale["k"].isnan().all())
    check_clean()


# ----------------------------------------------------------------- attend

def attend_bounds(kval, vval, q, p, scale, dtype, d, vscale_max):
    """Error bounds (out, lse, p) of one KV head.

    A logit is a sum of d products in 32 bits; each step is off by at most
    2^-22 (an ulp where the tensor core truncates) of the sum of magnitudes,
    and scaling rounds three times.  exp turns a logit error into twice that,
    relative, in p (numerator and sum); ex2 and the sums add 2^-20.  With bf16
    the probabilities of the second product are rounded to f16: 2^-11 relative,
    and 2^-25 absolute against at most 448 * the largest V scale (the reference
    is within a factor 2^8 of the largest p).  Sums over keys: 2^-20.
    """
    mag = scale * (q.double().abs() @ kval.abs().T)              # [G, n, L]
    eps_x = (d + 4) * 2.0 ** -22 * mag
    rel = 2.0 * eps_x.amax(-1, keepdim=True) + 2.0 ** -19 if kval.shape[0] else torch.zeros(1)
    av = p @ vval.abs()
    out = rel * av + 2.0 ** -20 * av
    if dtype == "bf16":
        pmax = p.amax(-1, keepdim=True) if kval.shape[0] else torch.zeros(1)
        out = out + 2.0 ** -11 * av + 2.0 ** -25 * 448 * vscale_max * pmax * kval.shape[0]
    lse = (rel[..., 0] if kval.shape[0] else 0.0) + 2.0 ** -20
    return out, lse, rel * p


def run_attend(dtype, S, Hq, H, d, block, T, lens, n_new, weights, seed, decay=1.0, scale=0.0,
               shape_values=None, q_mag=1.0, with_lse=True, in_place=False, cap=None):
    g = gen(seed)
    cap = cap or (max(max(lens), 1) + block - 1) // block * block + block
    rc = ref.Cache(S, H, cap, d, block)
    x = torch.randn(2, S, H, cap, d, generator=g) * 2.0 ** (2 * torch.randn(2, S, H, cap, 1, generator=g))
    if shape_values is not None:
        shape_values(x)
    rc.append([cap] * S, [cap] * S, x[0], x[1])
    dev = Dev(S, Hq, H, cap, d, block, dtype)
    dev.fill(rc, lens)
    q = (q_mag * torch.randn(S, Hq, T, d, generator=g)).to(DT[dtype])
    for s, n in enumerate(n_new or []):
        q[s, :, n:] = math.nan                       # rows of nobody
    qd = q.cuda()
    out = torch.full((S, Hq, T, d), 7.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((S, Hq, T), 7.0, device="cuda") if with_lse else None
    w_in = w_out = None
    if weights:
        w0 = torch.rand(S, H, cap, generator=g)
        for s, L in enumerate(lens):
            n = T if n_new is None else n_new[s]
            w0[s, :, max(L - n, 0):] = math.nan      # rows that hold no weight yet
        w_in = w0.cuda() if weights != "fresh" else None
        w_out = w_in if in_place else torch.full((S, H, cap), 7.0, device="cuda")
    ml = max(max(lens), 1)
    need = bkv.bkv_cache8_workspace_size(dev.geom, ml, T, 0, bool(weights))
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    bkv.bkv_cache8_attend(dev.geom, *dev.bufs, i32(lens), ml, qd, T,
                          None if n_new is None else i32(n_new), scale, out, lse, w_in, w_out,
                          decay, ws)
    check_clean()
    u = ref.U_BF16 if dtype == "bf16" else ref.U_F32
    G = Hq // H
    sc = scale or 1.0 / math.sqrt(d)
    out, lse = out.double().cpu(), None if lse is None else lse.double().cpu()
    wo = w_out.double().cpu() if weights else None
    for s, L in enumerate(lens):
        n = T if n_new is None else n_new[s]
        assert bool((out[s, :, n:] == 7.0).all())
        if lse is not None:
            assert bool((lse[s, :, n:] == 7.0).all())
        if n == 0:
            if weights and not in_place:
                assert bool((wo[s] == 7.0).all())
            continue
        for h in range(H):
            kv, vv = rc.values("k", s, h, L), rc.values("v", s, h, L)
            qh = q[s, h * G:(h + 1) * G, :n]
            o, z, p = ref.attend(kv, vv, qh, L, n, sc)
            vmax = float(rc.scale["v"][s, h].max())
            bo, bz, bp = attend_bounds(kv, vv, qh, p, sc, dtype, d, vmax)
            got = out[s, h * G:(h + 1) * G, :n]
            err = (got - o).abs() - (bo + u * (o.abs() + bo))
            assert bool((err <= 0).all()), (s, h, float(err.max()))
            if lse is not None:
                gz = lse[s, h * G:(h + 1) * G, :n]
                empty = z == -math.inf
                assert bool((gz[empty] == -math.inf).all())
                tol = (bz + 4 * ref.U_F32 * z.abs())[~empty]
                assert bool(((gz - z)[~empty].abs() <= tol).all())
            if weights:
                total, tol = p.sum((0, 1)), bp.sum((0, 1))
                if weights != "fresh":
                    old = decay * w0[s, h, :L].double()
                    old[max(L - n, 0):] = 0
                    total = total + old
                # a sum of G n + 1 terms in 32 bits, and a probability under the
                # smallest normal float (2^-126) may count as zero: ex2 flushes
                # subnormal results, so each is off by less than 2^-126
                tol = tol + (G * n + 3) * ref.U_F32 * total + G * n * 2.0 ** -126
                assert bool(((wo[s, h, :L] - total).abs() <= tol).all()), (s, h)
                if not in_place:
                    assert bool((wo[s, h, L:] == 7.0).all())
    return dev


LENS = [0, 1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 640, 1000]
ATTENDS = [
    # dtype, S, Hq, H, d, block, T, lens, n_new, weights
    ("bf16", 14, 5, 1, 128, 64, 1, LENS, None, True),
    ("bf16", 14, 8, 8, 64, 16, 1, LENS, None, True),
    ("f32", 14, 4, 2, 64, 16, 1, LENS, None, True),
    ("f32", 3, 7, 1, 96, 32, 3, [2, 130, 300], None, True),
    ("bf16", 3, 3, 1, 96, 32, 3, [2, 130, 300], None, "fresh"),   # CUDA cores in bf16
    ("bf16", 4, 16, 2, 128, 32, 1, [1, 33, 500, 129], None, False),
    ("bf16", 5, 14, 2, 128, 128, 2, [0, 1, 2, 300, 129], None, True),   # rows that see nothing
    ("bf16", 5, 10, 2, 64, 64, 6, [9, 0, 700, 6, 130], [6, 3, 0, 5, 1], True),
    ("bf16", 2, 8, 1, 128, 64, 9, [200, 640], [9, 4], True),       # 72 rows: the keys again
    ("bf16", 2, 2, 1, 64, 16, 70, [300, 70], None, True),
    ("f32", 2, 2, 1, 64, 16, 70, [300, 70], [70, 41], True),
    ("f32", 2, 1, 1, 128, 128, 40, [40, 17], [40, 17], "fresh"),
    ("bf16", 1, 1, 1, 128, 16, 1, [1], None, True),
    ("bf16", 70, 4, 1, 64, 32, 1, [(37 * i) % 400 for i in range(70)], None, True),
    ("bf16", 70, 4, 1, 128, 32, 2, [0 if i % 3 else 5 * i for i in range(70)],
     [i % 3 for i in range(70)], True),
]


@pytest.mark.parametrize("i", range(len(ATTENDS)))
def test_attend(i):
    dtype, S, Hq, H, d, block, T, lens, n_new, weights = ATTENDS[i]
    run_attend(dtype, S, Hq, H, d, block, T, lens, n_new, weights, 200 + i,
               decay=0.75 if i % 2 else 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_split_over_every_cta(dtype):
    """One head over many CTAs, weights in place, no lse."""
    run_attend(dtype, 1, 3, 1, 128 if dtype == "bf16" else 64, 128, 1, [20011], None, True, 300,
               decay=0.5, with_lse=False, in_place=True)


def test_attend_large_logits():
    """Logits of several hundred: one key takes nearly everything, and the
    softmax reference moves along the cache."""
    run_attend("bf16", 2, 4, 1, 128, 64, 1, [700, 2000], None, True, 301, q_mag=20.0)
    run_attend("f32", 1, 4, 1, 64, 64, 1, [700], None, True, 302, q_mag=20.0)


def test_attend_v_scales_far_apart():
    """Blocks of V many binades apart, some all zero."""
    def shape(x):
        for b in range(0, x.shape[3], 16):
            x[1, :, :, b:b + 16] *= 0.0 if b % 80 == 0 else 2.0 ** ((b // 16 * 7) % 30 - 15)
    for dtype in ("bf16", "f32"):
        run_attend(dtype, 1, 4, 1, 128, 16, 1, [500], None, True, 303, shape_values=shape)


def test_attend_nan_in_a_visible_row_spreads_and_in_a_hidden_one_does_not():
    g = gen(304)
    S, Hq, H, d, block, cap = 2, 4, 1, 128, 16, 64
    rc = ref.Cache(S, H, cap, d, block)
    x = torch.randn(2, S, H, cap, d, generator=g)
    rc.append([cap] * S, [cap] * S, x[0], x[1])
    for T, lens in ((1, [20, 33]), (3, [20, 33])):
        dev = Dev(S, Hq, H, cap, d, block, "bf16")
        dev.fill(rc, lens)                           # the rest of the block holds NaN codes
        dev.codes["v"][1, 0, 5, 3] = POISON
        q = torch.randn(S, Hq, T, d, generator=g).bfloat16().cuda()
        out = torch.zeros_like(q)
        ws = torch.empty(bkv.bkv_cache8_workspace_size(dev.geom, cap, T, 0, False),
                         dtype=torch.uint8, device="cuda")
        bkv.bkv_cache8_attend(dev.geom, *dev.bufs, i32(lens), cap, q, T, None, 0.0, out, None,
                              None, None, 1.0, ws)
        assert bool(out[0].isfinite().all())
        assert bool(out[1, :, :, 3].isnan().all())
        rest = torch.cat([out[1, :, :, :3], out[1, :, :, 4:]], -1)
        assert bool(rest.isfinite().all())
    check_clean()


def test_attend_reports_bad_lengths():
    dev = Dev(4, 2, 1, 64, 64, 16, "bf16")
    rc = ref.Cache(4, 1, 64, 64, 16)
    x = torch.randn(2, 4, 1, 64, 64, generator=gen(5))
    rc.append([64] * 4, [64] * 4, x[0], x[1])
    dev.fill(rc, [64] * 4)
    q = torch.randn(4, 2, 2, 64, generator=gen(6)).bfloat16().cuda()
    out = torch.full_like(q, 7.0)
    ws = torch.empty(bkv.bkv_cache8_workspace_size(dev.geom, 48, 2, 0, False), dtype=torch.uint8,
                     device="cuda")
    bkv.bkv_cache8_attend(dev.geom, *dev.bufs, i32([49, -1, 20, 48]), 48, q, 2,
                          i32([1, 1, 3, 2]), 0.0, out, None, None, None, 1.0, ws)
    assert bkv.bkv_read_device_status() == (6, 611)
    assert bool((out[:3] == 7.0).all()) and bool((out[3] != 7.0).any())
    check_clean()


# ------------------------------------------------------------------ evict

EVICTS = [
    # S, H, d, block, lens, K, sink, recent
    (3, 2, 128, 64, [300, 256, 1000], 256, 4, 32),
    (4, 1, 64, 16, [0, 1, 100, 37], 36, 0, 0),
    (2, 2, 16, 128, [500, 129], 129, 0, 129),          # only the recent rows
    (2, 1, 32, 32, [900, 33], 32, 32, 0),              # only the sink
    (2, 3, 96, 32, [700, 2000], 333, 3, 100),
    (1, 1, 128, 128, [5000], 2500, 16, 256),
    (2, 1, 64, 16, [64, 64], 100, 5, 5),               # budgets above the lengths
    (1, 2, 128, 16, [3000], 1, 0, 1),
    (1, 2, 128, 16, [3000], 1, 0, 0),
    (1, 1, 16, 16, [46000], 9001, 7, 1000),            # a crowded threshold bin (ties)
    (1, 1, 16, 16, [40000], 39000, 0, 0),
]


def make_evict(i, special=True):
    S, H, d, block, lens, K, sink, recent = EVICTS[i]
    g = gen(400 + i)
    cap = (max(max(lens), K) + block - 1) // block * block + block
    rc = ref.Cache(S, H, cap, d, block)
    # blocks up to 2^24 apart: codes that leave the normal range under the new scale
    mag = torch.exp2(24 * torch.rand(2, S, H, cap // block, generator=g) ** 3 - 12)
    x = torch.randn(2, S, H, cap, d, generator=g) * mag.repeat_interleave(block, 3)[..., None]
    x[:, :, :, ::19, 1] = math.nan
    x[1, :, :, :block] = 0.0
    rc.append([cap] * S, [cap] * S, x[0], x[1])
    dev = Dev(S, H, H, cap, d, block, "bf16")
    dev.fill(rc, lens)
    w = torch.exp(2 * torch.randn(S, H, cap, generator=g))
    w[torch.rand(S, H, cap, generator=g) < 0.3] = 0.0              # ties
    w = torch.where(torch.rand(S, H, cap, generator=g) < 0.2, torch.round(w), w)
    if special:
        w[:, :, 11::97] = math.nan
        w[:, :, 13::101] = math.inf
        w[:, :, 17::103] = -0.0
        w[:, :, 23::107] = -1.5
        w[:, :, 29::109] = -math.inf
    return dev, rc, w, cap


def check_evict(i, rc, w, got_codes, got_scale, got_w, got_idx, got_lens):
    S, H, d, block, lens, K, sink, recent = EVICTS[i]
    for s, L in enumerate(lens):
        n = min(L, K)
        assert int(got_lens[s]) == n
        for h in range(H):
            idx = ref.kept_positions(w[s, h], L, K, sink, recent)
            assert len(idx) == n
            if got_idx is not None:
                assert got_idx[s, h, :n].tolist() == idx
                assert bool((got_idx[s, h, n:] == -3).all())
            assert same(got_w[s, h, :n], w[s, h, idx])
            for c in "kv":
                val = rc.values(c, s, h, L)[idx]
                for b in range(-(-n // block)):
                    rows = val[b * block:(b + 1) * block]
                    want = ref.scale_for(ref.finite_amax(rows))
                    assert float(got_scale[c][s, h, b]) == float(want), (s, h, c, b)
                    code = ref.decode(got_codes[c][s, h, b * block:b * block + len(rows)])
                    assert same(code, ref.round_e4m3(rows / want)), (s, h, c, b)


@pytest.mark.parametrize("i", range(len(EVICTS)))
def test_evict(i):
    S, H, d, block, lens, K, sink, recent = EVICTS[i]
    dev, rc, w, cap = make_evict(i)
    wd = w.cuda()
    dcap = (min(K, cap) + block - 1) // block * block
    dst = Dev(S, H, H, dcap, d, block, "bf16")
    idx = torch.full((S, H, K), -3, dtype=torch.int32, device="cuda")
    nl = i32([-9] * S)
    ml = max(lens)
    ws = torch.full((bkv.bkv_cache8_workspace_size(dev.geom, ml, 0, K, False),), 0xff,
                    dtype=torch.uint8, device="cuda")
    bkv.bkv_cache8_evict(dev.geom, *dev.bufs, wd, i32(lens), ml, K, sink, recent, dst.geom,
                         *dst.bufs, dst.weights, idx, nl, ws)
    check_clean()
    check_evict(i, rc, w, dst.codes, dst.scale, dst.weights.cpu(), idx.cpu(), nl.cpu())
    for s, L in enumerate(lens):                     # rows behind the last were left
        n = min(L, K)
        nb = -(-n // block)
        for c in "kv":
            assert bool((dst.codes[c][s, :, n:] == POISON).all())
            assert bool(dst.scale[c][s, :, nb:].isnan().all())
        assert bool(dst.weights[s, :, n:].isnan().all())


@pytest.mark.parametrize("i", range(len(EVICTS)))
def test_evict_in_place(i):
    """The same rows in the same buffers, lengths replaced, positions not asked for."""
    S, H, d, block, lens, K, sink, recent = EVICTS[i]
    dev, rc, w, cap = make_evict(i)
    wd = w.cuda()
    ld = i32(lens)
    ws = torch.full((bkv.bkv_cache8_workspace_size(dev.geom, max(lens), 0, K, False),), 0xff,
                    dtype=torch.uint8, device="cuda")
    bkv.bkv_cache8_evict(dev.geom, *dev.bufs, wd, ld, max(lens), K, sink, recent, dev.geom,
                         *dev.bufs, wd, None, ld, ws)
    check_clean()
    check_evict(i, rc, w, dev.codes, dev.scale, wd.cpu(), None, ld.cpu())


def test_evict_reports_bad_lengths():
    dev, rc, w, cap = make_evict(1)
    S, H, d, block, lens, K, sink, recent = EVICTS[1]
    dst = Dev(S, H, H, 48, d, block, "bf16")
    nl = i32([-9] * S)
    ws = torch.empty(bkv.bkv_cache8_workspace_size(dev.geom, 60, 0, K, False), dtype=torch.uint8,
                     device="cuda")
    bkv.bkv_cache8_evict(dev.geom, *dev.bufs, w.cuda(), i32([-1, 1, 61, 37]), 60, K, sink, recent,
                         dst.geom, *dst.bufs, dst.weights, None, nl, ws)
    assert bkv.bkv_read_device_status() == (6, 621)
    assert nl.tolist() == [-9, 1, -9, 36]
    for s in (0, 2):
        assert bool((dst.codes["k"][s] == POISON).all()) and bool((dst.codes["v"][s] == POISON).all())
    check_clean()


# ------------------------------------------------- as a decode loop uses them

def loop_state(dtype="bf16", S=2, Hq=10, H=2, d=128, block=32, cap=256):
    dev = Dev(S, Hq, H, cap, d, block, dtype)
    n = max(bkv.bkv_cache8_workspace_size(dev.geom, cap, 1, 160, True),
            bkv.bkv_cache8_workspace_size(dev.geom, cap, 140, 160, True))
    return dev, torch.empty(n, dtype=torch.uint8, device="cuda")


def test_decode_loop_with_eviction():
    """A prompt, decode steps, an eviction in place, more decode steps: every
    output against the definitions, on the cache as the definitions have it."""
    S, Hq, H, d, block, cap, K, sink, recent = 2, 10, 2, 128, 32, 256, 96, 4, 24
    G = Hq // H
    dev, ws = loop_state()
    rc = ref.Cache(S, H, cap, d, block)
    g = gen(500)
    lens = [0, 0]
    w = torch.zeros(S, H, cap, dtype=torch.float64)
    tol_w = torch.zeros(S, H, cap, dtype=torch.float64)

    def step(T, n):
        nonlocal lens
        lens = [a + b for a, b in zip(lens, n)]
        k = torch.randn(S, H, T, d, generator=g).bfloat16()
        v = torch.randn(S, H, T, d, generator=g).bfloat16()
        q = (2 * torch.randn(S, Hq, T, d, generator=g)).bfloat16()
        out = torch.zeros(S, Hq, T, d, dtype=torch.bfloat16, device="cuda")
        L, N = i32(lens), None if all(x == T for x in n) else i32(n)
        bkv.bkv_cache8_append(dev.geom, *dev.bufs, L, k.cuda(), v.cuda(), T, N)
        bkv.bkv_cache8_attend(dev.geom, *dev.bufs, L, cap, q.cuda(), T, N, 0.0, out, None,
                              dev.weights, dev.weights, 0.9, ws)
        rc.append(lens, n, k, v)
        out = out.double().cpu()
        for s in range(S):
            for h in range(H):
                kv, vv = rc.values("k", s, h, lens[s]), rc.values("v", s, h, lens[s])
                qh = q[s, h * G:(h + 1) * G, :n[s]]
                o, _, p = ref.attend(kv, vv, qh, lens[s], n[s], 1 / math.sqrt(d))
                bo, _, bp = attend_bounds(kv, vv, qh, p, 1 / math.sqrt(d), "bf16", d,
                                          float(rc.scale["v"][s, h].max()))
                err = (out[s, h * G:(h + 1) * G, :n[s]] - o).abs()
                assert bool((err <= bo + ref.U_BF16 * (o.abs() + bo)).all())
                a = lens[s] - n[s]
                old, old_tol = 0.9 * w[s, h, :a], tol_w[s, h, :a]
                w[s, h, :lens[s]] = p.sum((0, 1))
                w[s, h, :a] += old
                tol_w[s, h, :lens[s]] = (bp.sum((0, 1)) + G * T * 2.0 ** -126
                                          + (G * T + 4) * ref.U_F32 * w[s, h, :lens[s]])
                tol_w[s, h, :a] += old_tol
                got = dev.weights[s, h, :lens[s]].double().cpu()
                assert bool(((got - w[s, h, :lens[s]]).abs() <= tol_w[s, h, :lens[s]]).all())

    step(140, [140, 77])
    for _ in range(5):
        step(1, [1, 1])
    before = dev.weights.double().cpu()              # the kernel's own: near ties fall as it sees them
    L = i32(lens)
    bkv.bkv_cache8_evict(dev.geom, *dev.bufs, dev.weights, L, cap, K, sink, recent, dev.geom,
                         *dev.bufs, dev.weights, None, L, ws)
    for s in range(S):
        n = min(lens[s], K)
        for h in range(H):
            idx = ref.kept_positions(before[s, h], lens[s], K, sink, recent)
            for c in "kv":
                val = rc.values(c, s, h, lens[s])[idx]
                for b in range(-(-n // block)):
                    rows = val[b * block:(b + 1) * block]
                    sc = ref.scale_for(ref.finite_amax(rows))
                    rc.scale[c][s, h, b] = sc
                    rc.code[c][s, h, b * block:b * block + len(rows)] = ref.round_e4m3(rows / sc)
            w[s, h, :n], tol_w[s, h, :n] = w[s, h, idx], tol_w[s, h, idx]
        lens[s] = n
    assert L.tolist() == lens
    for _ in range(4):
        step(1, [1, 1])
    check_clean()


def test_captured_loop_replays_with_new_lengths():
    """One decode step captured in a graph: a replay serves the lengths, rows
    and queries of the moment, and equals the eager calls bit for bit."""
    S, Hq, H, d, cap = 2, 10, 2, 128, 256
    res = []
    for graphed in (False, True):
        dev, ws = loop_state()
        g = gen(501)
        k, v = (torch.randn(S, H, 140, d, generator=g).bfloat16().cuda() for _ in range(2))
        lens = i32([140, 33])
        bkv.bkv_cache8_append(dev.geom, *dev.bufs, lens, k, v, 140, i32([140, 33]))
        dev.weights.zero_()
        kn, vn = (torch.zeros(S, H, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        q = torch.zeros(S, Hq, 1, d, dtype=torch.bfloat16, device="cuda")
        out = torch.zeros_like(q)

        def step():
            lens.add_(1)
            bkv.bkv_cache8_append(dev.geom, *dev.bufs, lens, kn, vn, 1)
            bkv.bkv_cache8_attend(dev.geom, *dev.bufs, lens, cap, q, 1, None, 0.0, out, None,
                                  dev.weights, dev.weights, 1.0, ws)

        def evict():
            bkv.bkv_cache8_evict(dev.geom, *dev.bufs, dev.weights, lens, cap, 100, 4, 16, dev.geom,
                                 *dev.bufs, dev.weights, None, lens, ws)

        if graphed:
            torch.cuda.synchronize()
            side = torch.cuda.Stream()
            gs, ge = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
            with torch.cuda.graph(gs, stream=side):
                step()
            with torch.cuda.graph(ge, stream=side):
                evict()
        outs = []
        for i in range(24):
            kn.copy_(torch.randn(kn.shape, generator=g))
            vn.copy_(torch.randn(kn.shape, generator=g))
            q.copy_(torch.randn(q.shape, generator=g))
            gs.replay() if graphed else step()
            outs.append(out.clone())
            if i == 15:
                ge.replay() if graphed else evict()
        torch.cuda.synchronize()
        res.append([torch.stack(outs)] + [t.clone() for t in dev.bufs] + [lens.clone()])
    check_clean()
    assert res[0][-1].tolist() == [108, 57]
    for a, b in zip(*res):
        assert same(a, b)


def test_two_streams_at_once():
    """Calls on two streams with a workspace each do not disturb one another,
    and repeated calls give the same bits."""
    states = []
    for s in range(2):
        g = gen(510 + s)
        dev = Dev(3, 8, 2, 2048, 128, 64, "bf16")
        rc_lens = i32([2000 - 31 * s, 900, 1500])
        k, v = (torch.randn(3, 2, 2048, 128, generator=g).bfloat16().cuda() for _ in range(2))
        bkv.bkv_cache8_append(dev.geom, *dev.bufs, i32([2048] * 3), k, v, 2048)
        q = torch.randn(3, 8, 1, 128, generator=g).bfloat16().cuda()
        ws = torch.empty(bkv.bkv_cache8_workspace_size(dev.geom, 2048, 1, 0, True),
                         dtype=torch.uint8, device="cuda")
        states.append((dev, rc_lens, q, ws, torch.cuda.Stream()))

    def call(i, stream):
        dev, lens, q, ws, _ = states[i]
        out, w = torch.empty_like(q), torch.zeros(3, 2, 2048, device="cuda")
        torch.cuda.synchronize()
        return out, w, lambda: bkv.bkv_cache8_attend(dev.geom, *dev.bufs, lens, 2048, q, 1, None,
                                                     0.0, out, None, None, w, 1.0, ws, stream)

    alone = []
    for i in range(2):
        out, w, f = call(i, None)
        f()
        torch.cuda.synchronize()
        alone.append((out, w))
    both = [call(i, states[i][4]) for i in range(2)]
    for _ in range(20):
        for _, _, f in both:
            f()
    torch.cuda.synchronize()
    for (o, w, _), (ao, aw) in zip(both, alone):
        assert same(o, ao) and same(w, aw)
    check_clean()


def nan_case(dtype, S, Hq, H, d, block, T, lens, n_new, poke):
    """Outputs, lse and weights with and without NaN codes at poke: (which,
    sequence, KV head, row, elements)."""
    g = gen(700)
    cap = (max(lens) + block - 1) // block * block
    rc = ref.Cache(S, H, cap, d, block)
    x = torch.randn(2, S, H, cap, d, generator=g)
    rc.append([cap] * S, [cap] * S, x[0], x[1])
    q = torch.randn(S, Hq, T, d, generator=g).to(DT[dtype]).cuda()
    res = []
    for bad in (False, True):
        dev = Dev(S, Hq, H, cap, d, block, dtype)
        dev.fill(rc, lens)
        for c, s, h, j, elements in poke if bad else ():
            for e in elements:
                dev.codes[c][s, h, j, e] = POISON | (0x80 if e % 2 else 0)
        out, lse = torch.full_like(q, 7.0), torch.full((S, Hq, T), 7.0, device="cuda")
        w = torch.full((S, H, cap), 7.0, device="cuda")
        ws = torch.full((bkv.bkv_cache8_workspace_size(dev.geom, cap, T, 0, True),), 0xff,
                        dtype=torch.uint8, device="cuda")
        bkv.bkv_cache8_attend(dev.geom, *dev.bufs, i32(lens), cap, q, T,
                              None if n_new is None else i32(n_new), 0.0, out, lse, None, w, 1.0, ws)
        check_clean()
        res.append((out.double().cpu(), lse.double().cpu(), w.double().cpu()))
    return res


NANS = [
    # dtype, S, Hq, H, d, block, T, lens, n_new: every kernel, one tile and many
    ("f32", 2, 4, 2, 96, 16, 5, [40, 900], None),
    ("bf16", 2, 2, 2, 64, 32, 7, [40, 300], [7, 5]),
    ("bf16", 2, 4, 2, 128, 64, 4, [133, 700], None),
    ("bf16", 2, 8, 2, 128, 16, 5, [133, 700], [5, 4]),
    ("bf16", 2, 8, 2, 64, 16, 8, [40, 300], None),
    ("bf16", 2, 2, 1, 128, 64, 64, [130, 400], [64, 40]),
    ("bf16", 1, 2, 1, 64, 32, 50, [50], None),
    ("bf16", 2, 2, 1, 64, 32, 100, [260, 900], [90, 100]),
    ("bf16", 2, 2, 1, 128, 32, 128, [260, 900], [128, 77]),
    ("bf16", 1, 1, 1, 128, 128, 200, [20300], None),
    ("bf16", 2, 2, 1, 128, 32, 300, [300, 900], [300, 201]),
    ("bf16", 1, 3, 1, 64, 64, 300, [2000], None),
]


@pytest.mark.parametrize("i", range(len(NANS)))
def test_attend_nan_in_a_new_row_reaches_the_tokens_that_see_it(i):
    """NaN in K and V rows among the call's own tokens: every other output is
    the same bits as without."""
    dtype, S, Hq, H, d, block, T, lens, n_new = NANS[i]
    G = Hq // H
    for c in "vk":
        poke, hit = [], torch.zeros(S, Hq, T, d, dtype=torch.bool)
        for s, L in enumerate(lens):
            n = n_new[s] if n_new else T
            rows = {L - 1: [0, 17, d - 1], L - n // 2: [3, 17], L - n + 1: [16, 31], L - n // 3: [40]}
            for j, elements in rows.items():
                h = (s + j) % H
                poke.append((c, s, h, j, elements))
                t0 = j - (L - n)                     # the first token that sees row j
                cols = elements if c == "v" else range(d)
                for e in cols:
                    hit[s, h * G:(h + 1) * G, max(t0, 0):n, e] = True
        (o0, z0, w0), (o1, z1, w1) = nan_case(dtype, S, Hq, H, d, block, T, lens, n_new, poke)
        assert bool(o0.isfinite().all())
        assert same(o1, torch.where(hit, math.nan, o0))
        if c == "v":
            assert same(z1, z0) and same(w1, w0)
        else:
            assert same(z1, torch.where(hit[..., 0], math.nan, z0))


MANY_ROWS = [
    # dtype, S, Hq, H, d, block, T, lens, n_new, weights: more than 32 query rows a
    # KV head (one and two row tiles, expanded tiles), parts of segments
    ("bf16", 1, 5, 1, 128, 64, 7, [30011], None, True),            # 35 rows, over every CTA
    ("bf16", 3, 2, 1, 64, 128, 64, [20000, 64, 5001], [64, 64, 17], True),
    ("bf16", 2, 2, 2, 128, 16, 128, [9000, 130], [100, 128], "fresh"),
    ("bf16", 1, 3, 1, 128, 32, 80, [25000], None, False),          # 240 rows, two row tiles
    ("bf16", 4, 4, 2, 64, 16, 64, [64, 0, 12000, 700], [64, 0, 1, 33], True),
    ("bf16", 2, 2, 1, 128, 64, 129, [129, 6000], [129, 128], True),
    ("bf16", 2, 1, 1, 128, 128, 513, [9000, 513], [513, 300], True),   # expanded tiles
    ("bf16", 3, 4, 2, 64, 32, 70, [5000, 1, 71], [70, 1, 70], True),
    ("bf16", 2, 5, 1, 128, 16, 60, [40, 20], [60, 20], True),      # rows that see nothing
    ("bf16", 1, 40, 1, 128, 64, 1, [15000], None, True),           # a wide group, one token
    ("bf16", 40, 2, 1, 64, 16, 20, [(61 * i) % 333 for i in range(40)],
     [min(i % 21, 20) for i in range(40)], True),
    # up to 32 rows, many tiles a CTA
    ("bf16", 1, 12, 1, 128, 64, 1, [90001], None, True),
    ("bf16", 1, 3, 1, 64, 32, 7, [60000], None, True),
    ("bf16", 1, 8, 1, 128, 16, 4, [50000], None, "fresh"),
]


@pytest.mark.parametrize("i", range(len(MANY_ROWS)))
def test_attend_many_rows(i):
    dtype, S, Hq, H, d, block, T, lens, n_new, weights = MANY_ROWS[i]
    run_attend(dtype, S, Hq, H, d, block, T, lens, n_new, weights, 800 + i, decay=0.875)


def test_attend_many_rows_large_logits_and_scales_far_apart():
    """Softmax references that move while the outputs stand in TMEM, and K and V
    scales of one tile binades apart."""
    def shape(x):
        for b in range(0, x.shape[3], 16):
            x[1, :, :, b:b + 16] *= 0.0 if b % 80 == 0 else 2.0 ** ((b // 16 * 7) % 30 - 15)
            x[0, :, :, b:b + 16] *= 2.0 ** ((b // 16 * 5) % 9 - 6)
    for Hq, T in ((10, 5), (6, 40), (2, 200)):
        run_attend("bf16", 2, Hq, 1, 128, 64, T, [700, 2000], None, True, 820, q_mag=20.0)
        run_attend("bf16", 1, Hq, 1, 64, 16, T, [900], None, True, 821, shape_values=shape)


@pytest.mark.parametrize("T", [3, 12, 50, 200])
def test_captured_chunk_replays_with_new_lengths(T):
    """A padded call of several tokens in a graph: replays with other lengths,
    counts and rows equal the eager calls bit for bit, the workspace shared with
    another captured call in between."""
    S, Hq, H, d, cap = 3, 4, 2, 128, 1024
    res = []
    for graphed in (False, True):
        g = gen(830)
        dev = Dev(S, Hq, H, cap, d, 32, "bf16")
        ws = torch.empty(max(bkv.bkv_cache8_workspace_size(dev.geom, cap, t, 0, True) for t in (1, T)),
                         dtype=torch.uint8, device="cuda")
        lens, n_new = i32([0] * S), i32([0] * S)
        kn, vn = (torch.zeros(S, H, T, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        q = torch.zeros(S, Hq, T, d, dtype=torch.bfloat16, device="cuda")
        q1 = torch.zeros(S, Hq, 1, d, dtype=torch.bfloat16, device="cuda")
        out, out1 = torch.zeros_like(q), torch.zeros_like(q1)
        dev.weights.zero_()

        def chunk():
            lens.add_(n_new)
            bkv.bkv_cache8_append(dev.geom, *dev.bufs, lens, kn, vn, T, n_new)
            bkv.bkv_cache8_attend(dev.geom, *dev.bufs, lens, cap, q, T, n_new, 0.0, out, None,
                                  dev.weights, dev.weights, 1.0, ws)

        def one():
            bkv.bkv_cache8_attend(dev.geom, *dev.bufs, lens, cap, q1, 1, None, 0.0, out1, None,
                                  None, None, 1.0, ws)

        if graphed:
            torch.cuda.synchronize()
            side = torch.cuda.Stream()
            gc, go = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
            with torch.cuda.graph(gc, stream=side):
                chunk()
            with torch.cuda.graph(go, stream=side):
                one()
        outs = []
        for i in range(4):
            for t in (kn, vn, q, q1):
                t.copy_(torch.randn(t.shape, generator=g))
            n_new.copy_(torch.tensor([T, (i * 7) % (T + 1), 1 if i else T], dtype=torch.int32))
            gc.replay() if graphed else chunk()
            go.replay() if graphed else one()
            outs += [out.clone(), out1.clone()]
        torch.cuda.synchronize()
        res.append(outs + [dev.weights[s, :, :int(lens[s])].clone() for s in range(S)] + [lens.clone()])
    check_clean()
    for a, b in zip(*res):
        assert same(a, b)


def test_offsets_past_32_bits():
    """A head of more than 2^32 codes, all zeros but its last rows: these appended,
    attended to and kept by an eviction.

    Every zero key has logit 0, so with n0 of them the denominators are n0 plus the
    last rows' terms.  Bounds as in attend_bounds, and for the denominator a lane's
    sum of at most cap / 128 / 296 tiles x 8 terms, below 2^13 steps of 2^-24."""
    d, block, T = 128, 64, 40
    cap = (1 << 25) + 128
    codes = {n: torch.zeros(1, 1, cap, d, dtype=torch.uint8, device="cuda") for n in "kv"}
    scale = {n: torch.full((1, 1, cap // block), 2.0 ** -10, device="cuda") for n in "kv"}
    bufs = codes["k"], codes["v"], scale["k"], scale["v"]
    geom = bkv.geometry8_of(codes["k"], scale["k"], 2, torch.bfloat16)
    g = gen(840)
    k, v = (torch.randn(1, 1, T, d, generator=g).bfloat16() for _ in range(2))
    lens = i32([cap])
    bkv.bkv_cache8_append(geom, *bufs, lens, k.cuda(), v.cuda(), T)
    rc = ref.Cache(1, 1, block, d, block)
    rc.append([T], [T], k, v)
    for n in "kv":
        assert float(scale[n][0, 0, -1]) == float(rc.scale[n][0, 0, 0])
        assert same(ref.decode(codes[n][0, 0, cap - T:]), rc.code[n][0, 0, :T])
        assert not bool(codes[n][0, 0, cap - block:cap - T].any())
    kv, vv = rc.values("k", 0, 0, T), rc.values("v", 0, 0, T)
    w = torch.zeros(1, 1, cap, device="cuda")
    ws = torch.empty(max(bkv.bkv_cache8_workspace_size(geom, cap, t, 1024, True) for t in (1, 2, 20)),
                     dtype=torch.uint8, device="cuda")
    for T2 in (1, 2, 20):
        q = torch.randn(1, 2, T2, d, generator=g).bfloat16()
        out = torch.empty_like(q, device="cuda")
        bkv.bkv_cache8_attend(geom, *bufs, lens, cap, q.cuda(), T2, None, 0.0, out, None, None, w, 1.0, ws)
        z = q[0].double() @ kv.T / math.sqrt(d)
        see = torch.arange(T)[None, None] <= T - T2 + torch.arange(T2)[None, :, None]
        p = torch.where(see, z.exp(), 0.0)
        p = p / (p.sum(-1, keepdim=True) + cap - T)
        eps = (d + 4) * 2.0 ** -22 / math.sqrt(d) * (q[0].double().abs() @ kv.abs().T)
        rel = 2.0 * eps.amax(-1, keepdim=True) + 2.0 ** -19 + 2.0 ** -11
        av = p @ vv.abs()
        tol = (rel + 2.0 ** -20 + 2.0 ** -11) * av + T * 2.0 ** -25 * 448 * float(rc.scale["v"][0, 0, 0]) * \
            p.amax(-1, keepdim=True)
        o = p @ vv
        err = (out[0].double().cpu() - o).abs()
        assert bool((err <= tol + ref.U_BF16 * (o.abs() + tol)).all()), float((err / o.abs()).max())
        want = p.sum((0, 1))
        got = w[0, 0, cap - T:].double().cpu()
        assert bool(((got - want).abs() <= ((rel + 2.0 ** -20) * p).sum((0, 1)) + 2 * T2 * 2.0 ** -24 * want).all())
    w.zero_()
    inner = torch.randperm(cap - 64, generator=g)[:970] + 14
    keep = torch.cat([inner, torch.arange(cap - 40, cap - 10)])
    w[0, 0, keep.cuda()] = 1.0 + torch.rand(1000, generator=g).cuda()
    idx, nl = torch.full((1, 1, 1024), -3, dtype=torch.int32, device="cuda"), i32([-1])
    bkv.bkv_cache8_evict(geom, *bufs, w, lens, cap, 1024, 14, 10, geom, *bufs, w, idx, nl, ws)
    check_clean()
    assert nl.tolist() == [1024]
    assert idx[0, 0].tolist() == sorted(list(range(14)) + keep.tolist() + list(range(cap - 10, cap)))
    for n in "kv":
        assert float(scale[n][0, 0, 15]) == float(rc.scale[n][0, 0, 0])
        assert same(ref.decode(codes[n][0, 0, 1024 - T:1024]), rc.code[n][0, 0, :T])


def test_attend_many_segments_joined():
    """More rows to join than are dealt one by one, in two parts and in more."""
    g = gen(850)
    lens = torch.randint(1, 1500, (16,), generator=g).tolist()
    n_new = torch.randint(0, 101, (16,), generator=g).tolist()
    run_attend("bf16", 16, 4, 4, 64, 32, 100, lens, n_new, True, 851)
    run_attend("bf16", 2, 16, 8, 128, 16, 40, [5000, 9000], [40, 33], True, 852)


@pytest.mark.parametrize("dtype,T", [("f32", 2), ("bf16", 1), ("bf16", 20), ("bf16", 100), ("bf16", 300)])
def test_attend_workspace_of_16_byte_alignment(dtype, T):
    """The same bits from a workspace that is aligned to 16 bytes only."""
    S, Hq, H, d, block, cap = 2, 2, 1, 64, 32, 1024
    g = gen(860)
    rc = ref.Cache(S, H, cap, d, block)
    x = torch.randn(2, S, H, cap, d, generator=g)
    rc.append([cap] * S, [cap] * S, x[0], x[1])
    dev = Dev(S, Hq, H, cap, d, block, dtype)
    dev.fill(rc, [1000, 700])
    q = torch.randn(S, Hq, T, d, generator=g).to(DT[dtype]).cuda()
    need = bkv.bkv_cache8_workspace_size(dev.geom, cap, T, 0, True)
    res = []
    for off in (0, 16):
        ws = torch.full((need + 16,), 0xff, dtype=torch.uint8, device="cuda")[off:off + need]
        out, w = torch.empty_like(q), torch.zeros(S, H, cap, device="cuda")
        bkv.bkv_cache8_attend(dev.geom, *dev.bufs, i32([1000, 700]), cap, q, T, None, 0.0, out, None,
                              None, w, 1.0, ws)
        check_clean()
        res.append((out, w))
    assert bool(res[0][0].isfinite().all())
    assert same(res[0][0], res[1][0]) and same(res[0][1], res[1][1])


def test_calls_follow_copies_and_joined_streams_in_a_graph():
    """A captured step whose calls follow a memset, a copy and an event of another
    stream instead of kernels, replayed back to back."""
    S, Hq, H, d, cap = 2, 8, 2, 128, 512
    dev = Dev(S, Hq, H, cap, d, 32, "bf16")
    want = Dev(S, Hq, H, cap, d, 32, "bf16")
    g = gen(870)
    n = 24
    k, v, q = (torch.randn(n, S, h, 1, d, generator=g).bfloat16().cuda() for h in (H, H, Hq))
    all_lens = torch.tensor([[i + 1, 2 * i + 1] for i in range(n)], dtype=torch.int32).pin_memory()
    ws = torch.empty(bkv.bkv_cache8_workspace_size(dev.geom, cap, 1, 300, True), dtype=torch.uint8,
                     device="cuda")
    res = []
    for c, graphed in ((want, False), (dev, True)):
        lens = i32([0, 0])
        kn, vn, qn = torch.empty_like(k[0]), torch.empty_like(v[0]), torch.empty_like(q[0])
        out = torch.empty_like(qn)
        w = torch.zeros(S, H, cap, device="cuda")
        host = torch.zeros(2, dtype=torch.int32).pin_memory()
        torch.cuda.synchronize()

        def step(side):
            lens.copy_(host, non_blocking=True)          # a copy straight before the append
            bkv.bkv_cache8_append(c.geom, *c.bufs, lens, kn, vn, 1, i32_one)
            if side is not None:                         # a join straight before attend
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    out.zero_()
                torch.cuda.current_stream().wait_stream(side)
            bkv.bkv_cache8_attend(c.geom, *c.bufs, lens, cap, qn, 1, i32_one, 0.0, out, None, w, w,
                                  1.0, ws)
            out2.copy_(out)

        i32_one = i32([1, 1])
        out2 = torch.empty_like(out)
        if graphed:
            st, other = torch.cuda.Stream(), torch.cuda.Stream()
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=st):
                step(other)
        outs = []
        for i in range(n):
            torch.cuda.synchronize()
            host.copy_(all_lens[i])
            # sequence 1 gets every second row only: the rows between stay zero codes
            kn.copy_(k[i]), vn.copy_(v[i]), qn.copy_(q[i])
            c.codes["k"][1].masked_fill_(c.codes["k"][1] == POISON, 0)
            c.codes["v"][1].masked_fill_(c.codes["v"][1] == POISON, 0)
            c.scale["k"][1].nan_to_num_(2.0 ** -8), c.scale["v"][1].nan_to_num_(2.0 ** -8)
            w.nan_to_num_(0.0)
            gr.replay() if graphed else step(None)
            outs.append(out2.clone())
        torch.cuda.synchronize()
        res.append([torch.stack(outs), w, *c.bufs])
    check_clean()
    assert bool(res[0][0].isfinite().all())
    for a, b in zip(*res):
        assert same(a, b)


def test_a_loop_without_a_pause():
    """Append, attend and evict back to back, each call's input the one before's
    output, against the same calls with a synchronisation after each."""
    S, Hq, H, d, cap = 3, 8, 2, 128, 512
    res = []
    for pause in (False, True):
        g = gen(880)
        dev = Dev(S, Hq, H, cap, d, 32, "bf16")
        ws = torch.empty(bkv.bkv_cache8_workspace_size(dev.geom, cap, 1, 100, True), dtype=torch.uint8,
                         device="cuda")
        k, v = (torch.randn(S, H, 128, d, generator=g).bfloat16().cuda() for _ in range(2))
        q = torch.randn(S, Hq, 1, d, generator=g).bfloat16().cuda()
        lens, one = i32([128, 90, 101]), i32([1, 1, 1])
        dev.weights.zero_()
        out = torch.zeros_like(q)
        kn, vn = k[:, :, :1].contiguous(), v[:, :, :1].contiguous()
        wait = torch.cuda.synchronize if pause else lambda: None
        bkv.bkv_cache8_append(dev.geom, *dev.bufs, lens, k, v, 128, i32([128, 90, 101]))
        for i in range(60):
            # the output of a call is the next one's query and new row
            bkv.bkv_cache8_attend(dev.geom, *dev.bufs, lens, cap, q, 1, None, 0.0, out, None,
                                  dev.weights, dev.weights, 0.9, ws)
            wait()
            bkv.bkv_cache8_attend(dev.geom, *dev.bufs, lens, cap, out, 1, None, 0.0, q, None,
                                  dev.weights, dev.weights, 0.9, ws)
            wait()
            bkv.bkv_cache8_append(dev.geom, *dev.bufs, lens, kn, vn, 1, one)
            wait()
            bkv.bkv_cache8_evict(dev.geom, *dev.bufs, dev.weights, lens, cap, 100 - i % 7, 4, 16,
                                 dev.geom, *dev.bufs, dev.weights, None, lens, ws)
            wait()
        torch.cuda.synchronize()
        n = int(lens[0])
        res.append([q, out, lens] + [dev.codes[c][:, :, :n].clone() for c in "kv"] +
                   [dev.weights[:, :, :min(lens.tolist())].clone()])
    check_clean()
    for a, b in zip(*res):
        assert same(a, b)


@pytest.mark.parametrize("Hq,T,n_new", [(4, 8, [8, 5, 1]), (7, 4, [4, 3, 0]), (13, 2, None), (31, 1, None)])
def test_attend_two_row_blocks(Hq, T, n_new):
    """25 to 32 query rows of 128 elements, a row block that may have none."""
    run_attend("bf16", 3, Hq, 1, 128, 32, T, [3000, 257, 90], n_new, True, 900, decay=0.5)
    run_attend("bf16", 3, Hq, 1, 128, 32, T, [700, 8, 0], n_new, "fresh", 901)


def test_attend_nan_in_a_new_row_and_two_row_blocks():
    S, Hq, T, d, lens = 2, 4, 7, 128, [130, 700]
    poke = [("v", 0, 0, 126, [3, 90]), ("v", 1, 0, 699, [0]), ("v", 1, 0, 694, [127])]
    hit = torch.zeros(S, Hq, T, d, dtype=torch.bool)
    for _, s, _, j, elements in poke:
        for e in elements:
            hit[s, :, j - (lens[s] - T):, e] = True
    (o0, z0, w0), (o1, z1, w1) = nan_case("bf16", S, Hq, 1, d, 16, T, lens, None, poke)
    assert same(o1, torch.where(hit, math.nan, o0)) and same(z1, z0) and same(w1, w0)


@pytest.mark.parametrize("dtype,d", [("f32", 96), ("bf16", 112), ("f32", 16), ("f32", 128)])
@pytest.mark.parametrize("Hq,T,n_new", [(1, 1, None), (2, 1, None), (1, 3, [3, 2, 0]), (4, 1, None),
                                        (2, 2, [2, 1, 2]), (1, 5, [5, 4, 1])])
def test_attend_few_rows_on_cuda_cores(dtype, d, Hq, T, n_new):
    """Row blocks of 2, 4 and 8 rows, full and not."""
    run_attend(dtype, 3, Hq, 1, d, 16, T, [5, 700, 4001], n_new, True, 910, decay=0.5)


def test_attend_nan_in_a_new_row_of_few():
    for Hq, T in ((1, 2), (2, 2), (1, 4)):
        poke = [("v", 0, 0, 699, [3, 90]), ("v", 1, 0, 128, [0])]
        lens = [700, 129]
        hit = torch.zeros(2, Hq, T, 96, dtype=torch.bool)
        for _, s, _, j, elements in poke:
            for e in elements:
                hit[s, :, j - (lens[s] - T):, e] = True
        (o0, z0, w0), (o1, z1, w1) = nan_case("f32", 2, Hq, 1, 96, 16, T, lens, None, poke)
        assert same(o1, torch.where(hit, math.nan, o0)) and same(z1, z0) and same(w1, w0)


@pytest.mark.parametrize("Hq,T,n_new", [
    (4, 10, [10, 7, 0]), (3, 127, [127, 1, 60]), (3, 128, [128, 128, 5]), (7, 45, None),
    (40, 1, None), (129, 1, None), (13, 20, [20, 0, 19]), (2, 100, [100, 64, 33])])
def test_attend_weights_of_many_rows(Hq, T, n_new):
    """Tiles of query rows that hold several heads' tokens, or end inside one."""
    run_attend("bf16", 3, Hq, 1, 64, 32, T, [900, 129, 3001], n_new, True, 920, decay=0.5)
    run_attend("bf16", 3, Hq, 1, 128, 16, T, [T, 200, 40], n_new, "fresh", 921)
