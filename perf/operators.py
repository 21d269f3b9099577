"""The operators of the 8-bit KV cache, as they are measured.

Three operators that a decode loop runs one after another:

append   new K/V rows into a cache of e4m3 codes with one power-of-two scale
         for each block of rows and head;
attend   attention of the newest T tokens over that cache, with the sum of
         each cached key's probabilities (its attention weight) on the side;
evict    the rows with the most accumulated attention weight are kept, next to
         the first `sink` and the last `recent` ones, and compacted.

`run` computes them in elementary torch operations in 32 bits, or, where `own`
is set, by this repository's entry points.  `exact` is the definition in 64
bits, written apart from the plain form.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3_MAX = 448.0
MIN_EXP = -117  # the smallest scale is 2^-117


# ------------------------------------------------------------------ the cases

def listed():
    def append(name, n_seqs, hkv, d, block, T, lo, hi, ragged=False, dtype="bf16"):
        return {"name": name, "op": "append", "n_seqs": n_seqs, "hq": hkv, "hkv": hkv, "d": d,
                "block": block, "T": T, "lo": lo, "hi": hi, "ragged": ragged, "dtype": dtype}

    def attend(name, n_seqs, hq, hkv, d, block, T, lo, hi, weights, ragged=False, decay=1.0,
               dtype="bf16"):
        return {"name": name, "op": "attend", "n_seqs": n_seqs, "hq": hq, "hkv": hkv, "d": d,
                "block": block, "T": T, "lo": lo, "hi": hi, "weights": weights,
                "ragged": ragged, "decay": decay, "dtype": dtype}

    def evict(name, n_seqs, hkv, d, block, lo, hi, K, sink, recent):
        return {"name": name, "op": "evict", "n_seqs": n_seqs, "hq": hkv, "hkv": hkv, "d": d,
                "block": block, "lo": lo, "hi": hi, "K": K, "sink": sink, "recent": recent,
                "dtype": "bf16"}

    return [
        # one decode step's new rows of a ragged batch, one layer: latency counts
        append("append one token", 24, 8, 128, 64, 1, 700, 8192),
        # four prompts written whole into empty caches
        append("append prompts", 4, 8, 128, 64, 8192, 8192, 8192),
        # a padded chunk in 32 bits: lengths and counts that end inside a block
        append("append odd chunk", 5, 1, 64, 16, 37, 101, 1024, ragged=True, dtype="f32"),
        # the smallest model's decode step, in 32 bits
        attend("attend tiny", 1, 4, 1, 64, 16, 1, 1024, 1024, False, dtype="f32"),
        # one sequence's decode step with its weights (7 query heads to a KV head)
        attend("attend decode", 1, 28, 4, 128, 64, 1, 8192, 8192, True),
        # the decode step of a ragged batch that keeps no weights
        attend("attend ragged batch", 32, 32, 8, 128, 64, 1, 517, 16384, False),
        # a few long sequences, 5 query heads to a KV head, weights that fade
        attend("attend long", 4, 40, 8, 128, 128, 1, 32768, 32768, True, decay=0.99),
        # drafted tokens verified at once: a padded batch, up to six each
        attend("attend drafts", 8, 32, 8, 128, 32, 6, 1009, 8192, True, ragged=True),
        # a chunk of a long prompt over what is cached of it
        attend("attend chunk", 1, 40, 8, 128, 64, 1024, 16384, 16384, True),
        # one layer's cache down to its budget
        evict("evict one layer", 1, 4, 128, 64, 8192, 8192, 2048, 4, 256),
        # every layer's cache halved
        evict("evict 36 layers", 36, 8, 128, 64, 8192, 8192, 4096, 4, 512),
        # every layer of a long cache down to a small budget
        evict("evict 40 layers", 40, 8, 128, 128, 32768, 32768, 6144, 16, 1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["append", "attend", "attend", "evict"])
        dtype = "bf16" if op == "evict" or rng.random() < 0.8 else "f32"
        d = rng.choice([64, 128, 128]) if dtype == "bf16" else rng.choice([32, 64, 96, 128])
        hkv = rng.choice([1, 2, 4, 8])
        c = {"op": op, "n_seqs": _log(rng, 1, 32), "hq": hkv, "hkv": hkv, "d": d,
             "block": rng.choice([16, 32, 64, 128])}
        hi = _log(rng, 64, 32768)
        lo = hi if rng.random() < 0.3 else rng.randint(max(1, hi // 16), hi)
        if op == "evict":
            if rng.random() < 0.5:
                c["n_seqs"] = _log(rng, 1, 40)
            K = rng.randint(max(4, hi // 8), max(5, hi - hi // 4))
            sink = rng.choice([0, 0, 4, min(16, K // 4)])
            c |= {"lo": lo, "hi": hi, "K": K, "sink": sink, "recent": rng.randint(0, K // 2),
                  "dtype": "bf16"}
        else:
            T = 1 if rng.random() < 0.5 else _log(rng, 2, 1024)
            T = min(T, lo)
            if op == "append" and rng.random() < 0.3:
                T = lo
            c |= {"T": T, "lo": lo, "hi": hi, "ragged": T > 1 and rng.random() < 0.4,
                  "dtype": dtype}
        if op == "attend":
            c["hq"] = hkv * rng.choice([1, 2, 4, 5, 7, 8])
            c |= {"weights": rng.random() < 0.5, "decay": rng.choice([1.0, 0.97])}
            # what the largest listed cases take, of memory and of arithmetic
            if c["n_seqs"] * c["hq"] * c["T"] * hi > 40 * 1024 * 16384:
                continue
            if dtype == "f32" and c["n_seqs"] * c["hq"] * c["T"] * hi > 1 << 25:
                continue
        if work(c)["bytes"] <= 1.0e9 and _cache_bytes(c) <= 2.5e9:
            return c


def _lens(case):
    """The sequences' lengths, from lo to hi in equal steps, and the number of
    new tokens of each (T, or from T down to none in a padded batch)."""
    n, lo, hi = case["n_seqs"], case["lo"], case["hi"]
    lens = [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]
    T = case.get("T", 0)
    new = [T - i * (T + 1) // n if case.get("ragged") else T for i in range(n)]
    return lens, [min(a, b) for a, b in zip(new, lens)]


def _capacity(case):
    b = case["block"]
    return (case["hi"] + b - 1) // b * b + 2 * b


def _cache_bytes(case):
    return 2 * case["n_seqs"] * case["hkv"] * _capacity(case) * case["d"]


def work(case):
    """Each input read once, each output written once; multiplications and
    additions of the two products over the visible keys."""
    lens, new = _lens(case)
    hkv, hq, d, block = case["hkv"], case["hq"], case["d"], case["block"]
    e = 2 if case["dtype"] == "bf16" else 4
    row = 2 * d + 8.0 / block  # codes of K and V and their share of the scales
    if case["op"] == "append":
        rows = sum(new) * hkv
        return {"bytes": rows * (2 * d * e + row), "flops": 4.0 * rows * d}
    if case["op"] == "attend":
        b = sum(lens) * hkv * row + sum(new) * hq * (2 * d * e + 4)
        if case["weights"]:
            b += 8.0 * sum(lens) * hkv
        vis = sum(n * (L - n) + n * (n + 1) // 2 for L, n in zip(lens, new))
        return {"bytes": b, "flops": 4.0 * d * hq * vis}
    kept = sum(min(L, case["K"]) for L in lens) * hkv
    return {"bytes": 4.0 * sum(lens) * hkv + kept * (2 * row + 4 + 4 + 4), "flops": 2.0 * kept * d}


# ------------------------------------------------------------------ the inputs

def _pow2_scale(amax):
    """The smallest power of two s (not under 2^-117) with amax <= 448 s."""
    m, e = torch.frexp(amax)  # amax = m 2^e, 1/2 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=MIN_EXP)
    e = torch.where(amax == 0, torch.full_like(e, MIN_EXP), e)
    return torch.ldexp(torch.ones_like(amax), e)


def _quantised(x, block):
    """[..., rows, d] in 32 bits -> codes and the blocks' scales."""
    b = x.reshape(*x.shape[:-2], x.shape[-2] // block, block, x.shape[-1])
    s = _pow2_scale(b.abs().amax(dim=(-2, -1)))
    return (b / s[..., None, None]).to(torch.float8_e4m3fn).reshape(x.shape), s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(seed)
    S, H, d, block, cap = case["n_seqs"], case["hkv"], case["d"], case["block"], _capacity(case)
    dt = DT[case["dtype"]]
    lens, new = _lens(case)
    perm = torch.randperm(S, generator=g, device=dev)
    st = {"case": case, "max_len": max(lens),
          "lens": torch.tensor(lens, dtype=torch.int32, device=dev)[perm].contiguous(),
          "n_new": torch.tensor(new, dtype=torch.int32, device=dev)[perm].contiguous()}
    f8 = torch.float8_e4m3fn
    st["k8"] = torch.empty(S, H, cap, d, dtype=f8, device=dev)
    st["v8"] = torch.empty(S, H, cap, d, dtype=f8, device=dev)
    st["ks"] = torch.empty(S, H, cap // block, device=dev)
    st["vs"] = torch.empty(S, H, cap // block, device=dev)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    # a few outlier channels of the keys, one direction that the queries of a
    # head like and a share of its keys have, and magnitudes that drift along
    # the cache, so that neighbouring blocks have other scales
    heavy = 1.0 + 5.0 * (torch.rand(H, 1, d, generator=g, device=dev) < 0.03)
    liked = torch.nn.functional.normalize(randn(H, 1, d), dim=-1)
    drift = torch.exp2(torch.sin(torch.arange(cap, device=dev) / 97.0))[:, None]
    for s in range(S):  # rows past a sequence's length hold rows of an older one
        share = (torch.rand(H, cap, 1, generator=g, device=dev) < 0.02).float()
        k = (randn(H, cap, d) + 4.0 * share * liked) * heavy
        st["k8"][s], st["ks"][s] = _quantised(k, block)
        st["v8"][s], st["vs"][s] = _quantised(randn(H, cap, d) * drift, block)
    if case["op"] == "append":
        T = case["T"]
        st["k_new"] = (randn(S, H, T, d) * heavy).to(dt)
        st["v_new"] = (2.0 * randn(S, H, T, d)).to(dt)
    elif case["op"] == "attend":
        T, hq = case["T"], case["hq"]
        q = (randn(S, H, hq // H, T, d) + 3.0 * liked[:, None]) / heavy[:, None]
        st["q"] = q.reshape(S, hq, T, d).to(dt)
        st["out"] = torch.zeros(S, hq, T, d, dtype=dt, device=dev)
        st["lse"] = torch.zeros(S, hq, T, device=dev)
        if case["weights"]:
            st["w_in"] = torch.rand(S, H, cap, generator=g, device=dev)
            st["w_out"] = torch.zeros(S, H, cap, device=dev)
    else:
        # accumulated weights are heavy-tailed, and many positions have none
        w = torch.exp(2.0 * randn(S, H, cap) - 4.0)
        st["w"] = torch.where(torch.rand(S, H, cap, generator=g, device=dev) < 0.15, 0.0, w)
        dcap = (case["K"] + block - 1) // block * block
        st["dst"] = {"k8": torch.zeros(S, H, dcap, d, dtype=f8, device=dev),
                     "v8": torch.zeros(S, H, dcap, d, dtype=f8, device=dev),
                     "ks": torch.zeros(S, H, dcap // block, device=dev),
                     "vs": torch.zeros(S, H, dcap // block, device=dev),
                     "w": torch.zeros(S, H, dcap, device=dev),
                     "idx": torch.zeros(S, H, case["K"], dtype=torch.int32, device=dev),
                     "lens": torch.zeros(S, dtype=torch.int32, device=dev)}
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    if own:
        return _run_own(st)
    return {"append": _append, "attend": _attend, "evict": _evict}[st["case"]["op"]](st)


def _run_own(st):
    from kv_cache_compression_bkv_b200 import bkv

    c = st["case"]
    if "geom" not in st:  # the handle and the workspace that a decode loop keeps
        st["geom"] = bkv.geometry8_of(st["k8"], st["ks"], c["hq"], DT[c["dtype"]])
        if c["op"] == "attend":
            n = bkv.bkv_cache8_workspace_size(st["geom"], st["max_len"], c["T"], 0, c["weights"])
        elif c["op"] == "evict":
            n = bkv.bkv_cache8_workspace_size(st["geom"], st["max_len"], 0, c["K"], False)
            st["dst_geom"] = bkv.geometry8_of(st["dst"]["k8"], st["dst"]["ks"], c["hq"],
                                              DT[c["dtype"]])
        else:
            n = 0
        st["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device=st["k8"].device)
    n_new = st["n_new"] if c.get("ragged") else None
    if c["op"] == "append":
        bkv.bkv_cache8_append(st["geom"], st["k8"], st["v8"], st["ks"], st["vs"], st["lens"],
                              st["k_new"], st["v_new"], c["T"], n_new)
        return {"k": st["k8"], "v": st["v8"], "k_scale": st["ks"], "v_scale": st["vs"]}
    if c["op"] == "attend":
        bkv.bkv_cache8_attend(st["geom"], st["k8"], st["v8"], st["ks"], st["vs"], st["lens"],
                              st["max_len"], st["q"], c["T"], n_new, 0.0, st["out"], st["lse"],
                              st.get("w_in"), st.get("w_out"), c["decay"], st["ws"])
        return {"out": st["out"], "lse": st["lse"], "weights": st.get("w_out")}
    o = st["dst"]
    bkv.bkv_cache8_evict(st["geom"], st["k8"], st["v8"], st["ks"], st["vs"], st["w"], st["lens"],
                         st["max_len"], c["K"], c["sink"], c["recent"], st["dst_geom"], o["k8"],
                         o["v8"], o["ks"], o["vs"], o["w"], o["idx"], o["lens"], st["ws"])
    return {"k": o["k8"], "v": o["v8"], "k_scale": o["ks"], "v_scale": o["vs"],
            "weights": o["w"], "idx": o["idx"], "lens": o["lens"]}


def _append(st):
    c = st["case"]
    block, T = c["block"], c["T"]
    nb = (T + block - 2) // block + 1  # blocks that T rows can touch
    lens, n = st["lens"].long()[:, None], st["n_new"].long()[:, None]
    first = lens - n
    # [S, nb] block numbers, the last ones of the cache where the rows end there
    b = (first // block).clamp(max=st["ks"].shape[2] - nb) + torch.arange(nb, device=lens.device)
    rows = (b[:, :, None] * block + torch.arange(block, device=lens.device)).flatten(1)
    fresh = (rows >= first) & (rows < lens)                          # [S, rows]
    touched = fresh.view(-1, nb, block).any(2)
    held = b * block < first                                         # blocks with older rows
    s_idx = torch.arange(lens.shape[0], device=lens.device)[:, None]
    keep = (rows < first) & touched.repeat_interleave(block, 1)
    for codes, scales, x in ((st["k8"], st["ks"], st["k_new"]), (st["v8"], st["vs"], st["v_new"])):
        raw = codes.view(torch.uint8)
        old = raw[s_idx, :, rows]                                    # [S, rows, H, d]
        t = (rows - first).clamp(0, T - 1)
        new = x.float()[s_idx, :, t] * fresh[..., None, None]
        shape = (-1, nb, block) + new.shape[2:]
        amax = new.view(shape).abs().amax(dim=(2, 4))                # [S, nb, H]
        was = scales[s_idx, :, b]
        s = _pow2_scale(amax)
        s = torch.where(held[..., None], torch.maximum(s, was), s)
        before = old.view(torch.float8_e4m3fn).float() * was.repeat_interleave(block, 1)[..., None]
        val = torch.where(fresh[..., None, None], new, before)
        val = (val / s.repeat_interleave(block, 1)[..., None]).to(torch.float8_e4m3fn)
        put = (fresh | keep)[..., None, None]
        raw[s_idx, :, rows] = torch.where(put, val.view(torch.uint8), old)
        scales[s_idx, :, b] = torch.where(touched[..., None], s, was)
    return {"k": st["k8"], "v": st["v8"], "k_scale": st["ks"], "v_scale": st["vs"]}


def _attend(st):
    c = st["case"]
    S, H, d, T, Lm, block = c["n_seqs"], c["hkv"], c["d"], c["T"], st["max_len"], c["block"]
    G = c["hq"] // H
    lens, n = st["lens"].view(-1, 1, 1, 1), st["n_new"].view(-1, 1, 1, 1)
    j = torch.arange(Lm, device=lens.device)
    t = torch.arange(T, device=lens.device)
    there = (j < lens)[..., None].view(S, 1, Lm, 1)

    def values(codes, scales):
        x = codes[:, :, :Lm].float() * scales.repeat_interleave(block, 2)[:, :, :Lm, None]
        return torch.where(there, x, 0.0)

    q = st["q"].float().view(S, H, G * T, d)
    x = q @ values(st["k8"], st["ks"]).transpose(2, 3) * (1.0 / math.sqrt(d))
    sees = (t[:, None] < n) & (j < lens - n + t[:, None] + 1)        # [S, 1, T, Lm]
    sees = sees[:, :, None].expand(S, 1, G, T, Lm).reshape(S, 1, G * T, Lm)
    x = torch.where(sees, x, -math.inf)
    m = x.amax(3, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(3, keepdim=True)
    p = p / torch.where(l == 0, 1.0, l)
    o = (p @ values(st["v8"], st["vs"])).view(S, c["hq"], T, d)
    lse = (m + torch.log(l)).view(S, c["hq"], T)
    live = (t < n.view(S, 1, 1))
    out = torch.where(live[..., None], o.to(st["out"].dtype), st["out"])
    lse = torch.where(live, lse, st["lse"])
    w = None
    if c["weights"]:
        lens, n = lens[..., 0], n[..., 0]                            # [S, 1, 1]
        w = st["w_out"].clone()
        older = torch.where(j < lens - n, c["decay"] * st["w_in"][:, :, :Lm], 0.0)
        w[:, :, :Lm] = torch.where((j < lens) & (n > 0), older + p.sum(2), w[:, :, :Lm])
    return {"out": out, "lse": lse, "weights": w}


def _evict(st):
    c, o = st["case"], st["dst"]
    block, K, Lm = c["block"], c["K"], st["max_len"]
    lens = st["lens"].view(-1, 1, 1)
    j = torch.arange(Lm, device=lens.device)
    rank = torch.where((j < c["sink"]) | (j >= lens - c["recent"]), math.inf, st["w"][:, :, :Lm])
    rank = torch.where(j < lens, rank, -math.inf)
    # the K best, ties to the lower position, in ascending order
    idx = torch.sort(rank, dim=2, descending=True, stable=True).indices[:, :, :K]
    idx = torch.sort(idx, dim=2).values                              # [S, H, min(K, Lm)]
    kept = torch.minimum(lens, torch.full_like(lens, K))             # [S, 1, 1]
    i = torch.arange(idx.shape[2], device=lens.device)
    nb = (idx.shape[2] + block - 1) // block
    full = torch.arange(nb * block, device=lens.device) < kept       # [S, 1, nb*block]
    some = torch.arange(nb, device=lens.device) * block < kept       # blocks with a row
    src = torch.nn.functional.pad(idx, (0, nb * block - idx.shape[2]))
    got = {}
    for name, codes, scales in (("k", st["k8"], st["ks"]), ("v", st["v8"], st["vs"])):
        at = src[..., None].expand(*src.shape, codes.shape[3])
        raw = codes.view(torch.uint8).gather(2, at).view(torch.float8_e4m3fn)
        x = raw.float() * scales.gather(2, src // block)[..., None]
        new, s = _quantised(torch.where(full[..., None], x, 0.0), block)
        rows = o[name + "8"].view(torch.uint8).clone()
        rows[:, :, :nb * block] = torch.where(full[..., None], new.view(torch.uint8),
                                              rows[:, :, :nb * block])
        got[name] = rows.view(torch.float8_e4m3fn)
        got[name + "_scale"] = o[name + "s"].clone()
        got[name + "_scale"][:, :, :nb] = torch.where(some, s, got[name + "_scale"][:, :, :nb])
    got["weights"] = o["w"].clone()
    live = i < kept
    got["weights"][:, :, :idx.shape[2]] = torch.where(
        live, st["w"].gather(2, idx), got["weights"][:, :, :idx.shape[2]])
    got["idx"] = o["idx"].clone()
    got["idx"][:, :, :idx.shape[2]] = torch.where(live, idx.int(), got["idx"][:, :, :idx.shape[2]])
    got["lens"] = kept.view(-1).int()
    return got


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "evict": _exact_evict}[case["op"]](st)


def _e4m3_exact(x):
    """The e4m3 value next to x, ties to even: steps of 2^(e-3) in the binade
    2^e, and of 2^-9 below 2^-6."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    e = torch.where(x.abs() < torch.exp2(e), e - 1, e)       # log2 rounded up
    e = torch.where(x.abs() >= torch.exp2(e + 1), e + 1, e)  # log2 rounded down
    step = torch.exp2(e.clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _scale_exact(amax):
    e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / E4M3_MAX))
    e = torch.where(amax > E4M3_MAX * torch.exp2(e), e + 1, e)
    e = torch.where(amax <= E4M3_MAX * torch.exp2(e - 1), e - 1, e)
    return torch.exp2(e.clamp(min=MIN_EXP))


def _exact_append(st):
    block = st["case"]["block"]
    got = {}
    for name, codes, scales, x in (("k", st["k8"], st["ks"], st["k_new"]),
                                   ("v", st["v8"], st["vs"], st["v_new"])):
        code, scale = codes.double(), scales.double()
        for s, (L, n) in enumerate(zip(st["lens"].tolist(), st["n_new"].tolist())):
            for b in range((L - n) // block, -(-L // block) if n else 0):
                r0, r1 = max(b * block, L - n), min((b + 1) * block, L)
                new = x[s, :, r0 - (L - n):r1 - (L - n)].double()
                want = _scale_exact(new.abs().amax(dim=(1, 2)))
                if r0 > b * block:  # older rows stay, moved to a larger scale where one is needed
                    want = torch.maximum(want, scale[s, :, b])
                    old = code[s, :, b * block:r0] * (scale[s, :, b] / want)[:, None, None]
                    code[s, :, b * block:r0] = _e4m3_exact(old)
                code[s, :, r0:r1] = _e4m3_exact(new / want[:, None, None])
                scale[s, :, b] = want
        got[name], got[name + "_scale"] = code, scale
    return {k: got[k] for k in ("k", "v", "k_scale", "v_scale")}


def _exact_attend(st):
    c = st["case"]
    H, G, T, block = c["hkv"], c["hq"] // c["hkv"], c["T"], c["block"]
    out, lse = st["out"].double(), st["lse"].double()
    w = st["w_out"].double() if c["weights"] else None
    for s, (L, n) in enumerate(zip(st["lens"].tolist(), st["n_new"].tolist())):
        if n == 0:
            continue
        row = torch.arange(L, device=out.device) // block
        hidden = torch.arange(L, device=out.device) > torch.arange(L - n, L, device=out.device)[:, None]
        for h in range(H):
            k = st["k8"][s, h, :L].double() * st["ks"][s, h].double()[row, None]
            v = st["v8"][s, h, :L].double() * st["vs"][s, h].double()[row, None]
            total = torch.zeros(L, dtype=torch.float64, device=out.device)
            for hq in range(h * G, (h + 1) * G):
                x = st["q"][s, hq, :n].double() @ k.T / math.sqrt(c["d"])
                x[hidden] = -math.inf
                z = torch.logsumexp(x, dim=1)
                p = torch.exp(x - z[:, None])
                out[s, hq, :n], lse[s, hq, :n] = p @ v, z
                total += p.sum(0)
            if w is not None:
                total[:L - n] += c["decay"] * st["w_in"][s, h, :L - n].double()
                w[s, h, :L] = total
    return {"out": out, "lse": lse, "weights": w}


def _exact_evict(st):
    c, o = st["case"], st["dst"]
    block, K, sink = c["block"], c["K"], c["sink"]
    got = {"k": o["k8"].double(), "v": o["v8"].double(), "k_scale": o["ks"].double(),
           "v_scale": o["vs"].double(), "weights": o["w"].double(), "idx": o["idx"].clone(),
           "lens": o["lens"].clone()}
    for s, L in enumerate(st["lens"].tolist()):
        n = min(L, K)
        got["lens"][s] = n
        for h in range(c["hkv"]):
            w = st["w"][s, h, :L].double()
            if L > K:
                tail = L - c["recent"]
                # by weight, then by position: the order of (-w, j)
                order = torch.argsort(-w[sink:tail], stable=True)[:K - sink - c["recent"]] + sink
                every = torch.arange(L, device=w.device)
                idx = torch.cat([every[:sink], order.sort().values, every[tail:]])
            else:
                idx = torch.arange(L, device=w.device)
            got["idx"][s, h, :n] = idx.int()
            got["weights"][s, h, :n] = w[idx]
            nb = -(-n // block)
            for name, codes, scales in (("k", st["k8"], st["ks"]), ("v", st["v8"], st["vs"])):
                x = codes[s, h, :L].double()[idx] * scales[s, h].double()[idx // block, None]
                full = torch.zeros(nb * block, c["d"], dtype=torch.float64, device=w.device)
                full[:n] = x
                sc = _scale_exact(full.view(nb, -1).abs().amax(1))
                got[name][s, h, :n] = _e4m3_exact(full / sc.repeat_interleave(block)[:, None])[:n]
                got[name + "_scale"][s, h, :nb] = sc
    return got
