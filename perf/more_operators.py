"""Rotary positions, the 8-bit cache's append with them, decode attention of sequences that share a prefix, and the groups of
such sequences, as measured cases: inputs, the plain form of each operator in elementary torch operations, and the framework's
calls.

A cache page holds 16 tokens of every KV head: codes [Hkv][2 = K, V][16][D] of one byte (e4m3 or int8) and one fp32 scale,
a power of two, per (KV head, K | V).  A value is code * scale.

Rotary positions turn the pair i of a head's first rotary_dim channels, (i, i + rotary_dim / 2) or, interleaved, (2 i, 2 i + 1),
by position * frequency_i."""

import math
import random

import torch

own = False

P = 16
E4M3, INT8 = 0, 1
FMAX = (448.0, 127.0)       # largest magnitude of a code
EXP_LO, EXP_HI = -100, (119, 121)  # a block's scale is 2^e with e in this range
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # the queries and keys of one step of a serving batch, before they go to a cache that takes rotated keys
        dict(name="rope 64 tokens", kind="rope", tokens=64, hq=32, hkv=8, d=128, rotary=128, interleaved=False, dtype="bf16",
             base=10000.0, scaling="none", top=16384, fused=True),
        # a small model with half of each head rotated, in fp32, at positions far behind what it was trained on
        dict(name="rope fp32 part of the head", kind="rope", tokens=777, hq=6, hkv=2, d=64, rotary=32, interleaved=True,
             dtype="fp32", base=10000.0, scaling="linear", top=2000000000, fused=False),
        # a long prompt, its queries and keys slices of one projection's output, frequencies scaled for long contexts
        dict(name="rope prompt 16384", kind="rope", tokens=16384, hq=32, hkv=8, d=128, rotary=128, interleaved=False,
             dtype="bf16", base=1000000.0, scaling="yarn", top=131072, fused=True),
        # every running sequence of a serving batch adds the token it has just produced
        dict(name="rope append 64 x 1 e4m3", kind="append", fmt=E4M3, batch=64, hq=32, hkv=8, d=128, rotary=128,
             interleaved=False, base=500000.0, scaling="bands", new_lo=1, new_hi=1, old_lo=1000, old_hi=16000, lens_seed=1),
        # a few drafted tokens of each of eight sequences, a quarter of each head without positions
        dict(name="rope append drafts int8", kind="append", fmt=INT8, batch=8, hq=16, hkv=4, d=128, rotary=96,
             interleaved=True, base=10000.0, scaling="none", new_lo=1, new_hi=8, old_lo=100, old_hi=3000, lens_seed=2),
        # prompts (and a follow-up turn) of several users, written at once
        dict(name="rope append prompts e4m3", kind="append", fmt=E4M3, batch=6, hq=32, hkv=8, d=128, rotary=128,
             interleaved=False, base=1000000.0, scaling="yarn", new_lo=500, new_hi=16384, old_lo=0, old_hi=100, lens_seed=3),
        # a small model's few samples of one short prompt
        dict(name="shared 6 small int8", kind="shared", fmt=INT8, hq=6, hkv=2, d=64, groups=1, size_lo=6, size_hi=6, alone=0,
             prefix_lo=700, prefix_hi=700, own_lo=1, own_hi=100, lens_seed=4),
        # users of a few assistants with their instructions, and some without
        dict(name="shared 4 groups int8", kind="shared", fmt=INT8, hq=32, hkv=8, d=128, groups=4, size_lo=3, size_hi=12,
             alone=5, prefix_lo=1000, prefix_hi=8192, own_lo=0, own_hi=2000, lens_seed=5),
        # parallel samples of one long prompt
        dict(name="shared 64 of 16384 e4m3", kind="shared", fmt=E4M3, hq=32, hkv=8, d=128, groups=1, size_lo=64, size_hi=64,
             alone=0, prefix_lo=16384, prefix_hi=16384, own_lo=1, own_hi=1024, lens_seed=6),
        # many candidates over long documents
        dict(name="shared 2 x 128 of 32768 e4m3", kind="shared", fmt=E4M3, hq=64, hkv=8, d=128, groups=2, size_lo=128,
             size_hi=128, alone=0, prefix_lo=30000, prefix_hi=32768, own_lo=1, own_hi=512, lens_seed=7),
        # the same batches' page tables, before the first layer of a step
        dict(name="groups of 37", kind="groups", groups=4, size_lo=3, size_hi=12, alone=5, prefix_lo=1000, prefix_hi=8192,
             own_lo=0, own_hi=2000, min_pages=1, max_groups=16, lens_seed=5),
        dict(name="groups of 512", kind="groups", groups=24, size_lo=1, size_hi=40, alone=20, prefix_lo=100, prefix_hi=32768,
             own_lo=0, own_hi=512, min_pages=8, max_groups=32, lens_seed=8),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** rng.random())) - 1))


def _draw_rotary(rng, d):
    return dict(rotary=16 * rng.randint(1, d // 16), interleaved=rng.random() < 0.5,
                base=rng.choice([10000.0, 500000.0, 1000000.0]), scaling=rng.choice(["none", "linear", "yarn", "bands"]))


def draw(rng):
    kind = rng.choice(["rope", "append", "append", "shared", "shared", "shared", "groups"])
    seed = rng.randrange(1 << 30)
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.randint(1, 8)
    if kind == "rope":
        return dict(kind=kind, tokens=_spread(rng, 1, 12000), hq=min(hq, 32), hkv=hkv if hq <= 32 else 8, d=d,
                    dtype=rng.choice(list(TYPES)), top=_spread(rng, 100, 2000000000), fused=rng.random() < 0.5,
                    **_draw_rotary(rng, d))
    if kind == "append":
        c = dict(kind=kind, fmt=rng.choice([E4M3, INT8]), batch=_spread(rng, 1, 96), hq=hq, hkv=hkv, d=d,
                 new_lo=rng.choice([0, 1]), new_hi=_spread(rng, 1, 12000), old_lo=0, old_hi=_spread(rng, 1, 8000),
                 lens_seed=seed, **_draw_rotary(rng, d))
        while c["batch"] > 1 and c["batch"] * ((c["new_hi"] + c["old_hi"] / 4) * hkv + c["new_hi"] * hq / 2) * d > 4e7:
            c["batch"] = c["batch"] // 2
        return c
    c = dict(kind=kind, groups=_spread(rng, 1, 12), size_lo=1, size_hi=_spread(rng, 2, 100), alone=_spread(rng, 0, 20),
             prefix_lo=rng.choice([16, 500]), prefix_hi=_spread(rng, 600, 30000), own_lo=rng.choice([0, 1, 50]),
             own_hi=_spread(rng, 60, 2000), lens_seed=seed)
    if kind == "groups":
        return dict(c, min_pages=_spread(rng, 1, 40), max_groups=rng.choice([2, 8, 64]))
    c.update(fmt=rng.choice([E4M3, INT8]), hq=hq, hkv=hkv, d=d)
    while c["size_hi"] > 2 and (c["groups"] * c["size_hi"] + c["alone"]) * hq * c["prefix_hi"] > 1e8:
        c["size_hi"] = c["size_hi"] // 2
    while c["groups"] > 1 and c["groups"] * c["size_hi"] * hq * c["prefix_hi"] > 1e8:
        c["groups"] = c["groups"] // 2
    while c["own_hi"] > 60 and (c["groups"] * c["size_hi"] + c["alone"]) * c["own_hi"] * hkv * d > 1.5e8:
        c["own_hi"] = max(60, c["own_hi"] // 2)
    return c


# ---- sizes: the same for every seed, so that the work of a case is known -------------------------------------------------


def _lengths(case):
    """append: per sequence (tokens in the cache, of which new)."""
    rng = random.Random(case["lens_seed"])
    got = []
    for _ in range(case["batch"]):
        new = rng.randint(case["new_lo"], case["new_hi"])
        got.append((rng.randint(case["old_lo"], case["old_hi"]) + new, new))
    if not any(n for _, n in got):
        got[0] = (got[0][0] + case["new_hi"], case["new_hi"])
    return got


def _families(case):
    """Per group (tokens in the shared pages, the members' tokens behind them); the sequences alone are a group without a
    prefix."""
    rng = random.Random(case["lens_seed"])
    got = []
    for _ in range(case["groups"]):
        prefix = rng.randint(case["prefix_lo"], case["prefix_hi"]) // P * P  # what a fork shares: whole pages
        size = rng.randint(case["size_lo"], case["size_hi"])
        got.append((prefix, [rng.randint(case["own_lo"], case["own_hi"]) for _ in range(size)]))
    got.append((0, [rng.randint(case["own_lo"], case["own_hi"]) for _ in range(case["alone"])]))
    return got


def _pages(n):
    return -(-n // P)


def work(case):
    kind = case["kind"]
    if kind == "rope":
        size = 4 if case["dtype"] == "fp32" else 2
        part = case["tokens"] * (case["hq"] + case["hkv"])
        return {"bytes": part * case["d"] * size * 2 + case["tokens"] * 4, "flops": part * case["rotary"] * 3}
    if kind == "append":
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        lens = _lengths(case)
        t = sum(n for _, n in lens)
        blocks = sum(_pages(L) - (L - n) // P for L, n in lens if n)
        return {"bytes": t * d * (hq * 2 * 2 + hkv * 2 * 3) + blocks * hkv * 2 * 4, "flops": t * (hq + hkv) * case["rotary"] * 3}
    families = _families(case)
    if kind == "groups":
        entries = sum(len(m) * (p // P) + sum(n // P for n in m) for p, m in families)
        members = sum(len(m) for _, m in families)
        return {"bytes": 4 * (entries + 2 * members), "flops": 0}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    rows = sum(len(m) for _, m in families)
    tokens = sum((p if m else 0) + sum(m) for p, m in families)
    pairs = sum(p * len(m) + sum(m) for p, m in families)
    return {"bytes": tokens * hkv * 2 * (d + 4 / P) + rows * hq * d * 4, "flops": 4 * d * hq * pairs}


# ---- inputs -----------------------------------------------------------------------------------------------------------

SCALINGS = {
    "none": None,
    "linear": dict(kind="linear", factor=8.0),
    "yarn": dict(kind="yarn", factor=4.0, original_max_position=32768),
    "bands": dict(kind="bands", factor=8.0, original_max_position=8192, low_freq_factor=1.0, high_freq_factor=4.0),
}


def _scale_of(amax, fmt):
    """The smallest power of two 2^e with amax <= largest code * 2^e, e within its range (fp32, exact)."""
    m, x = torch.frexp(amax)
    top = 0.875 if fmt == E4M3 else 0.9921875
    e = torch.where(m <= top, x - (9 if fmt == E4M3 else 7), x - (8 if fmt == E4M3 else 6))
    e = torch.where(amax > 0, e, torch.full_like(e, EXP_LO)).clamp(EXP_LO, EXP_HI[fmt])
    return ((e.int() + 127) << 23).view(torch.float32)


def _round(x, fmt):
    """Codes (as uint8) of x, in units of its block's scale."""
    x = x.clamp(-FMAX[fmt], FMAX[fmt])
    if fmt == E4M3:
        return x.to(torch.float8_e4m3fn).view(torch.uint8)
    return x.round().to(torch.int8).view(torch.uint8)


def _values(codes, fmt):
    return codes.view(torch.float8_e4m3fn if fmt == E4M3 else torch.int8).float()


def _keys(n, hkv, d, mean, factor, g):
    """Keys with per-channel means and a few channels that are 15 times the others, as trained models have them."""
    return (torch.randn(n, hkv, d, device="cuda", generator=g) + mean) * factor


def _key_shape(hkv, d, g):
    mean = 3 * torch.randn(hkv, d, device="cuda", generator=g)
    factor = torch.ones(hkv, d, device="cuda")
    factor.scatter_(1, torch.rand(hkv, d, device="cuda", generator=g).argsort(1)[:, :6], 15.0)
    return mean, factor


def _cache(num_pages, hkv, d, fmt, mean, factor, g):
    codes = torch.empty(num_pages, hkv, 2, P, d, dtype=torch.uint8, device="cuda")
    scales = torch.empty(num_pages, hkv, 2, dtype=torch.float32, device="cuda")
    step = max(1, (1 << 27) // (hkv * P * d))
    for p0 in range(0, num_pages, step):
        n = min(step, num_pages - p0)
        k = _keys(n * P, hkv, d, mean, factor, g).view(n, P, hkv, d).transpose(1, 2)
        v = torch.randn(n, hkv, P, d, device="cuda", generator=g)
        x = torch.stack([k, v], 2).bfloat16().float()
        s = _scale_of(x.abs().amax((3, 4)), fmt)
        codes[p0:p0 + n] = _round(x / s[..., None, None], fmt)
        scales[p0:p0 + n] = s
    return codes, scales


def _cuda32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _rows(case, tokens, g, heads):
    """Rows of each of the heads' counts: slices of one projection's output."""
    d = case["d"]
    x = torch.randn(tokens, sum(heads), d, device="cuda", generator=g)
    mean, factor = _key_shape(case["hkv"], d, g)
    x[:, heads[0]:heads[0] + heads[1]] = _keys(tokens, heads[1], d, mean, factor, g)
    return torch.split(x.to(TYPES[case.get("dtype", "bf16")]), heads, 1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 29)
    kind = case["kind"]
    st = dict(case=case)
    if kind == "rope":
        t, hq, hkv = case["tokens"], case["hq"], case["hkv"]
        st["dims"] = dict(num_q_heads=hq, num_kv_heads=hkv, head_dim=case["d"], page_size=P, group_size=64, num_pages=1,
                          max_pages_per_seq=1)
        st["pos"] = torch.randint(0, case["top"], (t,), device="cuda", generator=g, dtype=torch.int32)
        parts = _rows(case, t, g, [hq, hkv, hkv])
        st["q"], st["k"] = parts[:2] if case["fused"] else [x.contiguous() for x in parts[:2]]
        return st
    if kind == "append":
        return _prepare_append(case, g, st)
    families = _families(case)
    lens = [p + n for p, m in families for n in m]
    order = torch.randperm(len(lens), device="cuda", generator=g)  # the slots of a batch in no order
    shared = [p // P for p, m in families if m]
    n_pages = sum(shared) + sum(_pages(n) for _, m in families for n in m) + 5
    ids = torch.randperm(n_pages, device="cuda", generator=g).to(torch.int32)
    table = torch.full((len(lens), max([1] + [_pages(n) for n in lens])), -1, dtype=torch.int32, device="cuda")
    at = b = 0
    for p, m in families:
        if m:
            table[b:b + len(m), :p // P] = ids[at:at + p // P]
            at += p // P
        for n in m:
            table[b, p // P:p // P + _pages(n)] = ids[at:at + _pages(n)]
            at += _pages(n)
            b += 1
    st["table"], st["lens"] = table[order].contiguous(), _cuda32(lens)[order].contiguous()
    hq, hkv, d = case.get("hq", 8), case.get("hkv", 8), case.get("d", 128)
    st["dims"] = dict(num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=P, group_size=64, num_pages=n_pages,
                      max_pages_per_seq=table.shape[1])
    if kind == "groups":
        return st
    st["codes"], st["scales"] = _cache(n_pages, hkv, d, case["fmt"], *_key_shape(hkv, d, g), g)
    st["q"] = torch.randn(len(lens), hq, d, device="cuda", generator=g).bfloat16()
    starts = [0]
    for _, m in families:
        starts.append(starts[-1] + len(m))
    st["members"] = torch.argsort(order).to(torch.int32)  # the slots of group after group
    st["start"], st["prefix"] = _cuda32(starts), _cuda32([p for p, _ in families])
    st["max_len"] = max(lens)
    st["max_prefix"] = max(p for p, m in families if m)
    st["max_own"] = max(n for _, m in families for n in m)
    return st


def _prepare_append(case, g, st):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    pairs = _lengths(case)
    lens = [n for n, _ in pairs]
    n_pages = sum(_pages(n) for n in lens) + 5
    ids = torch.randperm(n_pages, device="cuda", generator=g).to(torch.int32)
    table = torch.full((len(lens), max(_pages(n) for n in lens)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        table[b, :_pages(n)] = ids[at:at + _pages(n)]
        at += _pages(n)
    start = [0]
    for _, n in pairs:
        start.append(start[-1] + n)
    st.update(table=table, lens=_cuda32(lens), start=_cuda32(start), max_new=max(n for _, n in pairs),
              dims=dict(num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=P, group_size=64, num_pages=n_pages,
                        max_pages_per_seq=table.shape[1]))
    st["codes"], st["scales"] = _cache(n_pages, hkv, d, case["fmt"], *_key_shape(hkv, d, g), g)
    st["q"], st["k"], st["v"] = _rows(case, start[-1], g, [hq, hkv, hkv])
    b, pos = _places(st, start[-1])
    st["touched"] = torch.unique(table[b, pos // P]).long()
    return st


# ---- one pass ----------------------------------------------------------------------------------------------------------


def run(st):
    kind = st["case"]["kind"]
    if kind == "rope":
        return _rope_own(st) if own else _rope(st)
    if kind == "append":
        q = _append_own(st) if own else _append(st)
        if st["case"]["fmt"] == E4M3:
            return q, st["codes"].view(torch.float8_e4m3fn), st["scales"]
        at = st["touched"]  # the values that the int8 codes stand for (exact in bf16)
        return q, (_values(st["codes"][at], INT8) * st["scales"][at][..., None, None]).bfloat16(), st["scales"]
    if kind == "shared":
        return _shared_own(st) if own else _shared(st)
    return _groups_own(st) if own else _groups(st)


def _rope_plan_own(oscar, st):
    """The frequencies that a program keeps for its model."""
    c = st["case"]
    if "rope" not in st:
        st["rope"] = oscar.Rope(c["rotary"], base=c["base"], interleaved=c["interleaved"], scaling=SCALINGS[c["scaling"]])
    return st["rope"]


def _rope_own(st):
    import int2_rotated_kv_append_gb300 as oscar
    q = torch.empty(st["q"].shape, dtype=st["q"].dtype, device="cuda")
    k = torch.empty(st["k"].shape, dtype=st["k"].dtype, device="cuda")
    oscar.oscar_rope(st["dims"], _rope_plan_own(oscar, st), st["pos"], st["q"], st["k"], q, k)
    return q, k


def _append_own(st):
    import int2_rotated_kv_append_gb300 as oscar
    c = st["case"]
    q = torch.empty(st["q"].shape, dtype=torch.bfloat16, device="cuda")
    oscar.oscar_kv8_rope_append(st["dims"], _rope_plan_own(oscar, st), c["fmt"], c["batch"], st["max_new"], st["q"], st["k"],
                                st["v"], st["start"], None, st["table"], st["lens"], st["codes"], st["scales"], q)
    return q


def _shared_own(st):
    import int2_rotated_kv_append_gb300 as oscar
    batch, groups = st["q"].shape[0], st["prefix"].shape[0]
    bounds = (st["max_len"], st["max_prefix"], st["max_own"])
    if "work" not in st:
        st["work"] = torch.empty(oscar.oscar_kv8_decode_shared_workspace_bytes(st["dims"], batch, *bounds, batch, groups),
                                 dtype=torch.uint8, device="cuda")
    out = torch.empty_like(st["q"])
    oscar.oscar_kv8_decode_shared(st["dims"], st["case"]["fmt"], batch, *bounds, st["q"], st["codes"], st["scales"],
                                  st["table"], st["lens"], st["members"], st["start"], st["prefix"], 0.0, out, st["work"])
    return out


def _groups_own(st):
    import int2_rotated_kv_append_gb300 as oscar
    c, batch = st["case"], st["lens"].shape[0]
    if "work" not in st:
        st["work"] = torch.empty(oscar.oscar_pages_groups_workspace_bytes(st["dims"], batch), dtype=torch.uint8, device="cuda")
    members = torch.empty(batch, dtype=torch.int32, device="cuda")
    start = torch.empty(c["max_groups"] + 1, dtype=torch.int32, device="cuda")
    prefix = torch.empty(c["max_groups"], dtype=torch.int32, device="cuda")
    oscar.oscar_pages_groups(st["dims"], c["min_pages"], st["table"], st["lens"], members, start, prefix, st["work"])
    return members, start, prefix


# ---- the plain forms ---------------------------------------------------------------------------------------------------


def _frequencies(rotary, base, scaling):
    """Radians per position of every pair, and the factor on what is rotated."""
    f = [base ** (-2 * i / rotary) for i in range(rotary // 2)]
    if scaling is None:
        return f, 1.0
    s = scaling["factor"]
    if scaling["kind"] == "linear":
        return [x / s for x in f], 1.0
    length = scaling["original_max_position"]
    if scaling["kind"] == "yarn":
        turns = lambda n: rotary * math.log(length / (n * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        low, high = max(math.floor(turns(32.0)), 0), min(math.ceil(turns(1.0)), rotary - 1)
        ramp = [min(max((i - low) / max(high - low, 0.001), 0.0), 1.0) for i in range(len(f))]
        return [x / s * r + x * (1 - r) for x, r in zip(f, ramp)], 0.1 * math.log(s) + 1
    lo, hi = scaling["low_freq_factor"], scaling["high_freq_factor"]
    share = [min(max((length * x / (2 * math.pi) - lo) / (hi - lo), 0.0), 1.0) for x in f]
    return [x * w + x / s * (1 - w) for x, w in zip(f, share)], 1.0


def _turn(x, pos, st):
    """Rows x [tokens][heads][D], rotated, in 32 bits; the angles in 64."""
    c = st["case"]
    n = c["rotary"]
    if "f" not in st:  # kept for the model
        f, st["magnitude"] = _frequencies(n, c["base"], SCALINGS[c["scaling"]])
        st["f"] = torch.tensor(f, dtype=torch.float64, device="cuda")
    angle = pos.double()[:, None] * st["f"]
    cos, sin = (st["magnitude"] * angle.cos()).float()[:, None], (st["magnitude"] * angle.sin()).float()[:, None]
    x = x.float()
    if c["interleaved"]:
        a, b = x[..., 0:n:2], x[..., 1:n:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :n // 2], x[..., n // 2:n]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., n:]], -1)


def _rope(st):
    return _turn(st["q"], st["pos"], st).to(st["q"].dtype), _turn(st["k"], st["pos"], st).to(st["k"].dtype)


def _places(st, tokens):
    """Sequence and position of each of the rows that are the last of their sequences."""
    start = st["start"].long()
    t = torch.arange(tokens, device="cuda")
    b = torch.searchsorted(start[1:], t, right=True)
    return b, st["lens"].long()[b] - start[b + 1] + t


def _append(st):
    fmt, codes, scales = st["case"]["fmt"], st["codes"], st["scales"]
    b, pos = _places(st, st["k"].shape[0])
    x = torch.stack([_turn(st["k"], pos, st), st["v"].float()], 2)
    page, row = st["table"][b, pos // P].long(), pos % P
    amax = torch.zeros_like(scales).index_reduce_(0, page, x.abs().amax(3), "amax")
    first = torch.full((scales.shape[0],), P, device="cuda").index_reduce_(0, page, row, "amin")
    last = torch.full((scales.shape[0],), -1, device="cuda").index_reduce_(0, page, row, "amax")
    at = (first < P).nonzero().flatten()
    old, need = scales[at], _scale_of(amax[at], fmt)
    new = torch.where((first[at] > 0)[:, None, None], torch.maximum(old, need), need)
    block = torch.zeros(scales.shape[0], dtype=torch.long, device="cuda")
    block[at] = torch.arange(at.numel(), device="cuda")
    vals = _values(codes[at], fmt) * (old / new)[..., None, None]
    vals[block[page], :, :, row] = x / new[block[page]][..., None]
    kept = torch.arange(P, device="cuda") > last[at, None]
    codes[at] = torch.where(kept[:, None, None, :, None], codes[at], _round(vals, fmt))
    scales[at] = new
    return _turn(st["q"], pos, st).bfloat16()


def _tokens(st, table, side):
    """K or V of the pages of a table [n][pages], [n][Hkv][positions][D]."""
    table = table.long().clamp(min=0)
    x = _values(st["codes"][:, :, side][table], st["case"]["fmt"]) * st["scales"][:, :, side][table][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _part(st, q, table, seen):
    """Queries q [n][rows][Hq][D] over the first seen[n] positions of the tables: largest logit, sum, weighted values."""
    n, rows, hq, d = q.shape
    hkv = st["case"]["hkv"]
    q = q.float().view(n, rows, hkv, hq // hkv, d).transpose(1, 2).reshape(n, hkv, -1, d)
    s = torch.matmul(q, _tokens(st, table, 0).transpose(2, 3)).mul_(d ** -0.5)
    hidden = torch.arange(s.shape[-1], device="cuda") >= seen[:, None]
    s.masked_fill_(hidden[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True).clamp(min=-1e30)
    s = s.sub_(m).exp_()
    got = [m, s.sum(-1, keepdim=True), torch.matmul(s, _tokens(st, table, 1))]
    return [x.view(n, hkv, rows, hq // hkv, -1).transpose(1, 2).reshape(n, rows, hq, -1) for x in got]


def _shared(st):
    members, start, prefix = st["members"].long(), st["start"].long(), st["prefix"].long()
    q, lens = st["q"][members], st["lens"].long()[members]
    n = members.numel()
    i = torch.arange(n, device="cuda")
    group = torch.searchsorted(start[1:], i, right=True)
    place = i - start[group]
    size = (start[1:] - start[:-1]) * (prefix > 0)
    # every group's prefix, once for all its members
    rows = q.new_zeros(prefix.numel(), int(size.max()), *q.shape[1:])
    has = prefix[group] > 0
    rows[group[has], place[has]] = q[has]
    first = st["table"][members[start[:-1].clamp(max=n - 1)], :max(1, st["max_prefix"] // P)]
    m0, l0, o0 = (x[group, place * has] for x in _part(st, rows, first, prefix))
    # every sequence's own positions
    j = torch.arange(max(1, _pages(st["max_own"])), device="cuda")
    at = (prefix[group] // P)[:, None] + j
    tail = st["table"][members[:, None], at.clamp(max=st["table"].shape[1] - 1)]
    m1, l1, o1 = (x[:, 0] for x in _part(st, q[:, None], tail, lens - prefix[group]))
    has = has[:, None, None]
    m0, l0, o0 = torch.where(has, m0, -1e30), l0 * has, o0 * has
    m = torch.maximum(m0, m1)
    w0, w1 = (m0 - m).exp(), (m1 - m).exp()
    out = torch.empty_like(st["q"])
    out[members] = ((o0 * w0 + o1 * w1) / (l0 * w0 + l1 * w1).clamp(min=1e-30)).bfloat16()
    return out


def _groups(st):
    """The sequences with the same first min_pages full pages, groups in the order of their first members and as many as there
    is room for; then all others."""
    c, table = st["case"], st["table"]
    k, room = c["min_pages"], c["max_groups"]
    full = st["lens"].long() // P
    b = torch.arange(table.shape[0], device="cuda")
    head = table[:, :k]
    same = (head[:, None] == head[None]).all(-1) & (full >= k)[:, None] & (full >= k)
    leader = torch.where(same.any(1), same.int().argmax(1), b)
    size = torch.zeros_like(b).index_add_(0, leader, torch.ones_like(b))
    leads = size > 1
    number = torch.where(leads, leads.long().cumsum(0) - 1, room)
    count = number[leads].amax(0, keepdim=True) + 1 if bool(leads.any()) else torch.zeros(1, dtype=torch.long, device="cuda")
    count = count.clamp(max=room - 1)
    group = torch.minimum(number[leader], count)
    j = torch.arange(table.shape[1], device="cuda")
    alike = (table == table[leader]) & (j < torch.minimum(full, full[leader])[:, None])
    depth = alike.long().cumprod(1).sum(1)
    prefix = torch.full((room + 1,), table.shape[1], device="cuda").index_reduce_(0, group, depth, "amin")
    g = torch.arange(room, device="cuda")
    prefix = torch.where(g < count, prefix[:room] * P, 0)
    members = torch.argsort(group * b.numel() + b)
    ends = torch.zeros(room, dtype=torch.long, device="cuda").index_add_(0, group, torch.ones_like(b)).cumsum(0)
    start = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), ends])
    return members.int(), start.int(), prefix.int()


# ---- 64 bits -----------------------------------------------------------------------------------------------------------


def exact(case, seed):
    kind = case["kind"]
    if kind == "groups":
        return None  # whole numbers
    st = prepare(case, seed)
    if kind == "rope":
        return _exact_turn(st["q"], st["pos"], case), _exact_turn(st["k"], st["pos"], case)
    return _exact_append(st) if kind == "append" else _exact_shared(st)


def _exact_turn(x, pos, case):
    """Every pair as a complex number, times magnitude * e^(i angle)."""
    n, base, how = case["rotary"], case["base"], SCALINGS[case["scaling"]]
    f = torch.exp(torch.arange(0, n, 2, device="cuda", dtype=torch.float64) * (-math.log(base) / n))
    magnitude = 1.0
    if how is not None and how["kind"] == "linear":
        f = f / how["factor"]
    elif how is not None and how["kind"] == "yarn":
        i = torch.arange(n // 2, device="cuda", dtype=torch.float64)
        at = [n * math.log(how["original_max_position"] / (b * 2 * math.pi)) / (2 * math.log(base)) for b in (32, 1)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), n - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        f = f * (1 - ramp * (1 - 1 / how["factor"]))
        magnitude = 1 + math.log(how["factor"]) / 10
    elif how is not None:
        wave = 2 * math.pi / f
        length, lo, hi = how["original_max_position"], how["low_freq_factor"], how["high_freq_factor"]
        smooth = (length / wave - lo) / (hi - lo)
        mid = (1 - smooth) * f / how["factor"] + smooth * f
        f = torch.where(wave < length / hi, f, torch.where(wave > length / lo, f / how["factor"], mid))
    angle = torch.outer(pos.double(), f)
    turn = torch.polar(torch.full_like(angle, magnitude), angle)
    y = x.double().clone()
    even, odd = (slice(0, n, 2), slice(1, n, 2)) if case["interleaved"] else (slice(0, n // 2), slice(n // 2, n))
    z = torch.complex(y[..., even], y[..., odd]) * turn[:, None]
    y[..., even], y[..., odd] = z.real, z.imag
    return y


def _two_to(e):
    """2^e as doubles, exactly (a power function may be off by a rounding)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _coded(x, fmt):
    """The nearest values that codes stand for (ties to even)."""
    if fmt == INT8:
        return x.round().clamp(-127, 127)
    m, e = torch.frexp(x)  # |m| in [0.5, 1): four bits of it are kept, fewer below 2^-6
    step = _two_to((e - 1).clamp(min=-6) - 3)
    return ((x / step).round() * step).clamp(-448, 448)


def _exact_append(st):
    case = st["case"]
    fmt = case["fmt"]
    codes, scales = _values(st["codes"], fmt).double(), st["scales"].double()
    start, table, lens = st["start"].tolist(), st["table"].tolist(), st["lens"].tolist()
    pos = torch.cat([torch.arange(L - start[b + 1] + start[b], L, device="cuda") for b, L in enumerate(lens)])
    kv = torch.stack([_exact_turn(st["k"], pos, case), st["v"].double()], 2)
    for b, L in enumerate(lens):
        t0, t1 = start[b], start[b + 1]
        p = L - (t1 - t0)
        while p < L:  # page by page
            n = min(L, (p // P + 1) * P) - p
            t = t1 - (L - p)
            page, r = table[b][p // P], p % P
            x = kv[t:t + n]
            m, e = torch.frexp((x.abs().amax((0, 3)) / FMAX[fmt]).clamp(min=2.0 ** -100))
            s = _two_to(torch.where(m == 0.5, e - 1, e))
            if r:
                s = torch.maximum(s, scales[page])
                codes[page, :, :, :r] = _coded(codes[page, :, :, :r] * (scales[page] / s)[..., None, None], fmt)
            codes[page, :, :, r:r + n] = _coded(x / s[..., None], fmt).permute(1, 2, 0, 3)
            scales[page] = s
            p += n
    q = _exact_turn(st["q"], pos, case)
    if fmt == E4M3:
        return q, codes, scales
    return q, (codes * scales[..., None, None])[st["touched"]], scales


def _exact_shared(st):
    c = st["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    if sum(st["lens"].tolist()) * hq * d * 4 > 4e12:
        return None
    for b, L in enumerate(st["lens"].tolist()):
        if L == 0:
            continue
        ids = st["table"][b, :_pages(L)].long()
        kv = _values(st["codes"][ids], c["fmt"]).double() * st["scales"][ids].double()[..., None, None]
        kv = kv.permute(1, 2, 0, 3, 4).reshape(hkv, 2, -1, d)[:, :, :L]
        q = st["q"][b].double().view(hkv, hq // hkv, d)
        w = torch.softmax(q @ kv[:, 0].transpose(1, 2) / d ** 0.5, -1)
        out[b] = (w @ kv[:, 1]).reshape(hq, d)
    return out
