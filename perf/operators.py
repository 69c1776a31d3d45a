"""The 8-bit paged KV cache, its attention (full, or a sliding window with sinks) and the operations on cache pages, as
measured cases: inputs, the plain form of each operator in elementary torch operations, and the framework's calls.

A cache page holds 16 tokens of every KV head: codes [Hkv][2 = K, V][16][D] of one byte (e4m3 or int8) and one fp32 scale,
a power of two, per (KV head, K | V).  A value is code * scale."""

import random

import torch

own = False

P = 16
E4M3, INT8 = 0, 1
FMAX = (448.0, 127.0)       # largest magnitude of a code
EXP_LO, EXP_HI = -100, (119, 121)  # a block's scale is 2^e with e in this range


def listed():
    return [
        # every running sequence of a serving batch adds the token it has just produced
        dict(name="append 64 x 1 e4m3", kind="append", fmt=E4M3, batch=64, hkv=8, d=128, new_lo=1, new_hi=1, old_lo=1000,
             old_hi=16000, lens_seed=1),
        # prompts (and a follow-up turn) of several users, written at once
        dict(name="append prompts int8", kind="append", fmt=INT8, batch=6, hkv=8, d=128, new_lo=500, new_hi=16384, old_lo=0,
             old_hi=100, lens_seed=2),
        # a small model answering a few short chats, with a window and sinks; one slot of the batch is empty
        dict(name="decode short int8 window", kind="decode", fmt=INT8, batch=5, hq=6, hkv=2, d=64, len_lo=0, len_hi=700,
             sink=4, window=200, lens_seed=3),
        # one user, long context
        dict(name="decode 1 x 32768 e4m3", kind="decode", fmt=E4M3, batch=1, hq=32, hkv=8, d=128, len_lo=32768, len_hi=32768,
             sink=0, window=0, lens_seed=4),
        # a full serving batch of mixed lengths
        dict(name="decode 64 mixed e4m3", kind="decode", fmt=E4M3, batch=64, hq=32, hkv=8, d=128, len_lo=1024, len_hi=16384,
             sink=0, window=0, lens_seed=5),
        # checking a few drafted tokens of each of eight sequences
        dict(name="extend drafts int8", kind="extend", fmt=INT8, batch=8, hq=64, hkv=8, d=128, rows_lo=1, rows_hi=8,
             len_lo=1000, len_hi=32768, sink=0, window=0, lens_seed=6),
        # chunks of prompts under a sliding window with sinks, an odd number of query heads per KV head
        dict(name="extend window int8", kind="extend", fmt=INT8, batch=4, hq=28, hkv=4, d=64, rows_lo=512, rows_hi=2048,
             len_lo=2048, len_hi=8192, sink=16, window=1024, lens_seed=7),
        # the second half of a long prompt
        dict(name="extend 8192 of 16384 e4m3", kind="extend", fmt=E4M3, batch=1, hq=32, hkv=8, d=128, rows_lo=8192,
             rows_hi=8192, len_lo=16384, len_hi=16384, sink=0, window=0, lens_seed=8),
        # parallel samples of a few long prompts over a BF16 cache: the last samples are dropped, new ones forked
        dict(name="fork 24 bf16", kind="fork", pool="bf16", hkv=8, d=128, sources=8, forks=24, len_lo=1024, len_hi=16384,
             lens_seed=9),
        # many short candidates over an 8-bit cache
        dict(name="fork 252 int8", kind="fork", pool="int8", hkv=2, d=64, sources=4, forks=252, len_lo=100, len_hi=4096,
             lens_seed=10),
        # a small pool after some sequences have ended
        dict(name="compact small bf16", kind="compact", pool="bf16", hkv=1, d=64, batch=7, len_lo=1, len_hi=900, spare=0.6,
             lens_seed=11),
        # the pool of a serving batch, packed to the front before a part of it is given back
        dict(name="compact batch int8", kind="compact", pool="int8", hkv=8, d=128, batch=64, len_lo=1024, len_hi=16384,
             spare=0.5, lens_seed=12),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** rng.random())) - 1))


def draw(rng):
    kind = rng.choice(["append", "decode", "decode", "extend", "extend", "fork", "compact"])
    seed = rng.randrange(1 << 30)
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 4, 8])
    if kind == "append":
        c = dict(kind=kind, fmt=rng.choice([E4M3, INT8]), batch=_spread(rng, 1, 96), hkv=hkv, d=d,
                 new_lo=rng.choice([0, 1]), new_hi=_spread(rng, 1, 12000), old_lo=0, old_hi=_spread(rng, 1, 8000), lens_seed=seed)
        while c["batch"] > 1 and c["batch"] * (c["new_hi"] + c["old_hi"] / 4) * hkv * d > 4e7:
            c["batch"] = c["batch"] // 2
        return c
    if kind in ("decode", "extend"):
        hi = _spread(rng, 17, 40000)
        c = dict(kind=kind, fmt=rng.choice([E4M3, INT8]), batch=_spread(rng, 1, 100), hq=hkv * rng.randint(1, 8), hkv=hkv, d=d,
                 len_lo=rng.choice([0, 1, hi // 3, hi]), len_hi=hi, sink=0, window=0, lens_seed=seed)
        if rng.random() < 0.5:
            c["window"] = _spread(rng, 1, 6000)
            c["sink"] = rng.choice([0, 1, 4, 64, rng.randint(2, 200)])
        if kind == "extend":
            c["rows_hi"] = _spread(rng, 1, 5000)
            c["rows_lo"] = rng.choice([0, 1, c["rows_hi"]])
        rows = c.get("rows_hi", 1)
        while c["batch"] > 1 and (c["batch"] * hi * hkv * d > 5e8 or c["batch"] * rows * hi * c["hq"] > 1.5e9):
            c["batch"] = c["batch"] // 2
        return c
    if kind == "fork":
        return dict(kind=kind, pool=rng.choice(["bf16", "int8"]), hkv=min(hkv, 4), d=d, sources=_spread(rng, 1, 20),
                    forks=_spread(rng, 1, 300), len_lo=rng.choice([0, 1, 50]), len_hi=_spread(rng, 51, 9000), lens_seed=seed)
    return dict(kind=kind, pool=rng.choice(["bf16", "int8"]), hkv=min(hkv, 4), d=d, batch=_spread(rng, 1, 60),
                len_lo=rng.choice([0, 1, 50]), len_hi=_spread(rng, 51, 9000), spare=rng.choice([0.1, 0.5, 1.0, 2.0]),
                lens_seed=seed)


# ---- lengths: the same for every seed, so that the work of a case is known ---------------------------------------------


def _lengths(case):
    """Per sequence: (tokens in the cache, of which new rows)."""
    rng = random.Random(case["lens_seed"])
    kind = case["kind"]
    if kind == "append":
        got = []
        for _ in range(case["batch"]):
            new = rng.randint(case["new_lo"], case["new_hi"])
            got.append((rng.randint(case["old_lo"], case["old_hi"]) + new, new))
        if not any(n for _, n in got):
            got[0] = (got[0][0] + case["new_hi"], case["new_hi"])
        return got
    count = case["sources"] if kind == "fork" else case["batch"]
    lens = [rng.randint(case["len_lo"], case["len_hi"]) for _ in range(count)]
    if kind == "decode" and case["len_lo"] == 0 and count > 2:
        lens[count // 2] = 0
    if kind != "extend":
        return [(n, 1) for n in lens]
    rows = [min(n, rng.randint(case["rows_lo"], case["rows_hi"])) for n in lens]
    if not any(rows):
        lens[0], rows[0] = max(lens[0], 1), 1
    return list(zip(lens, rows))


def _pages(n):
    return -(-n // P)


def _seen(n, row, sink, window):
    """Positions that the query at position `row` of a sequence sees."""
    if not window:
        return row + 1
    low = max(0, row - window + 1)
    return row + 1 - low + min(sink, low)


def work(case):
    kind, hkv, d = case["kind"], case["hkv"], case["d"]
    lens = _lengths(case)
    if kind == "append":
        t = sum(n for _, n in lens)
        blocks = sum(_pages(L) - (L - n) // P for L, n in lens if n)
        return {"bytes": t * hkv * d * 2 * 3 + blocks * hkv * 2 * 4, "flops": 0}
    if kind in ("decode", "extend"):
        hq, sink, window = case["hq"], case["sink"], case["window"]
        rows = pairs = tokens = 0
        for L, n in lens:
            n = min(n, L)
            if n == 0:
                rows += kind == "decode"
                continue
            rows += n
            pairs += sum(_seen(L, r, sink, window) for r in range(L - n, L))
            low = max(0, L - n - window + 1) if window else 0
            tokens += L - low + min(sink, low)
        return {"bytes": tokens * hkv * 2 * (d + 4 / P) + rows * hq * d * 4, "flops": 4 * d * hq * pairs}
    page = hkv * 2 * P * d * 2 if case["pool"] == "bf16" else hkv * 2 * (P * d + 4)
    entries = sum(_pages(n) for n, _ in lens)
    if kind == "fork":
        each = case["forks"] / case["sources"]
        return {"bytes": case["forks"] * page * 2 + each * entries * 4 * 4, "flops": 0}
    n = _pool_pages(case)
    moved = entries * (n - entries) / n
    return {"bytes": moved * page * 2 + entries * 8 + n * 8, "flops": 0}


def _pool_pages(case):
    used = sum(_pages(n) for n, _ in _lengths(case))
    if case["kind"] == "fork":
        return used + case["forks"] + 8
    if case["kind"] == "compact":
        return used + max(1, int(used * case["spare"]))
    return used + 5


# ---- inputs -----------------------------------------------------------------------------------------------------------


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


def _typed(codes, fmt):
    return codes.view(torch.float8_e4m3fn if fmt == E4M3 else torch.int8)


def _keys(n, hkv, d, mean, factor, g):
    """Keys with per-channel means and a few channels that are 15 times the others, as trained models have them."""
    return (torch.randn(n, hkv, d, device="cuda", generator=g) + mean) * factor


def _key_shape(hkv, d, g):
    mean = 3 * torch.randn(hkv, d, device="cuda", generator=g)
    factor = torch.ones(hkv, d, device="cuda")
    factor.scatter_(1, torch.rand(hkv, d, device="cuda", generator=g).argsort(1)[:, :6], 15.0)
    return mean, factor


def _tables(lens, num_pages, rows, g):
    """A page table of `rows` rows over a random order of the pool's pages, and how often each page is referred to."""
    order = torch.randperm(num_pages, device="cuda", generator=g).to(torch.int32)
    table = torch.full((rows, max([1] + [_pages(n) for n in lens])), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        table[b, :_pages(n)] = order[at:at + _pages(n)]
        at += _pages(n)
    count = torch.zeros(num_pages, dtype=torch.int32, device="cuda")
    count[order[:at].long()] = 1
    return table, count


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


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    kind, hkv, d = case["kind"], case["hkv"], case["d"]
    pairs = _lengths(case)
    lens = [n for n, _ in pairs]
    n_pages = _pool_pages(case)
    rows = len(lens) + (case["forks"] if kind == "fork" else 0)
    table, count = _tables(lens, n_pages, rows, g)
    cuda32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    hq = case.get("hq", hkv)
    st = dict(case=case, table=table, lens=cuda32(lens + [0] * (rows - len(lens))), max_len=max(lens),
              dims=dict(num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=P, group_size=64, num_pages=n_pages,
                        max_pages_per_seq=table.shape[1]))
    if kind in ("append", "decode", "extend"):
        mean, factor = _key_shape(hkv, d, g)
        st["codes"], st["scales"] = _cache(n_pages, hkv, d, case["fmt"], mean, factor, g)
    if kind == "append" or kind == "extend":
        new = [n for _, n in pairs]
        start = [0]
        for n in new:
            start.append(start[-1] + n)
        st["start"], st["max_new"] = cuda32(start), max(new)
    if kind == "append":
        st["k"] = _keys(start[-1], hkv, d, mean, factor, g).bfloat16()
        st["v"] = torch.randn(start[-1], hkv, d, device="cuda", generator=g).bfloat16()
    elif kind in ("decode", "extend"):
        n = start[-1] if kind == "extend" else len(lens)
        st["q"] = torch.randn(n, hq, d, device="cuda", generator=g).bfloat16()
    else:
        if case["pool"] == "bf16":
            st["pools"] = [torch.randn(n_pages, hkv, 2, P, d, device="cuda", generator=g, dtype=torch.bfloat16)]
        else:
            st["pools"] = [torch.randint(-127, 128, (n_pages, hkv, 2, P, d), device="cuda", generator=g, dtype=torch.int8),
                           torch.rand(n_pages, hkv, 2, device="cuda", generator=g)]
        st["count"] = count
    if kind == "fork":
        st["src"] = torch.randint(0, case["sources"], (case["forks"],), device="cuda", generator=g, dtype=torch.int32)
        st["dst"] = torch.arange(case["sources"], rows, device="cuda", dtype=torch.int32)
        st["granted"] = torch.zeros(case["forks"], dtype=torch.int32, device="cuda")
    if kind == "compact":
        st["table0"], st["count0"] = table.clone(), count.clone()
        st["live"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return st


# ---- one pass ----------------------------------------------------------------------------------------------------------


def run(st):
    kind = st["case"]["kind"]
    if kind == "append":
        return _append_own(st) if own else _append(st)
    if kind == "decode":
        return _decode_own(st) if own else _decode(st)
    if kind == "extend":
        return _extend_own(st) if own else _extend(st)
    if kind == "fork":
        return _fork_own(st) if own else _fork(st)
    return _compact_own(st) if own else _compact(st)


def _append_own(st):
    import int2_rotated_kv_append_gb300 as oscar
    c = st["case"]
    oscar.oscar_kv8_append(st["dims"], c["fmt"], c["batch"], st["max_new"], st["k"], st["v"], st["start"], st["table"],
                           st["lens"], st["codes"], st["scales"])
    return _typed(st["codes"], c["fmt"]), st["scales"]


def _decode_own(st):
    import int2_rotated_kv_append_gb300 as oscar
    c = st["case"]
    if "work" not in st:
        st["work"] = torch.empty(oscar.oscar_kv8_decode_workspace_bytes(st["dims"], c["batch"], st["max_len"], 0, c["sink"],
                                                                        c["window"]), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(st["q"])
    oscar.oscar_kv8_decode(st["dims"], c["fmt"], c["batch"], st["max_len"], 0, st["q"], st["codes"], st["scales"], st["table"],
                           st["lens"], c["sink"], c["window"], 0.0, out, st["work"])
    return out


def _extend_own(st):
    import int2_rotated_kv_append_gb300 as oscar
    c = st["case"]
    if "work" not in st:
        st["work"] = torch.empty(oscar.oscar_kv8_extend_varlen_workspace_bytes(
            st["dims"], c["batch"], st["q"].shape[0], st["max_len"], st["max_new"], 0, c["sink"], c["window"]),
            dtype=torch.uint8, device="cuda")
    out = torch.empty_like(st["q"])
    oscar.oscar_kv8_extend_varlen(st["dims"], c["fmt"], c["batch"], st["max_len"], st["max_new"], 0, st["q"], st["start"],
                                  st["codes"], st["scales"], st["table"], st["lens"], c["sink"], c["window"], 0.0, out,
                                  st["work"])
    return out


def _page_work(oscar, st):
    if "work" not in st:
        st["work"] = torch.empty(oscar.oscar_pages_workspace_bytes(st["dims"], st["table"].shape[0],
                                                                   st["case"].get("forks", 0)),
                                 dtype=torch.uint8, device="cuda")
    return st["work"]


def _fork_own(st):
    import int2_rotated_kv_append_gb300 as oscar
    oscar.oscar_pages_free(st["dims"], st["dst"], st["table"], st["lens"], st["count"])
    oscar.oscar_pages_fork(st["dims"], st["pools"], st["src"], st["dst"], st["table"], st["lens"], st["count"], st["granted"],
                           _page_work(oscar, st))
    return [st["table"], st["lens"], st["count"], st["granted"], *st["pools"]]


def _compact_own(st):
    import int2_rotated_kv_append_gb300 as oscar
    st["table"].copy_(st["table0"])  # the pool as it was before: its pages are all still there
    st["count"].copy_(st["count0"])
    oscar.oscar_pages_compact(st["dims"], st["pools"], st["table"], st["lens"], st["count"], st["live"], _page_work(oscar, st))
    return [st["table"], st["count"], st["live"], *st["pools"]]


# ---- the plain forms ---------------------------------------------------------------------------------------------------


def _places(st, tokens):
    """Sequence and position of each of the rows that are the last of their sequences."""
    start = st["start"].long()
    t = torch.arange(tokens, device="cuda")
    b = torch.searchsorted(start[1:], t, right=True)
    return b, st["lens"].long()[b] - start[b + 1] + t


def _append(st):
    fmt, codes, scales = st["case"]["fmt"], st["codes"], st["scales"]
    x = torch.stack([st["k"], st["v"]], 2).float()
    b, pos = _places(st, x.shape[0])
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
    return _typed(codes, fmt), scales


def _dense(st, side):
    """K or V of every sequence in a row of its own, [B][Hkv][positions][D]."""
    table = st["table"].long().clamp(min=0)
    x = _values(st["codes"][:, :, side][table], st["case"]["fmt"]) * st["scales"][:, :, side][table][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _attend(st, q, pos):
    """q [B][rows][Hq][D] at positions pos [B][rows] (-1: none) over the cache."""
    c = st["case"]
    B, R, hq, d = q.shape
    hkv = c["hkv"]
    q = q.float().view(B, R, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, d)
    s = torch.matmul(q, _dense(st, 0).transpose(2, 3)).mul_(d ** -0.5)
    n = s.shape[-1]
    j = torch.arange(n, device="cuda")
    see = j <= pos[..., None]
    if c["window"]:
        see &= (j < c["sink"]) | (j > pos[..., None] - c["window"])
    s = s.view(B, hkv, hq // hkv, R, n).masked_fill_(~see[:, None, None], float("-inf"))
    s = s.sub_(s.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(B, hkv, -1, n), _dense(st, 1))
    o = o.view(B, hkv, hq // hkv, R, d) / total.clamp(min=1e-30)
    return o.permute(0, 3, 1, 2, 4).reshape(B, R, hq, d)


def _decode(st):
    return _attend(st, st["q"][:, None], st["lens"].long()[:, None] - 1)[:, 0].bfloat16()


def _extend(st):
    c, q = st["case"], st["q"]
    b, pos = _places(st, q.shape[0])
    r = torch.arange(q.shape[0], device="cuda") - st["start"].long()[b]
    qq = torch.zeros(c["batch"], st["max_new"], *q.shape[1:], dtype=q.dtype, device="cuda")
    pp = torch.full((c["batch"], st["max_new"]), -1, device="cuda")
    qq[b, r], pp[b, r] = q, pos
    return _attend(st, qq, pp)[b, r].bfloat16()


def _fork(st):
    table, lens, count = st["table"], st["lens"], st["count"]
    src, dst = st["src"].long(), st["dst"].long()
    j = torch.arange(table.shape[1], device="cuda") * P
    held = j < lens[dst][:, None]
    gone = table[dst][held].long()
    count.index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
    table[dst] = torch.where(held, -1, table[dst])
    lens[dst] = 0
    n = lens[src]
    held = j < n[:, None]
    ids = table[src]
    part = n % P != 0
    fresh = (count == 0).nonzero().flatten()[:int(part.sum())]  # lowest first, in the order of the forks
    last = (n // P).clamp(max=table.shape[1] - 1).long()[part]
    from_page = ids[part, last].long()
    for pool in st["pools"]:
        pool[fresh] = pool[from_page]
    ids[part, last] = fresh.int()
    table[dst] = torch.where(held, ids, table[dst])
    used = ids[held].long()
    count.index_add_(0, used, torch.ones_like(used, dtype=torch.int32))
    lens[dst] = n
    st["granted"].fill_(1)
    return [table, lens, count, st["granted"], *st["pools"]]


def _compact(st):
    table, count = st["table"], st["count"]
    table.copy_(st["table0"])
    count.copy_(st["count0"])
    live = count > 0
    k = live.sum()
    i = torch.arange(count.numel(), device="cuda")
    src, dst = (live & (i >= k)).nonzero().flatten(), (~live & (i < k)).nonzero().flatten()
    for pool in st["pools"]:
        pool[dst] = pool[src]
    count[dst] = count[src]
    count[src] = 0
    i[src] = dst
    held = torch.arange(table.shape[1], device="cuda") * P < st["lens"][:, None]
    table.copy_(torch.where(held, i[table.long().clamp(min=0)].int(), table))
    st["live"].copy_(k)
    return [table, count, st["live"], *st["pools"]]


# ---- 64 bits -----------------------------------------------------------------------------------------------------------


def exact(case, seed):
    if case["kind"] in ("fork", "compact"):
        return None  # copies and whole numbers
    if case["kind"] == "append" and case["fmt"] == INT8:
        return None
    st = prepare(case, seed)
    return _exact_append(st) if case["kind"] == "append" else _exact_attention(st)


def _two_to(e):
    """2^e as doubles, exactly (a power function may be off by a rounding)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3(x):
    """The nearest e4m3 value (ties to even) of doubles within its range."""
    m, e = torch.frexp(x)  # |m| in [0.5, 1): four bits of it are kept, fewer below 2^-6
    step = _two_to((e - 1).clamp(min=-6) - 3)
    return ((x / step).round() * step).clamp(-448, 448)


def _exact_append(st):
    codes = st["codes"].view(torch.float8_e4m3fn).double()
    scales = st["scales"].double()
    start, table, lens = st["start"].tolist(), st["table"].tolist(), st["lens"].tolist()
    kv = torch.stack([st["k"], st["v"]], 2).double()
    for b, L in enumerate(lens):
        t0, t1 = start[b], start[b + 1]
        p = L - (t1 - t0)
        while p < L:  # page by page
            n = min(L, (p // P + 1) * P) - p
            t = t1 - (L - p)
            page, r = table[b][p // P], p % P
            x = kv[t:t + n]
            a = x.abs().amax((0, 3))
            m, e = torch.frexp((a / 448).clamp(min=2.0 ** -100))
            s = _two_to(torch.where(m == 0.5, e - 1, e))
            if r:
                s = torch.maximum(s, scales[page])
                codes[page, :, :, :r] = _e4m3(codes[page, :, :, :r] * (scales[page] / s)[..., None, None])
            codes[page, :, :, r:r + n] = _e4m3(x / s[..., None]).permute(1, 2, 0, 3)
            scales[page] = s
            p += n
    return codes, scales


def _exact_attention(st):
    c = st["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    lens = st["lens"].tolist()
    if c["kind"] == "extend":
        start = st["start"].tolist()
    else:
        start = list(range(c["batch"] + 1))
    if sum((start[b + 1] - start[b]) * lens[b] for b in range(c["batch"])) * hq * d * 4 > 6e12:
        return None
    out = torch.zeros(start[-1], hq, d, dtype=torch.float64, device="cuda")
    as_type = torch.float8_e4m3fn if c["fmt"] == E4M3 else torch.int8
    for b, L in enumerate(lens):
        rows = start[b + 1] - start[b]
        if L == 0 or rows == 0:
            continue
        ids = st["table"][b, :_pages(L)].long()
        kv = st["codes"][ids].view(as_type).double() * st["scales"][ids].double()[..., None, None]
        kv = kv.permute(1, 2, 0, 3, 4).reshape(hkv, 2, -1, d)[:, :, :L]
        j = torch.arange(L, device="cuda")
        for r0 in range(0, rows, 2048):
            r1 = min(rows, r0 + 2048)
            p = torch.arange(L - rows + r0, L - rows + r1, device="cuda")[:, None]
            hidden = j > p
            if c["window"]:
                hidden |= (j >= c["sink"]) & (j <= p - c["window"])
            for h in range(hq):
                s = st["q"][start[b] + r0:start[b] + r1, h].double() @ kv[h * hkv // hq, 0].T / d ** 0.5
                w = torch.softmax(s.masked_fill(hidden, float("-inf")), 1)
                out[start[b] + r0:start[b] + r1, h] = w @ kv[h * hkv // hq, 1]
    return out
