"""Rotary positions on the host: frequencies against their formulas in many digits, refusals (nothing is launched)."""

import ctypes
import math
from decimal import Decimal, getcontext

import pytest
import torch

import int2_rotated_kv_append_gb300 as ok
from int2_rotated_kv_append_gb300 import build

BAD, UNS, OK = ok.OSCAR_ERR_INVALID_ARG, ok.OSCAR_ERR_UNSUPPORTED, ok.OSCAR_OK
P, ODD = ctypes.c_void_p(256), ctypes.c_void_p(24)
getcontext().prec = 60
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return ok.load_library()


def fractions(turns):
    return [Decimal(int(t) % 2 ** 64) / 2 ** 64 for t in turns]


@pytest.mark.parametrize("rotary", [16, 32, 96, 128])
@pytest.mark.parametrize("base", [10000.0, 500000.0, 1.5])
def test_plain_frequencies(rotary, base):
    turns, magnitude = ok.oscar_rope_turns(rotary, base)
    assert magnitude == 1.0 and turns.shape == (rotary // 2,)
    for i, t in enumerate(fractions(turns)):
        f = (Decimal(base).ln() * (Decimal(-2 * i) / rotary)).exp() / (2 * PI)
        # the power is a double, off by a step at most (2^-52), the fraction two units of 2^-64
        assert abs(t - f) <= f * Decimal(2) ** -52 + Decimal(2) ** -63
    assert abs(int(turns[0]) - int(Decimal(2) ** 64 / (2 * PI))) <= 2  # a radian a position


def expected(rotary, base, kind, s):
    f = [base ** (-2 * i / rotary) for i in range(rotary // 2)]
    if kind == "linear":
        return [x / s["factor"] for x in f]
    if kind == "ntk":
        return [(base * s["factor"] ** (rotary / (rotary - 2))) ** (-2 * i / rotary) for i in range(rotary // 2)]
    if kind == "divisors":
        return [x / d for x, d in zip(f, s["divisors"])]
    n = s["original_max_position"]
    if kind == "yarn":
        at = [rotary * math.log(n / (r * 2 * math.pi)) / (2 * math.log(base)) for r in (s.get("beta_fast", 32), s.get("beta_slow", 1))]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rotary - 1)
        g = [min(1, max(0, (i - lo) / max(hi - lo, 0.001))) for i in range(rotary // 2)]
        return [x / s["factor"] * w + x * (1 - w) for x, w in zip(f, g)]
    out = []
    for x in f:
        t = n * x / (2 * math.pi)
        w = min(1, max(0, (t - s["low_freq_factor"]) / (s["high_freq_factor"] - s["low_freq_factor"])))
        out.append(x * w + x / s["factor"] * (1 - w))
    return out


@pytest.mark.parametrize("s", [
    dict(kind="linear", factor=8.0), dict(kind="linear", factor=0.25), dict(kind="ntk", factor=4.0),
    dict(kind="yarn", factor=4.0, original_max_position=32768),
    dict(kind="yarn", factor=40.0, original_max_position=4096, beta_slow=2.0, beta_fast=16.0),
    dict(kind="yarn", factor=0.5, original_max_position=7),
    dict(kind="bands", factor=8.0, original_max_position=8192, low_freq_factor=1.0, high_freq_factor=4.0),
    dict(kind="divisors", divisors=[1.0 + i / 3 for i in range(32)])], ids=lambda s: s["kind"])
def test_scaled_frequencies(s):
    rotary, base = 64, 10000.0
    turns, magnitude = ok.oscar_rope_turns(rotary, base, s)
    assert magnitude == pytest.approx(0.1 * math.log(s["factor"]) + 1 if s["kind"] == "yarn" and s["factor"] > 1 else 1.0, rel=2 ** -24)
    for t, f in zip(fractions(turns), expected(rotary, base, s["kind"], s)):
        want = Decimal(f) / (2 * PI)
        want -= int(want)
        # a handful of operations in double on either side
        assert abs(t - want) <= Decimal(f) * Decimal(2) ** -48 + Decimal(2) ** -63


def test_the_last_ntk_pair_is_slowed_by_the_factor_and_the_first_is_not():
    (a, _), (b, _) = ok.oscar_rope_turns(64), ok.oscar_rope_turns(64, scaling=dict(kind="ntk", factor=4.0))
    a, b = fractions(a), fractions(b)
    assert a[0] == b[0] and abs(a[-1] / b[-1] - 4) < Decimal("1e-12")


def test_frequency_refusals(lib):
    out, mag = (ctypes.c_uint64 * 64)(), ctypes.c_float()

    def call(rotary=64, base=10000.0, turns=out, magnitude=mag, **s):
        c = None
        if s:
            div = s.pop("divisors", None)
            c = ok.oscar_rope_scaling_t(**s)
            if div:
                c.divisors = (ctypes.c_double * len(div))(*div)
        return lib.oscar_rope_turns(rotary, base, ctypes.byref(c) if c else None, ctypes.cast(turns, ctypes.c_void_p) if turns is not None else None,
                                    ctypes.byref(magnitude) if magnitude is not None else None)
    inf, nan = math.inf, math.nan
    assert call() == OK and call(kind=0) == OK
    assert call(rotary=0) == BAD and call(rotary=-16) == BAD and call(rotary=24) == UNS and call(rotary=144) == UNS
    for b in (1.0, 0.0, -3.0, inf, nan):
        assert call(base=b) == BAD
    assert call(turns=None) == BAD and call(magnitude=None) == BAD
    assert call(kind=6, factor=2.0) == BAD and call(kind=-1, factor=2.0) == BAD
    for kind in (1, 2, 3, 4):
        for f in (0.0, -1.0, inf, nan):
            assert call(kind=kind, factor=f, original_max_position=100, low=1.0, high=2.0) == BAD
    for kind in (3, 4):
        good = dict(kind=kind, factor=2.0, original_max_position=100, low=1.0, high=2.0)
        assert call(**good) == OK
        for bad in (dict(original_max_position=0), dict(low=0.0), dict(high=1.0), dict(high=inf), dict(low=nan)):
            assert call(**{**good, **bad}) == BAD
    assert call(kind=5) == BAD and call(kind=5, divisors=[1.0] * 31 + [0.0]) == BAD
    assert call(kind=1, factor=1e-7) == BAD  # 10^7 radians a position
    assert call(kind=2, factor=1e300) == BAD  # a base beyond doubles


def test_scaling_dicts():
    for s in (dict(kind="cubic"), dict(factor=2.0), dict(kind="linear"), dict(kind="linear", factor=2.0, low=1),
              dict(kind="yarn", factor=2.0), dict(kind="divisors", divisors=[1.0] * 5)):
        with pytest.raises(ValueError):
            ok.oscar_rope_turns(64, scaling=s)


def dims(**kw):
    d = dict(num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16, group_size=64, num_pages=100, max_pages_per_seq=20)
    d.update(kw)
    return ctypes.byref(ok.make_dims(**d))


def rope(rotary=64, interleaved=0, magnitude=1.0, turns=256):
    return ctypes.byref(ok.oscar_rope_t(rotary, interleaved, magnitude, turns))


BAD_DIMS = [(None, BAD), (dims(head_dim=96, group_size=32), UNS), (dims(page_size=32), UNS), (dims(num_q_heads=7), BAD)]
BAD_ROPES = [(None, BAD), (rope(0), BAD), (rope(-16), BAD), (rope(144), BAD), (rope(24), UNS), (rope(interleaved=2), BAD),
             (rope(magnitude=math.inf), BAD), (rope(magnitude=math.nan), BAD), (rope(turns=None), BAD), (rope(turns=260), BAD)]


def test_rope_refusals(lib):
    def call(d=None, r=None, type=0, tokens=3, **kw):
        a = dict(pos=P, q=P, qs=1024, k=P, ks=256, qo=P, qos=1024, ko=P, kos=256)
        a.update(kw)
        return lib.oscar_rope(dims() if d is None else d[0], rope() if r is None else r[0], type, tokens, a["pos"], a["q"], a["qs"],
                              a["k"], a["ks"], a["qo"], a["qos"], a["ko"], a["kos"], None)
    for d, want in BAD_DIMS:
        assert call((d,)) == want
    for r, want in BAD_ROPES:
        assert call(r=(r,)) == want
    assert call(tokens=0) == OK and call(tokens=0, q=None, k=None) == OK
    assert call(tokens=-1) == BAD and call(tokens=1 << 31) == BAD and call(type=3) == BAD and call(type=-1) == BAD
    assert call(pos=None) == BAD and call(q=None) == BAD and call(ko=None) == BAD and call(q=None, qo=None, k=None, ko=None) == BAD
    for n in ("q", "k", "qo", "ko"):
        assert call(**{n: ODD}) == BAD
    for n, row in (("qs", 1024), ("ks", 256), ("qos", 1024), ("kos", 256)):
        assert call(**{n: row - 8}) == BAD and call(**{n: row + 4}) == BAD and call(**{n: -row}) == BAD
        assert call(type=2, **{n: row + 2}) == BAD


def test_rows_that_go_over_rows_still_to_be_read_are_refused(lib):
    for qs, qos, ks, kos in ((2048, 1024, 256, 256), (1024, 1024, 256, 512)):
        assert lib.oscar_rope(dims(), rope(), 0, 2, P, P, qs, 1 << 24, ks, P, qos, 1 << 24, kos, None) == BAD
    assert lib.oscar_kv8_rope_append(dims(), rope(), 0, 1, 2, 2, P, 2048, P, 256, P, 256, P, None, P, P, None, P, P, P, 1024, None) == BAD


def test_append_refusals(lib):
    def call(d=None, r=None, fmt=0, batch=2, tokens=4, most=3, **kw):
        a = {n: P for n in "q k v start table lens pages scales qo".split()}
        a.update(qs=1024, ks=256, vs=256, qos=1024, pos=None, granted=None)
        a.update(kw)
        return lib.oscar_kv8_rope_append(dims() if d is None else d[0], rope() if r is None else r[0], fmt, batch, tokens, most, a["q"],
                                         a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["start"], a["pos"], a["table"], a["lens"],
                                         a["granted"], a["pages"], a["scales"], a["qo"], a["qos"], None)
    for d, want in BAD_DIMS:
        assert call((d,)) == want
    for r, want in BAD_ROPES:
        assert call(r=(r,)) == want
    assert call(tokens=0) == OK and call(tokens=0, batch=0, k=None) == OK
    assert call(fmt=2) == BAD and call(fmt=-1) == BAD and call(batch=-1) == BAD and call(batch=0) == BAD
    assert call(tokens=-1) == BAD and call(tokens=1 << 31) == BAD and call(most=0) == BAD and call(most=-1) == BAD
    assert call(batch=65536) == UNS and call((dims(max_pages_per_seq=1 << 28),)) == UNS
    for n in "q k v start table lens pages scales qo".split():
        assert call(**{n: None}) == BAD
    for n in "q k v pages scales qo".split():
        assert call(**{n: ODD}) == BAD
    for n, row in (("qs", 1024), ("ks", 256), ("vs", 256), ("qos", 1024)):
        assert call(**{n: row - 8}) == BAD and call(**{n: row + 4}) == BAD


def test_binding_refuses_rows_that_are_not_rows(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)  # (where tensors of the CPU are)
    r = ok.Rope(64, device="cpu")
    d = dict(num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16, group_size=64, num_pages=9, max_pages_per_seq=4)
    pos = torch.zeros(3, dtype=torch.int32)
    q, k = torch.zeros(3, 8, 128, dtype=torch.bfloat16), torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    cases = [(pos, q.double(), None, q.double(), None), (pos, q, k.half(), q, k), (pos, q, k[:2], q, k[:2]), (pos, None, None, None, None),
             (pos[:2], q, k, q, k), (pos.long(), q, k, q, k), (pos, q[:, :7], k, q, k), (pos, q[..., ::2], k, q, k),
             (pos, q.transpose(0, 1).contiguous().transpose(0, 1), k, q, k)]
    for c in cases:
        with pytest.raises(ValueError):
            ok.oscar_rope(d, r, *c, stream=0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError):
        ok.oscar_rope(d, r, pos, q, k, q, k, stream=0)
