"""Cosine and sine of oscar_rope by themselves: relative to their own size, however small an angle is or how near a quarter turn."""

import math

import numpy as np
import pytest
import torch

import int2_rotated_kv_append_gb300 as ok

pytestmark = pytest.mark.gpu


def cos_sin(turns, positions):
    """float64 [T][pairs] each: the nearest quarter turn is taken off in whole numbers, so neither loses to cancellation."""
    c, s = np.empty((len(positions), len(turns))), np.empty((len(positions), len(turns)))
    for i, p in enumerate(positions):
        for j, t in enumerate(turns):
            whole = int(p) * int(t) % 2 ** 64
            quarter = (whole + 2 ** 61) >> 62
            a = 2 * math.pi * ((whole - (quarter << 62)) / 2.0 ** 64)
            c[i, j], s[i, j] = [(math.cos(a), math.sin(a)), (-math.sin(a), math.cos(a)), (-math.cos(a), -math.sin(a)),
                                (math.sin(a), -math.cos(a))][quarter % 4]
    return c, s


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("base,rotary", [(1e6, 128), (1e4, 64), (1.5, 32)])
def test_cosines_and_sines_to_a_rounding_of_their_own(base, rotary, interleaved):
    """Pairs (1, 0) become (cos, sin) exactly.  The angle's conversion to fp32 is half a step (2^-24) of what is left within an eighth
    of a turn, which cosine and sine of it pass on at most as it is; the function is off by a step at most (2^-23): 2^-22 together.  A
    sine or cosine below 2^-62 of a turn is left out: the fraction itself ends at 2^-64."""
    rope = ok.Rope(rotary, base=base, interleaved=interleaved)
    near = [round(n * 2 ** 62 / (int(t) % 2 ** 62)) for t in rope.turns.tolist() if int(t) % 2 ** 62 for n in (1, 2, 3, 4, 1001)]
    pos = [0, 1, -1, 2, 3, 17, 1000, 2 ** 31 - 1, -2 ** 31] + [p for p in near if p < 2 ** 31]  # and a step from quarter turns
    x = torch.zeros(len(pos), 1, rotary, device="cuda")
    first = torch.arange(rotary // 2, device="cuda") * (2 if interleaved else 1)
    x[:, 0, first] = 1.0
    d = ok.make_dims(1, 1, 64 if rotary <= 64 else 128, 16, 64, 1, 1)
    rows = torch.zeros(len(pos), 1, d.head_dim, device="cuda")
    rows[..., :rotary] = x
    y = torch.empty_like(rows)
    ok.oscar_rope(d, rope, torch.tensor(pos, dtype=torch.int32, device="cuda"), rows, None, y, None)
    got = y[:, 0].double().cpu().numpy()
    first = first.cpu().numpy()
    second = first + (1 if interleaved else rotary // 2)
    for value, want in zip((got[:, first], got[:, second]), cos_sin([t % 2 ** 64 for t in rope.turns.tolist()], pos)):
        assert (np.abs(value - want) <= 2.0 ** -22 * np.abs(want))[np.abs(want) >= 2.0 ** -62].all()
        assert (value[want == 0] == 0).all()
