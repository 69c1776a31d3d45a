"""The bits of oscar_kv8_decode_shared's weights in each of its forms: rows against 64-bit attention within what that form's own
roundings allow (kv8_shared_ref), a position's error in proportion to what it contributes."""

import numpy as np
import pytest
import torch

import int2_rotated_kv_append_gb300 as ok
import kv8_ref as R
import kv8_shared_ref as S
from test_gpu_kv8_shared import Case

pytestmark = pytest.mark.gpu

# each by itself, and in tiles of 64, 128 and 256 rows; D = 64 and 128 (about 20 members of each group are looked at)
FORMS = [((4, 2, 128), 0, [(512, [20, 30, 40, 50]), (256, [0, 4])]), ((10, 2, 64), 0, [(3200, [20, 0]), (0, [700])]),
         ((8, 8, 128), 64, [(16000, [5, 0, 300, 16] * 9), (768, [9, 3])]), ((6, 2, 64), 64, [(40000, [700, 9, 1, 0] * 5)]),
         ((5, 1, 64), 128, [(40000, [7 * i for i in range(24)])]), ((3, 1, 128), 128, [(24000, [7 * i for i in range(30)])]),
         ((4, 2, 128), 256, [(20000, [20, 30, 40, 50] * 20), (256, [0, 4])]), ((4, 1, 64), 256, [(24000, [20, 30, 40, 50] * 20)])]


def make(shape, rows, groups, fmt, **kw):
    c = Case(*shape, fmt, groups, seed=rows + shape[0], **kw)
    assert c.tile_rows() == rows
    return c


def check(c, rows):
    out = c.run()
    assert ok.oscar_device_errors(reset=True) == 0
    for g, p in enumerate(c.prefix):
        members = c.members[c.start[g]:c.start[g + 1]]
        for b in members[::max(1, len(members) // 20)]:
            n = int(c.lens[b])
            if n == 0:
                assert (out[b] == 0).all()
                continue
            want, tol = S.rows(c.codes, c.scales, c.q, b, n, c.table, c.fmt, p // 16 * 16, rows > 0)
            over = ((out[b].double() - want).abs() / tol).max().item()
            assert over <= 1, (g, b, over)


def forms(test):
    test = pytest.mark.parametrize("shape,rows,groups", FORMS, ids=["%d-%d" % (f[1], f[0][2]) for f in FORMS])(test)
    return pytest.mark.parametrize("fmt", [R.E4M3, R.INT8])(test)


@forms
@pytest.mark.parametrize("spread,sharp", [(0, 1), (3, 20), (9, 20), (40, 1)])
def test_rows_within_their_own_forms_roundings(shape, rows, groups, fmt, spread, sharp):
    c = make(shape, rows, groups, fmt, spread=spread)
    c.q *= sharp
    check(c, rows)


def plant(c, pages, k, v, k_scale, v_scale):
    """In the named pages, of every head: K codes k [P] in channel 0 and zeros, V codes v [P][D]."""
    codes = torch.zeros(2, 16, c.D, dtype=torch.int8)
    codes[0, :, 0], codes[1] = torch.from_numpy(np.asarray(k).astype(np.int8)), torch.from_numpy(np.asarray(v).astype(np.int8))
    ids = torch.as_tensor(pages).long().cuda()
    c.codes[ids] = codes.view(torch.uint8).cuda()
    c.scales[ids] = torch.tensor([k_scale, v_scale], device="cuda")


def blank(shape, rows, groups):
    """A cache whose tokens weigh nothing, in 64 bits, beside planted ones, and have the value 0."""
    c = make(shape, rows, groups, R.INT8)
    plant(c, range(c.codes.shape[0]), [-127] * 16, np.zeros((16, c.D)), float(c.D), 1.0)
    c.q.zero_()
    c.q[:, :, 0] = 1.0
    return c


@pytest.mark.parametrize("shape,rows,groups", FORMS, ids=["%d-%d" % (f[1], f[0][2]) for f in FORMS])
@pytest.mark.parametrize("seed", range(3))
def test_pages_that_cancel(shape, rows, groups, seed):
    # in a page of the first group's prefix, and in every page that a member has behind its prefix (tests/test_kv8_shared_ref.py: fewer
    # bits are outside the tolerances)
    c = blank(shape, rows, groups)
    k, v, _ = R.cancelling_page(c.D, seed)
    # (the page's weights are those at a scale of 1/8)
    factor = 2.0 ** -4 if c.D == 64 else 2.0 ** -3
    keep = c.codes.clone(), c.scales.clone()
    b, full = c.members[0], c.prefix[0] // 16
    plant(c, c.table[b, [0, full // 2, full - 1][seed]:][:1].copy(), k, v, factor, 1.0)
    check(c, rows)
    c.codes.copy_(keep[0]), c.scales.copy_(keep[1])
    own = [int(c.table[m, j]) for g, p in enumerate(c.prefix) for m in c.members[c.start[g]:c.start[g + 1]]
           for j in range(p // 16, int(c.lens[m]) // 16)]
    plant(c, own, k, v, factor, 1.0)
    check(c, rows)


@pytest.mark.parametrize("shape,rows,groups", FORMS, ids=["%d-%d" % (f[1], f[0][2]) for f in FORMS])
@pytest.mark.parametrize("where", ["own", "prefix"])
def test_light_tokens_of_large_values(shape, rows, groups, where):
    # a token of the first page weighs most and has the value 0, others weigh 2^-10 to 2^-26 of it and have scales that make up for it
    c = blank(shape, rows, groups)
    plant(c, c.table[c.members, 0].copy(), [0] + [-127] * 15, np.zeros((16, c.D)), float(c.D), 1.0)
    rng = np.random.default_rng(rows)
    for g, p in enumerate(c.prefix):
        members = c.members[c.start[g]:c.start[g + 1]]
        for m in members if where == "own" else members[:1]:
            pages = range(p // 16, int(c.lens[m]) // 16) if where == "own" else range(1, p // 16, 97)
            for j in pages:
                e = int(rng.integers(10, 26))
                # logits of -ln(2) e / sqrt(D) apart, within a step of the codes
                step = 2.0 ** (1 if c.D == 64 else 2)
                k = -np.rint(np.log(2.0) * (e + rng.random(16)) * np.sqrt(c.D) / step)
                plant(c, [int(c.table[m, j])], k, rng.integers(-127, 128, (16, c.D)), step, 2.0 ** e)
    check(c, rows)
