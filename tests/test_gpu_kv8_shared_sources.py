"""oscar_kv8_decode_shared where the first sequence that a group lists is no good source of the group's pages: out of range, freed, or
shorter than the prefix.  The other members' rows are those of dense 64-bit attention over their own pages."""

import numpy as np
import pytest
import torch

import int2_rotated_kv_append_gb300 as ok
import kv8_ref as R
from test_gpu_kv8_shared import Case

pytestmark = pytest.mark.gpu

# each by itself, and in tiles of 64, 128 and 256 rows
FORMS = [((4, 2, 128), 0, [(512, [20, 30, 40, 50]), (256, [0, 4])]),
         ((8, 8, 128), 64, [(16000, [5, 0, 300, 16] * 9), (768, [9, 3])]),
         ((5, 1, 64), 128, [(40000, [7 * i for i in range(24)])]),
         ((4, 2, 128), 256, [(20000, [20, 30, 40, 50] * 20), (256, [0, 4])])]


def forms(test):
    test = pytest.mark.parametrize("shape,rows,groups", FORMS, ids=["list", "64", "128", "256"])(test)
    return pytest.mark.parametrize("fmt", [R.E4M3, R.INT8])(test)


def make(shape, rows, groups, fmt):
    c = Case(*shape, fmt, groups, seed=rows + 21)
    assert c.tile_rows() == rows
    return c


def of(c, g):
    """Members of group g."""
    return c.members[c.start[g]:c.start[g + 1]]


def shorten(c, lens, b, n):
    """Sequence b ends after n tokens: its other pages are given back."""
    lens[b] = n
    c.table[b, -(-n // 16):] = -1
    c.t_table.copy_(torch.from_numpy(c.table))


def run(c, lens):
    return c.run(lens=torch.from_numpy(lens).cuda())


@forms
def test_first_members_out_of_range(shape, rows, groups, fmt):
    c = make(shape, rows, groups, fmt)
    for bad in (-1, c.batch, 2 ** 31 - 1):
        m = list(c.members)
        for g in range(len(groups)):
            m[c.start[g]] = bad
        out = c.run(lists=(m, c.start, c.prefix))
        assert ok.oscar_device_errors(reset=True) == ok.OSCAR_DEVERR_POSITION
        c.check(out, members=[b for b in m if b != bad])


@forms
def test_first_members_freed(shape, rows, groups, fmt):
    c = make(shape, rows, groups, fmt)
    lens = c.lens.copy()
    for g in range(len(groups)):
        shorten(c, lens, of(c, g)[0], 0)
    out = run(c, lens)
    for g in range(len(groups)):
        assert (out[of(c, g)[0]] == 0).all()
    c.check(out, lens=lens)


@forms
def test_first_members_shorter_than_the_prefix(shape, rows, groups, fmt):
    c = make(shape, rows, groups, fmt)
    lens = c.lens.copy()
    for i, b in enumerate(of(c, 0)[:-1]):  # all but the last: more of them than a warp has lanes, where there are
        shorten(c, lens, b, (37 * i + 100) % groups[0][0])
    c.check(run(c, lens), lens=lens)


@forms
@pytest.mark.parametrize("longest", [0, 1, 100, 240])
def test_every_member_shorter_than_the_prefix(shape, rows, groups, fmt, longest):
    # nobody has the prefix's last pages: they are not looked up, and what lies behind the longest member's last token is not read
    c = make(shape, rows, groups, fmt)
    lens = c.lens.copy()
    for i, b in enumerate(of(c, 0)):
        shorten(c, lens, b, longest if i == 2 else min(longest, 7 * i))
    b = of(c, 0)[2]
    if longest % 16:
        c.codes[int(c.table[b, longest // 16]), :, :, longest % 16:] = 0x7f  # NaN in e4m3
    c.check(run(c, lens), lens=lens)


@forms
def test_first_members_out_of_range_and_the_others_short(shape, rows, groups, fmt):
    c = make(shape, rows, groups, fmt)
    lens = c.lens.copy()
    for i, b in enumerate(of(c, 0)):
        shorten(c, lens, b, 50 + i)
    m = list(c.members)
    m[0] = -1
    out = c.run(lists=(m, c.start, c.prefix), lens=torch.from_numpy(lens).cuda())
    assert ok.oscar_device_errors(reset=True) == ok.OSCAR_DEVERR_POSITION
    c.check(out, members=m[1:], lens=lens)


@forms
def test_nobody_in_range(shape, rows, groups, fmt):
    c = make(shape, rows, groups, fmt)
    m = list(c.members)
    m[:c.start[1]] = [-1] * c.start[1]
    out = c.run(lists=(m, c.start, c.prefix))
    assert ok.oscar_device_errors(reset=True) == ok.OSCAR_DEVERR_POSITION
    c.check(out, members=m[c.start[1]:])


def test_lists_found_before_a_member_was_freed():
    from int2_rotated_kv_append_gb300.cache import Kv8Cache
    B, n = 64, 6000
    c = Kv8Cache(8, 2, 128, num_pages=n // 16 + 3 * B, batch=B, max_seq_len=n + 64)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    g = torch.Generator("cuda").manual_seed(1)

    def append(new):
        assert c.reserve(i32(new)).all()
        k, v = (torch.randn(sum(new), 2, 128, device="cuda", generator=g).bfloat16() for _ in range(2))
        c.append(k, v, i32(np.concatenate([[0], np.cumsum(new)])), max(new))

    append([n] + [0] * (B - 1))
    c.fork(i32([0] * (B - 1)), i32(list(range(1, B))))
    append([1] * B)
    groups = c.groups(max_groups=2)
    assert ok.oscar_kv8_decode_shared_plan(c.dims, B, c.max_seq_len, n, 64, B, 2)["tile_rows"] > 0
    c.free(i32([0, 5]))
    q = torch.randn(B, 8, 128, device="cuda", generator=g).bfloat16()
    out = c.decode_shared(q, groups, max_prefix_len=n, max_own_len=64)
    want, tol = R.attention(c.pages, c.scales, q, list(range(B)), [x - 1 for x in c.seq_lens.tolist()], c.page_table.tolist(), R.E4M3, 0, 0)
    assert ((out.double() - want).abs() <= tol).all() and (out[[0, 5]] == 0).all()
    assert ok.oscar_device_errors(reset=True) == 0
