"""oscar_kv8_decode_shared and oscar_pages_groups against dense 64-bit attention and lists in Python."""

import numpy as np
import pytest
import torch

import int2_rotated_kv_append_gb300 as ok
import kv8_ref as R
from int2_rotated_kv_append_gb300.cache import Kv8Cache, SharedPrefixes

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Case:
    """A cache of groups [(prefix tokens, [own tokens of each member])], sequences in a random order, `idle` more that are no
    member."""

    def __init__(self, hq, H, D, fmt, groups, seed=0, idle=2, spread=0):
        rng = np.random.default_rng(seed)
        self.fmt, self.D = fmt, D
        total = sum(len(m) for _, m in groups)
        self.batch = B = total + idle
        lens = [p + n for p, m in groups for n in m]
        per = max([1] + [-(-n // 16) for n in lens]) + 1
        need = sum(p // 16 for p, _ in groups) + sum(-(-n // 16) + 1 for p, m in groups for n in m) + 2
        ids = rng.permutation(need).astype(np.int32)
        self.order = rng.permutation(B)
        self.table = np.full((B, per), -1, np.int32)
        self.lens = np.zeros(B, np.int32)
        at = i = 0
        for p, m in groups:
            full = p // 16
            shared = ids[at:at + full]
            at += full
            for n in m:
                b = self.order[i]
                own = -(-(p + n) // 16) - full
                self.table[b, :full] = shared
                self.table[b, full:full + own] = ids[at:at + own]
                at += own
                self.lens[b] = p + n
                i += 1
        self.members = [int(x) for x in self.order[:total]]
        self.start = np.cumsum([0] + [len(m) for _, m in groups]).tolist()
        self.prefix = [p for p, _ in groups]
        g = torch.Generator("cuda").manual_seed(seed)
        x = torch.randn(need, H, 2, 16, D, device="cuda", generator=g)
        if fmt == R.E4M3:
            self.codes = (x * 60).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            self.codes = (x * 30).round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
        e = torch.randint(-6, -3, (need, H, 2), device="cuda", generator=g)
        e[..., 1] += torch.randint(-spread, spread + 1, (need, H), device="cuda", generator=g)
        self.scales = torch.ldexp(torch.ones(need, H, 2, device="cuda"), e)
        self.q = torch.randn(B, hq, D, device="cuda", generator=g).bfloat16()
        self.dims = ok.make_dims(hq, H, D, 16, 64, need, per)
        self.t_table, self.t_lens = torch.from_numpy(self.table).cuda(), torch.from_numpy(self.lens).cuda()

    def run(self, max_prefix=None, max_own=None, lists=None, lens=None, out=None, max_len=None, stream=None, work=None):
        members, start, prefix = (i32(x) for x in (lists or (self.members, self.start, self.prefix)))
        top = int(self.lens.max()) if max_len is None else max_len
        max_prefix = max(self.prefix) if max_prefix is None else max_prefix
        if max_own is None:
            used = {b: min(p, max_prefix) // 16 * 16 for g, p in enumerate(self.prefix) for b in self.members[self.start[g]:self.start[g + 1]]}
            max_own = max([0] + [int(self.lens[b]) - p for b, p in used.items()])
        if out is None:
            out = torch.full_like(self.q, 7.0)
        bounds = (top, max_prefix, max_own)
        n = ok.oscar_kv8_decode_shared_workspace_bytes(self.dims, self.batch, *bounds, len(members), len(prefix))
        assert n > 0
        if work is None:
            work = torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")  # NaN wherever nothing is written
        ok.oscar_kv8_decode_shared(self.dims, self.fmt, self.batch, *bounds, self.q, self.codes, self.scales, self.t_table,
                                   self.t_lens if lens is None else lens, members, start, prefix, 0.0, out, work, stream)
        return out

    def tile_rows(self):
        """Of the prefix kernel's tiles; 0 where members attend their prefixes by themselves."""
        own = max(int(self.lens[b]) - p for g, p in enumerate(self.prefix) for b in self.members[self.start[g]:self.start[g + 1]])
        return ok.oscar_kv8_decode_shared_plan(self.dims, self.batch, int(self.lens.max()), max(self.prefix), own, len(self.members),
                                               len(self.prefix))["tile_rows"]

    def check(self, out, members=None, lens=None):
        members = self.members if members is None else members
        lens = self.lens if lens is None else lens
        rows = [b for b in members]
        want, tol = R.attention(self.codes, self.scales, self.q[rows], rows, [int(lens[b]) - 1 for b in rows], self.table, self.fmt, 0, 0)
        got = out[rows].double()
        assert torch.isfinite(got).all()
        assert ((got - want).abs() <= tol).all(), ((got - want).abs() / tol).max()
        rest = [b for b in range(self.batch) if b not in set(rows)]
        assert (out[rest] == 7).all()
        assert ok.oscar_device_errors(reset=True) == 0


SHAPES = [(1, 1, 64), (6, 2, 64), (5, 1, 128), (32, 4, 128), (7, 7, 128)]


@pytest.mark.parametrize("fmt", [R.E4M3, R.INT8])
@pytest.mark.parametrize("hq,H,D", SHAPES)
@pytest.mark.parametrize("groups", [
    [(16, [1])], [(16, [0, 1, 17])], [(400, [5, 0, 300, 16])], [(2048, list(range(40)))],
    [(1024, [3] * 90), (0, [50, 0, 1]), (160, [7, 8])], [(3000 // 16 * 16, [100] * 17), (16, [900, 2])], [(0, [40, 700, 0])],
    [(0, [])], [(640, []), (640, [30])]], ids=lambda g: "+".join("%dx%d" % (len(m), p) for p, m in g))
def test_shared(hq, H, D, fmt, groups):
    c = Case(hq, H, D, fmt, groups, seed=len(groups) + hq)
    if not c.members:
        out = torch.full_like(c.q, 7.0)
        ok.oscar_kv8_decode_shared(c.dims, fmt, c.batch, 16, 16, 16, c.q, c.codes, c.scales, c.t_table, c.t_lens, i32([]), i32([0, 0]),
                                   i32([0]), 0.0, out, torch.empty(4096, dtype=torch.uint8, device="cuda"))
        assert (out == 7).all()
        return
    c.check(c.run())


# large enough for the kernel over prefixes: tiles of 64, 128 and 256 rows, ragged ones, queries of a member in two tiles, groups of
# one, prefixes of fewer blocks than a split
TILED = [((8, 8, 128), 64, [(16000, [5, 0, 300, 16] * 9)] + [(48 * 16, [9])] * 4 + [(0, [700, 0])]),
         ((32, 8, 128), 64, [(8192, list(range(11))), (8016, [0, 1000]), (12000, [90] * 13), (4000, [2, 3]), (11104, [1] * 15)]),
         ((5, 1, 64), 128, [(40000, [7 * i for i in range(24)])]),
         ((24, 8, 128), 128, [(9600, [40] * 41), (9008, [17])]),
         ((7, 1, 128), 256, [(30000, [3] * 90), (16, [40, 1])]),
         ((20, 4, 64), 256, [(20000, [100, 0, 33] * 40), (0, [64, 1]), (15888, [5] * 77)]),
         ((64, 8, 128), 256, [(4096, [50] * 37), (100, [1, 2])])]


@pytest.mark.parametrize("fmt", [R.E4M3, R.INT8])
@pytest.mark.parametrize("shape,rows,groups", TILED, ids=lambda x: str(x)[:24])
def test_shared_over_tiles(shape, rows, groups, fmt):
    groups = [(p // 16 * 16, m) for p, m in groups]
    c = Case(*shape, fmt, groups, seed=rows + shape[0])
    assert c.tile_rows() == rows
    c.check(c.run())


@pytest.mark.parametrize("fmt", [R.E4M3, R.INT8])
def test_more_groups_than_a_warp_has_lanes(fmt):
    rng = np.random.default_rng(1)
    groups = [(int(rng.integers(0, 30)) * 16, rng.integers(0, 90, rng.integers(0, 6)).tolist()) for _ in range(75)]
    c = Case(4, 2, 128, fmt, groups, seed=5)
    c.check(c.run())


def test_more_groups_than_a_warp_has_lanes_over_tiles():
    rng = np.random.default_rng(1)
    groups = [(int(rng.integers(0, 200)) * 16, rng.integers(0, 90, rng.integers(0, 9)).tolist()) for _ in range(75)] + [(8000, [5] * 99)]
    c = Case(8, 2, 128, R.E4M3, groups, seed=5)
    assert c.tile_rows() > 0
    c.check(c.run())


def test_more_groups_than_tiles_may_be_and_more_members_than_a_chunk():
    # 384 members' pages are dealt out together
    c = Case(4, 1, 64, R.INT8, [(6400, list(range(60)) * 10), (48, [1, 2])] + [(32, [3])] * 5, seed=14)
    assert c.tile_rows() > 0
    c.check(c.run())
    c = Case(4, 1, 64, R.INT8, [(32, [3])] * 1100 + [(6400, list(range(60))), (48, [1, 2])], seed=14)
    assert c.tile_rows() == 0
    c.check(c.run())


@pytest.mark.parametrize("heads", [1, 40, 200])
def test_heads_fewer_and_more_than_fit_a_wave(heads):
    c = Case(heads, heads, 64, R.INT8, [(1600, [9] * 5), (800, [40, 0, 3])], seed=heads)
    c.check(c.run())
    c = Case(heads, heads, 64, R.INT8, [(16000, [9] * 70), (800, [40, 0, 3])], seed=heads)
    assert c.tile_rows() > 0
    c.check(c.run())


def test_long_prefix_over_many_splits_and_own_parts_in_splits():
    for hq, D in ((8, 128), (3, 64)):  # few rows of many partials, and one of few
        c = Case(hq, 1, D, R.E4M3, [(20000 // 16 * 16, [9000, 1, 16, 0, 333])], seed=3)
        c.check(c.run())
        c = Case(hq, 1, D, R.INT8, [(20000 // 16 * 16, [0])], seed=4)
        assert c.tile_rows() == 0
        c.check(c.run())


def test_bounds_below_the_prefixes_leave_the_rest_to_the_members():
    c = Case(6, 2, 128, R.INT8, [(512, [20, 0]), (96, [1, 5, 9])], seed=4)
    for bound in (0, 15, 16, 100, 511):
        c.check(c.run(max_prefix=bound))
    c.check(c.run(max_own=532, max_len=544))  # far above what there is
    c = Case(6, 2, 128, R.INT8, [(20000, [20, 0] * 30), (96, [1, 5, 9])], seed=4)
    assert c.tile_rows() > 0
    for bound in (15000, 19999):
        c.check(c.run(max_prefix=bound))
    c.check(c.run(max_own=20016, max_len=20032))


def test_prefixes_that_are_not_whole_pages():
    c = Case(4, 2, 64, R.E4M3, [(320, [20, 40])], seed=6)
    for p in (319, 311, 5, -3):
        c.check(c.run(max_own=360, lists=(c.members, c.start, [p])))


def test_v_scales_far_apart():
    for spread in (9, 40):
        for prefix in (512, 12000):
            c = Case(8, 2, 128, R.E4M3, [(prefix, [20] * 99), (256, [50] * 3)], seed=7, spread=spread)
            assert (c.tile_rows() > 0) == (prefix > 512)
            c.check(c.run())


# the same cases small (every member by itself) and over tiles
SMALL, LARGE = [(512, [20, 30, 40, 50]), (256, [0, 4])], [(20000, [20, 30, 40, 50] * 20), (256, [0, 4])]


@pytest.mark.parametrize("groups", [SMALL, LARGE], ids=["small", "tiles"])
def test_members_shorter_than_the_prefix_and_empty_ones(groups):
    c = Case(4, 2, 128, R.INT8, groups, seed=8)
    assert (c.tile_rows() > 0) == (groups is LARGE)
    lens = c.lens.copy()
    lens[c.members[0]], lens[c.members[2]], lens[c.members[-2]] = 300, 0, 17
    c.check(c.run(lens=torch.from_numpy(lens).cuda()), lens=lens)
    lens[:] = 0
    out = c.run(lens=torch.from_numpy(lens).cuda())
    assert (out[c.members] == 0).all() and ok.oscar_device_errors(reset=True) == 0


@pytest.mark.parametrize("groups", [SMALL, LARGE], ids=["small", "tiles"])
def test_some_of_the_sequences_in_any_order(groups):
    c = Case(4, 2, 128, R.E4M3, groups, seed=9)
    m, p = c.members, groups[0][0]
    some = [m[3], m[0], m[-1]]
    c.check(c.run(lists=(some, [0, 2, 3], [p, 0]), max_own=300), members=some)
    # fewer members than entries: those behind the last group are none
    c.check(c.run(lists=(m, [0, 2, 2], [p, 0])), members=m[:2])


@pytest.mark.parametrize("groups", [SMALL, LARGE], ids=["small", "tiles"])
def test_a_sequence_named_twice(groups):
    c = Case(4, 2, 128, R.INT8, groups, seed=15)
    m, n = c.members, len(groups[0][1])
    c.check(c.run(lists=([m[0]] + m[:n] + [m[1]] + m[n:], [0, n + 2, len(m) + 2], c.prefix)))


@pytest.mark.parametrize("groups", [SMALL, LARGE], ids=["small", "tiles"])
def test_bad_numbers_are_flagged_and_nothing_else_is_touched(groups):
    c = Case(4, 2, 128, R.INT8, groups, seed=10)
    m, P, n, t, p = c.members, ok.OSCAR_DEVERR_POSITION, len(groups[0][1]), len(c.members), groups[0][0]
    for start in ([0, n, n - 1], [0, n, t + 1], [1, n, t], [0, -1, t], [0, t + 1, t], [0, 2 ** 31 - 1, t]):
        out = c.run(lists=(m, start, c.prefix))
        assert (out == 7).all() and ok.oscar_device_errors(reset=True) == P, start
    for bad in (-1, c.batch, 2 ** 31 - 1):
        out = c.run(lists=(m[:2] + [bad] + m[3:], c.start, c.prefix))
        assert ok.oscar_device_errors(reset=True) == P
        c.check(out, members=m[:2] + m[3:])
    lens = c.t_lens.clone()
    lens[m[1]] = 100000
    c.run(lens=lens)
    assert ok.oscar_device_errors(reset=True) & ok.OSCAR_DEVERR_SEQ_LEN
    out = c.run(max_own=32)  # 40 and 50 tokens are cut off
    assert ok.oscar_device_errors(reset=True) == ok.OSCAR_DEVERR_SEQ_LEN
    cut = np.minimum(c.lens, [p + 32 if b in m[:n] else 10 ** 6 for b in range(c.batch)])
    c.check(out, lens=cut)
    keep = c.t_table.clone()
    c.t_table[m[0], 3] = c.dims.num_pages
    c.t_table[m[-2], 16:] = -1
    c.table = c.t_table.cpu().numpy()
    for b in m[1:n] if groups is LARGE else ():  # over tiles the prefix is read through the first member's pages
        c.table[b, 3] = -1
    out = c.run()
    assert ok.oscar_device_errors(reset=True) == ok.OSCAR_DEVERR_PAGE_ID
    c.check(out)
    c.t_table = keep


@pytest.mark.parametrize("groups", [SMALL, LARGE], ids=["small", "tiles"])
def test_nan_queries_and_pages_behind_the_tokens(groups):
    c = Case(4, 2, 128, R.E4M3, groups, seed=11)
    clean = c.run()
    for b in range(c.batch):  # NaN codes behind every last token
        n = int(c.lens[b])
        if n % 16:
            c.codes[int(c.table[b, n // 16]), :, :, n % 16:] = 0x7f
    assert torch.equal(c.run(), clean)
    c.q[c.members[1], 2] = float("nan")
    out = c.run()
    assert out[c.members[1], 2].isnan().all()
    out[c.members[1], 2] = clean[c.members[1], 2]
    assert torch.equal(out, clean)


def test_the_same_call_twice_on_two_streams_and_captured():
    a = Case(8, 2, 128, R.E4M3, [(20000, [100] * 40), (512, [9, 700])], seed=12)
    b = Case(8, 2, 128, R.E4M3, [(10240, [10] * 70)], seed=13)
    assert a.tile_rows() > 0 and b.tile_rows() > 0
    want = a.run(), b.run()
    a.check(want[0])
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        for c, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                outs.append(c.run(stream=s))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, want[i % 2])
    # two calls back to back share a workspace, in a graph
    bounds = [(int(c.lens.max()), max(c.prefix), int(c.lens.max())) for c in (a, b)]
    n = max(ok.oscar_kv8_decode_shared_workspace_bytes(c.dims, c.batch, *t, len(c.members), len(c.prefix)) for c, t in zip((a, b), bounds))
    work = torch.empty(n, dtype=torch.uint8, device="cuda")
    lists = [tuple(i32(x) for x in (c.members, c.start, c.prefix)) for c in (a, b)]
    outs = [torch.zeros_like(c.q) for c in (a, b)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for c, t, l, o in zip((a, b), bounds, lists, outs):
            ok.oscar_kv8_decode_shared(c.dims, c.fmt, c.batch, *t, c.q, c.codes, c.scales, c.t_table, c.t_lens, *l, 0.0, o, work)
    for _ in range(3):
        for o in outs:
            o.zero_()
        g.replay()
        for c, o, w in zip((a, b), outs, want):
            for r in c.members:
                assert ((o[r].double() - w[r].double()).abs() <= 2.0 ** -7 * w[r].double().abs() + 1e-2).all()
            o[[x for x in range(c.batch) if x not in set(c.members)]] = 7
            c.check(o)


# ---- groups -------------------------------------------------------------------------------------------------------------


def find(table, lens, k, room):
    """Lists from the definition."""
    full = [n // 16 if 0 <= n <= table.shape[1] * 16 else 0 for n in lens]
    heads = {}
    for b in range(len(lens)):
        key = tuple(table[b, :k]) if full[b] >= k and min(table[b, :k]) >= 0 else ("alone", b)
        heads.setdefault(key, []).append(b)
    groups = [m for m in heads.values() if len(m) > 1][:room - 1]
    members, start, prefix = [], [0], []
    for m in groups:
        n = 0
        while n < min(full[b] for b in m) and table[m[0], n] >= 0 and all(table[b, n] == table[m[0], n] for b in m):
            n += 1
        members += m
        start.append(len(members))
        prefix.append(16 * n)
    members += [b for b in range(len(lens)) if b not in set(members)]
    return members, start + [len(lens)] * (room - len(groups)), prefix + [0] * (room - len(groups))


def groups(table, lens, k, room, pages=1 << 20):
    B = len(lens)
    d = ok.make_dims(8, 8, 128, 16, 64, pages, table.shape[1])
    work = torch.full((ok.oscar_pages_groups_workspace_bytes(d, B),), 0xff, dtype=torch.uint8, device="cuda")
    got = [torch.full((n,), -9, dtype=torch.int32, device="cuda") for n in (B, room + 1, room)]
    ok.oscar_pages_groups(d, k, torch.from_numpy(table).cuda(), i32(lens), *got, work)
    return [x.tolist() for x in got]


def check_groups(table, lens, k, room):
    got, want = groups(table, lens, k, room), find(table, lens, k, room)
    assert got[0] == want[0] and got[1] == want[1] and got[2] == want[2]


@pytest.mark.parametrize("B,pages", [(1, 1), (2, 3), (33, 40), (300, 70), (1100, 9), (70, 2500)])
def test_groups(B, pages):
    rng = np.random.default_rng(B)
    for room in (1, 2, 5, 2000):
        for k in (1, 2, 7):
            table = rng.integers(0, 1 << 20, (B, pages)).astype(np.int32)
            for b in range(1, B):  # most rows begin as another one does, for a while
                if rng.random() < 0.8:
                    a = rng.integers(0, b)
                    n = rng.integers(0, pages + 1)
                    table[b, :n] = table[a, :n]
            table[rng.random((B, pages)) < 0.3 / pages] = -1
            lens = rng.integers(0, 16 * pages + 1, B).tolist() if rng.random() < 0.5 else [16 * pages - int(x) for x in rng.integers(0, 20, B)]
            lens = [max(n, 0) for n in lens]
            check_groups(table, lens, k, room)
    assert ok.oscar_device_errors(reset=True) == 0


def test_groups_of_many_sequences_and_the_same_last_page_in_other_prefixes():
    rng = np.random.default_rng(2)
    B = 5000
    table = np.zeros((B, 3), np.int32)
    table[:, 0] = rng.integers(0, 40, B)  # the third page is everyone's: only the first two tell
    table[:, 1] = rng.integers(0, 3, B)
    table[:, 2] = 77
    check_groups(table, [48] * B, 3, 200)
    check_groups(table, [47] * B, 2, 50)


def test_groups_with_bad_lengths_and_none():
    table = np.tile(np.arange(4, dtype=np.int32), (5, 1))
    lens = [64, -1, 65, 40, 2 ** 31 - 1]
    check_groups(table, lens, 1, 3)
    assert ok.oscar_device_errors(reset=True) == ok.OSCAR_DEVERR_POSITION
    check_groups(table, [0] * 5, 1, 3)
    check_groups(table, [64] * 5, 9, 3)


# ---- together ------------------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("fmt", [R.E4M3, R.INT8])
@pytest.mark.parametrize("D,interleaved", [(64, True), (128, False)])
def test_a_prompt_its_samples_and_their_steps(fmt, D, interleaved):
    """Reserve, rotate and append a prompt, extend over it, fork it to samples, and steps of all of them with shared prefixes:
    each against dense attention over the same codes with queries rotated in 64 bits, and near the step without groups."""
    import rope_ref as RR
    hq, H, B = 8, 2, 12
    c = Kv8Cache(hq, H, D, num_pages=400, batch=B, max_seq_len=1500, kv_format=fmt)
    rope = ok.Rope(D // 2, interleaved=interleaved, scaling=dict(kind="linear", factor=2.0))
    g = torch.Generator("cuda").manual_seed(4)

    def step(new, sharing):
        T = sum(new)
        rows = torch.randn(T, hq + 2 * H, D, device="cuda", generator=g).bfloat16()
        q, k, v = torch.split(rows, [hq, H, H], 1)
        start = i32(np.concatenate([[0], np.cumsum(new)]))
        assert c.reserve(i32(new)).all()
        qr = c.rope_append(q, k, v, rope, start, max(new))
        lens = c.seq_lens.tolist()
        seq = [b for b, n in enumerate(new) for _ in range(n)]
        pos = [lens[b] - n + i for b, n in enumerate(new) for i in range(n)]
        want, err = RR.rotate(q.double().cpu().numpy(), pos, rope)
        assert (np.abs(qr.double().cpu().numpy() - want) <= err + 2.0 ** -8 * (np.abs(want) + err)).all()
        if not sharing:
            out = c.extend(qr, start, max(new))
        else:
            groups = c.groups(min_pages=2, max_groups=4)
            out = c.decode_shared(qr, groups, max_prefix_len=1024, max_own_len=1100)
        ref, tol = R.attention(c.pages, c.scales, qr, seq, pos, c.page_table.tolist(), fmt, 0, 0)
        assert ((out.double() - ref).abs() <= tol).all()
        if sharing:
            plain = c.decode(qr)
            assert ((plain.double() - ref).abs() <= tol).all()
            return groups
        return None

    step([1001, 77] + [0] * (B - 2), False)
    c.fork(i32([0] * 7 + [1] * 2), i32([2, 3, 4, 5, 6, 7, 8, 9, 10]))
    for i in range(20):
        groups = step([1] * B, True)
    members, start, prefix = (x.tolist() for x in groups)
    assert members[:start[1]] == [0, 2, 3, 4, 5, 6, 7, 8] and prefix == [992, 64, 0, 0] and members[start[1]:start[2]] == [1, 9, 10]
    c.free(i32([0, 3]))  # the prompt's own sequence ends, its pages live on
    c.seq_lens[5] -= 5
    groups = c.groups(min_pages=2)
    assert groups.members.tolist() == [1, 9, 10, 2, 4, 5, 6, 7, 8, 0, 3, 11] and groups.group_start.tolist()[:3] == [0, 3, 9]
    q = torch.randn(B, hq, D, device="cuda", generator=g).bfloat16()
    lens = c.seq_lens.tolist()
    ref, tol = R.attention(c.pages, c.scales, q, list(range(B)), [n - 1 for n in lens], c.page_table.tolist(), fmt, 0, 0)
    out = c.decode_shared(q, groups)
    assert ((out.double() - ref).abs() <= tol).all() and (out[0] == 0).all()
    assert ok.oscar_device_errors(reset=True) == 0
    assert isinstance(groups, SharedPrefixes)
    with pytest.raises(ValueError):
        c.decode_shared(q, groups, max_own_len=c.max_seq_len + 1)


@pytest.mark.parametrize("B,prompt", [(5, 300), (64, 6000)])
def test_captured_steps_read_what_the_step_before_wrote(B, prompt):
    """Whole steps replayed without a pause, two at a time, and the last one's output, over the list and over tiles: the queries,
    lengths, tables and lists that its kernels read are written by the kernels just before them."""
    hq, H, D, steps = 8, 2, 128, 6
    c = Kv8Cache(hq, H, D, num_pages=prompt // 16 + 5 * B, batch=B, max_seq_len=prompt + 2 * steps + 16)
    g = torch.Generator("cuda").manual_seed(B)
    rope = ok.Rope(D)
    x = torch.randn(prompt, hq + 2 * H, D, device="cuda", generator=g).bfloat16()
    assert c.reserve(i32([prompt] + [0] * (B - 1))).all()
    c.rope_append(*torch.split(x, [hq, H, H], 1), rope, i32([0] + [prompt] * B), prompt)
    c.fork(i32([0] * (B - 1)), i32(list(range(1, B))))
    rows = torch.zeros(B, hq + 2 * H, D, dtype=torch.bfloat16, device="cuda")
    source = torch.randn(2 * steps + 3, B, hq + 2 * H, D, device="cuda", generator=g).bfloat16()
    at = torch.zeros(1, dtype=torch.int64, device="cuda")
    start, ones = torch.arange(B + 1, dtype=torch.int32, device="cuda"), i32([1] * B)
    out, qr = (torch.zeros(B, hq, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def step():
        rows.copy_(source.index_select(0, at)[0])
        at.add_(1)
        c.reserve(ones)
        c.rope_append(*torch.split(rows, [hq, H, H], 1), rope, start, 1, q_out=qr)
        c.decode_shared(qr, c.groups(max_groups=2), out, max_prefix_len=prompt, max_own_len=64)

    assert (ok.oscar_kv8_decode_shared_plan(c.dims, B, c.max_seq_len, prompt, 64, B, 2)["tile_rows"] > 0) == (B == 64)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(steps):
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        lens = c.seq_lens.tolist()
        assert lens == [prompt + 3 + 2 * i] * B
        ref, tol = R.attention(c.pages, c.scales, qr, list(range(B)), [n - 1 for n in lens], c.page_table.tolist(), R.E4M3, 0, 0)
        assert ((out.double() - ref).abs() <= tol).all()
    assert ok.oscar_device_errors(reset=True) == 0


def test_a_cache_with_a_window_refuses():
    c = Kv8Cache(4, 2, 64, num_pages=8, batch=2, max_seq_len=64, window_len=16)
    with pytest.raises(ValueError):
        c.decode_shared(torch.zeros(2, 4, 64, device="cuda", dtype=torch.bfloat16), SharedPrefixes(i32([0]), i32([0, 1]), i32([0])))
