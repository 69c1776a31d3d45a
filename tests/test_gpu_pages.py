"""Page operations against an allocator in plain Python lists: tables, lengths and counts have to be equal."""

import random

import numpy as np
import pytest
import torch

import int2_rotated_kv_append_gb300 as ok
import kv8_ref as R

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Both:
    """The device state and its model, taken through the same calls."""

    def __init__(self, num_pages, batch, max_pages, pools=()):
        self.m = R.Pages(num_pages, batch, max_pages)
        self.dims = ok.make_dims(1, 1, 64, 16, 64, num_pages, max_pages)
        self.table, self.lens, self.refs = i32(self.m.table), i32(self.m.lens), i32(self.m.refs)
        self.pools = list(pools)
        self.want = [p.clone() for p in self.pools]
        self.ws = torch.full((ok.oscar_pages_workspace_bytes(self.dims, batch, 600),), 0xff, dtype=torch.uint8, device="cuda")

    def check(self, errors=0):
        held = torch.arange(self.table.shape[1])[None] * 16 < torch.tensor(self.m.lens)[:, None]
        assert self.lens.tolist() == self.m.lens
        assert self.refs.tolist() == self.m.refs
        assert torch.equal(torch.where(held, self.table.cpu(), -1), torch.where(held, torch.tensor(self.m.table, dtype=torch.int32), -1))
        for p, w in zip(self.pools, self.want):
            assert torch.equal(p, w)
        assert ok.oscar_device_errors(reset=True) == errors

    def reserve(self, new, errors=0):
        granted = torch.full((len(new),), 9, dtype=torch.int32, device="cuda")
        ok.oscar_pages_reserve(self.dims, i32(new), self.table, self.lens, self.refs, granted, self.ws)
        assert granted.tolist() == self.m.reserve(new)
        self.check(errors)

    def fork(self, src, dst, errors=0):
        granted = torch.full((len(src),), 9, dtype=torch.int32, device="cuda")
        ok.oscar_pages_fork(self.dims, self.pools, i32(src), i32(dst), self.table, self.lens, self.refs, granted, self.ws)
        want, copies = self.m.fork(src, dst)
        for w in self.want:
            for s, d in copies:
                w[d] = w[s]
        assert granted.tolist() == want
        self.check(errors)

    def free(self, seqs):
        ok.oscar_pages_free(self.dims, i32(seqs), self.table, self.lens, self.refs)
        self.m.free(seqs)
        self.check()

    def trim(self, sink, window):
        ok.oscar_pages_trim(self.dims, sink, window, self.table, self.lens, self.refs)
        self.m.trim(sink, window)
        self.check()

    def compact(self):
        used = i32([77])
        ok.oscar_pages_compact(self.dims, self.pools, self.table, self.lens, self.refs, used, self.ws)
        n, moves = self.m.compact()
        for w in self.want:
            for s, d in moves:
                w[d] = w[s]
        assert used.item() == n
        # a page that moved away may hold anything
        for p, w in zip(self.pools, self.want):
            assert torch.equal(p[:n], w[:n])
            p[n:], w[n:] = 0, 0
        self.check()


def pools(n, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    return [torch.randn(n, 2, 2, 16, 64, device="cuda", generator=g).bfloat16(),
            torch.randint(0, 256, (n, 3, 4), device="cuda", generator=g).byte(),       # 12 bytes a page
            torch.randn(n, 1, device="cuda", generator=g),                             # 4
            torch.randint(0, 256, (n, 70000 // 16 * 16), device="cuda", generator=g).byte()]


@pytest.mark.parametrize("seed", range(8))
def test_random_calls(seed):
    r = random.Random(seed)
    n, batch, max_pages = r.choice([(60, 9, 20), (7, 3, 9), (5000, 40, 200), (4096, 12, 700)])
    b = Both(n, batch, max_pages, pools(n, seed) if n < 100 else [torch.randn(n, 64, device="cuda")])
    for _ in range(40):
        what = r.choice(["reserve", "reserve", "fork", "free", "trim", "compact"])
        lens = b.m.lens
        if what == "reserve":
            top = r.choice([1, 20, 16 * n // batch])
            new = [min(r.randint(0, top), max_pages * 16 - L) for L in lens]
            asked = sum(-(-(L + k) // 16) - -(-L // 16) for L, k in zip(lens, new))
            b.reserve(new, ok.OSCAR_DEVERR_NO_PAGES if asked > len(b.m.free_ids()) else 0)
        elif what == "fork":
            empty = [i for i in range(batch) if lens[i] == 0]
            dst = r.sample(empty, r.randint(0, len(empty)))
            src = [r.choice([s for s in range(batch) if s != d]) for d in dst]
            part = sum(lens[s] % 16 != 0 and b.m.table[s][lens[s] // 16] >= 0 for s in src)
            if dst:
                b.fork(src, dst, ok.OSCAR_DEVERR_NO_PAGES if part > len(b.m.free_ids()) else 0)
        elif what == "free":
            b.free([r.randrange(batch) for _ in range(r.randint(1, batch))])  # some twice
        elif what == "trim":
            b.trim(r.choice([0, 3, 16, 40]), r.choice([1, 16, 50, 300]))
        else:
            b.compact()


def test_reserve_serves_in_order_and_refuses_the_rest():
    b = Both(10, 5, 10)
    b.reserve([16 * 4, 16 * 4, 16 * 3, 0, 1], ok.OSCAR_DEVERR_NO_PAGES)  # 4, 4, refused, nothing, refused
    assert b.m.lens == [64, 64, 0, 0, 0]
    b.reserve([0, 0, 1, 16, 0])
    b.reserve([0, 0, 15, 0, 0])  # within the page
    b.reserve([0, 0, 1, 0, 0], ok.OSCAR_DEVERR_NO_PAGES)


def test_reserve_of_more_pages_than_32_bits_count():
    dims = ok.make_dims(1, 1, 64, 16, 64, 4, 1 << 26)
    lens, refs, granted = i32([0] * 100), i32([0] * 4), i32([5] * 100)
    table = torch.full((100, 1), -1, dtype=torch.int32, device="cuda")  # no row is written: nothing is granted
    ws = torch.empty(ok.oscar_pages_workspace_bytes(dims, 100, 0), dtype=torch.uint8, device="cuda")
    ok.oscar_pages_reserve(dims, i32([1 << 30] * 100), table, lens, refs, granted, ws)
    assert granted.tolist() == [0] * 100 and not lens.any() and not refs.any()
    assert ok.oscar_device_errors(reset=True) == ok.OSCAR_DEVERR_NO_PAGES


def test_fork_refusals():
    b = Both(30, 8, 6, pools(30))
    b.reserve([20, 32, 0, 5, 0, 0, 0, 0])
    P = ok.OSCAR_DEVERR_POSITION
    b.fork([0, 0, 1, 2], [2, 3, 2, 4], P)       # 3 is in use; 2 named twice; 4 becomes empty again
    b.fork([0, 9, -1, 6, 5], [9, 4, 5, 6, -3], P)  # ids out of range, a fork of itself
    b.fork([1, 1, 0], [4, 5, 6])


def test_fork_of_a_trimmed_sequence_and_many_forks():
    b = Both(600, 520, 8, [torch.randn(600, 64, device="cuda")])
    b.reserve([100, 63] + [0] * 518)
    b.trim(16, 20)
    b.fork([i % 2 for i in range(518)], list(range(2, 520)), ok.OSCAR_DEVERR_NO_PAGES if 518 > 589 else 0)
    b.free(list(range(520)))
    assert not b.refs.any()


def test_copy_pages_and_per_sequence_buffers():
    n = 40
    dims = ok.make_dims(1, 1, 64, 16, 64, n, 4)
    ps = pools(n, 3)
    want = [p.clone() for p in ps]
    src, dst = [3, 3, -1, 5, 39, 7], [10, 11, 12, -2, 0, 7]
    for w in want:
        for s, d in ((3, 10), (3, 11), (39, 0)):
            w[d] = w[s]
    ok.oscar_pages_copy(dims, ps, i32(src), i32(dst))
    assert all(torch.equal(p, w) for p, w in zip(ps, want))
    ok.oscar_pages_copy(dims, ps, i32([40, 0]), i32([1, 40]))
    assert ok.oscar_device_errors(reset=True) == ok.OSCAR_DEVERR_PAGE_ID
    assert all(torch.equal(p, w) for p, w in zip(ps, want))


def test_bad_device_values_are_skipped_and_flagged():
    b = Both(20, 4, 5, pools(20))
    b.reserve([50, 40, 16, 0])
    P, I = ok.OSCAR_DEVERR_POSITION, ok.OSCAR_DEVERR_PAGE_ID
    ok.oscar_pages_free(b.dims, i32([4, -1]), b.table, b.lens, b.refs)
    b.check(P)
    lens = i32([81, -1, 16, 0])
    ok.oscar_pages_free(b.dims, i32([0, 1]), b.table, lens, b.refs)
    b.check(P)
    ok.oscar_pages_trim(b.dims, 0, 1, b.table, i32([81, -1, 0, 0]), b.refs)
    b.check(P)
    ok.oscar_pages_reserve(b.dims, i32([-1, 60, 0, 81]), b.table, b.lens, b.refs, None, b.ws)
    b.check(P)
    bad = b.table.clone()
    bad[0, 0], bad[1, 0] = 20, 19  # out of range; a free page
    ok.oscar_pages_free(b.dims, i32([0, 1]), bad, b.lens.clone(), b.refs)
    assert ok.oscar_device_errors(reset=True) == I
    assert b.refs.tolist()[0] == 1 and b.refs.tolist()[19] == 0


def test_compact_of_a_large_pool():
    n = 300000
    g = torch.Generator("cuda").manual_seed(1)
    refs = (torch.rand(n, device="cuda", generator=g) < 0.4).int()
    used = refs.nonzero().flatten()
    pool = torch.arange(n, dtype=torch.int32, device="cuda")[:, None].repeat(1, 4).contiguous()
    batch, width = 50, -(-used.numel() // 50)
    table = torch.full((batch * width,), -1, dtype=torch.int32, device="cuda")
    table[:used.numel()] = used[torch.randperm(used.numel(), device="cuda")].int()
    table = table.view(batch, width)
    before = table.clone()
    lens = i32([width * 16] * batch)
    dims = ok.make_dims(1, 1, 64, 16, 64, n, width)
    num = i32([0])
    ws = torch.empty(ok.oscar_pages_workspace_bytes(dims, batch, 0), dtype=torch.uint8, device="cuda")
    ok.oscar_pages_compact(dims, [pool], table, lens, refs, num, ws)
    k = num.item()
    assert k == used.numel() and refs[:k].all() and not refs[k:].any()
    assert int(table.max()) < k
    ids = table[table >= 0].long()
    assert torch.equal(pool[ids, 0], before[before >= 0])
    assert torch.equal(ids.sort()[0], torch.arange(k, device="cuda"))
    ok.oscar_pages_compact(dims, [pool], table, lens, refs, num, ws)  # nothing to do
    assert torch.equal(pool[ids, 0], before[before >= 0]) and num.item() == k


def test_free_pages_far_into_a_full_pool():
    n = 50000
    dims = ok.make_dims(1, 1, 64, 16, 64, n, 100)
    refs = torch.ones(n, dtype=torch.int32, device="cuda")
    refs[[17, 40000, 49999]] = 0
    table, lens = torch.full((3, 100), -1, dtype=torch.int32, device="cuda"), i32([0, 0, 0])
    ws = torch.empty(ok.oscar_pages_workspace_bytes(dims, 3, 0), dtype=torch.uint8, device="cuda")
    granted = i32([0, 0, 0])
    ok.oscar_pages_reserve(dims, i32([1, 17, 1]), table, lens, refs, granted, ws)
    assert table[:, :2].tolist() == [[17, -1], [40000, 49999], [-1, -1]] and granted.tolist() == [1, 1, 0]
    assert ok.oscar_device_errors(reset=True) == ok.OSCAR_DEVERR_NO_PAGES


@pytest.mark.parametrize("chunks", [1, 4, 6, 7, 9])
@pytest.mark.parametrize("more", [-1, 0, 1, 5])
def test_compact_around_whole_chunks_of_the_count(chunks, more):
    n = 4096 * chunks + more
    b = Both(n, 5, n // 4 + 2, pools=pools(n, seed=chunks))
    b.reserve([16 * (n // 5), 16 * (n // 6) + 3, 40, 16 * (n // 5), 16 * (n // 5)])
    b.compact()  # nothing moves
    b.free([0, 2])
    b.compact()
    b.free([3])
    b.fork([1], [0])
    b.compact()
    b.reserve([1, 1, 17, 0, 0])
    b.compact()
