"""oscar_kv8_append against the 64-bit reference: codes and scales have to be equal."""

import numpy as np
import pytest
import torch

import int2_rotated_kv_append_gb300 as ok
import kv8_ref as R

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, H, D, fmt, capacity, seed):
        """Sequences of at most `capacity` tokens each, pages in a random order, pools filled with a pattern."""
        self.H, self.D, self.fmt, self.rng = H, D, fmt, np.random.default_rng(seed)
        per = [max(1, -(-c // 16)) for c in capacity]
        n = sum(per) + 3
        order = self.rng.permutation(n)
        self.table = np.full((len(per), max(per)), -1, np.int32)
        at = 0
        for b, c in enumerate(per):
            self.table[b, :c] = order[at:at + c]
            at += c
        self.dims = ok.make_dims(H, H, D, 16, D, n, max(per))
        self.codes = np.full((n, H, 2, 16, D), 0x2b, np.uint8)
        self.scales = np.full((n, H, 2), 2.0 ** 30, np.float32)  # stale: a page's first token replaces it
        self.g_codes, self.g_scales = torch.from_numpy(self.codes).cuda(), torch.from_numpy(self.scales).cuda()
        self.lens = [0] * len(per)

    def kv(self, T, spread=1.0):
        x = self.rng.normal(size=(2, T, self.H, self.D)) * spread
        x *= 2.0 ** self.rng.integers(-3, 4, size=(2, T, 1, 1))
        x[:, :, :, :3] *= 20
        return [torch.from_numpy(a).to(torch.bfloat16) for a in x]

    def append(self, new, k=None, v=None):
        self.lens = [a + n for a, n in zip(self.lens, new)]
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        if k is None:
            k, v = self.kv(int(start[-1]))
        R.append(self.codes, self.scales, k.double().numpy(), v.double().numpy(), start, self.table, self.lens, self.fmt)
        ok.oscar_kv8_append(self.dims, self.fmt, len(new), max(new), k.cuda(), v.cuda(), torch.from_numpy(start).cuda(),
                            torch.from_numpy(self.table).cuda(), torch.tensor(self.lens, dtype=torch.int32, device="cuda"),
                            self.g_codes, self.g_scales)

    def check(self):
        assert np.array_equal(self.g_scales.cpu().numpy(), self.scales)
        got = self.g_codes.cpu().numpy()
        if self.fmt == R.E4M3:  # a zero's sign says nothing
            got, want = np.where(got == 0x80, 0, got), np.where(self.codes == 0x80, 0, self.codes)
        else:
            want = self.codes
        assert np.array_equal(got, want)


@pytest.mark.parametrize("fmt", [R.E4M3, R.INT8])
@pytest.mark.parametrize("H,D", [(1, 64), (3, 128), (8, 128)])
def test_append_in_pieces(H, D, fmt):
    c = Case(H, D, fmt, [100, 1, 64, 33, 40], seed=H * D + fmt)
    for new in ([17, 0, 16, 1, 5], [1, 1, 1, 1, 0], [40, 0, 15, 30, 1], [1, 0, 1, 1, 1], [0, 0, 0, 0, 1]):
        c.append(new)
        c.check()
    assert ok.oscar_device_errors(reset=True) == 0


@pytest.mark.parametrize("fmt", [R.E4M3, R.INT8])
def test_append_single_tokens_with_growing_and_falling_scales(fmt):
    c = Case(2, 64, fmt, [40, 40], seed=5)
    for i, e in enumerate([0, 3, -4, 9, 9, -20, 11, 30, -30, 31] + list(range(-8, 12))):
        k, v = c.kv(2, 2.0 ** e)
        c.append([1, 1], k, v)
        c.check()


@pytest.mark.parametrize("fmt", [R.E4M3, R.INT8])
def test_append_extremes(fmt):
    # zeros, the border magnitudes of each scale, bf16's largest and smallest values, infinities
    big = torch.finfo(torch.bfloat16).max
    rows = [0.0, 448.0, 450.0, 127.0, 128.0, big, -big, float("inf"), -float("inf"), 1e-38, 9e-41, 2.0 ** -100]
    c = Case(1, 64, fmt, [16] * len(rows) + [64], seed=6)
    T = len(rows) + 48
    k = torch.zeros(T, 1, 64, dtype=torch.bfloat16)
    for i, r in enumerate(rows):
        k[i, 0, ::2] = r
        k[i, 0, 1::2] = r / 3 if abs(r) < 1e38 else 1.0
    k[len(rows):] = torch.randn(48, 1, 64, generator=torch.Generator().manual_seed(1)).bfloat16()
    k[len(rows) + 20, 0, 5] = float("inf")
    c.append([1] * len(rows) + [48], k, -k)
    c.check()
    vals = c.g_codes.view(torch.float8_e4m3fn if fmt == R.E4M3 else torch.int8).float() * c.g_scales[..., None, None]
    assert torch.isfinite(vals[torch.from_numpy(c.table[:len(rows), 0]).cuda().long(), :, :, :1]).all()
    assert ok.oscar_device_errors(reset=True) == 0


@pytest.mark.parametrize("fmt", [R.E4M3, R.INT8])
def test_append_nan_becomes_zero_and_is_flagged(fmt):
    c = Case(2, 128, fmt, [32], seed=7)
    k, v = c.kv(20)
    k[3, 1, 7] = float("nan")
    v[18, 0, 0] = float("nan")
    c.append([20], k, v)
    c.check()
    assert ok.oscar_device_errors(reset=True) == ok.OSCAR_DEVERR_VALUE


def test_append_skips_what_is_out_of_range():
    c = Case(2, 64, R.INT8, [32, 32, 32, 32], seed=8)
    before = c.g_codes.clone()
    k, v = (x.cuda() for x in c.kv(12))
    def call(start, lens, table=None, max_new=6):
        ok.oscar_kv8_append(c.dims, R.INT8, 4, max_new, k, v, torch.tensor(start, dtype=torch.int32, device="cuda"),
                            torch.from_numpy(c.table if table is None else table).cuda(),
                            torch.tensor(lens, dtype=torch.int32, device="cuda"), c.g_codes, c.g_scales)
        return ok.oscar_device_errors(reset=True)
    P = ok.OSCAR_DEVERR_POSITION
    assert call([0, 3, 6, 9, 12], [2, 2, 2, 2]) == P      # more rows than tokens
    assert call([0, 12, 12, 12, 12], [12, 0, 0, 0]) == P  # above max_tokens_per_seq
    assert call([0, 3, 6, 9, 12], [40] * 4) == P          # beyond the table row
    assert call([0, 0, 0, 0, 13], [0, 0, 0, 13], max_new=13) == P
    assert call([5, 3, 3, 3, 3], [4, 0, 0, 0]) == P       # decreasing
    bad = c.table.copy()
    bad[:, 0] = [-1, 10 ** 6, c.dims.num_pages, -7]
    assert call([0, 3, 6, 9, 12], [3] * 4, bad) == ok.OSCAR_DEVERR_PAGE_ID
    assert torch.equal(c.g_codes, before)


def test_append_prompt_of_many_pages_equals_the_reference_on_a_sample():
    c = Case(8, 128, R.E4M3, [5000, 3001], seed=9)
    k, v = (torch.randn(8001, 8, 128, device="cuda", generator=torch.Generator("cuda").manual_seed(2)).bfloat16()
            for _ in range(2))
    start = torch.tensor([0, 5000, 8001], dtype=torch.int32, device="cuda")
    lens = torch.tensor([5000, 3001], dtype=torch.int32, device="cuda")
    ok.oscar_kv8_append(c.dims, R.E4M3, 2, 5000, k, v, start, torch.from_numpy(c.table).cuda(), lens, c.g_codes,
                        c.g_scales)
    R.append(c.codes, c.scales, k.double().cpu().numpy(), v.double().cpu().numpy(), [0, 5000, 8001], c.table,
             [5000, 3001], R.E4M3)
    c.check()


@pytest.mark.parametrize("most", [5, 1000, 2 ** 31 - 1])
def test_append_with_a_bound_far_above_the_tokens(most):
    # the grid goes by the tokens that there are
    c = Case(2, 64, R.INT8, [40, 40], seed=10)
    k, v = c.kv(6)
    start, lens = torch.tensor([0, 5, 6], dtype=torch.int32, device="cuda"), torch.tensor([5, 1], dtype=torch.int32, device="cuda")
    R.append(c.codes, c.scales, k.double().numpy(), v.double().numpy(), [0, 5, 6], c.table, [5, 1], R.INT8)
    t0, t1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    t0.record()
    ok.oscar_kv8_append(c.dims, R.INT8, 2, most, k.cuda(), v.cuda(), start, torch.from_numpy(c.table).cuda(), lens, c.g_codes,
                        c.g_scales)
    t1.record()
    torch.cuda.synchronize()
    c.check()
    assert t0.elapsed_time(t1) < 100  # (2^28 empty blocks took longer)
