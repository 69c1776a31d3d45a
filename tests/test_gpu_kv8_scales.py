"""V scales that differ between pages by far: what a row gets depends on what it sees alone, for the decode and the
extend over the 8-bit cache.  Reference and tolerance: kv8_ref.attention_of_rows."""

import numpy as np
import pytest
import torch

import int2_rotated_kv_append_gb300 as ok
import kv8_ref as R
from test_gpu_kv8_attention import Cache

pytestmark = pytest.mark.gpu


def check(c, out, q, seq, pos, sink, window, decode=False):
    assert torch.isfinite(out).all()
    ref, tol = R.attention_of_rows(c.codes, c.scales, q, seq, pos, c.table.tolist(), c.fmt, sink, window, decode)
    err = (out.double() - ref).abs()
    worst = (err / tol).max().item()
    assert (err <= tol).all(), f"{worst:.3g} times the tolerance, at {(err > tol).nonzero()[:4].tolist()}"


def scaled(c, exponents):
    """The V scales of each sequence's pages times 2^exponents[page]."""
    for b, L in enumerate(c.lens):
        for j in range(-(-L // 16)):
            c.scales[c.table[b, j].item(), :, 1] *= 2.0 ** int(exponents[j])


PATTERNS = {
    "one large page": lambda n: np.where(np.arange(n) == n // 2, 40, 0),
    "every seventh": lambda n: np.where(np.arange(n) % 7 == 3, 26, 0),
    "rising": lambda n: np.linspace(0, 40, n).round(),
    "falling": lambda n: np.linspace(10, -30, n).round(),
    "within 2^7": lambda n: np.random.default_rng(n).integers(0, 7, n),
    "any": lambda n: np.random.default_rng(n).integers(-60, 60, n),
    "large at both ends": lambda n: np.where((np.arange(n) == 0) | (np.arange(n) == n - 1), 30, 0),
}


@pytest.mark.parametrize("pattern", list(PATTERNS))
@pytest.mark.parametrize("D,gqa,fmt", [(64, 5, R.INT8), (128, 8, R.E4M3), (128, 1, R.INT8), (64, 2, R.E4M3)])
@pytest.mark.parametrize("sink,window", [(0, 0), (0, 64), (20, 100)])
def test_page_scales_far_apart(pattern, D, gqa, fmt, sink, window):
    lens = [1100, 333]
    c = Cache(2, D, fmt, lens, seed=D + gqa + fmt + window)
    scaled(c, PATTERNS[pattern](-(-max(lens) // 16)))
    for rows in ([700, 333], [100, 40], [5, 2], [1, 1]):  # two row tiles, one (or two at D = 128), half a tile
        seq = [b for b, r in enumerate(rows) for _ in range(r)]
        pos = [lens[b] - r + i for b, r in enumerate(rows) for i in range(r)]
        q = c.q(len(seq), 2 * gqa)
        for pps in (0, 16):
            check(c, c.extend(q, rows, sink, window, pps=pps), q, seq, pos, sink, window)
    for pps in (0, 3):
        check(c, c.decode(q, sink, window, pps=pps), q, seq, pos, sink, window, decode=True)
    assert ok.oscar_device_errors(reset=True) == 0


@pytest.mark.parametrize("fmt", [R.E4M3, R.INT8])
@pytest.mark.parametrize("sink,window", [(0, 0), (0, 48), (37, 48)])
@pytest.mark.parametrize("at", [[200], [40, 41], [200, 201, 500, 39]])
def test_infinite_values_are_seen_by_the_rows_that_see_them_alone(fmt, sink, window, at):
    # the append saturates them and their pages get the largest scale: the other rows of these pages keep what their
    # codes hold, the other pages' rows all of it
    H, D, L = 2, 128, 600
    c = Cache(H, D, fmt, [L], seed=fmt + window + len(at))
    k, v = (torch.randn(L, H, D, device="cuda", generator=c.g).bfloat16() for _ in range(2))
    v[at, :, 3] = float("inf")
    v[at, 1, 70] = -float("inf")
    start = torch.tensor([0, L], dtype=torch.int32, device="cuda")
    ok.oscar_kv8_append(c.dims(2 * H), fmt, 1, L, k, v, start, c.table_d, c.lens_d, c.codes, c.scales)
    for rows in (600, 60, 25, 1):
        q = c.q(rows, 2 * H)
        check(c, c.extend(q, [rows], sink, window), q, [0] * rows, list(range(L - rows, L)), sink, window)
        check(c, c.extend(q, [rows], sink, window, pps=8), q, [0] * rows, list(range(L - rows, L)), sink, window)
    # rows that end the sequence early: a decode of each length
    for n in (30, 39, 40, 42, 45, 190, 200, 205, 500, 520):
        c.lens_d[0] = n
        q = c.q(1, 2 * H)
        check(c, c.extend(q, [1], sink, window), q, [0], [n - 1], sink, window)


def test_weights_on_pages_of_small_values():
    # the logits favour the pages with the smallest V, by up to what their scale lacks: every page's share counts
    c = Cache(1, 128, R.E4M3, [900], seed=31)
    n = -(-900 // 16)
    e = np.random.default_rng(5).integers(-20, 1, n)
    scaled(c, e)
    for j in range(n):
        page = c.table[0, j].item()
        x = c.codes[page, 0, 0].view(torch.float8_e4m3fn).float()
        x[:, 0] = float(-e[j])  # q's first channel times this: about log 2 per step of the exponent
        c.codes[page, 0, 0] = x.to(torch.float8_e4m3fn).view(torch.uint8)
        c.scales[page, 0, 0] = 2.0 ** -5
    for rows in (300, 10, 1):
        q = c.q(rows, 4, 0.05)
        q[:, :, 0] = 256.0
        pos = list(range(900 - rows, 900))
        check(c, c.extend(q, [rows]), q, [0] * rows, pos, 0, 0)
        check(c, c.extend(q, [rows], 0, 200, pps=8), q, [0] * rows, pos, 0, 200)
    check(c, c.decode(q), q, [0], [899], 0, 0, decode=True)


def test_values_of_zero_scale_beside_others():
    c = Cache(2, 64, R.INT8, [500], seed=32)
    for j in (3, 4, 20):
        c.scales[c.table[0, j].item()] = 0.0
    for j in (7, 9):
        c.scales[c.table[0, j].item(), :, 1] = 2.0 ** -100
        c.codes[c.table[0, j].item(), :, 1] = 0
    for rows in (200, 9, 1):
        q = c.q(rows, 6)
        check(c, c.extend(q, [rows]), q, [0] * rows, list(range(500 - rows, 500)), 0, 0)
    check(c, c.decode(q), q, [0], [499], 0, 0, decode=True)


@pytest.mark.parametrize("fmt", [R.E4M3, R.INT8])
def test_jumps_of_different_sizes_within_a_warp(fmt):
    # rows that see a page 2^110 above the ones before them beside rows that see one 2^188 above
    c = Cache(1, 128, fmt, [192], seed=33 + fmt)
    scaled(c, [-70] * 8 + [40, 118, -70, 0])
    for rows, hq in ((64, 1), (64, 2), (64, 4), (40, 1), (192, 3)):
        q = c.q(rows, hq)
        pos = list(range(192 - rows, 192))
        check(c, c.extend(q, [rows]), q, [0] * rows, pos, 0, 0)
        check(c, c.extend(q, [rows], pps=8), q, [0] * rows, pos, 0, 0)
        check(c, c.extend(q, [rows], 5, 17), q, [0] * rows, pos, 5, 17)


@pytest.mark.parametrize("fmt", [R.E4M3, R.INT8])
@pytest.mark.parametrize("sink,window", [(0, 0), (37, 48)])
@pytest.mark.parametrize("pps", [0, 1, 4])
def test_decode_of_several_infinite_values(fmt, sink, window, pps):
    # their weighted sum is beyond fp32 before it is divided by the weights' sum
    c = Cache(2, 128, fmt, [900, 400, 50], seed=fmt + window + 40)
    k, v = (torch.randn(1350, 2, 128, device="cuda", generator=c.g).bfloat16() for _ in range(2))
    v[[5, 30, 31, 870, 880, 899, 900, 901, 930, 1299, 1310, 1311], :, 3] = float("inf")
    v[[20, 890, 1290, 1305], 1, 70:90] = -float("inf")
    start = torch.tensor([0, 900, 1300, 1350], dtype=torch.int32, device="cuda")
    ok.oscar_kv8_append(c.dims(8), fmt, 3, 900, k, v, start, c.table_d, c.lens_d, c.codes, c.scales)
    for factor in (0.01, 1.0, 8.0):  # even weights (the sum of many), and a few large ones
        q = c.q(3, 8, factor)
        check(c, c.decode(q, sink, window, pps=pps), q, [0, 1, 2], [899, 399, 49], sink, window, decode=True)
        check(c, c.extend(q, [1, 1, 1], sink, window, pps=8 * pps), q, [0, 1, 2], [899, 399, 49], sink, window)


def test_decode_beside_a_token_of_a_large_scale_behind_the_window():
    # the window's first page has its scale from a token that is out of the window
    c = Cache(1, 64, R.INT8, [300], seed=45)
    scaled(c, [-60] * 19)
    page = c.table[0, 10].item()
    c.scales[page, 0, 1] = 2.0 ** 118
    c.codes[page, 0, 1, 8:] = 0
    q = c.q(1, 4)
    check(c, c.decode(q, 0, 300 - 168), q, [0], [299], 0, 300 - 168, decode=True)
    check(c, c.decode(q, 0, 300 - 168, pps=3), q, [0], [299], 0, 300 - 168, decode=True)
    check(c, c.extend(q, [1], 0, 300 - 168), q, [0], [299], 0, 300 - 168)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("gqa", [1, 5, 8])
def test_decode_holds_weights_in_two_parts(D, gqa):
    # (tests/test_kv8_ref.py: one part alone is outside the tolerance)
    lens = [16] * 5
    c = Cache(1, D, R.INT8, lens, seed=D + gqa)
    pages = [R.cancelling_page(D, seed) for seed in range(5)]
    for b, (k, v, _) in enumerate(pages):
        page = c.table[b, 0].item()
        codes = torch.zeros(2, 16, D, dtype=torch.int8)
        codes[0, :, 0], codes[1] = torch.from_numpy(k), torch.from_numpy(v)
        c.codes[page, 0] = codes.view(torch.uint8).cuda()
        c.scales[page, 0] = torch.tensor([2.0 ** -4, 1.0], device="cuda")
    q = torch.zeros(5, gqa, D, device="cuda", dtype=torch.bfloat16)
    q[:, :, 0] = 1.0
    out = c.decode(q, sm_scale=0.125).double().cpu().numpy()
    for b, (k, v, w) in enumerate(pages):
        want, tol = R.cancelling_tolerance(v, w)
        assert (np.abs(out[b] - want) <= tol).all()


@pytest.mark.parametrize("fmt", [R.E4M3, R.INT8])
@pytest.mark.parametrize("D,gqa", [(128, 4), (64, 7)])
@pytest.mark.parametrize("pps", [0, 40])
def test_one_chunk_beside_many_single_rows(fmt, D, gqa, pps):
    # one varlen call of a prompt chunk and of sequences that decode, as a mixed serving step makes it
    g = np.random.default_rng(gqa)
    lens = [4100] + [int(n) for n in g.integers(1, 6000, 40)]
    rows = [700] + [1] * 40
    rows[7] = 0
    c = Cache(2, D, fmt, lens, seed=fmt + gqa)
    q = c.q(sum(rows), 2 * gqa)
    seq = [b for b, r in enumerate(rows) for _ in range(r)]
    pos = [lens[b] - r + i for b, r in enumerate(rows) for i in range(r)]
    check(c, c.extend(q, rows, pps=pps), q, seq, pos, 0, 0)
    check(c, c.extend(q, rows, 8, 500, pps=pps), q, seq, pos, 8, 500)
    assert ok.oscar_device_errors(reset=True) == 0


@pytest.mark.parametrize("fmt", [R.E4M3, R.INT8])
@pytest.mark.parametrize("at", [[300], [20, 21], [599, 130, 131]])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_infinite_keys_take_or_lose_all_the_weight(fmt, at, sign):
    # saturated, their logits are around 1e37: finite, and far beyond where a float tells neighbours apart
    H, D, L = 2, 128, 600
    c = Cache(H, D, fmt, [L], seed=fmt + len(at) + 50)
    k, v = (torch.randn(L, H, D, device="cuda", generator=c.g).bfloat16() for _ in range(2))
    for i, t in enumerate(at):
        k[t, :, 5 + i % 2] = sign * float("inf")
    start = torch.tensor([0, L], dtype=torch.int32, device="cuda")
    ok.oscar_kv8_append(c.dims(2 * H), fmt, 1, L, k, v, start, c.table_d, c.lens_d, c.codes, c.scales)
    for rows in (600, 50, 1):
        q = c.q(rows, 2 * H, 0.5)
        q[:, :, 5] = q[:, :, 5].abs().clamp(max=1.0) + 0.25
        q[:, :, 6] = 2 * q[:, :, 5]  # no two such keys have the same logit
        pos = list(range(L - rows, L))
        for pps, window in ((0, 0), (8, 0), (0, 100), (8, 100)):
            check(c, c.extend(q, [rows], 0, window, pps=pps), q, [0] * rows, pos, 0, window)
            if rows == 1:
                check(c, c.decode(q, 0, window, pps=pps // 2), q, [0], pos, 0, window, decode=True)


@pytest.mark.parametrize("fmt", [R.E4M3, R.INT8])
def test_large_queries_that_an_infinite_key_does_not_touch(fmt):
    # its page's K scale times the query's size is beyond fp32; the logits of that page are 0
    H, D, L = 1, 64, 300
    c = Cache(H, D, fmt, [L], seed=fmt + 60)
    k, v = (torch.randn(L, H, D, device="cuda", generator=c.g).bfloat16() for _ in range(2))
    k[[100, 250], :, 5] = float("inf")
    start = torch.tensor([0, L], dtype=torch.int32, device="cuda")
    ok.oscar_kv8_append(c.dims(4), fmt, 1, L, k, v, start, c.table_d, c.lens_d, c.codes, c.scales)
    for rows in (300, 60, 10, 1):
        q = c.q(rows, 4, 2.0 ** 14)
        q[:, :, 5] = 0.0
        pos = list(range(L - rows, L))
        check(c, c.extend(q, [rows]), q, [0] * rows, pos, 0, 0)
        check(c, c.extend(q, [rows], 3, 70, pps=8), q, [0] * rows, pos, 3, 70)
    check(c, c.decode(q), q, [0], pos, 0, 0, decode=True)
    check(c, c.decode(q, 3, 70, pps=2), q, [0], pos, 3, 70, decode=True)
