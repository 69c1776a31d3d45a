"""oscar_kv8_decode and oscar_kv8_extend_varlen against dense 64-bit attention over the same codes."""

import numpy as np
import pytest
import torch

import int2_rotated_kv_append_gb300 as ok
import kv8_ref as R

pytestmark = pytest.mark.gpu


class Cache:
    """Random codes of plausible keys and values; every page that no sequence holds, and every row behind a
    sequence's last token, holds codes that would ruin a result that reads them (e4m3 NaN, int8 -128)."""

    def __init__(self, H, D, fmt, lens, seed, shared=False):
        g = torch.Generator("cuda").manual_seed(seed)
        self.H, self.D, self.fmt, self.lens = H, D, fmt, lens
        per = [-(-n // 16) for n in lens]
        n = sum(per) + 4
        order = torch.randperm(n, generator=torch.Generator().manual_seed(seed))
        self.table = torch.full((len(lens), max([1] + per)), -1, dtype=torch.int32)
        at = 0
        for b, c in enumerate(per):
            self.table[b, :c] = order[at:at + c]
            at += c
        x = torch.randn(n, H, 2, 16, D, device="cuda", generator=g)
        x[:, :, 0] += 2 * torch.randn(H, 1, D, device="cuda", generator=g)
        x[:, :, 0, :, :4] *= 8
        x *= 2.0 ** torch.randint(-2, 3, (n, H, 2, 1, 1), device="cuda", generator=g)
        e = torch.ceil(torch.log2(x.abs().amax((3, 4)) / R.FMAX[fmt])).int()
        s = ((e + 127) << 23).view(torch.float32)  # a power of two to the bit
        x = x / s[..., None, None]
        self.codes = (x.to(torch.float8_e4m3fn) if fmt == R.E4M3 else x.round().to(torch.int8)).view(torch.uint8)
        bad = 0x7f if fmt == R.E4M3 else 0x80
        self.codes[order[at:].cuda()] = bad
        for b, L in enumerate(lens):
            if L % 16:
                self.codes[self.table[b, L // 16].item(), :, :, L % 16:] = bad
        self.scales = s
        self.dims = lambda hq: ok.make_dims(hq, H, D, 16, D, n, self.table.shape[1])
        self.table_d = self.table.cuda()
        self.lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.g = g

    def q(self, rows, hq, factor=1.0):
        return (torch.randn(rows, hq, self.D, device="cuda", generator=self.g) * factor).bfloat16()

    def decode(self, q, sink=0, window=0, pps=0, sm_scale=0.0, max_len=None, table=None, lens=None):
        d = self.dims(q.shape[1])
        m = max(self.lens) if max_len is None else max_len
        ws = torch.full((ok.oscar_kv8_decode_workspace_bytes(d, len(self.lens), m, pps, sink, window),), 0xff,
                        dtype=torch.uint8, device="cuda")
        out = torch.full_like(q, float("nan"))
        ok.oscar_kv8_decode(d, self.fmt, len(self.lens), m, pps, q, self.codes, self.scales,
                            self.table_d if table is None else table, self.lens_d if lens is None else lens, sink, window,
                            sm_scale, out, ws)
        return out

    def extend(self, q, rows, sink=0, window=0, pps=0, sm_scale=0.0, max_rows=None):
        d = self.dims(q.shape[1])
        start = torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device="cuda")
        m = max(rows) if max_rows is None else max_rows
        ws = torch.full((ok.oscar_kv8_extend_varlen_workspace_bytes(d, len(rows), q.shape[0], max(self.lens), m, pps, sink,
                                                                    window),), 0xff, dtype=torch.uint8, device="cuda")
        out = torch.full_like(q, float("nan"))
        ok.oscar_kv8_extend_varlen(d, self.fmt, len(rows), max(self.lens), m, pps, q, start, self.codes, self.scales,
                                   self.table_d, self.lens_d, sink, window, sm_scale, out, ws)
        return out

    def check(self, out, q, row_seq, row_pos, sink=0, window=0, sm_scale=None, table=None):
        ref, tol = R.attention(self.codes, self.scales, q, row_seq, row_pos, (self.table if table is None else table).tolist(),
                               self.fmt, sink, window, sm_scale)
        err = (out.double() - ref).abs()
        assert torch.isfinite(out).all()
        worst = (err / tol.clamp(min=1e-300)).max().item() if err.numel() else 0.0
        assert (err <= tol).all(), f"{worst:.3g} times the tolerance, at {(err > tol).nonzero()[:4].tolist()}"
        return worst

    def check_decode(self, out, q, **kw):
        return self.check(out, q, list(range(len(self.lens))), [n - 1 for n in self.lens], **kw)


EDGE = [0, 1, 2, 15, 16, 17, 31, 33, 127, 128, 129, 700, 1500]


@pytest.mark.parametrize("fmt", [R.E4M3, R.INT8])
@pytest.mark.parametrize("D,H,gqa", [(64, 2, 3), (64, 1, 8), (128, 2, 1), (128, 3, 4), (128, 1, 7), (128, 1, 8)])
@pytest.mark.parametrize("sink,window", [(0, 0), (0, 1), (4, 100), (17, 64), (300, 33), (0, 16), (5, 5000)])
def test_decode(D, H, gqa, fmt, sink, window):
    c = Cache(H, D, fmt, EDGE, seed=D + H + gqa + fmt + window)
    q = c.q(len(EDGE), H * gqa)
    c.check_decode(c.decode(q, sink, window), q, sink=sink, window=window)
    assert ok.oscar_device_errors(reset=True) == 0


@pytest.mark.parametrize("pps", [1, 3, 7, 40, 200, 100000])
def test_decode_split_sizes(pps):
    c = Cache(2, 128, R.E4M3, [5000, 0, 1, 2777], seed=pps)
    q = c.q(4, 8)
    c.check_decode(c.decode(q, pps=pps), q)
    c.check_decode(c.decode(q, 20, 1000, pps=pps), q, sink=20, window=1000)


@pytest.mark.parametrize("fmt", [R.E4M3, R.INT8])
def test_decode_long_and_large_batch(fmt):
    c = Cache(2, 128, fmt, [70001], seed=1)
    q = c.q(1, 16)
    c.check_decode(c.decode(q), q)
    c.check_decode(c.decode(q, 64, 4096), q, sink=64, window=4096)
    c = Cache(1, 64, fmt, [int(n) for n in np.random.default_rng(2).integers(0, 300, 300)], seed=3)
    q = c.q(300, 5)
    c.check_decode(c.decode(q), q)


def test_decode_scales_and_large_queries():
    c = Cache(2, 128, R.INT8, [900, 37], seed=4)
    for sm_scale, factor in ((0.5, 1.0), (1e-3, 300.0), (1e-6, 1e6), (1e-30, 1e30), (1.0, 1e-30)):
        q = c.q(2, 8, factor)
        c.check_decode(c.decode(q, sm_scale=sm_scale), q, sm_scale=sm_scale)


def test_decode_flags_lengths_and_pages():
    c = Cache(2, 128, R.E4M3, [300, 100, 200], seed=5)
    q = c.q(3, 8)
    lens = torch.tensor([300, -4, 1000], dtype=torch.int32, device="cuda")
    out = c.decode(q, lens=lens, max_len=200)
    assert ok.oscar_device_errors(reset=True) == ok.OSCAR_DEVERR_SEQ_LEN
    assert (out[1] == 0).all()
    ref, tol = R.attention(c.codes, c.scales, q, [0, 1, 2], [199, -1, 199], c.table.tolist(), c.fmt, 0, 0)
    assert ((out.double() - ref).abs() <= tol).all()
    table = c.table.clone()
    table[0, 3], table[2, 0], table[1, 6] = -1, 10 ** 6, c.dims(8).num_pages
    out = c.decode(q, table=table.cuda())
    assert ok.oscar_device_errors(reset=True) == ok.OSCAR_DEVERR_PAGE_ID
    c.check_decode(out, q, table=table)
    table[0, :] = -1  # a sequence of bad pages only
    assert (c.decode(q, table=table.cuda())[0] == 0).all()
    ok.oscar_device_errors(reset=True)


def test_decode_window_never_looks_up_pages_outside():
    c = Cache(2, 128, R.E4M3, [1000, 333], seed=6)
    q = c.q(2, 8)
    table = c.table.clone()
    table[0, 2:(1000 - 100) // 16] = -1
    table[1, 2:(333 - 100) // 16] = 10 ** 6
    c.check_decode(c.decode(q, 32, 100, table=table.cuda()), q, sink=32, window=100)
    assert ok.oscar_device_errors(reset=True) == 0


ROWS = [0, 1, 2, 15, 16, 17, 31, 33, 100, 128, 129, 0, 300]


@pytest.mark.parametrize("fmt", [R.E4M3, R.INT8])
@pytest.mark.parametrize("D,H,gqa", [(64, 2, 3), (64, 1, 8), (128, 2, 1), (128, 3, 4), (128, 1, 7), (128, 1, 8)])
@pytest.mark.parametrize("sink,window", [(0, 0), (0, 1), (4, 100), (17, 64), (300, 33), (0, 16), (5, 5000)])
def test_extend(D, H, gqa, fmt, sink, window):
    c = Cache(H, D, fmt, EDGE, seed=D + H + gqa + fmt + window + 1)
    rows = [min(r, n) for r, n in zip(ROWS, EDGE)]
    seq = [b for b, r in enumerate(rows) for _ in range(r)]
    pos = [EDGE[b] - r + i for b, r in enumerate(rows) for i in range(r)]
    q = c.q(len(seq), H * gqa)
    c.check(c.extend(q, rows, sink, window), q, seq, pos, sink=sink, window=window)
    assert ok.oscar_device_errors(reset=True) == 0


@pytest.mark.parametrize("fmt", [R.E4M3, R.INT8])
@pytest.mark.parametrize("sink,window", [(0, 0), (64, 700)])
@pytest.mark.parametrize("D,gqa", [(128, 4), (64, 5)])
def test_extend_whole_prompts(fmt, sink, window, D, gqa):
    lens = [2500, 1031]
    c = Cache(1, D, fmt, lens, seed=window + gqa)
    seq = [b for b, n in enumerate(lens) for _ in range(n)]
    pos = [i for n in lens for i in range(n)]
    q = c.q(len(seq), gqa)
    c.check(c.extend(q, lens, sink, window), q, seq, pos, sink=sink, window=window)


@pytest.mark.parametrize("rows", [[1, 8, 3, 0], [40, 2, 0, 7]])
@pytest.mark.parametrize("pps", [0, 1, 8, 16, 50])
def test_extend_few_rows_over_long_caches(rows, pps):
    lens = [9000, 333, 5000, 12000]
    c = Cache(2, 128, R.INT8, lens, seed=sum(rows))
    seq = [b for b, r in enumerate(rows) for _ in range(r)]
    pos = [lens[b] - r + i for b, r in enumerate(rows) for i in range(r)]
    q = c.q(len(seq), 16)
    c.check(c.extend(q, rows, pps=pps), q, seq, pos)
    c.check(c.extend(q, rows, 10, 2000, pps=pps), q, seq, pos, sink=10, window=2000)


def test_extend_rising_maxima():
    # keys grow along the sequence, so that running maxima move far again and again
    c = Cache(1, 128, R.INT8, [1200], seed=11)
    for j in range(75):
        c.scales[c.table[0, j].item(), :, 0] *= 2.0 ** (j // 12)
    q = c.q(200, 4)
    c.check(c.extend(q, [200]), q, [0] * 200, list(range(1000, 1200)))
    q = c.q(1, 4)
    c.check_decode(c.decode(q), q)


def test_extend_scales_and_large_queries():
    c = Cache(2, 128, R.E4M3, [900, 137], seed=12)
    seq, pos = [0] * 130 + [1] * 37, list(range(770, 900)) + list(range(100, 137))
    for sm_scale, factor in ((0.5, 1.0), (1e-3, 300.0), (1e-6, 1e6), (1.0, 1e-30)):
        q = c.q(167, 8, factor)
        c.check(c.extend(q, [130, 37], sm_scale=sm_scale), q, seq, pos, sm_scale=sm_scale)


def test_extend_of_one_row_is_a_decode():
    c = Cache(2, 128, R.E4M3, [1000, 17, 1], seed=13)
    q = c.q(3, 8)
    c.check_decode(c.extend(q, [1, 1, 1], 4, 300), q, sink=4, window=300)


def test_extend_flags_bad_rows():
    c = Cache(2, 128, R.E4M3, [20, 300], seed=14)
    q = c.q(33, 8)
    out = c.extend(q, [25, 8])  # five rows before the first token
    assert ok.oscar_device_errors(reset=True) == ok.OSCAR_DEVERR_POSITION
    assert (out[:5] == 0).all()
    c.check(out, q, [0] * 25 + [1] * 8, [-1] * 5 + list(range(20)) + list(range(292, 300)))
    out = c.extend(q, [25, 8], max_rows=10)  # the first sequence has more rows than the call says
    assert ok.oscar_device_errors(reset=True) == ok.OSCAR_DEVERR_POSITION
    c.check(out[25:], q[25:], [1] * 8, list(range(292, 300)))


@pytest.mark.parametrize("kind", ["decode", "extend"])
def test_unaligned_tables_and_other_streams(kind):
    c = Cache(2, 128, R.E4M3, [700, 90], seed=15)
    wide = torch.full((2, c.table.shape[1] + 3), 7, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = c.table_d
    c.table_d = wide[:, :].contiguous()
    n = c.dims(8).num_pages
    c.dims = lambda hq: ok.make_dims(hq, 2, 128, 16, 128, n, wide.shape[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        q = c.q(2 if kind == "decode" else 60, 8)
        out = c.decode(q) if kind == "decode" else c.extend(q, [40, 20])
    s.synchronize()
    if kind == "decode":
        c.check_decode(out, q)
    else:
        c.check(out, q, [0] * 40 + [1] * 20, list(range(660, 700)) + list(range(70, 90)))


def test_captured_and_replayed_with_growing_lengths():
    c = Cache(2, 128, R.INT8, [3000, 40], seed=16)
    q = c.q(2, 8)
    c.decode(q)  # everything is loaded before the capture
    torch.cuda.synchronize()
    d, sizes = c.dims(8), (2, 3000, 0, 8, 500)
    ws = torch.empty(ok.oscar_kv8_decode_workspace_bytes(d, *sizes), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):  # two calls share the workspace
            ok.oscar_kv8_decode(d, c.fmt, 2, 3000, 0, q, c.codes, c.scales, c.table_d, c.lens_d, 8, 500, 0.0, out, ws)
    for lens in ([3000, 40], [17, 33], [2999, 0]):
        c.lens_d.copy_(torch.tensor(lens))
        graph.replay()
        c.check(out, q, [0, 1], [n - 1 for n in lens], sink=8, window=500)


@pytest.mark.parametrize("D,rows", [(128, [1, 8, 3, 0]), (64, [1, 8, 3, 0]), (128, [300, 200, 100, 77])])
def test_extend_is_the_same_on_cold_caches(D, rows):
    # the first pass after other data went through L2 meets every copy late: results have to be the same bits
    import time
    lens = [9000, 333, 5000, 12000]
    c = Cache(2, D, R.INT8, lens, seed=17)
    q = c.q(sum(rows), 16)
    big = torch.empty(300 << 20, dtype=torch.uint8, device="cuda")
    for pps in (8, 16, 64):
        want = c.extend(q, rows, pps=pps)
        for i in range(25):
            big.fill_(i)
            torch.cuda.synchronize()
            time.sleep(0.001)
            assert torch.equal(c.extend(q, rows, pps=pps), want), (pps, i)


def test_pages_far_into_a_large_pool():
    # byte offsets beyond 32 bits: 150000 pages of 32 KB, the cache in the last ones
    n, H, D, L = 150000, 8, 128, 300
    small = Cache(H, D, R.E4M3, [L], seed=18)
    ids = torch.tensor([n - 1 - 3 * i for i in range(19)], dtype=torch.int32)
    codes = torch.empty(n, H, 2, 16, D, dtype=torch.uint8, device="cuda")
    scales = torch.empty(n, H, 2, device="cuda")
    codes[ids.cuda().long()] = small.codes[small.table_d[0].long()]
    scales[ids.cuda().long()] = small.scales[small.table_d[0].long()]
    big = Cache(H, D, R.E4M3, [L], seed=18)
    big.codes, big.scales, big.table_d = codes, scales, ids.cuda()[None].contiguous()
    big.dims = lambda hq: ok.make_dims(hq, H, D, 16, D, n, 19)
    q, qx = small.q(1, 32), small.q(150, 32)
    assert torch.equal(big.decode(q), small.decode(q))
    assert torch.equal(big.extend(qx, [150]), small.extend(qx, [150]))
    assert torch.equal(big.extend(qx[:20], [20]), small.extend(qx[:20], [20]))
    k, v = (torch.randn(1, H, D, device="cuda").bfloat16() for _ in range(2))
    lens = torch.tensor([L + 1], dtype=torch.int32, device="cuda")
    for c in (big, small):
        ok.oscar_kv8_append(c.dims(32), R.E4M3, 1, 1, k, v, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), c.table_d, lens,
                            c.codes, c.scales)
    assert torch.equal(codes[ids[-1].item()], small.codes[small.table[0, -1].item()])


@pytest.mark.parametrize("D,fmt", [(64, R.E4M3), (64, R.INT8), (128, R.E4M3), (128, R.INT8)])
@pytest.mark.parametrize("gqa,most", [(1, 64), (1, 65), (7, 9), (7, 10), (8, 8), (8, 9), (3, 21), (3, 22)])
@pytest.mark.parametrize("sink,window", [(0, 0), (5, 40), (70, 1), (0, 500)])
def test_extend_around_64_rows_of_a_tile(D, fmt, gqa, most, sink, window):
    lens = [1, 64, 65, 129, 128, 700, 1500, 0, 63]
    rows = [min(n, r) for n, r in zip(lens, (1, most, most, most, 1, most, 2, 0, most))]
    c = Cache(2, D, fmt, lens, seed=D + fmt + gqa + most + window)
    seq = [b for b, r in enumerate(rows) for _ in range(r)]
    pos = [lens[b] - r + i for b, r in enumerate(rows) for i in range(r)]
    q = c.q(len(seq), 2 * gqa)
    for pps in (0, 8):
        c.check(c.extend(q, rows, sink, window, pps=pps), q, seq, pos, sink=sink, window=window)
    assert ok.oscar_device_errors(reset=True) == 0


@pytest.mark.parametrize("batch,length", [(8, 8192), (32, 4096), (3, 16384), (1, 16), (1, 17), (70, 300)])
def test_decode_split_rule(batch, length):
    lens = [length - 5 * b for b in range(batch)]
    lens = [max(n, 1) for n in lens]
    c = Cache(2, 64, R.INT8, lens, seed=batch)
    q = c.q(batch, 4)
    c.check_decode(c.decode(q), q)
    c.check_decode(c.decode(q, 16, 900), q, sink=16, window=900)


def test_nan_queries_stay_in_their_rows():
    c = Cache(2, 128, R.E4M3, [700, 90], seed=19)
    q = c.q(2, 8)
    want = c.decode(q)
    bad = q.clone()
    bad[0, 3, 5] = float("nan")
    out = c.decode(bad)
    assert out[0, 3].isnan().all()
    out[0, 3] = want[0, 3]
    assert torch.equal(out, want)
    for rows, pps in (([40, 2], 0), ([300, 90], 0), ([3, 1], 8)):
        q = c.q(sum(rows), 8)
        want = c.extend(q, rows, pps=pps)
        bad = q.clone()
        bad[1, 6, 100] = float("nan")
        out = c.extend(bad, rows, pps=pps)
        assert out[1, 6].isnan().all()
        out[1, 6] = want[1, 6]
        assert torch.equal(out, want)


@pytest.mark.parametrize("window", [700, 10 ** 6, 2 ** 31 - 1])
def test_a_window_over_the_whole_cache_is_no_window(window):
    c = Cache(2, 64, R.INT8, [700, 90], seed=20)
    q, qx = c.q(2, 8), c.q(200, 8)
    assert torch.equal(c.decode(q, 2 ** 31 - 1, window), c.decode(q))
    assert torch.equal(c.extend(qx, [150, 50], 3, window), c.extend(qx, [150, 50]))


def test_calls_on_two_streams_at_once():
    c = Cache(2, 128, R.INT8, [3000, 1500], seed=21)
    q, qx = c.q(2, 8), c.q(300, 8)
    want, wantx = c.decode(q), c.extend(qx, [200, 100])
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(20):
        with torch.cuda.stream(a):
            got.append((c.decode(q), want))
        with torch.cuda.stream(b):
            got.append((c.extend(qx, [200, 100]), wantx))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in got)


def test_a_reserved_token_without_an_append_is_zero():
    # zeroed pools: code 0 and scale 0
    c = Cache(1, 128, R.E4M3, [40], seed=22)
    c.codes.zero_()
    c.scales.zero_()
    assert (c.decode(c.q(1, 4)) == 0).all() and (c.extend(c.q(40, 4), [40]) == 0).all()
    assert (c.extend(c.q(3, 4), [3]) == 0).all()
