"""oscar_rope and oscar_kv8_rope_append against rotations in 64 bits."""

import numpy as np
import pytest
import torch

import int2_rotated_kv_append_gb300 as ok
import kv8_ref as R
import rope_ref as RR

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]
YARN = dict(kind="yarn", factor=4.0, original_max_position=2048)


def dims(hq, hkv, d, pages=1, most=1):
    return ok.make_dims(hq, hkv, d, 16, 64, pages, most)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def far_positions(T, rng):
    p = rng.integers(-2 ** 31, 2 ** 31, T)
    p[:min(T, 6)] = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 131072][:min(T, 6)]
    return p


def check(got, x, positions, rope):
    """`got` against x (a tensor of the same type): the arithmetic's error and half a step of the type."""
    want, err = RR.rotate(x.double().cpu().numpy(), positions, rope)
    fi = torch.finfo(got.dtype)
    tol = err + (fi.eps / 2) * (np.abs(want) + err) + fi.tiny * fi.eps
    assert (np.abs(got.double().cpu().numpy() - want) <= tol).all()
    n = rope.rotary_dim
    assert torch.equal(got[..., n:], x[..., n:])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,hkv,d,rotary", [(1, 1, 1, 64, 64), (3, 6, 2, 64, 16), (5, 8, 1, 128, 128), (40, 7, 7, 128, 96),
                                               (1300, 5, 5, 64, 48), (1223, 24, 3, 128, 112)])
def test_rope(T, hq, hkv, d, rotary, interleaved, dtype):
    rng = np.random.default_rng(T + rotary)
    g = torch.Generator("cuda").manual_seed(T)
    rope = ok.Rope(rotary, interleaved=interleaved, scaling=YARN if T % 2 else None)
    pos = far_positions(T, rng)
    q, k = (torch.randn(T, h, d, device="cuda", generator=g).to(dtype) for h in (hq, hkv))
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    ok.oscar_rope(dims(hq, hkv, d), rope, i32(pos), q, k, qo, ko)
    check(qo, q, pos, rope)
    check(ko, k, pos, rope)


@pytest.mark.parametrize("T", [7, 2000])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope_of_slices_in_place_and_of_one_side(T, interleaved, dtype):
    rope = ok.Rope(32, interleaved=interleaved)
    pos = np.arange(T) * 37
    g = torch.Generator("cuda").manual_seed(3)
    whole = torch.randn(T, 6 + 2 + 2, 64, device="cuda", generator=g).to(dtype)
    before = whole.clone()
    q, k, v = torch.split(whole, [6, 2, 2], 1)
    q0, k0, v0 = torch.split(before, [6, 2, 2], 1)
    wide = torch.full((T, 9, 64), 5.0, device="cuda", dtype=dtype)
    ok.oscar_rope(dims(6, 2, 64), rope, i32(pos), q, k, wide[:, :6], k)  # keys in place
    check(wide[:, :6], q0, pos, rope)
    check(k, k0, pos, rope)
    assert torch.equal(q, q0) and torch.equal(v, v0) and (wide[:, 6:] == 5).all()
    ok.oscar_rope(dims(6, 2, 64), rope, i32(pos), q, None, q, None)
    check(q, q0, pos, rope)
    whole.copy_(before)
    ok.oscar_rope(dims(6, 2, 64), rope, i32(pos), None, k, None, k)
    check(k, k0, pos, rope)
    assert torch.equal(q, q0) and torch.equal(v, v0)


def test_rope_back_and_forth_moves_keys():
    # the rotation by p - n of a key rotated by n is that by p, and a NaN stays in its pair
    rope = ok.Rope(64)
    T = 50
    x = torch.randn(T, 2, 64, device="cuda")
    p, n = np.arange(T) * 1000003, np.arange(T)[::-1] * 70001
    y, z, w = (torch.empty_like(x) for _ in range(3))
    d = dims(2, 2, 64)
    ok.oscar_rope(d, rope, i32(n), None, x, None, y)
    ok.oscar_rope(d, rope, i32(p - n), None, y, None, z)
    ok.oscar_rope(d, rope, i32(p), None, x, None, w)
    # each of the three is off by 2^-21 (|a| + |b|) at most, and |a| + |b| <= sqrt(2) times the pair's length
    length = (x[..., :32] ** 2 + x[..., 32:] ** 2).sqrt().repeat(1, 1, 2)
    assert ((z - w).abs() <= 3 * 2 ** 0.5 * 2.0 ** -21 * 1.01 * length).all()
    x[3, 1, 5] = float("nan")
    ok.oscar_rope(d, rope, i32(p), None, x, None, y)
    bad = torch.zeros_like(x, dtype=torch.bool)
    bad[3, 1, 5] = bad[3, 1, 37] = True
    assert torch.equal(y.isnan(), bad)


def test_rope_empty_and_rows_beyond_2_31_elements():
    rope = ok.Rope(128)
    d = dims(1, 1, 128)
    e = torch.empty(0, 1, 128, device="cuda", dtype=torch.bfloat16)
    ok.oscar_rope(d, rope, i32([]), e, e, e, e)
    # rows so far apart that the last one lies beyond 2^31 elements
    T, stride = 70, 32 * 1024 * 1024
    flat = torch.empty(stride * (T - 1) + 128, device="cuda", dtype=torch.bfloat16)
    rows = flat.as_strided((T, 1, 128), (stride, 128, 1))
    x = torch.randn(T, 1, 128, device="cuda").bfloat16()
    rows.copy_(x)
    pos = np.arange(T) * 30000001
    ok.oscar_rope(d, rope, i32(pos), rows, None, rows, None)
    check(rows.clone(), x, pos, rope)


# ---- the append -------------------------------------------------------------------------------------------------------


class Case:
    """Sequences of at most `capacity` tokens each, pages in a random order, pools filled with a pattern."""

    def __init__(self, hq, H, D, fmt, capacity, rope, seed):
        self.hq, self.H, self.D, self.fmt, self.rope, self.rng = hq, H, D, fmt, rope, np.random.default_rng(seed)
        per = [max(1, -(-c // 16)) for c in capacity]
        n = sum(per) + 3
        order = self.rng.permutation(n)
        self.table = np.full((len(per), max(per)), -1, np.int32)
        at = 0
        for b, c in enumerate(per):
            self.table[b, :c] = order[at:at + c]
            at += c
        self.dims = dims(hq, H, D, n, max(per))
        self.codes = torch.full((n, H, 2, 16, D), 0x2b, dtype=torch.uint8, device="cuda")
        self.scales = torch.full((n, H, 2), 2.0 ** 30, device="cuda")  # stale: a page's first token replaces it
        self.lens = [0] * len(per)

    def rows(self, T, spread=1.0):
        x = self.rng.normal(size=(T, self.hq + 2 * self.H, self.D)) * spread
        x *= 2.0 ** self.rng.integers(-3, 4, size=(T, 1, 1))
        x[:, :, :3] *= 20
        return torch.from_numpy(x).to(torch.bfloat16).cuda()

    def append(self, new, x=None, positions=None, granted=None, with_q=True, lens=None):
        """One call and its check: queries, values' codes equal, keys' scales and codes as near as the arithmetic allows."""
        if lens is None:
            self.lens = [a + n for a, n in zip(self.lens, new)]
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        T = int(start[-1])
        x = self.rows(T) if x is None else x
        q, k, v = torch.split(x, [self.hq, self.H, self.H], 1)
        old_c, old_s = self.codes.cpu().numpy(), self.scales.cpu().numpy()
        out = torch.full((T, self.hq, self.D), 7.0, device="cuda", dtype=torch.bfloat16)
        table = torch.from_numpy(self.table).cuda()
        ok.oscar_kv8_rope_append(self.dims, self.rope, self.fmt, len(new), max(new), q if with_q else None, k, v, i32(start),
                                 None if positions is None else i32(positions), table, i32(self.lens if lens is None else lens),
                                 self.codes, self.scales, out if with_q else None, granted=None if granted is None else i32(granted))
        where = np.concatenate([np.arange(L - n, L) for L, n in zip(self.lens, new)]) if positions is None else positions
        live = [n if granted is None or granted[b] else 0 for b, n in enumerate(new)]
        rows = [t for b, n in enumerate(live) for t in range(start[b], start[b] + n)]
        if with_q:
            check(out[rows], q[rows], where[rows], self.rope)
            none = [t for t in range(T) if t not in set(rows)]
            assert (out[none] == 0).all()
        else:
            assert (out == 7).all()
        got_c, got_s = self.codes.cpu().numpy(), self.scales.cpu().numpy()
        want_c, want_s = old_c.copy(), old_s.copy()
        kr, err = RR.rotate(k.double().cpu().numpy(), where, self.rope)
        if granted is None:  # values: every bit
            R.append(want_c, want_s, np.zeros_like(kr), v.double().cpu().numpy(), start, self.table, self.lens, self.fmt)
            zero = lambda c: np.where(c == 0x80, 0, c) if self.fmt == R.E4M3 else c  # noqa: E731
            assert np.array_equal(got_s[:, :, 1], want_s[:, :, 1])
            assert np.array_equal(zero(got_c[:, :, 1]), zero(want_c[:, :, 1]))
        touched = np.zeros(old_c.shape[0], bool)
        for b, n in enumerate(live):
            L = self.lens[b]
            for j in range((L - n) // 16, -(-L // 16)) if n else ():
                page = self.table[b, j]
                touched[page] = True
                o0, o1 = max(L - n - j * 16, 0), min(L - j * 16, 16)
                t0 = start[b] + j * 16 + o0 - (L - n)
                for h in range(self.H):
                    y, e = kr[t0:t0 + o1 - o0, h], err[t0:t0 + o1 - o0, h]
                    s, was = float(got_s[page, h, 0]), float(old_s[page, h, 0])
                    allowed = {R.scale_of((np.abs(y) - e).max(), self.fmt), R.scale_of((np.abs(y) + e).max(), self.fmt)}
                    assert s in ({max(a, was) for a in allowed} if o0 else allowed)
                    c = got_c[page, h, 0]
                    val = R.code_values(c, self.fmt) * s
                    # half a step: of a value, and of the smallest values' fixed step; int8 steps are all alike
                    half = 0.5 * s if self.fmt == R.INT8 else 2.0 ** -4 * (np.abs(y) + e) + 2.0 ** -10 * s
                    over = R.FMAX[self.fmt] * s
                    assert (np.abs(val[o0:o1] - np.clip(y, -over, over)) <= half + e).all()
                    # earlier rows: as they were, or under the larger scale; rows behind: as they were
                    kept = old_c[page, h, 0, :o0]
                    if s != was and o0:
                        kept = R.encode(R.code_values(kept, self.fmt) * (was / s), self.fmt)
                    assert np.array_equal(R.code_values(c[:o0], self.fmt), R.code_values(kept, self.fmt))
                    assert np.array_equal(c[o1:], old_c[page, h, 0, o1:])
        assert np.array_equal(got_c[~touched], old_c[~touched]) and np.array_equal(got_s[~touched], old_s[~touched])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("fmt", [R.E4M3, R.INT8])
@pytest.mark.parametrize("hq,H,D,rotary", [(1, 1, 64, 64), (6, 3, 128, 96), (8, 8, 128, 128), (16, 2, 64, 16)])
def test_append_in_pieces(hq, H, D, rotary, fmt, interleaved):
    c = Case(hq, H, D, fmt, [100, 1, 64, 33, 40], ok.Rope(rotary, interleaved=interleaved, scaling=YARN), seed=H * D + fmt)
    for new in ([17, 0, 16, 1, 5], [1, 1, 1, 1, 0], [40, 0, 15, 30, 1], [1, 0, 1, 1, 1], [0, 0, 0, 0, 1]):
        c.append(new)
    assert ok.oscar_device_errors(reset=True) == 0


def test_append_of_many_pages_with_positions_of_its_own():
    c = Case(8, 2, 128, R.E4M3, [900, 333, 1], ok.Rope(128), seed=1)
    c.append([880, 300, 0], positions=far_positions(1180, np.random.default_rng(2)))
    c.append([20, 33, 1], positions=np.arange(54) * -40000001, with_q=False)
    assert ok.oscar_device_errors(reset=True) == 0


@pytest.mark.parametrize("fmt", [R.E4M3, R.INT8])
def test_append_single_tokens_with_growing_and_falling_scales(fmt):
    c = Case(2, 2, 64, fmt, [40, 40], ok.Rope(64), seed=5)
    for e in [0, 3, -4, 9, 9, -20, 11, 30, -30, 31] + list(range(-8, 12)):
        c.append([1, 1], c.rows(2, 2.0 ** e))


def test_append_skips_what_reserve_refused_and_zeroes_its_queries():
    c = Case(4, 2, 128, R.INT8, [64, 64, 64], ok.Rope(32, interleaved=True), seed=6)
    c.append([20, 10, 3])
    c.lens = [21, 10, 6]  # the second has not grown
    c.append([1, 40, 3], granted=[1, 0, 1], lens=c.lens)
    assert ok.oscar_device_errors(reset=True) == 0


def test_append_extremes():
    # infinities saturate or, in a pair, become NaN as their formula does; NaN is stored as 0 and flagged; zeros
    for fmt in (R.E4M3, R.INT8):
        rope = ok.Rope(32)
        d = dims(1, 1, 64, 4, 1)
        T = 4
        k = torch.zeros(T, 1, 64, device="cuda", dtype=torch.bfloat16)
        k[1, 0, 40] = float("inf")      # behind the rotated channels
        k[1, 0, 41] = -1.0
        k[2, 0, 3] = float("nan")       # with channel 19
        k[2, 0, 50] = 2.0
        k[3, 0, 0] = torch.finfo(torch.bfloat16).max
        k[3, 0, 16] = torch.finfo(torch.bfloat16).max  # the sum of two such is infinite
        codes = torch.zeros(4, 1, 2, 16, 64, device="cuda", dtype=torch.uint8)
        scales = torch.zeros(4, 1, 2, device="cuda")
        ok.oscar_kv8_rope_append(d, rope, fmt, T, 1, None, k, torch.zeros_like(k), i32(range(T + 1)), i32([0, 0, 7, 1]),
                                 i32([[0], [1], [2], [3]]), i32([1] * T), codes, scales, None)
        assert ok.oscar_device_errors(reset=True) == ok.OSCAR_DEVERR_VALUE
        val = codes.view(torch.float8_e4m3fn if fmt == R.E4M3 else torch.int8).double() * scales.double()[..., None, None]
        assert torch.isfinite(val).all() and (val[0] == 0).all() and scales[0, 0, 0] == 2.0 ** -100
        top = [float(R.FMAX[fmt] * 2.0 ** R.EXP_HI[fmt])] * 2
        assert val[1, 0, 0, 0, 40] == top[0] and val[1, 0, 0, 0, 41] == 0
        # (2 and the NaN pair's zeros)
        assert val[2, 0, 0, 0, 3] == 0 and val[2, 0, 0, 0, 19] == 0 and abs(val[2, 0, 0, 0, 50] - 2) <= 2 * 2.0 ** -4
        # cos 1 - sin 1 < 0 of the largest value, and cos 1 + sin 1 > 1 of it: beyond fp32's or the codes' largest, saturated
        assert val[3, 0, 0, 0, 16] == top[0] and val[3, 0, 0, 0, 0] < 0


def test_append_skips_what_is_out_of_range():
    c = Case(2, 2, 64, R.INT8, [32, 32, 32, 32], ok.Rope(64), seed=8)
    before = c.codes.clone()
    x = c.rows(12)
    q, k, v = torch.split(x, 2, 1)
    out = torch.full((12, 2, 64), 7.0, device="cuda", dtype=torch.bfloat16)

    def call(start, lens, table=None, max_new=6):
        ok.oscar_kv8_rope_append(c.dims, c.rope, R.INT8, 4, max_new, q, k, v, i32(start), None,
                                 torch.from_numpy(c.table if table is None else table).cuda(), i32(lens), c.codes, c.scales, out)
        return ok.oscar_device_errors(reset=True)
    P = ok.OSCAR_DEVERR_POSITION
    assert call([0, 3, 6, 9, 12], [2, 2, 2, 2]) == P      # more rows than tokens
    assert call([0, 12, 12, 12, 12], [12, 0, 0, 0]) == P  # above max_tokens_per_seq
    assert call([0, 3, 6, 9, 12], [40] * 4) == P          # beyond the table row
    assert call([0, 0, 0, 0, 13], [0, 0, 0, 13], max_new=13) == P
    assert call([5, 3, 3, 3, 3], [4, 0, 0, 0]) == P       # decreasing
    assert (out == 7).all()
    bad = c.table.copy()
    bad[:, 0] = [-1, 10 ** 6, c.dims.num_pages, -7]
    assert call([0, 3, 6, 9, 12], [3] * 4, bad) == ok.OSCAR_DEVERR_PAGE_ID
    assert torch.equal(c.codes, before)
    check(out, q, np.array([0, 1, 2] * 4), c.rope)


def test_append_on_a_stream_of_its_own_and_captured():
    rope = ok.Rope(128)
    d = dims(4, 2, 128, 6, 3)
    x = torch.randn(3, 8, 128, device="cuda").bfloat16()
    q, k, v = torch.split(x, [4, 2, 2], 1)
    start, lens, table = i32([0, 1, 3]), i32([5, 20]), i32([[3, -1, -1], [0, 4, -1]])
    codes, scales = torch.zeros(6, 2, 2, 16, 128, device="cuda", dtype=torch.uint8), torch.zeros(6, 2, 2, device="cuda")
    out = torch.empty(3, 4, 128, device="cuda", dtype=torch.bfloat16)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ok.oscar_kv8_rope_append(d, rope, R.E4M3, 2, 2, q, k, v, start, None, table, lens, codes, scales, out)
    for _ in range(3):
        lens += 1
        g.replay()
    want = [torch.zeros_like(codes), torch.zeros_like(scales)]
    lens -= 3
    for _ in range(3):
        lens += 1
        q2 = torch.empty_like(out)
        ok.oscar_kv8_rope_append(d, rope, R.E4M3, 2, 2, q, k, v, start, None, table, lens, *want, q2, stream=s)
        torch.cuda.synchronize()
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1]) and torch.equal(out, q2)


def test_append_and_decode_in_pages_beyond_4_gb():
    H, D, n = 8, 128, 140000  # pages of 32 KB
    rope = ok.Rope(128)
    codes, scales = torch.empty(n, H, 2, 16, D, device="cuda", dtype=torch.uint8), torch.empty(n, H, 2, device="cuda")
    far = [n - 1, n - 3, 131072]
    small = [torch.zeros(3, H, 2, 16, D, device="cuda", dtype=torch.uint8), torch.zeros(3, H, 2, device="cuda")]
    x = torch.randn(40, 16 + 2 * H, D, device="cuda").bfloat16()
    q, k, v = torch.split(x, [16, H, H], 1)
    outs = []
    for pool, ids, pages in (((codes, scales), far, n), (small, [0, 1, 2], 3)):
        d = dims(16, H, D, pages, 3)
        qo = torch.empty(40, 16, D, device="cuda", dtype=torch.bfloat16)
        ok.oscar_kv8_rope_append(d, rope, R.INT8, 1, 40, q, k, v, i32([0, 40]), None, i32([ids]), i32([40]), *pool, qo)
        out = torch.empty(1, 16, D, device="cuda", dtype=torch.bfloat16)
        w = torch.empty(ok.oscar_kv8_decode_shared_workspace_bytes(d, 1, 48, 0, 48, 1, 1), dtype=torch.uint8, device="cuda")
        ok.oscar_kv8_decode_shared(d, R.INT8, 1, 48, 0, 48, qo[-1:], *pool, i32([ids]), i32([40]), i32([0]), i32([0, 1]), i32([0]), 0.0,
                                   out, w)
        outs += [pool[0][ids, :, :, :8].clone(), pool[1][ids].clone(), out]
    for a, b in zip(outs[:3], outs[3:]):
        assert torch.equal(a, b)
    assert ok.oscar_device_errors(reset=True) == 0


def test_int2_cache_takes_keys_without_positions():
    from int2_rotated_kv_append_gb300 import synth
    from int2_rotated_kv_append_gb300.cache import Int2Cache
    w = synth.make_workload(num_q_heads=8, num_kv_heads=2, head_dim=128, group_size=64, sink_len=16, window_len=64, seq_lens=[700], seed=3)
    rope = ok.Rope(64, interleaved=True)
    rows = torch.cat([w.k, w.v], 1).cuda()
    k, v = rows[:, :2], w.v.cuda()
    pos = w.tok_pos.cuda()
    a, b = Int2Cache(w), Int2Cache(w)
    a.append(k, v, w.slot_mapping.cuda(), rope=rope, positions=pos)
    turned = torch.empty(k.shape, dtype=k.dtype, device="cuda")
    ok.oscar_rope(w.dims, rope, pos, None, k, None, turned)
    check(turned, k, w.tok_pos.numpy(), rope)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    b.append(turned, v, w.slot_mapping.cuda(), stream=s)
    torch.cuda.synchronize()
    assert torch.equal(a.int2_pages, b.int2_pages) and torch.equal(a.scale_zero.view(torch.int16), b.scale_zero.view(torch.int16))
    assert torch.equal(rows[:, :2], w.k.cuda())
    b.append(k, v, w.slot_mapping.cuda(), stream=s, rope=rope, positions=pos)
    torch.cuda.synchronize()
    assert torch.equal(a.int2_pages, b.int2_pages)
    with pytest.raises(ValueError):
        a.append(k, v, w.slot_mapping.cuda(), rope=rope)
