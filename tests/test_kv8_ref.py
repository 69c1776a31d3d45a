"""The 8-bit reference against torch's own e4m3 conversion and hand-worked cases (CPU)."""

import numpy as np
import torch

import kv8_ref as R


def test_e4m3_codes_are_torchs():
    g = np.random.default_rng(1)
    x = np.concatenate([g.normal(size=4000) * 2.0 ** g.integers(-12, 9, 4000), R.E4M3_VALUES[:127],
                        (R.E4M3_VALUES[:126] + R.E4M3_VALUES[1:127]) / 2, [0.0, -0.0, 448.0, -448.0]])
    x = np.clip(x, -448, 448).astype(np.float32)
    ours = R.encode(x.astype(np.float64), R.E4M3)
    theirs = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ours, theirs)
    back = torch.from_numpy(ours).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.code_values(ours, R.E4M3), back)


def test_scales():
    assert R.scale_of(448.0, R.E4M3) == 1.0 and R.scale_of(449.0, R.E4M3) == 2.0
    assert R.scale_of(127.0, R.INT8) == 1.0 and R.scale_of(128.0, R.INT8) == 2.0
    assert R.scale_of(0.0, R.INT8) == 2.0 ** -100


def test_append_takes_earlier_codes_to_the_larger_scale():
    codes, scales = np.zeros((2, 1, 2, 16, 64), np.uint8), np.ones((2, 1, 2), np.float32)
    table = [[1]]
    x = np.ones((1, 1, 64))
    R.append(codes, scales, x * 0.5, x, [0, 1], table, [1], R.INT8)
    assert scales[1, 0, 0] == 2.0 ** -7 and codes[1, 0, 0, 0, 0] == 64
    R.append(codes, scales, x * 3.0, x, [0, 1], table, [2], R.INT8)
    assert scales[1, 0, 0] == 2.0 ** -5 and codes[1, 0, 0, 0, 0] == 16 and codes[1, 0, 0, 1, 0] == 96


def test_pages_fork_then_free_gives_everything_back():
    m = R.Pages(8, 3, 4)
    assert m.reserve([40, 0, 0]) == [1, 1, 1] and m.table[0][:3] == [0, 1, 2]
    granted, copies = m.fork([0, 0], [1, 2])
    assert granted == [1, 1] and copies == [(2, 3), (2, 4)] and m.refs[:5] == [3, 3, 1, 1, 1]
    m.free([0, 1, 2])
    assert not any(m.refs)


def test_a_cancelling_page_shows_the_second_part_of_the_weights():
    # the decode's weights, emulated in numpy: two fp16 parts hold the tolerance, one alone, or one mis-scaled, does not
    for seed in range(5):
        k, v, w = R.cancelling_page(128, seed)
        want, tol = R.cancelling_tolerance(v, w)
        s = (k * 2.0 ** -7 * np.log2(np.e)).astype(np.float32)
        p = np.exp2(s - np.ceil(s.max())).astype(np.float32)
        hi = (p * np.float32(2 ** 14)).astype(np.float16)
        lo = ((p * np.float32(2 ** 14) - hi.astype(np.float32)) * np.float32(2 ** 12)).astype(np.float16)

        def out(second):
            o = ((hi.astype(np.float64) + second * lo.astype(np.float64)) / 2 ** 14) @ v / p.astype(np.float64).sum()
            return torch.from_numpy(o).bfloat16().double().numpy()
        assert (np.abs(out(2.0 ** -12) - want) <= tol).all()
        for planted in (0.0, 2.0 ** -11, 2.0 ** -14):
            assert (np.abs(out(planted) - want) > tol).sum() > 30, planted
