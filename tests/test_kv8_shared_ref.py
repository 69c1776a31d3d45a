"""The tolerances of kv8_shared_ref against weights rounded as each form does, and against weights of fewer bits, which they show."""

import numpy as np
import pytest
import torch

import kv8_ref as R
import kv8_shared_ref as S


def rounded(w, part):
    """Weights w (relative to the largest) as a form holds them, or as one of fewer bits would."""
    t = torch.from_numpy(w)
    if part == "list":
        hi = (t * 2.0 ** 14).half().double()
        return ((hi + ((t * 2.0 ** 14 - hi) * 2.0 ** 12).half().double() * 2.0 ** -12) * 2.0 ** -14).numpy()
    if part == "one part":
        return ((t * 2.0 ** 14).half().double() * 2.0 ** -14).numpy()
    if part == "fp16":
        return ((t * 2.0 ** 6).half().double() * 2.0 ** -6).numpy()
    if part == "fp16 without boost":
        return t.half().double().numpy()
    return t.bfloat16().double().numpy()


def misses(k, v, bits, part):
    q = torch.zeros(1, v.shape[1], dtype=torch.float64)
    q[0, 0] = 1.0
    kk = torch.zeros(len(k), v.shape[1], dtype=torch.float64)
    kk[:, 0] = torch.from_numpy(np.asarray(k, float))
    want, tol = S.attend(q, kk, torch.from_numpy(np.asarray(v, float)), 0.125, torch.tensor(bits, dtype=torch.float64).repeat(len(k), 1))
    w = np.exp((np.asarray(k) - np.max(k)) * 0.125)
    got = torch.from_numpy(rounded(w, part) @ v / w.sum()).bfloat16().double()
    return int(((got - want[0]).abs() > tol[0]).sum())


@pytest.mark.parametrize("seed", range(5))
def test_cancelling_pages(seed):
    k, v, _ = R.cancelling_page(64, seed)
    k = k * 2.0 ** -4
    assert misses(k, v, S.LIST, "list") == 0 and misses(k, v, S.LIST, "one part") > 5
    for bits in (S.OWN, S.TAME):
        assert misses(k, v, bits, "fp16") == 0 and misses(k, v, bits, "bf16") > 5
    assert misses(k, v, S.WILD, "bf16") == 0


def test_light_tokens_of_large_values():
    # weights of 2^-24 to 2^-26 of the largest, whose own value is 0
    k = np.array([0.0] + [-8 * np.log(2.0) * e for e in np.linspace(24, 26, 30)])
    v = np.ones((31, 64)) * 2.0 ** 26
    v[0] = 0
    assert misses(k, v, S.OWN, "fp16") == 0 and misses(k, v, S.OWN, "fp16 without boost") > 5
    assert misses(k, v, S.LIST, "list") == 0
