"""The binding's checks of the 8-bit cache's buffers: a pool of fewer pages than dims has, or scales of another type, would be read and
written past their ends.  Nothing is launched."""

import pytest
import torch

import int2_rotated_kv_append_gb300 as ok
from int2_rotated_kv_append_gb300 import build

DIMS = dict(num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16, group_size=64, num_pages=9, max_pages_per_seq=4)
PAGES, SCALES = torch.zeros(9, 2, 2, 16, 128, dtype=torch.uint8), torch.zeros(9, 2, 2)
BAD = [(PAGES[:8], SCALES), (PAGES[..., :64].contiguous(), SCALES), (PAGES.half()[:4], SCALES), (PAGES[..., ::2], SCALES),
       (torch.zeros(18, 2, 2, 16, 128, dtype=torch.uint8)[::2], SCALES), (PAGES, SCALES[:8]), (PAGES, SCALES.half()),
       (PAGES, SCALES.bfloat16()), (PAGES, SCALES.double()), (PAGES, torch.zeros(9, 4, 2)[:, ::2]),
       (PAGES, torch.zeros(72, dtype=torch.uint8))]


@pytest.fixture(autouse=True)
def on_the_cpu(monkeypatch):
    build.build()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)  # (where tensors of the CPU are)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


@pytest.mark.parametrize("pages,scales", BAD)
def test_rope_append_refuses_other_pools(pages, scales):
    q, k = torch.zeros(3, 8, 128, dtype=torch.bfloat16), torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ok.oscar_kv8_rope_append(DIMS, ok.Rope(64, device="cpu"), 0, 3, 1, q, k, k, i32(4), None, i32(3, 4), i32(3), pages, scales, q,
                                 stream=0)


@pytest.mark.parametrize("pages,scales", BAD)
def test_decode_shared_refuses_other_pools(pages, scales):
    q = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ok.oscar_kv8_decode_shared(DIMS, 0, 3, 64, 32, 32, q, pages, scales, i32(3, 4), i32(3), i32(3), i32(3), i32(2), 0.0, q,
                                   torch.zeros(1 << 20, dtype=torch.uint8), stream=0)


@pytest.mark.parametrize("pages", [PAGES, PAGES.view(torch.int8), PAGES.view(torch.float8_e4m3fn), torch.zeros(10, 2, 2, 16, 128, dtype=torch.uint8)])
def test_pools_that_are_large_enough_pass(pages):
    # (the call ends at its format, which comes after these checks)
    q, k = torch.zeros(3, 8, 128, dtype=torch.bfloat16), torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ok.OscarError):
        ok.oscar_kv8_rope_append(DIMS, ok.Rope(64, device="cpu"), 7, 3, 1, q, k, k, i32(4), None, i32(3, 4), i32(3), pages, SCALES, q,
                                 stream=0)
    with pytest.raises(ok.OscarError):
        ok.oscar_kv8_decode_shared(DIMS, 7, 3, 64, 32, 32, q, pages, SCALES, i32(3, 4), i32(3), i32(3), i32(3), i32(2), 0.0, q,
                                   torch.zeros(1 << 20, dtype=torch.uint8), stream=0)
