"""Kv8Cache up to the last token that it grants."""

import pytest
import torch

import int2_rotated_kv_append_gb300 as ok
import kv8_ref as R
from int2_rotated_kv_append_gb300.cache import Kv8Cache

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("max_seq_len,sink,window", [(200, 0, 0), (1, 0, 0), (33, 4, 20), (64, 0, 0), (207, 0, 30)])
def test_every_granted_token_is_attended(max_seq_len, sink, window):
    g = torch.Generator("cuda").manual_seed(max_seq_len)
    c = Kv8Cache(num_q_heads=4, num_kv_heads=2, head_dim=64, num_pages=40, batch=2, max_seq_len=max_seq_len, sink_len=sink,
                 window_len=window)
    room = 16 * -(-max_seq_len // 16)
    assert c.reserve(i32([room, 1])).tolist() == [1, 1]
    k, v = (torch.randn(room + 1, 2, 64, device="cuda", generator=g).bfloat16() for _ in range(2))
    c.append(k, v, i32([0, room, room + 1]), room)
    rows = min(room, 40)
    q = torch.randn(rows + 1, 4, 64, device="cuda", generator=g).bfloat16()
    ref, tol = R.attention(c.pages, c.scales, q, [0] * rows + [1], list(range(room - rows, room)) + [0], c.page_table.tolist(),
                           c.kv_format, sink, window)
    out = c.extend(q, i32([0, rows, rows + 1]), rows)
    assert ((out.double() - ref).abs() <= tol).all()
    assert ((c.decode(q[-2:]).double() - ref[-2:]).abs() <= tol[-2:]).all()
    assert ok.oscar_device_errors(reset=True) == 0
    assert c.reserve(i32([1, 1])).tolist() == [0, 1]  # not one token more
    assert c.seq_lens.tolist() == [room, 2] and ok.oscar_device_errors(reset=True) == ok.OSCAR_DEVERR_POSITION
