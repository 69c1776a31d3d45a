"""An append after a reservation that was refused: nothing of the sequence, or of those that share its pages, changes."""

import pytest
import torch

import int2_rotated_kv_append_gb300 as ok
import kv8_ref as R
from int2_rotated_kv_append_gb300.cache import Kv8Cache

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def rows(c, n, g):
    return [torch.randn(n, c.dims.num_kv_heads, c.dims.head_dim, device="cuda", generator=g).bfloat16() for _ in range(2)]


def decode_of(c, q, out, seqs):
    lens = c.seq_lens.tolist()
    ref, tol = R.attention(c.pages, c.scales, q[seqs], seqs, [lens[b] - 1 for b in seqs], c.page_table.tolist(), c.kv_format,
                           c.sink_len, c.window_len)
    assert ((out[seqs].double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("fmt", [R.E4M3, R.INT8])
def test_step_without_free_pages_leaves_shared_pages(captured, fmt):
    g = torch.Generator("cuda").manual_seed(1)
    c = Kv8Cache(num_q_heads=4, num_kv_heads=2, head_dim=64, num_pages=6, batch=4, max_seq_len=320, kv_format=fmt)
    assert c.reserve(i32([48, 0, 0, 5])).all()
    c.append(*rows(c, 53, g), i32([0, 48, 48, 48, 53]), 48)
    c.fork(i32([0, 0]), i32([1, 2]))  # three sequences of three full pages
    assert c.seq_lens.tolist() == [48, 48, 48, 5] and c.page_refs.tolist() == [3, 3, 3, 1, 0, 0]
    one, start = i32([1, 1, 1, 1]), i32([0, 1, 2, 3, 4])
    k, v = rows(c, 4, g)
    k *= 50  # a larger scale: earlier codes of a page would change with it
    q = torch.randn(4, 4, 64, device="cuda", generator=g).bfloat16()
    out = torch.empty_like(q)

    def step():
        c.reserve(one)
        c.append(k, v, start, 1)
        c.decode(q, out)

    shared = c.page_table[0, :3].long()
    codes, scales = c.pages[shared].clone(), c.scales[shared].clone()
    if captured:
        c.decode(q, out)
        c.reserve(i32([0, 0, 0, 0]))
        c.append(k, v, i32([0, 0, 0, 0, 0]), 1)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        step = graph.replay
    for i in range(3):  # two of the three get a page, the third is refused each time
        step()
        assert ok.oscar_device_errors(reset=True) == ok.OSCAR_DEVERR_NO_PAGES
        assert c.granted.tolist() == [1, 1, 0, 1] and c.seq_lens.tolist() == [49 + i, 49 + i, 48, 6 + i]
        assert torch.equal(c.pages[shared], codes) and torch.equal(c.scales[shared], scales)
        decode_of(c, q, out, [0, 1, 2, 3])
    c.free(i32([0]))
    assert c.reserve(i32([0, 0, 1, 0])).tolist() == [1, 1, 1, 1]
    c.append(k[:1], v[:1], i32([0, 0, 0, 1, 1]), 1)
    c.decode(q, out)
    assert c.seq_lens.tolist() == [0, 51, 49, 8]
    assert torch.equal(c.pages[shared], codes) and torch.equal(c.scales[shared], scales)
    decode_of(c, q, out, [1, 2, 3])


def test_append_of_several_tokens_skips_refused_sequences_alone():
    g = torch.Generator("cuda").manual_seed(2)
    c = Kv8Cache(num_q_heads=2, num_kv_heads=1, head_dim=128, num_pages=7, batch=3, max_seq_len=128)
    c.reserve(i32([20, 20, 20]))
    c.append(*rows(c, 60, g), i32([0, 20, 40, 60]), 20)
    before = c.pages.clone(), c.scales.clone()
    granted = c.reserve(i32([12, 40, 12]))  # the second needs two pages, one is free
    assert granted.tolist() == [1, 0, 1] and c.seq_lens.tolist() == [32, 20, 32]
    k, v = rows(c, 64, g)
    c.append(k, v, i32([0, 12, 52, 64]), 40)
    own = c.page_table[1, :2].long()
    assert torch.equal(c.pages[own], before[0][own]) and torch.equal(c.scales[own], before[1][own])
    for b, at in ((0, 0), (2, 52)):
        last = c.page_table[b, 1].item()
        got = c.pages[last, 0, 1].view(torch.float8_e4m3fn).float() * c.scales[last, 0, 1]
        assert ((got[4:] - v[at:at + 12, 0].float()).abs() <= c.scales[last, 0, 1] * 16).all()  # half a step of the largest codes
    assert ok.oscar_device_errors(reset=True) == ok.OSCAR_DEVERR_NO_PAGES


def test_append_without_a_reservation_goes_by_the_lengths():
    c = Kv8Cache(num_q_heads=2, num_kv_heads=1, head_dim=64, num_pages=4, batch=1, max_seq_len=32)
    c.page_table[0, 0] = 2
    c.seq_lens[0] = 3
    k = torch.ones(3, 1, 64, device="cuda", dtype=torch.bfloat16)
    c.append(k, k, i32([0, 3]), 3)
    assert (c.pages[2, 0, :, :3] != 0).all() and not c.pages[[0, 1, 3]].any()
