"""What Kv8Cache passes to the library, on the host: the calls are recorded, nothing is launched."""

import pytest
import torch

from int2_rotated_kv_append_gb300 import build, cache


@pytest.fixture
def recorded(monkeypatch):
    build.build()
    calls = []
    for name, ws, stream in (("oscar_kv8_decode", 14, 15), ("oscar_kv8_extend_varlen", 16, 17), ("oscar_pages_reserve", 6, 7),
                             ("oscar_pages_fork", 8, 9), ("oscar_pages_compact", 6, 7)):
        def call(*args, name=name, ws=ws, stream=stream):
            calls.append((name, args[ws], args[stream]))
        monkeypatch.setattr(cache, name, call)
    return calls


def make(**kw):
    return cache.Kv8Cache(num_q_heads=8, num_kv_heads=2, head_dim=64, num_pages=300, batch=2, max_seq_len=2000, device="cpu", **kw)


def test_streams_have_workspaces_of_their_own(recorded):
    c = make()
    q = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    start = torch.tensor([0, 1, 2], dtype=torch.int32)
    for stream in (3, 5, 3):
        c.decode(q, stream=stream)
        c.extend(q, start, 1, stream=stream)
        c.reserve(start[:2], stream=stream)
        c.fork(start[:1], start[1:2], stream=stream)
        c.compact(stream=stream)
    spans = {}
    for name, ws, stream in recorded:
        spans.setdefault(stream, set()).add((ws.data_ptr(), ws.data_ptr() + ws.numel()))
    assert set(spans) == {3, 5}
    for a0, a1 in spans[3]:
        assert all(a1 <= b0 or b1 <= a0 for b0, b1 in spans[5])


def test_a_grown_workspace_leaves_the_smaller_one_to_captured_graphs(recorded):
    c = make()
    q = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    c.reserve(torch.zeros(2, dtype=torch.int32), stream=3)
    c.decode(q, stream=3, pages_per_split=1)
    c.reserve(torch.zeros(2, dtype=torch.int32), stream=3)
    small, large, again = (ws for _, ws, _ in recorded)
    assert small.numel() < large.numel() and again.data_ptr() == large.data_ptr()
    assert any(w.data_ptr() == small.data_ptr() for w in c._ws[3])


def test_attention_is_planned_for_the_longest_length_that_the_caller_names(recorded, monkeypatch):
    sizes = []
    for name in ("oscar_kv8_decode_workspace_bytes", "oscar_kv8_extend_varlen_workspace_bytes"):
        real = getattr(cache, name)
        monkeypatch.setattr(cache, name, lambda *a, real=real: sizes.append(a) or real(*a))
    lengths = []
    for name, at in (("oscar_kv8_decode", 3), ("oscar_kv8_extend_varlen", 3)):
        monkeypatch.setattr(cache, name, lambda *a, at=at: lengths.append(a[at]))
    c = make()
    q = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    start = torch.tensor([0, 1, 2], dtype=torch.int32)
    for given, want in ((None, 2000), (700, 700), (2000, 2000)):
        c.decode(q, max_seq_len=given, stream=3)
        c.extend(q, start, 1, max_seq_len=given, stream=3)
        assert lengths[-2:] == [want, want] and sizes[-2][2] == want and sizes[-1][3] == want
    for given in (2001, -1):
        with pytest.raises(ValueError):
            c.decode(q, max_seq_len=given, stream=3)
        with pytest.raises(ValueError):
            c.extend(q, start, 1, max_seq_len=given, stream=3)
