"""Refusals of oscar_kv8_decode_shared and oscar_pages_groups on the host: nothing is launched."""

import ctypes

import pytest
import torch

import int2_rotated_kv_append_gb300 as ok
from int2_rotated_kv_append_gb300 import build
from test_kv8_abi import BAD, BAD_DIMS, ODD, OK, P, UNS, WS, dims


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ok.load_library()


def test_decode_shared_refusals(lib):
    def size(d, batch=4, max_len=300, prefix=200, own=100, members=4, groups=2):
        return lib.oscar_kv8_decode_shared_workspace_bytes(d, batch, max_len, prefix, own, members, groups)

    def call(d=None, fmt=0, batch=4, max_len=300, prefix=200, own=100, members=4, groups=2, ws=1 << 40, **ptr):
        a = {n: P for n in "q pages scales table lens members start prefixes out work".split()}
        a.update({k.replace("p_", ""): v for k, v in ptr.items()})
        return lib.oscar_kv8_decode_shared(dims() if d is None else d[0], fmt, batch, max_len, prefix, own, members, groups, a["q"],
                                           a["pages"], a["scales"], a["table"], a["lens"], a["members"], a["start"], a["prefixes"], 0.0,
                                           a["out"], a["work"], ws, None)
    for d, want in BAD_DIMS:
        assert call((d,)) == want and size(d) == 0
    for kw in (dict(batch=-1), dict(max_len=-1), dict(prefix=-1), dict(own=-1), dict(members=-1), dict(groups=-1), dict(max_len=321),
               dict(prefix=301), dict(own=301), dict(members=65536), dict(groups=65536)):
        assert call(**kw) == BAD and size(dims(), **kw) == 0, kw
    assert call(fmt=2) == BAD and call(fmt=-1) == BAD and call(batch=0) == BAD
    assert call(members=0) == OK and call(groups=0) == OK
    need = size(dims())
    assert need > 0 and call(ws=need - 1) == WS
    for n in "q pages scales table lens p_members start prefixes out work".split():
        assert call(**{n: None}) == BAD, n
    for n in "q pages scales out work".split():
        assert call(**{n: ODD}) == BAD
    assert call((dims(num_pages=1 << 29),)) == UNS


@pytest.mark.parametrize("kw", [dict(), dict(prefix=0), dict(own=0), dict(members=65535, groups=65535), dict(members=1, groups=65535),
                                dict(members=65535, groups=1)])
def test_decode_shared_workspaces(lib, kw):
    a = {**dict(max_len=300, prefix=200, own=100, members=4, groups=2), **kw}
    for heads in ((32, 8), (1, 1), (200, 200), (1600, 200)):
        d = dims(num_q_heads=heads[0], num_kv_heads=heads[1])
        n = lib.oscar_kv8_decode_shared_workspace_bytes(d, 4, *a.values())
        assert 0 < n < 1 << 40
        t, p, o = (ctypes.c_int32(-1) for _ in range(3))
        assert lib.oscar_kv8_decode_shared_plan(d, 4, *a.values(), ctypes.byref(t), ctypes.byref(p), ctypes.byref(o)) == OK
        assert t.value in (0, 64, 128, 256) and (t.value > 0) == (p.value > 0) and o.value > 0
        assert lib.oscar_kv8_decode_shared_plan(d, 4, *a.values(), None, None, None) == OK
    assert lib.oscar_kv8_decode_shared_plan(d, 4, 300, 301, 0, 4, 2, None, None, None) == BAD
    assert lib.oscar_kv8_decode_shared_plan(None, 4, 300, 300, 0, 4, 2, None, None, None) == BAD


def test_groups_refusals(lib):
    def call(d=None, batch=4, k=1, room=2, ws=1 << 20, **ptr):
        a = {n: P for n in "table lens members start prefixes work".split()}
        a.update(ptr)
        return lib.oscar_pages_groups(dims() if d is None else d[0], batch, k, room, a["table"], a["lens"], a["members"], a["start"],
                                      a["prefixes"], a["work"], ws, None)
    for d, want in ((None, BAD), (dims(page_size=32), UNS), (dims(num_pages=0), BAD)):
        assert call((d,)) == want and lib.oscar_pages_groups_workspace_bytes(d, 4) == 0
    assert call(batch=-1) == BAD and call(k=0) == BAD and call(room=0) == BAD and call(batch=0) == OK
    need = lib.oscar_pages_groups_workspace_bytes(dims(), 4)
    assert need > 0 and call(ws=need - 1) == WS
    for n in "table lens members start prefixes work".split():
        assert call(**{n: None}) == BAD
    assert call(work=ODD) == BAD


def test_binding_checks_lists(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)  # (where tensors of the CPU are)
    d = dict(num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16, group_size=64, num_pages=9, max_pages_per_seq=4)
    i = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    q = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    pages, scales, work = torch.zeros(9, 2, 2, 16, 128, dtype=torch.uint8), torch.zeros(9, 2, 2), torch.zeros(1 << 20, dtype=torch.uint8)
    good = dict(q=q, table=i((3, 4)), lens=i(3), members=i(3), start=i(3), prefix=i(2), out=q)
    for bad in (dict(q=q.half()), dict(q=q[:2]), dict(out=q[:, :4]), dict(start=i(2)), dict(members=i(3).long()), dict(lens=i(2)),
                dict(table=i((2, 4))), dict(prefix=i(2).float())):
        a = {**good, **bad}
        with pytest.raises(ValueError):
            ok.oscar_kv8_decode_shared(d, 0, 3, 64, 32, 32, a["q"], pages, scales, a["table"], a["lens"], a["members"], a["start"],
                                       a["prefix"], 0.0, a["out"], work, stream=0)
    for bad in (dict(members=i(2)), dict(start=i(2)), dict(prefix=i(0)), dict(table=i((2, 4)))):
        a = {**good, **bad}
        with pytest.raises(ValueError):
            ok.oscar_pages_groups(d, 1, a["table"], a["lens"], a["members"], a["start"], a["prefix"], work, stream=0)
    assert ctypes.sizeof(ok.oscar_rope_t) == 24
