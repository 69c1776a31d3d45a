"""Refusals of the 8-bit cache and page entry points, on the host: nothing is launched."""

import ctypes

import pytest
import torch

import int2_rotated_kv_append_gb300 as ok
from int2_rotated_kv_append_gb300 import build

BAD, UNS, WS, OK = ok.OSCAR_ERR_INVALID_ARG, ok.OSCAR_ERR_UNSUPPORTED, ok.OSCAR_ERR_WORKSPACE, ok.OSCAR_OK
P = ctypes.c_void_p(256)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p(24)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ok.load_library()


def dims(**kw):
    d = dict(num_q_heads=32, num_kv_heads=8, head_dim=128, page_size=16, group_size=64, num_pages=100, max_pages_per_seq=20)
    d.update(kw)
    return ctypes.byref(ok.make_dims(**d))


BAD_DIMS = [(None, BAD), (dims(head_dim=96, group_size=32), UNS), (dims(page_size=32), UNS), (dims(num_pages=0), BAD),
            (dims(num_q_heads=128), UNS), (dims(num_q_heads=30), BAD)]


def test_append_refusals(lib):
    def call(d=None, fmt=0, batch=2, tokens=4, most=3, **ptr):
        a = {n: P for n in "k v start table lens pages scales".split()}
        a.update(ptr)
        return lib.oscar_kv8_append(dims() if d is None else d[0], fmt, batch, tokens, most, a["k"], a["v"], a["start"],
                                    a["table"], a["lens"], a["pages"], a["scales"], None)
    for d, want in BAD_DIMS:
        assert call((d,)) == want
    assert call(tokens=0) == OK and call(tokens=0, batch=0, k=None) == OK
    assert call(fmt=2) == BAD and call(fmt=-1) == BAD and call(batch=-1) == BAD and call(batch=0) == BAD
    assert call(tokens=-1) == BAD and call(tokens=1 << 31) == BAD and call(most=0) == BAD and call(most=-1) == BAD
    assert call(batch=65536) == UNS
    for n in "k v start table lens pages scales".split():
        assert call(**{n: None}) == BAD
    for n in "k v pages scales".split():
        assert call(**{n: ODD}) == BAD


@pytest.mark.parametrize("extend", [False, True])
def test_attention_refusals(lib, extend):
    def size(d, batch=2, rows=9, max_len=300, most=5, pps=0, sink=4, window=8):
        if extend:
            return lib.oscar_kv8_extend_varlen_workspace_bytes(d, batch, rows, max_len, most, pps, sink, window)
        return lib.oscar_kv8_decode_workspace_bytes(d, batch, max_len, pps, sink, window)

    def call(d=None, fmt=0, batch=2, rows=9, max_len=300, most=5, pps=0, sink=4, window=8, ws=1 << 30, **ptr):
        a = {n: P for n in "q start pages scales table lens out work".split()}
        a.update(ptr)
        d = dims() if d is None else d[0]
        if extend:
            return lib.oscar_kv8_extend_varlen(d, fmt, batch, rows, max_len, most, pps, a["q"], a["start"], a["pages"],
                                               a["scales"], a["table"], a["lens"], sink, window, 0.0, a["out"], a["work"],
                                               ws, None)
        return lib.oscar_kv8_decode(d, fmt, batch, max_len, pps, a["q"], a["pages"], a["scales"], a["table"], a["lens"],
                                    sink, window, 0.0, a["out"], a["work"], ws, None)
    for d, want in BAD_DIMS:
        assert call((d,)) == want and size(d) == 0
    assert call(rows=0) == OK if extend else call(batch=0) == OK
    for kw in (dict(batch=-1), dict(max_len=-1), dict(pps=-1), dict(sink=-1), dict(window=-1), dict(max_len=321)):
        assert call(**kw) == BAD and size(dims(), **kw) == 0
    assert call(fmt=2) == BAD
    if extend:
        assert call(rows=-1) == BAD and call(most=-1) == BAD and call(most=0) == BAD and call(batch=0) == BAD
        assert size(dims(), rows=-1) == 0 and size(dims(), most=-1) == 0
    need = size(dims())
    assert need > 0 and call(ws=need - 1) == WS
    names = "q pages scales table lens out work".split() + (["start"] if extend else [])
    for n in names:
        assert call(**{n: None}) == BAD
    for n in "q pages scales out work".split():
        assert call(**{n: ODD}) == BAD


def test_page_refusals(lib):
    def pools(*entries):
        arr = (ok.oscar_page_pool_t * max(1, len(entries)))()
        for i, (base, n) in enumerate(entries):
            arr[i].base, arr[i].page_bytes = base, n
        return len(entries), arr
    good = pools((256, 4096), (512, 12))
    need = lib.oscar_pages_workspace_bytes(dims(), 4, 3)
    assert need > 0 and lib.oscar_pages_workspace_bytes(dims(), -1, 0) == 0 and lib.oscar_pages_workspace_bytes(dims(), 1, -1) == 0
    assert lib.oscar_pages_workspace_bytes(None, 1, 0) == 0

    def reserve(d=None, batch=4, new=P, table=P, lens=P, refs=P, ws=P, n=need):
        return lib.oscar_pages_reserve(dims() if d is None else d[0], batch, new, table, lens, refs, None, ws, n, None)

    def fork(d=None, pl=good, batch=4, n=3, src=P, dst=P, table=P, lens=P, refs=P, ws=P, nb=need):
        return lib.oscar_pages_fork(dims() if d is None else d[0], pl[0], pl[1], batch, n, src, dst, table, lens, refs, None,
                                    ws, nb, None)

    def free(d=None, batch=4, n=2, seqs=P, table=P, lens=P, refs=P):
        return lib.oscar_pages_free(dims() if d is None else d[0], batch, n, seqs, table, lens, refs, None)

    def trim(d=None, batch=4, sink=0, window=1, table=P, lens=P, refs=P):
        return lib.oscar_pages_trim(dims() if d is None else d[0], batch, sink, window, table, lens, refs, None)

    def compact(d=None, pl=good, batch=4, table=P, lens=P, refs=P, ws=P, nb=need):
        return lib.oscar_pages_compact(dims() if d is None else d[0], pl[0], pl[1], batch, table, lens, refs, None, ws, nb, None)

    def copy(d=None, pl=good, n=2, src=P, dst=P):
        return lib.oscar_pages_copy(dims() if d is None else d[0], pl[0], pl[1], n, src, dst, None)

    for call in (reserve, fork, free, trim, compact, copy):
        assert call((None,)) == BAD and call((dims(num_pages=0),)) == BAD and call((dims(max_pages_per_seq=0),)) == BAD
        assert call((dims(page_size=32),)) == UNS
    for call in (reserve, fork, free, trim, compact):
        assert call(batch=-1) == BAD and call(batch=65536) == UNS
        for n in ("table", "lens", "refs"):
            assert call(**{n: None}) == BAD
    for call in (reserve, fork, compact):
        assert call(refs=ODD) == BAD and call(ws=None) == BAD and call(ws=ODD) == BAD
    assert reserve(n=16) == WS and fork(nb=need - 1) == WS and compact(nb=16) == WS
    for call in (fork, compact, copy):
        assert call(pl=pools((24, 64))) == BAD and call(pl=pools((None, 64))) == BAD and call(pl=pools((256, 6))) == BAD
        assert call(pl=pools((256, 0))) == BAD and call(pl=(9, good[1])) == BAD and call(pl=(-1, good[1])) == BAD
        assert call(pl=(1, None)) == BAD
    assert fork(n=0) == OK and free(n=0) == OK and trim(batch=0) == OK and copy(n=0) == OK and reserve(batch=0) == OK
    assert fork(n=-1) == BAD and free(n=-1) == BAD and copy(n=-1) == BAD and fork(src=None) == BAD and fork(dst=None) == BAD
    assert free(seqs=None) == BAD and trim(sink=-1) == BAD and trim(window=0) == BAD and reserve(new=None) == BAD
    assert copy(src=None) == BAD and copy(dst=None) == BAD and free(batch=0) == BAD and fork(batch=0) == BAD


def test_python_pools_are_contiguous_tensors_of_equal_pages():
    with pytest.raises(ValueError):
        ok._pools([torch.zeros(10, 4).t()], 10)
    with pytest.raises(ValueError):
        ok._pools([torch.zeros(7)], 10)
    with pytest.raises(ValueError):
        ok._pools([torch.zeros(0)], 10)
    arr = ok._pools([torch.zeros(10, 4), torch.zeros(30, dtype=torch.bfloat16)], 10)
    assert (arr[0].page_bytes, arr[1].page_bytes) == (16, 6)


def test_append_granted_refuses_what_append_refuses(lib):
    def call(d=None, fmt=0, batch=2, tokens=4, most=3, **ptr):
        a = {n: P for n in "k v start table lens granted pages scales".split()}
        a.update(ptr)
        return lib.oscar_kv8_append_granted(dims() if d is None else d[0], fmt, batch, tokens, most, a["k"], a["v"], a["start"],
                                            a["table"], a["lens"], a["granted"], a["pages"], a["scales"], None)
    for d, want in BAD_DIMS:
        assert call((d,)) == want
    assert call(tokens=0) == OK and call(tokens=0, granted=None) == OK
    assert call(fmt=2) == BAD and call(batch=-1) == BAD and call(most=0) == BAD and call(batch=65536) == UNS
    for n in "k v start table lens pages scales".split():
        assert call(**{n: None}) == BAD
    with pytest.raises(ValueError):
        ok.oscar_kv8_append(None, 0, 2, 1, torch.zeros(2, 8, 128), None, None, None, None, None, None, granted=torch.ones(1))


def test_lengths_beyond_what_positions_can_count_are_refused(lib):
    d = dims(max_pages_per_seq=1 << 27)
    for n, fits in (((1 << 31) - 33, True), ((1 << 31) - 32, False), ((1 << 31) - 1, False)):
        assert (lib.oscar_kv8_decode_workspace_bytes(d, 1, n, 0, 0, 64) > 0) == fits
        assert (lib.oscar_kv8_extend_varlen_workspace_bytes(d, 1, 4, n, 4, 0, 0, 64) > 0) == fits
    assert lib.oscar_kv8_decode(d, 0, 1, (1 << 31) - 1, 0, P, P, P, P, P, 0, 64, 0.0, P, P, 1 << 30, None) == BAD
    assert lib.oscar_kv8_extend_varlen(d, 0, 1, 4, (1 << 31) - 1, 4, 0, P, P, P, P, P, P, 0, 64, 0.0, P, P, 1 << 30, None) == BAD
