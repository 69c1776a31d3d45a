"""The 8-bit cache as a serving program uses it: reserve, append, attention, fork, trim, compact, free."""

import numpy as np
import pytest
import torch

import int2_rotated_kv_append_gb300 as ok
import kv8_ref as R
from int2_rotated_kv_append_gb300 import synth
from int2_rotated_kv_append_gb300.cache import Int2Cache, Kv8Cache

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Server:
    """A Kv8Cache beside the bf16 tokens that went into each sequence."""

    def __init__(self, **kw):
        self.c = Kv8Cache(**kw)
        self.g = torch.Generator("cuda").manual_seed(3)
        d = self.c.dims
        self.shape = (d.num_kv_heads, d.head_dim)

    def add(self, new):
        c = self.c
        T = sum(new)
        k, v = (torch.randn(T, *self.shape, device="cuda", generator=self.g).bfloat16() for _ in range(2))
        c.reserve(i32(new))
        assert c.granted.all()
        c.append(k, v, i32(np.concatenate([[0], np.cumsum(new)])), max(new))
        return k, v

    def check(self, rows):
        """Query rows at the end of each sequence, by extend (and decode for one row each)."""
        c, d = self.c, self.c.dims
        lens = c.seq_lens.tolist()
        q = torch.randn(sum(rows), d.num_q_heads, d.head_dim, device="cuda", generator=self.g).bfloat16()
        start = np.concatenate([[0], np.cumsum(rows)])
        seq = [b for b, r in enumerate(rows) for _ in range(r)]
        pos = [lens[b] - r + i for b, r in enumerate(rows) for i in range(r)]
        ref, tol = R.attention(c.pages, c.scales, q, seq, pos, c.page_table.tolist(), c.kv_format, c.sink_len, c.window_len)
        out = c.extend(q, i32(start), max(rows))
        assert ((out.double() - ref).abs() <= tol).all()
        if all(r == 1 for r in rows):
            assert ((c.decode(q).double() - ref).abs() <= tol).all()
        assert ok.oscar_device_errors(reset=True) == 0


@pytest.mark.parametrize("fmt", [R.E4M3, R.INT8])
@pytest.mark.parametrize("sink,window", [(0, 0), (20, 64)])
def test_serving_loop(fmt, sink, window):
    s = Server(num_q_heads=8, num_kv_heads=2, head_dim=128, num_pages=120, batch=6, max_seq_len=600, kv_format=fmt,
               sink_len=sink, window_len=window)
    c = s.c
    s.add([300, 77, 0, 0, 0, 1])
    s.check([300, 77, 0, 0, 0, 1])
    c.fork(i32([0, 0, 1]), i32([2, 3, 4]))
    s.check([1, 1, 1, 1, 1, 1])
    for step in range(20):
        s.add([1, 1, 1, 1, 1, 1])  # the forks go their own ways
        if window:
            c.trim()
        s.check([1] * 6)
    shared = c.page_refs.max().item()
    assert shared == 3 if not window else shared >= 1
    c.free(i32([0, 4]))
    used = i32([0])
    c.compact(used)
    assert used.item() == int((c.page_refs > 0).sum()) and not c.page_refs[used.item():].any()
    s.check([0, 5, 1, 1, 0, 3])
    s.add([50, 0, 3, 0, 7, 1])
    s.check([50, 1, 3, 1, 7, 1])
    c.free(i32([0, 1, 2, 3, 4, 5]))
    assert not c.page_refs.any() and not c.seq_lens.any()


def test_values_survive_within_half_a_step():
    # what is stored is within half a code step of what was appended, also after a block's scale grew
    s = Server(num_q_heads=2, num_kv_heads=2, head_dim=64, num_pages=4, batch=1, max_seq_len=64, kv_format=R.INT8)
    kept = [s.add([n]) for n in (5, 1, 1, 20)]
    k = torch.cat([a for a, _ in kept]).double()
    c = s.c
    ids = c.page_table[0, :2].long()
    got = (c.pages[ids].view(torch.int8).double() * c.scales[ids].double()[..., None, None])[:, :, 0]
    got = got.permute(0, 2, 1, 3).reshape(32, 2, 64)[:27]
    step = c.scales[ids].double()[:, :, 0].repeat_interleave(16, 0)[:27, :, None]
    # each of the up to three roundings of the first rows is half a step of its time; steps at least doubled in between
    assert ((got - k).abs() <= step).all()


def test_whole_step_in_a_graph():
    s = Server(num_q_heads=4, num_kv_heads=1, head_dim=64, num_pages=40, batch=3, max_seq_len=200, sink_len=4, window_len=40)
    c = s.c
    s.add([30, 50, 1])
    k, v = (torch.randn(3, 1, 64, device="cuda", generator=s.g).bfloat16() for _ in range(2))
    q = torch.randn(3, 4, 64, device="cuda", generator=s.g).bfloat16()
    one, start = i32([1, 1, 1]), i32([0, 1, 2, 3])
    out = torch.empty_like(q)

    def step():
        c.reserve(one)
        c.append(k, v, start, 1)
        c.decode(q, out)
        c.trim()

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(40):
        k.normal_(generator=s.g)
        graph.replay()
        lens = c.seq_lens.tolist()
        assert lens == [32 + i, 52 + i, 3 + i]
        ref, tol = R.attention(c.pages, c.scales, q, [0, 1, 2], [n - 1 for n in lens], c.page_table.tolist(), c.kv_format, 4, 40)
        assert ((out.double() - ref).abs() <= tol).all()
    assert ok.oscar_device_errors(reset=True) == 0


def test_fork_of_an_int2_cache_decodes_the_same():
    # pages of the INT2 pools through oscar_pages_fork, the BF16 sink and window rows through oscar_pages_copy
    w = synth.make_workload(num_q_heads=8, num_kv_heads=2, head_dim=128, group_size=64, sink_len=16, window_len=64,
                            seq_lens=[500, 333, 0, 0], seed=3, spare_pages=6)
    c = Int2Cache(w)
    c.prefill()
    refs = torch.zeros(w.num_pages, dtype=torch.int32, device="cuda")
    for b, L in enumerate([500, 333]):
        refs[c.page_table[b, :-(-L // 16)].long()] = 1
    src, dst = i32([1, 0]), i32([2, 3])
    ws = torch.empty(ok.oscar_pages_workspace_bytes(c.dims, 4, 2), dtype=torch.uint8, device="cuda")
    pools = [c.int2_pages, c.scale_zero]
    ok.oscar_pages_fork(c.dims, pools, src, dst, c.page_table, c.seq_lens, refs, None, ws)
    per_seq = ok.make_dims(8, 2, 128, 16, 64, 4, 1)
    ok.oscar_pages_copy(per_seq, [c.sink, c.window], src, dst)
    q = w.q.cuda()
    q[2], q[3] = q[1], q[0]
    out = c.decode(q)
    assert torch.equal(out[2], out[1]) and torch.equal(out[3], out[0])
    used = i32([0])
    ok.oscar_pages_free(c.dims, i32([0, 1]), c.page_table, c.seq_lens, refs)
    ok.oscar_pages_compact(c.dims, pools, c.page_table, c.seq_lens, refs, used, ws)
    again = c.decode(q)
    assert torch.equal(again[2], out[2]) and torch.equal(again[3], out[3]) and not again[:2].any()
    assert used.item() == 32 + 21 and ok.oscar_device_errors(reset=True) == 0


def test_decode_and_extend_of_one_cache_on_two_streams():
    s = Server(num_q_heads=16, num_kv_heads=2, head_dim=128, num_pages=400, batch=2, max_seq_len=3000, kv_format=R.INT8)
    c = s.c
    s.add([3000, 1500])
    q, qx = (torch.randn(n, 16, 128, device="cuda", generator=s.g).bfloat16() for n in (2, 300))
    start = i32([0, 200, 300])
    want, wantx = c.decode(q), c.extend(qx, start, 200)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for i in range(20):
        got.append((c.decode(q, stream=a if i % 2 else a.cuda_stream), want))
        got.append((c.extend(qx, start, 200, stream=b), wantx))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in got)
    assert torch.equal(c.decode(q, stream=0), want)


def test_a_tight_length_bound_gives_the_same_rows():
    s = Server(num_q_heads=8, num_kv_heads=2, head_dim=64, num_pages=100, batch=2, max_seq_len=100000)
    s.add([1000, 333])
    q, qx = (torch.randn(n, 8, 64, device="cuda", generator=s.g).bfloat16() for n in (2, 50))
    c, start = s.c, i32([0, 40, 50])
    for bound in (None, 1000, 50000):
        ref, tol = R.attention(c.pages, c.scales, q, [0, 1], [999, 332], c.page_table.tolist(), c.kv_format, 0, 0)
        assert ((c.decode(q, max_seq_len=bound).double() - ref).abs() <= tol).all()
        pos = list(range(960, 1000)) + list(range(323, 333))
        ref, tol = R.attention(c.pages, c.scales, qx, [0] * 40 + [1] * 10, pos, c.page_table.tolist(), c.kv_format, 0, 0)
        assert ((c.extend(qx, start, 40, max_seq_len=bound).double() - ref).abs() <= tol).all()
    assert ok.oscar_device_errors(reset=True) == 0


@pytest.mark.parametrize("kept", [100, 96, 81, 80, 1])
def test_rejected_drafts_are_given_back_through_a_fork(kept):
    # 100 tokens, of which `kept` stay: the length is lowered, the sequence forked, the old one freed at its full length
    s = Server(num_q_heads=4, num_kv_heads=1, head_dim=64, num_pages=20, batch=3, max_seq_len=320, kv_format=R.INT8)
    c = s.c
    s.add([100, 30, 0])
    c.seq_lens[0] = kept
    c.fork(i32([0]), i32([2]), granted=c.granted)
    assert c.granted[0].item() == 1
    c.seq_lens[0] = 100
    c.free(i32([0]))
    assert c.seq_lens.tolist() == [0, 30, kept] and c.page_refs.sum().item() == -(-kept // 16) + 2
    assert c.page_refs.max().item() == 1
    s.check([0, 1, 1])
    s.add([0, 1, 40])
    s.check([0, 1, 7])
