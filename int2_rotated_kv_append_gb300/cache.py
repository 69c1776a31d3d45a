"""Device-side paged caches driven through the C ABI.

``Int2Cache`` owns the INT2 code pool, the fp16 scale/zero pool and the BF16
sink/window buffers of a workload; ``Bf16Cache`` owns the all-BF16 pool of the
speedup reference; ``Kv8Cache`` owns an 8-bit pool whose pages it manages itself
(reserve, fork, free, trim, compact), rotates keys on their way in and attends
shared prefixes once.  They only allocate torch memory and call the
library, as does ``calibrate`` (the offline step that produces R and the clipping
thresholds).

``Int2Cache`` and ``Bf16Cache`` have one workspace each: calls of one such cache are
made on one stream at a time.  ``Kv8Cache`` has one per stream.
"""

from __future__ import annotations

import contextlib
from typing import NamedTuple

import torch

from . import (OSCAR_KV8_E4M3, make_dims, oscar_append, oscar_append_mixed, oscar_bf16_append, oscar_bf16_decode,
               oscar_bf16_decode_workspace_bytes, oscar_calibrate, oscar_calibrate_workspace_bytes, oscar_decode,
               oscar_decode_workspace_bytes, oscar_extend, oscar_extend_varlen, oscar_extend_varlen_workspace_bytes,
               oscar_extend_workspace_bytes, oscar_kv8_append, oscar_kv8_decode, oscar_kv8_decode_shared,
               oscar_kv8_decode_shared_workspace_bytes, oscar_kv8_decode_workspace_bytes, oscar_kv8_extend_varlen,
               oscar_kv8_extend_varlen_workspace_bytes, oscar_kv8_rope_append, oscar_pages_compact, oscar_pages_fork,
               oscar_pages_free, oscar_pages_groups, oscar_pages_groups_workspace_bytes, oscar_pages_reserve,
               oscar_pages_trim, oscar_pages_workspace_bytes, oscar_rope, _stream)
from .synth import Workload

SENTINEL = 0xA5


def _allocating(device, stream):
    """The context in which what a call on ``stream`` uses is allocated."""
    if stream is None or device.type != "cuda":
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(stream)
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


class Int2Cache:
    def __init__(self, w: Workload, device="cuda", pages_per_split: int | None = None, fill: int = SENTINEL):
        self.w = w
        self.device = torch.device(device)
        H, D, P, G = w.num_kv_heads, w.head_dim, w.page_size, w.group_size
        self.dims = w.dims
        self.int2_pages = torch.full((w.num_pages * H * 2 * P * D // 4,), fill, dtype=torch.uint8,
                                     device=self.device)
        fill16 = fill * 0x101
        fill16 = fill16 - 0x10000 if fill16 >= 0x8000 else fill16
        self.scale_zero = torch.full((w.num_pages * H * 2 * P * (D // G) * 2,), fill16, dtype=torch.int16,
                                     device=self.device).view(torch.float16)
        self.page_table = w.page_table.to(self.device)
        self.seq_lens = w.seq_lens.to(self.device)
        self.R_k, self.R_v = w.R_k.to(self.device), w.R_v.to(self.device)
        self.clip_k, self.clip_v = w.clip_k.to(self.device), w.clip_v.to(self.device)
        self.offset_k = None if w.offset_k is None else w.offset_k.to(self.device).contiguous()
        self.pps = w.pages_per_split if pages_per_split is None else pages_per_split
        self.sink = None
        self.window = None
        self._ws = None

    def append(self, k, v, slot_mapping, stream=None, rope=None, positions=None):
        """With ``rope`` (a ``Rope``) the keys come without positions and are rotated by ``positions`` (int32 device [T])
        first; k may then be a slice of longer rows."""
        if rope is not None:
            if positions is None:
                raise ValueError("keys that are to be rotated have positions")
            with _allocating(self.device, stream):
                plain, k = k, torch.empty(k.shape, dtype=k.dtype, device=k.device)
            oscar_rope(self.dims, rope, positions, None, plain, None, k, stream)
        oscar_append(self.dims, k, v, self.R_k, self.R_v, self.clip_k, self.clip_v, self.page_table, slot_mapping,
                     self.int2_pages, self.scale_zero, stream, offset_k=self.offset_k)

    def prefill(self, stream=None):
        """Append every token of the workload and fill the BF16 sink/window buffers
        (with a key offset, both in one oscar_append_mixed call, which stores the
        offset keys in the BF16 rows)."""
        w = self.w
        if self.offset_k is not None:
            B, H, D = w.batch, w.num_kv_heads, w.head_dim
            self.sink = torch.zeros((B, 2, H, max(w.sink_len, 1), D), dtype=torch.bfloat16, device=self.device)
            self.window = torch.zeros((B, 2, H, max(w.window_len, 1), D), dtype=torch.bfloat16, device=self.device)
            d = self.device
            oscar_append_mixed(self.dims, w.k.to(d), w.v.to(d), self.R_k, self.R_v, self.clip_k, self.clip_v,
                               self.page_table, w.slot_mapping.to(d), w.tok_seq.to(d), w.tok_pos.to(d), self.seq_lens,
                               w.sink_len, w.window_len, self.int2_pages, self.scale_zero, self.sink, self.window,
                               stream, offset_k=self.offset_k)
            return
        self.append(w.k.to(self.device), w.v.to(self.device), w.slot_mapping.to(self.device), stream)
        sink, win = w.sink_window()
        self.sink, self.window = sink.to(self.device), win.to(self.device)

    def workspace(self, max_seq_len=None):
        w = self.w
        msl = w.max_seq_len if max_seq_len is None else max_seq_len
        nbytes = oscar_decode_workspace_bytes(self.dims, w.batch, msl, self.pps, w.sink_len, w.window_len)
        if nbytes == 0:
            raise ValueError("invalid decode arguments for workspace sizing")
        if self._ws is None or self._ws.numel() < nbytes:
            self._ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        return self._ws

    def decode(self, q, out=None, sm_scale=0.0, seq_lens=None, max_seq_len=None, stream=None):
        w = self.w
        msl = w.max_seq_len if max_seq_len is None else max_seq_len
        if out is None:
            out = torch.empty((w.batch, w.num_q_heads, w.head_dim), dtype=torch.float32, device=self.device)
        ws = self.workspace(msl)
        oscar_decode(self.dims, w.batch, msl, self.pps, q, self.R_k, self.R_v, self.int2_pages, self.scale_zero,
                     self.sink, self.window, self.page_table, self.seq_lens if seq_lens is None else seq_lens,
                     w.sink_len, w.window_len, sm_scale, out, ws, stream)
        return out


    def extend(self, q, row_seq, row_pos, out=None, sm_scale=0.0, max_seq_len=None, stream=None):
        """Causal attention of query rows q [rows][Hq][D]; row r belongs to sequence
        row_seq[r] at position row_pos[r] (int32 device tensors)."""
        w = self.w
        msl = w.max_seq_len if max_seq_len is None else max_seq_len
        rows = q.shape[0]
        if out is None:
            out = torch.empty((rows, w.num_q_heads, w.head_dim), dtype=torch.float32, device=self.device)
        nbytes = oscar_extend_workspace_bytes(self.dims, rows, msl, self.pps, w.sink_len, w.window_len)
        if nbytes == 0:
            raise ValueError("invalid extend arguments for workspace sizing")
        if self._ws is None or self._ws.numel() < nbytes:
            self._ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        oscar_extend(self.dims, w.batch, msl, self.pps, q, row_seq, row_pos, self.R_k, self.R_v, self.int2_pages,
                     self.scale_zero, self.sink, self.window, self.page_table, self.seq_lens, w.sink_len,
                     w.window_len, sm_scale, out, self._ws, stream)
        return out


    def extend_varlen(self, q, q_start, max_rows_per_seq, out=None, sm_scale=0.0, max_seq_len=None, stream=None):
        """Causal attention of the rows q [rows][Hq][D], rows q_start[b] .. q_start[b+1]-1
        being the last positions of sequence b (int32 device q_start [B+1])."""
        w = self.w
        msl = w.max_seq_len if max_seq_len is None else max_seq_len
        rows = q.shape[0]
        if out is None:
            out = torch.empty((rows, w.num_q_heads, w.head_dim), dtype=torch.float32, device=self.device)
        nbytes = oscar_extend_varlen_workspace_bytes(self.dims, rows, msl, self.pps, w.sink_len, w.window_len)
        if nbytes == 0:
            raise ValueError("invalid extend arguments for workspace sizing")
        if self._ws is None or self._ws.numel() < nbytes:
            self._ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        oscar_extend_varlen(self.dims, w.batch, msl, max_rows_per_seq, self.pps, q, q_start, self.R_k, self.R_v,
                            self.int2_pages, self.scale_zero, self.sink, self.window, self.page_table, self.seq_lens,
                            w.sink_len, w.window_len, sm_scale, out, self._ws, stream)
        return out


class Bf16Cache:
    def __init__(self, w: Workload, device="cuda", pages_per_split: int | None = None):
        self.w = w
        self.device = torch.device(device)
        self.dims = w.dims
        self.pages = torch.zeros((w.num_pages * w.num_kv_heads * 2 * w.page_size * w.head_dim,),
                                 dtype=torch.bfloat16, device=self.device)
        self.page_table = w.page_table.to(self.device)
        self.seq_lens = w.seq_lens.to(self.device)
        self.pps = w.pages_per_split if pages_per_split is None else pages_per_split
        self._ws = None

    def prefill(self, stream=None):
        w = self.w
        oscar_bf16_append(self.dims, w.k.to(self.device), w.v.to(self.device), w.slot_mapping.to(self.device),
                          self.pages, stream)

    def workspace(self):
        w = self.w
        nbytes = oscar_bf16_decode_workspace_bytes(self.dims, w.batch, w.max_seq_len, self.pps)
        if self._ws is None or self._ws.numel() < nbytes:
            self._ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        return self._ws

    def decode(self, q, out=None, sm_scale=0.0, stream=None):
        w = self.w
        if out is None:
            out = torch.empty((w.batch, w.num_q_heads, w.head_dim), dtype=torch.float32, device=self.device)
        oscar_bf16_decode(self.dims, w.batch, w.max_seq_len, self.pps, q, self.pages, self.page_table,
                          self.seq_lens, sm_scale, out, self.workspace(), stream)
        return out


class SharedPrefixes(NamedTuple):
    """Groups of sequences that share a prefix (int32 device tensors), as ``Kv8Cache.groups`` finds them."""

    members: torch.Tensor      # sequences, group after group
    group_start: torch.Tensor  # [groups + 1]
    prefix_lens: torch.Tensor  # [groups] tokens


class Kv8Cache:
    """An 8-bit paged cache for up to ``batch`` sequences of max_seq_len tokens (rounded up to whole
    pages of 16), with its page table, lengths and page counts.  With ``window_len`` >= 1 attention
    sees the last window_len positions and the first sink_len, and ``trim`` gives back the pages
    behind the window.

    Every method takes the stream of its call (a torch stream or a handle; None: the current one).
    Calls on different streams have workspaces of their own, so two that only read the cache may
    run at once; graphs captured on one stream share its workspace and are replayed one after
    another.  Outputs that a method makes belong to its stream."""

    def __init__(self, num_q_heads, num_kv_heads, head_dim, num_pages, batch, max_seq_len, kv_format=OSCAR_KV8_E4M3,
                 sink_len=0, window_len=0, device="cuda"):
        self.device = torch.device(device)
        self.batch, self.kv_format = batch, kv_format
        self.sink_len, self.window_len = sink_len, window_len
        self.dims = make_dims(num_q_heads, num_kv_heads, head_dim, 16, head_dim, num_pages, max(1, -(-max_seq_len // 16)))
        self.max_seq_len = 16 * self.dims.max_pages_per_seq  # what reserve grants, the attention sees
        d = self.device
        self.pages = torch.zeros((num_pages, num_kv_heads, 2, 16, head_dim), dtype=torch.uint8, device=d)
        self.scales = torch.zeros((num_pages, num_kv_heads, 2), dtype=torch.float32, device=d)
        self.page_table = torch.full((batch, self.dims.max_pages_per_seq), -1, dtype=torch.int32, device=d)
        self.seq_lens = torch.zeros(batch, dtype=torch.int32, device=d)
        self.page_refs = torch.zeros(num_pages, dtype=torch.int32, device=d)
        self.granted = torch.ones(batch, dtype=torch.int32, device=d)  # of the last reserve
        self._ws = {}  # by stream: the last one is used, smaller ones stay for captured graphs that point to them

    def _allocating(self, stream):
        return _allocating(self.device, stream)

    def _workspace(self, nbytes, stream):
        if nbytes == 0:
            raise ValueError("invalid arguments for workspace sizing")
        own = self._ws.setdefault(_stream(stream), [])
        if not own or own[-1].numel() < nbytes:
            with self._allocating(stream):
                own.append(torch.empty(nbytes, dtype=torch.uint8, device=self.device))
        return own[-1]

    def _output(self, q, stream):
        with self._allocating(stream):
            return torch.empty_like(q)

    def reserve(self, new_tokens, stream=None):
        """Pages for new_tokens[b] (int32 device [batch]) more tokens of each sequence; returns ``granted``."""
        oscar_pages_reserve(self.dims, new_tokens, self.page_table, self.seq_lens, self.page_refs, self.granted,
                            self._workspace(oscar_pages_workspace_bytes(self.dims, self.batch, 0), stream), stream)
        return self.granted

    def append(self, k, v, t_start, max_tokens_per_seq, stream=None):
        """Quantise the reserved tokens k, v [T][Hkv][D]; t_start int32 device [batch + 1].  Sequences that the
        last ``reserve`` refused are skipped and stay as they were."""
        oscar_kv8_append(self.dims, self.kv_format, self.batch, max_tokens_per_seq, k, v, t_start, self.page_table,
                         self.seq_lens, self.pages, self.scales, stream, granted=self.granted)

    def rope_append(self, q, k, v, rope, t_start, max_tokens_per_seq, q_out=None, positions=None, stream=None):
        """``append`` of keys that ``rope`` (a ``Rope``) rotates on the way, at their positions in the sequences or at
        ``positions`` (int32 device [T]); returns the rotated queries (``q_out``, which may be q; None where q is None).  q, k
        and v may be slices of one projection's rows."""
        if q is not None and q_out is None:
            with self._allocating(stream):
                q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        oscar_kv8_rope_append(self.dims, rope, self.kv_format, self.batch, max_tokens_per_seq, q, k, v, t_start, positions,
                              self.page_table, self.seq_lens, self.pages, self.scales, q_out, stream, granted=self.granted)
        return q_out

    def _bound(self, max_seq_len):
        if max_seq_len is None:
            return self.max_seq_len
        if not 0 <= max_seq_len <= self.max_seq_len:
            raise ValueError(f"max_seq_len is between 0 and the cache's {self.max_seq_len}")
        return max_seq_len

    def decode(self, q, out=None, sm_scale=0.0, pages_per_split=0, stream=None, max_seq_len=None):
        """One query row per sequence.  ``max_seq_len``: a bound on every length (None: the cache's room); the work is
        split for it, so a bound near the longest length is quicker than a large cache's room."""
        bound = self._bound(max_seq_len)
        if out is None:
            out = self._output(q, stream)
        ws = self._workspace(oscar_kv8_decode_workspace_bytes(self.dims, self.batch, bound, pages_per_split,
                                                              self.sink_len, self.window_len), stream)
        oscar_kv8_decode(self.dims, self.kv_format, self.batch, bound, pages_per_split, q, self.pages, self.scales,
                         self.page_table, self.seq_lens, self.sink_len, self.window_len, sm_scale, out, ws, stream)
        return out

    def groups(self, min_pages=1, max_groups=8, stream=None):
        """The sequences whose first min_pages pages are full and the same (as ``fork`` leaves them), max_groups - 1 groups of
        them at most, and the rest, which share nothing.  They hold while the sequences grow or end, until a slot that was freed is
        filled again: one call serves every layer of a step, and later steps that only append.  ``decode_shared`` is the quicker
        the nearer max_groups is to one more than there are."""
        with self._allocating(stream):
            new = lambda n: torch.empty(n, dtype=torch.int32, device=self.device)  # noqa: E731
            g = SharedPrefixes(new(self.batch), new(max_groups + 1), new(max_groups))
        oscar_pages_groups(self.dims, min_pages, self.page_table, self.seq_lens, *g,
                           self._workspace(oscar_pages_groups_workspace_bytes(self.dims, self.batch), stream), stream)
        return g

    def decode_shared(self, q, groups, out=None, sm_scale=0.0, stream=None, max_seq_len=None, max_prefix_len=None,
                      max_own_len=None):
        """``decode`` that attends what each group (a ``SharedPrefixes``) shares once for all its members, for caches without a
        window.  The bounds (None: max_seq_len's) size the work: on a group's prefix, of which more is attended by each
        member, and on what a member has behind it, of which more is cut off and flagged (of sequences in no group: on all they
        have).  Bounds near the truth make it up to twice as quick.  Rows of sequences that are no member are left as they are in
        ``out``, and mean nothing in an output made here."""
        if self.window_len:
            raise ValueError("decode_shared is for caches without a window")
        bound = self._bound(max_seq_len)
        prefix, own = (bound if x is None else x for x in (max_prefix_len, max_own_len))
        if not (0 <= prefix <= bound and 0 <= own <= bound):
            raise ValueError(f"bounds on parts of a sequence are between 0 and {bound}")
        if out is None:
            out = self._output(q, stream)
        ws = self._workspace(oscar_kv8_decode_shared_workspace_bytes(self.dims, self.batch, bound, prefix, own,
                                                                     groups.members.numel(), groups.prefix_lens.numel()),
                             stream)
        oscar_kv8_decode_shared(self.dims, self.kv_format, self.batch, bound, prefix, own, q, self.pages, self.scales,
                                self.page_table, self.seq_lens, *groups, sm_scale, out, ws, stream)
        return out

    def extend(self, q, q_start, max_rows_per_seq, out=None, sm_scale=0.0, pages_per_split=0, stream=None,
               max_seq_len=None):
        """The last rows of each sequence, q_start int32 device [batch + 1]; ``max_seq_len`` as in ``decode``."""
        bound = self._bound(max_seq_len)
        if out is None:
            out = self._output(q, stream)
        ws = self._workspace(oscar_kv8_extend_varlen_workspace_bytes(
            self.dims, self.batch, q.shape[0], bound, max_rows_per_seq, pages_per_split, self.sink_len,
            self.window_len), stream)
        oscar_kv8_extend_varlen(self.dims, self.kv_format, self.batch, bound, max_rows_per_seq, pages_per_split, q,
                                q_start, self.pages, self.scales, self.page_table, self.seq_lens, self.sink_len,
                                self.window_len, sm_scale, out, ws, stream)
        return out

    def fork(self, src_seq, dst_seq, granted=None, stream=None):
        oscar_pages_fork(self.dims, [self.pages, self.scales], src_seq, dst_seq, self.page_table, self.seq_lens,
                         self.page_refs, granted,
                         self._workspace(oscar_pages_workspace_bytes(self.dims, self.batch, src_seq.numel()), stream), stream)

    def free(self, seqs, stream=None):
        oscar_pages_free(self.dims, seqs, self.page_table, self.seq_lens, self.page_refs, stream)

    def trim(self, stream=None):
        oscar_pages_trim(self.dims, self.sink_len, self.window_len, self.page_table, self.seq_lens, self.page_refs,
                         stream)

    def compact(self, num_used=None, stream=None):
        oscar_pages_compact(self.dims, [self.pages, self.scales], self.page_table, self.seq_lens, self.page_refs,
                            num_used, self._workspace(oscar_pages_workspace_bytes(self.dims, self.batch, 0), stream), stream)


def calibrate(k=None, v=None, centered: bool = True, clip_quantile: float = 1.0, with_cov: bool = False,
              workspace=None, stream=None) -> dict:
    """R, clipping thresholds and eigenvalues per KV head from calibration samples
    (device bf16 [N][Hkv][D]); returns {"k": {...}, "v": {...}} for the sides given,
    each with R [Hkv][D][D], clip [Hkv][D], eigenvalues [Hkv][D], sweeps [Hkv] and,
    with ``with_cov``, cov [Hkv][D][D]."""
    x = k if k is not None else v
    if x is None:
        raise ValueError("calibrate needs k or v samples")
    N, H, D = x.shape
    dims = make_dims(H, H, D, 16, D, 1, 1)
    dev = x.device

    def outputs():
        o = {"R": torch.empty(H, D, D, dtype=torch.float32, device=dev),
             "clip": torch.empty(H, D, dtype=torch.float32, device=dev),
             "eigenvalues": torch.empty(H, D, dtype=torch.float32, device=dev),
             "sweeps": torch.empty(H, dtype=torch.int32, device=dev)}
        if with_cov:
            o["cov"] = torch.empty(H, D, D, dtype=torch.float32, device=dev)
        return o

    out_k = outputs() if k is not None else None
    out_v = outputs() if v is not None else None
    if workspace is None:
        workspace = torch.empty(oscar_calibrate_workspace_bytes(dims, N), dtype=torch.uint8, device=dev)
    oscar_calibrate(dims, N, k, v, int(centered), clip_quantile, out_k, out_v, workspace, stream)
    res = {}
    if out_k is not None:
        res["k"] = out_k
    if out_v is not None:
        res["v"] = out_v
    return res
