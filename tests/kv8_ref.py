"""Plain 64-bit reference of the 8-bit paged cache and of the page operations, written from
their definitions: element by element codes, dense attention with an explicit mask, a page
allocator in Python lists."""

import math

import numpy as np
import torch

P = 16
E4M3, INT8 = 0, 1
FMAX = (448.0, 127.0)
EXP_HI = (119, 121)


def _e4m3_table():
    out = np.empty(256)
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[c] = math.nan if (c & 127) == 127 else (-v if c & 128 else v)
    return out


E4M3_VALUES = _e4m3_table()


def code_values(codes, fmt):
    """uint8 numpy codes -> float64."""
    return E4M3_VALUES[codes] if fmt == E4M3 else codes.view(np.int8).astype(np.float64)


def encode(x, fmt):
    """float64 in units of the scale -> uint8 codes: the nearest value, ties to the even code, saturating."""
    if fmt == INT8:
        return np.clip(np.rint(x), -127, 127).astype(np.int8).view(np.uint8)
    pos = E4M3_VALUES[:127]
    a = np.minimum(np.abs(x), 448.0)
    hi = np.minimum(np.searchsorted(pos, a), 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (pick | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def scale_of(amax, fmt):
    """The smallest 2^e with amax <= M 2^e, by trial."""
    for e in range(-100, EXP_HI[fmt] + 1):
        if amax <= FMAX[fmt] * 2.0 ** e:
            return 2.0 ** e
    return 2.0 ** EXP_HI[fmt]


def append(codes, scales, k, v, t_start, table, lens, fmt):
    """In place on numpy codes [pages][H][2][P][D] uint8 and scales [pages][H][2] fp32; k, v float64 [T][H][D]."""
    for b, L in enumerate(lens):
        n = t_start[b + 1] - t_start[b]
        for j in range((L - n) // P, -(-L // P)) if n else ():
            page = table[b][j]
            o0, o1 = max(L - n - j * P, 0), min(L - j * P, P)
            t0 = t_start[b] + j * P + o0 - (L - n)
            for side, x in enumerate((k, v)):
                for h in range(codes.shape[1]):
                    blk = np.nan_to_num(x[t0:t0 + o1 - o0, h], nan=0.0, posinf=3.3895313892515355e38,
                                        neginf=-3.3895313892515355e38)
                    s = scale_of(np.abs(blk).max(), fmt)
                    old = float(scales[page, h, side])
                    if o0 and s <= old:
                        s = old
                    elif o0:
                        c = codes[page, h, side, :o0]
                        codes[page, h, side, :o0] = encode(code_values(c, fmt) * (old / s), fmt)
                    codes[page, h, side, o0:o1] = encode(blk / s, fmt)
                    scales[page, h, side] = s


def attention(codes, scales, q, row_seq, row_pos, table, fmt, sink, window, sm_scale=None):
    """float64 (out, tolerance) for bf16 rows q [R][Hq][D] at row_pos of row_seq (torch tensors, any device).

    The tolerance counts roundings: the weights may be held in bf16 (half a step 2^-8 each, so 2^-8 of
    A = sum w |v| / sum w), the output is bf16 (2^-8 of itself), logits are fp32 sums of D products
    (an error of d in a logit changes weights by a factor 1 + d, numerator and denominator).

    Weights held in fp16 have a smallest step.  Decode: two parts, a step of 2^-14 2^-12 2^-24 = 2^-50 of the largest
    weight beside them.  Extend: w 2^3 s / r, s the block's and r the largest V scale, has a step of 2^-24, so a
    weight is off by at most 2^-25 2^-3 r / s of one whose exponential is 1 (the sum has at least that); it
    meets |v| <= M s with M r < 2 max |v|, as a block's largest code is over M / 2: 2^-27 max |v| for each of n
    visible tokens.  There a V code c s' / s is held to a step of 2^-24 as well: 2^-25 r < 2^-31 max |v| once more
    (M / 2 > 2^5).  Both matter only where every larger weight meets a value of 0."""
    R, hq, D = q.shape
    H = codes.shape[1]
    out = torch.zeros(R, hq, D, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    scale = sm_scale if sm_scale else 1.0 / math.sqrt(D)
    as_type = torch.float8_e4m3fn if fmt == E4M3 else torch.int8
    for b in sorted(set(row_seq)):
        rows = [r for r in range(R) if row_seq[r] == b and row_pos[r] >= 0]
        if not rows:
            continue
        top = max(row_pos[r] for r in rows) + 1
        j = torch.arange(top, device=q.device)
        p = torch.tensor([row_pos[r] for r in rows], device=q.device)[:, None]
        see = j <= p
        if window:
            see &= (j < sink) | (j > p - window)
        used = see.any(0)
        ids = torch.as_tensor(table[b][:-(-top // P)], device=q.device).long()
        bad = (ids < 0) | (ids >= codes.shape[0])
        see &= ~bad.repeat_interleave(P)[:top]
        ids = torch.where(bad, 0, ids)
        kv = codes[ids].view(as_type).double() * scales[ids].double()[..., None, None]
        kv = kv.permute(1, 2, 0, 3, 4).reshape(H, 2, -1, D)[:, :, :top]
        kv = torch.where((used & see.any(0))[None, None, :, None], kv, 0.0)
        for h in range(hq):
            qq, kk, vv = q[rows, h].double(), kv[h * H // hq, 0], kv[h * H // hq, 1]
            s = (qq @ kk.T * scale).masked_fill(~see, -math.inf)
            w = torch.exp(s - s.amax(1, keepdim=True).clamp(min=-1e300))
            total = w.sum(1, keepdim=True).clamp(min=1e-300)
            o, a = w @ vv / total, w @ vv.abs() / total
            dlog = (D + 16) * 2.0 ** -24 * (qq.abs() @ kk.abs().T * scale).amax(1, keepdim=True)
            out[rows, h] = o
            tol[rows, h] = 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2.0 ** -12) * a + 2 * dlog * a + (see.sum(1, keepdim=True) + 1) * 2.0 ** -27 * vv.abs().max()
    return out, tol


class Pages:
    """The page allocator's state in Python: table rows of held entries, lengths, counts."""

    def __init__(self, num_pages, batch, max_pages):
        self.refs = [0] * num_pages
        self.table = [[-1] * max_pages for _ in range(batch)]
        self.lens = [0] * batch

    def held(self, b):
        return -(-self.lens[b] // P)

    def free_ids(self):
        return [i for i, r in enumerate(self.refs) if r == 0]

    def reserve(self, new):
        granted, asked, free = [], 0, self.free_ids()
        for b, n in enumerate(new):
            need = -(-(self.lens[b] + n) // P) - self.held(b)
            ok = need == 0 or asked + need <= len(free)
            if ok:
                for i in range(need):
                    self.table[b][self.held(b) + i] = free[asked + i]
                    self.refs[free[asked + i]] = 1
                self.lens[b] += n
            asked += need
            granted.append(int(ok))
        return granted

    def fork(self, src, dst):
        """Returns (granted, copies as (from, to) page pairs)."""
        granted, copies, asked, free = [], [], 0, self.free_ids()
        lens, B = list(self.lens), len(self.lens)
        for i, (s, d) in enumerate(zip(src, dst)):
            ok = 0 <= s < B and 0 <= d < B and s != d and lens[d] == 0 and d not in dst[:i]
            part = ok and lens[s] % P != 0 and self.table[s][lens[s] // P] >= 0
            if part and asked >= len(free):
                ok = False
            if ok:
                for j in range(lens[s] // P):
                    self.table[d][j] = self.table[s][j]
                    if self.table[s][j] >= 0:
                        self.refs[self.table[s][j]] += 1
                if lens[s] % P:
                    self.table[d][lens[s] // P] = free[asked] if part else -1
                if part:
                    self.refs[free[asked]] = 1
                    copies.append((self.table[s][lens[s] // P], free[asked]))
                self.lens[d] = lens[s]
            asked += bool(part)
            granted.append(int(ok))
        return granted, copies

    def _drop(self, b, j):
        if self.table[b][j] >= 0:
            self.refs[self.table[b][j]] -= 1
            self.table[b][j] = -1

    def free(self, seqs):
        for b in seqs:
            for j in range(self.held(b)):
                self._drop(b, j)
            self.lens[b] = 0

    def trim(self, sink, window):
        for b, L in enumerate(self.lens):
            for j in range(self.held(b)):
                if j * P >= sink and (j + 1) * P <= L - window:
                    self._drop(b, j)

    def compact(self):
        """Returns (pages in use, moves as (from, to) pairs)."""
        n = sum(r > 0 for r in self.refs)
        src = [i for i in range(n, len(self.refs)) if self.refs[i] > 0]
        dst = [i for i in range(n) if self.refs[i] == 0]
        moves = list(zip(src, dst))
        to = dict(moves)
        for b in range(len(self.lens)):
            for j in range(self.held(b)):
                self.table[b][j] = to.get(self.table[b][j], self.table[b][j])
        for s, d in moves:
            self.refs[d], self.refs[s] = self.refs[s], 0
        return n, moves


def attention_of_rows(codes, scales, q, row_seq, row_pos, table, fmt, sink, window, decode):
    """float64 (out, tolerance), the tolerance from what each row sees alone: a position that a row does not see, in
    the same page or in another, has no part in it.  A = sum w |v| / sum w over the visible positions, w = 1 for
    the largest logit.

    Both: the output is bf16 (half a step, 2^-8 of itself; 2^-133 where bf16 is subnormal), logits are fp32 sums of D
    exact products and three fp32 roundings, (D + 16) 2^-24 of sum |q k|, once in the numerator and once in the sum (of the
    positions that have a weight in 64 bits; a row's only one has the weight 1 whatever its logit is);
    exponentials and fp32 sums over n positions: 2^-20 + n 2^-24 of A.

    Decode: weights in two fp16 parts hold 2^-22 of themselves and at worst 2^-50 of the largest.
    Extend: weights as bf16 (2^-8 of themselves) where the V scales of pages are far apart; as fp16 (2^-11, less than
    that) where the largest so far is at most 2^8 times a block's smallest.  There w 2^4 s / r is what is held, r at
    most the largest w s so far, so r <= 2^8 s for every s in the block, and a step of 2^-24 leaves w off by 2^-25 r / (2^4
    s) <= 2^-21: of |v| at that position, whatever else is in its page."""
    R, hq, D = q.shape
    H = codes.shape[1]
    out = torch.zeros(R, hq, D, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    as_type = torch.float8_e4m3fn if fmt == E4M3 else torch.int8
    for b in sorted(set(row_seq)):
        rows = [r for r in range(R) if row_seq[r] == b and row_pos[r] >= 0]
        top = max(row_pos[r] for r in rows) + 1
        j = torch.arange(top, device=q.device)
        p = torch.tensor([row_pos[r] for r in rows], device=q.device)[:, None]
        see = j <= p
        if window:
            see &= (j < sink) | (j > p - window)
        ids = torch.as_tensor(table[b][:-(-top // P)], device=q.device).long().clamp(min=0)
        kv = codes[ids].view(as_type).double() * scales[ids].double()[..., None, None]
        kv = kv.permute(1, 2, 0, 3, 4).reshape(H, 2, -1, D)[:, :, :top]
        kv = torch.where(see.any(0)[None, None, :, None], kv, 0.0)
        n = see.sum(1, keepdim=True)
        for h in range(hq):
            qq, kk, vv = q[rows, h].double(), kv[h * H // hq, 0], kv[h * H // hq, 1]
            s = (qq @ kk.T / math.sqrt(D)).masked_fill(~see, -math.inf)
            w = torch.exp(s - s.amax(1, keepdim=True))
            total = w.sum(1, keepdim=True)
            w = w / total
            size = (qq.abs() @ kk.abs().T / math.sqrt(D)).masked_fill(w == 0, 0)
            dlog = (D + 16) * 2.0 ** -24 * size.amax(1, keepdim=True) * ((w > 0).sum(1, keepdim=True) > 1)
            o, a = w @ vv, w @ vv.abs()
            own, step = (2.0 ** -22, 2.0 ** -50) if decode else (2.0 ** -8, 2.0 ** -21)
            out[rows, h] = o
            tol[rows, h] = (2.0 ** -8 * o.abs() + 2.0 ** -133 + (own + 2.0 ** -20 + n * 2.0 ** -24 + 2 * dlog) * a * 1.01
                            + step / total * (see.double() @ vv.abs()))
    return out, tol


def cancelling_page(D, seed):
    """One int8 page whose values nearly cancel under the softmax of the query (1, 0, ...): (K codes of channel 0 [P], to
    be scaled by 2^-4; V codes [P][D]; exact weights [P] at sm_scale 1/8).  Tokens come in pairs of opposite signs, the
    second code the first times the quotient of their weights, rounded: the output is about 2^-9 of sum w |v|, so that its
    own rounding leaves the weights' errors to be seen."""
    g = np.random.default_rng(seed)
    k = -g.permutation(np.arange(3, 3 + 7 * P, 7))[:P]
    k = np.sort(k).reshape(2, P // 2).T.reshape(P)  # in each pair the first weighs less
    w = np.exp(k * 2.0 ** -4 / 8)
    c = g.integers(64, 128, (P // 2, D)) * g.choice([-1, 1], (P // 2, D))
    v = np.zeros((P, D))
    v[0::2], v[1::2] = c, -np.rint(c * (w[0::2] / w[1::2])[:, None])
    return k, v, w


def cancelling_tolerance(v, w):
    """Of the decode's output over a cancelling_page: it is bf16 (2^-8 of itself); weights in two fp16 parts hold 2^-22, exponentials
    2^-22, and their argument, one exact product, is rounded three times and subtracted from (4 2^-24 at |s| < 2), in the
    numerator and in the sum; 16 fp32 additions each: together below 2^-22 (1 + 1 + 2 + 2 + 4 + 4) of A = sum w |v| / sum w."""
    o, a = w @ v / w.sum(), w @ np.abs(v) / w.sum()
    return o, 2.0 ** -8 * np.abs(o) + 14 * 2.0 ** -22 * a
