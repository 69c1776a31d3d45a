"""What each form of oscar_kv8_decode_shared promises of a row, in 64 bits: the error that its own weights' bits and steps allow."""

import math

import torch

import kv8_ref as R

# Of a weight, relative to itself, and at worst, relative to the row's largest: half a step each.
# List: the decode's two fp16 parts.  Own tokens over tiles: fp16 (2^-11) of the weight times 2^6 and a maximum that lags upwards: a
# subnormal's half step 2^-25 2^-6.  Prefixes: the extend's (kv8_ref.attention_of_rows): fp16, and 2^-21 of the largest, where V scales are
# within 2^8 of one another; bf16 (2^-8), whose exponents reach further than weights do, in a block whose scales are not.  A block with scales
# near one another in a prefix that has others is held in one or the other.
LIST, OWN, TAME, WILD = (2.0 ** -22, 2.0 ** -50), (2.0 ** -11, 2.0 ** -31), (2.0 ** -11, 2.0 ** -21), (2.0 ** -8, 0.0)
EITHER = (WILD[0], TAME[1])
BLOCK = 8  # pages


def attend(q, k, v, scale, bits):
    """float64 (out, tolerance) of rows q [R][D] over k, v [n][D]; bits [n][2]: of the weight of each position.

    The output is bf16 (half a step, 2^-8 of itself; 2^-133 where it is subnormal).  Logits are fp32 sums of D exact products and three
    fp32 roundings, (D + 16) 2^-24 of sum |q k|, once in the numerator and once in the sum (nothing for a row's only position).
    Exponentials, fp32 sums over n positions and joins: 2^-20 + n 2^-24 of A = sum w |v| / sum w."""
    n, D = k.shape
    s = q @ k.T * scale
    w = torch.exp(s - s.amax(1, keepdim=True))
    total = w.sum(1, keepdim=True)
    w = w / total
    size = (q.abs() @ k.abs().T * scale).masked_fill(w == 0, 0)
    dlog = (D + 16) * 2.0 ** -24 * size.amax(1, keepdim=True) * ((w > 0).sum(1, keepdim=True) > 1)
    o, a = w @ v, w @ v.abs()
    tol = 2.0 ** -8 * o.abs() + 2.0 ** -133 + (2.0 ** -20 + n * 2.0 ** -24 + 2 * dlog) * a * 1.01
    tol += ((w * bits[:, 0]) @ v.abs()) * 1.01 + bits[:, 1][None] @ v.abs() / total
    return o, tol


def rows(codes, scales, q, b, length, table, fmt, shared, tiled):
    """(out, tolerance) [Hq][D] of sequence b, `shared` of whose tokens are attended with its group (`tiled`: over tiles)."""
    hq, D = q.shape[1:]
    H = codes.shape[1]
    ids = torch.as_tensor(table[b][:-(-length // R.P)], device=q.device).long()
    kv = codes[ids].view(torch.float8_e4m3fn if fmt == R.E4M3 else torch.int8).double() * scales[ids].double()[..., None, None]
    kv = kv.permute(1, 2, 0, 3, 4).reshape(H, 2, -1, D)[:, :, :length]
    out, tol = (torch.zeros(hq, D, dtype=torch.float64, device=q.device) for _ in range(2))
    for h in range(H):
        bits = torch.tensor(OWN if tiled else LIST, dtype=torch.float64, device=q.device).repeat(length, 1)
        if tiled and shared:
            vs = scales[ids[:shared // R.P], h, 1].tolist()
            tame = max(vs) <= 2 ** 8 * min(vs)
            for j in range(0, len(vs), BLOCK):
                blk = vs[j:j + BLOCK]
                kind = TAME if tame else WILD if max(blk) > 2 ** 8 * min(blk) else EITHER
                bits[j * R.P:(j + BLOCK) * R.P] = torch.tensor(kind, dtype=torch.float64, device=q.device)
            bits[shared:] = torch.tensor(OWN, dtype=torch.float64, device=q.device)
        at = slice(h * hq // H, (h + 1) * hq // H)
        out[at], tol[at] = attend(q[b, at].double(), kv[h, 0], kv[h, 1], 1 / math.sqrt(D), bits)
    return out, tol
