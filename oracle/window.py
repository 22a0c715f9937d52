"""Oracle of windowed attention and of the 4-bit cache, in float64 from their definitions.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

* ``u4_quantise``   a 16-bit row x: lo = min x, s = the smallest value of its type not below
  fl32(fl32(max - lo) / 15), or the one below that where fl32(15 s + lo) passes the type's
  largest value, code = rne(fl32(x - lo) / s) with the exact quotient.
* ``u4_values``   code s + lo.
* ``visible``   the tokens that a query at position p sees: t <= p and (no window, or t > p -
  window, or t < sinks).
* ``window_attention``   softmax attention of runs of queries over what each sees.
"""

from __future__ import annotations

from fractions import Fraction

import numpy as np

from .paged_attention import decode_kv


def _sixteen_bit_up(x: float, bf16: bool) -> float:
    """The smallest bf16 / fp16 value not below the float32 x >= 0."""
    if x == 0:
        return 0.0
    if bf16:
        bits = int(np.float32(x).view(np.uint32))
        bits = -(-bits // 65536) * 65536
        return float(np.uint32(bits).view(np.float32))
    _, e = np.frexp(np.float64(x))
    ulp = 2.0 ** max(int(e) - 11, -24)
    return float(np.ceil(np.float64(x) / ulp) * ulp)


# the largest value of the type, and what fp32 still rounds to it (half a step, to even)
_MOST = {True: (255 * 2**120, 2**103), False: (65504, Fraction(1, 512))}


def _sixteen_bit_below(s: float, bf16: bool) -> float:
    """The bf16 / fp16 value next below s > 0."""
    if bf16:
        return float(np.uint32(int(np.float32(s).view(np.uint32)) - 65536).view(np.float32))
    return float((np.float16(s).view(np.uint16) - np.uint16(1)).view(np.float16))


def u4_quantise(x):
    """Stored rows [..., D] (uint16: bf16 bits, float16) -> codes [..., D] uint8, pairs [..., 2]
    float64 (s, lo)."""
    bf16 = x.dtype == np.uint16
    f = decode_kv(x).astype(np.float32)
    flat = f.reshape(-1, f.shape[-1])
    codes = np.zeros(flat.shape, np.uint8)
    pairs = np.zeros((len(flat), 2))
    for r, row in enumerate(flat):
        lo, hi = row.min(), row.max()
        s = _sixteen_bit_up(float(np.float32(hi - lo) / np.float32(15)), bf16)
        most, half = _MOST[bf16]
        if s and 15 * Fraction(s) + Fraction(float(lo)) > most + half:
            s = _sixteen_bit_below(s, bf16)
        pairs[r] = s, lo
        if s:
            for i, d in enumerate(row - lo):
                codes[r, i] = round(Fraction(float(d)) / Fraction(s))    # ties to even, exact
    return codes.reshape(f.shape), pairs.reshape(f.shape[:-1] + (2,))


def u4_pack(codes):
    """Codes [..., D] -> bytes [..., D / 2], the even channel low."""
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def u4_values(codes, pairs):
    return codes.astype(np.float64) * pairs[..., :1] + pairs[..., 1:]


def visible(p, length, window, sinks):
    return [t for t in range(min(p + 1, length))
            if window == 0 or t > p - window or t < sinks]


def window_attention(q, k, v, counts, lens, scale, window, sinks, k_size=None, v_size=None):
    """Attention of counts[b] queries of sequence b, the last at position lens[b] - 1.

    q [total, Hq, D] stored; k, v: lists of float64 [lens[b], Hkv, D]; k_size, v_size: the same
    shapes, what |k| and |v| are made of (None: |k|, |v|). Returns (out, sum_t p_t v_size_t,
    max_t sum_d |q_d| k_size_td, largest number of visible tokens) in float64."""
    qf = decode_kv(q)
    total, Hq, D = q.shape
    out, size, dots = np.zeros((total, Hq, D)), np.zeros((total, Hq, D)), np.zeros((total, Hq))
    at = most = 0
    for b, (n, length) in enumerate(zip(counts, lens)):
        ks = np.abs(k[b]) if k_size is None else k_size[b]
        vs = np.abs(v[b]) if v_size is None else v_size[b]
        g = Hq // k[b].shape[1]
        for i in range(n):
            t = np.array(visible(length - n + i, length, window, sinks), np.int64)
            most = max(most, len(t))
            for h in range(Hq if len(t) else 0):
                e = float(scale) * (k[b][t, h // g] @ qf[at + i, h])
                w = np.exp(e - e.max())
                w /= w.sum()
                out[at + i, h] = w @ v[b][t, h // g]
                size[at + i, h] = w @ vs[t, h // g]
                dots[at + i, h] = (ks[t, h // g] @ np.abs(qf[at + i, h])).max()
        at += n
    return out, size, dots, most
