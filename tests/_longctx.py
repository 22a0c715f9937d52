"""Shared inputs of the long-context operators' tests: a scattered paged cache
with garbage in every row that no sequence owns, on the host and on the GPU."""

from __future__ import annotations

import numpy as np

from _pkv_helpers import to_dev
from paged_kv_decode_05_gb300.workloads import f32_to_bf16_bits

HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def stored(x, dtype):
    x = np.asarray(x, np.float32)
    return f32_to_bf16_bits(x) if dtype == "bf16" else x.astype(np.float16)


class Paged:
    """Sequences of the given lengths over a shuffled pool. Rows past a sequence's end, unused
    blocks and the scales of unused blocks hold NaN (INT8 codes: -128 and 127). ``more``: free
    blocks per sequence in ``new_tables``."""

    def __init__(self, lens, hkv, d, kv, seed=0, more=0, cols=1, q=None, g=1, std=1.0):
        rng = np.random.default_rng(seed)
        self.rng, self.hkv, self.d, self.kv, self.g = rng, hkv, d, kv, g
        self.qt = q or ("bf16" if kv == "i8" else kv)
        self.lens = np.asarray(lens, np.int32)
        nb = -(-self.lens // 16)
        self.mb = int(nb.max(initial=0)) + cols
        total = int(nb.sum()) + len(lens) * more + 3
        perm = rng.permutation(total).astype(np.int32)
        self.tables = np.full((len(lens), self.mb), -7, np.int32)      # never read past the end
        at = 0
        for b, n in enumerate(nb):
            self.tables[b, :n] = perm[at:at + n]
            at += n
        self.new_tables = perm[at:at + len(lens) * more].reshape(len(lens), more).copy()
        shape = (total, hkv, 16, d)
        live = np.zeros((total, 16), bool)
        for b, n in enumerate(self.lens):
            for j in range(int(nb[b])):
                live[self.tables[b, j], :min(16, n - 16 * j)] = True
        self.live = live
        mask = np.broadcast_to(live[:, None, :, None], shape)
        self.k_scales = self.v_scales = None
        if kv == "i8":
            def codes():
                x = np.clip(np.rint(rng.standard_normal(shape) * 42), -127, 127)
                junk = np.where(rng.random(shape) < 0.5, -128, 127)
                return np.where(mask, x, junk).astype(np.int8)
            self.k, self.v = codes(), codes()
            used = live.any(1)[:, None]

            def scales():
                s = (0.01 + 0.02 * rng.random(shape[:2])) * std
                return np.where(used, s, np.nan).astype(np.float32)
            self.k_scales, self.v_scales = scales(), scales()
        else:
            nan = np.uint16(0x7FC0) if kv == "bf16" else np.float16(np.nan)
            x = [stored(rng.standard_normal(shape) * std, kv) for _ in range(2)]
            self.k, self.v = (np.where(mask, a, nan).astype(a.dtype) for a in x)
        self.q = stored(rng.standard_normal((len(lens), hkv * g, d)), self.qt)
        self.scale = d ** -0.5

    def bounds(self):
        """Oracle bounds of every used block (others NaN or junk), in the cache's type."""
        out = np.zeros((len(self.k), self.hkv, 2, self.d), self.k.dtype)
        for blk in range(len(self.k)):
            n = int(self.live[blk].sum())
            if n:
                rows = self.k[blk, :, :n]
                x = rows if rows.dtype != np.uint16 else (rows.astype(np.uint32) << 16).view(
                    np.float32)
                for i, r in enumerate((x.argmin(1), x.argmax(1))):
                    out[blk, :, i] = np.take_along_axis(rows, r[:, None], 1)[:, 0]
        return out

    def gpu(self):
        import torch
        names = ("k", "v", "q", "tables", "lens", "k_scales", "v_scales", "new_tables")
        t = {n: None if getattr(self, n) is None else to_dev(getattr(self, n)) for n in names}
        t["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        t["out"] = torch.full(self.q.shape, float("nan"), device="cuda").to(t["q"].dtype)
        return t


def attention_tolerance(case, want, size, dots, tokens):
    """Bound of |kernel - exact| for outputs sum_t p_t v_t, by counting roundings.

    * the output's rounding: half a step of its type, relative to the value;
    * a weight: its score is a chain of at most 4 tensor-core products of 16
      terms, each cut off within 17 units of 2^-23 of the terms' absolute sum
      (dots), plus 3 fp32 roundings; exp2 within 2^-21; P in 16-bit parts within
      2^-16 (bf16 hi + lo), 2^-21 (fp16 hi + lo) or 2^-11 (one fp16 part, INT8
      under a bf16 output);
    * the sums over tokens: one product of 16 terms per 16 tokens and part, 17
      units of 2^-23 of what was summed so far, and as much for l, plus one
      rounding per rescaling, which the same count covers.
    * fp16 parts of P below fp16's normal range (2^-14): each is off by up to
      2^-25 in P's own units, whatever the weight. 16-bit caches keep P in
      [0, 1], so a token adds at most 2^-25 max|v| (l >= 1: the largest score's
      weight is 1). INT8 codes meet P v_scale 2^-e, with 2^-e >= 2^12 /
      max v_scale, so a token adds at most 2^-25 2^-12 127 max v_scale.
    INT8 under a bf16 query: q enters in fp16, exact but for values below 2^-14,
    which round by at most 2^-25 (dots of the codes: 127 scale d at most, within
    the score bound at these scales).
    """
    p = {"bf16": 2.0 ** -16, "f16": 2.0 ** -21}[case.kv] if case.kv != "i8" else (
        2.0 ** -21 if case.qt == "f16" else 2.0 ** -11)
    score = abs(case.scale) * dots * (4 * 17 + 3) * 2.0 ** -23
    steps = 2 * (tokens / 16 + 4) * 17 * 2.0 ** -23
    weight = 2 * score + 2.0 ** -20 + p + steps
    tiny = 0.0
    if case.kv == "f16":
        tiny = tokens * 2.0 ** -25 * float(np.nanmax(np.abs(case.v.astype(np.float64))))
    elif case.kv == "i8":
        tiny = tokens * 2.0 ** -37 * 127 * float(np.nanmax(case.v_scales))
    return HALF_STEP[case.qt] * np.abs(want) + weight[..., None] * size * 1.01 + tiny + 1e-30
