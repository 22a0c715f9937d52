"""Shared inputs of the windowed-attention and 4-bit cache tests."""

from __future__ import annotations

import numpy as np

from _longctx import HALF_STEP, Paged, stored
from oracle import decode_kv
from oracle import window as ow
from oracle.paged_attention import _gather_sequence


def packed_pairs(pairs, dtype):
    return stored(pairs, dtype)


class Windowed:
    """A paged cache of any type (``Paged``; ``u4``: its rows quantised by the oracle, random codes
    and NaN pairs in every other row) whose tokens hidden from every query hold NaN, and whose
    blocks without a visible token are named -9 in the table."""

    def __init__(self, lens, hkv, d, kv, window, sinks, seed=0, q=None, g=1, cols=1, counts=None,
                 std=1.0):
        base = Paged(lens, hkv, d, q if kv == "u4" else kv, seed=seed, cols=cols, q=q, g=g, std=std)
        self.__dict__.update(base.__dict__)
        self.kv, self.window, self.sinks = kv, window, sinks
        rng = np.random.default_rng(seed + 1000)
        self.counts = [min(1, n) for n in lens] if counts is None else list(counts)
        if counts is not None:
            self.q = stored(rng.standard_normal((sum(counts), hkv * g, d)), self.qt)
        self.cu = np.concatenate([[0], np.cumsum(self.counts)]).astype(np.int32)
        seen = np.zeros((len(self.k), 16), bool)
        keep_tables = self.tables.copy()
        for b, (n, length) in enumerate(zip(self.counts, self.lens.tolist())):
            tokens = set()
            for i in range(n):
                tokens.update(ow.visible(length - n + i, length, window, sinks))
            blocks = {t // 16 for t in tokens}
            for t in tokens:
                seen[self.tables[b, t // 16], t % 16] = True
            for j in range(-(-length // 16)):
                if j not in blocks:
                    keep_tables[b, j] = -9
        self.seen, self.true_tables = seen, self.tables
        self.tables = keep_tables
        hide = ~seen[:, None, :, None]
        self.pairs = [None, None]
        if kv == "u4":
            caches = []
            for i, x in enumerate((self.k, self.v)):
                codes, pairs = np.zeros(x.shape, np.uint8), np.zeros(x.shape[:3] + (2,))
                rows = np.broadcast_to(seen[:, None], x.shape[:3])
                codes[rows], pairs[rows] = ow.u4_quantise(x[rows])
                self.pairs[i] = (codes, pairs)
                junk = rng.integers(0, 256, x.shape[:3] + (d // 2,)).astype(np.uint8)
                caches.append(np.where(hide, junk, ow.u4_pack(codes)))
                pairs = np.where(hide, np.nan, pairs)
                if i:
                    self.v_scales = stored(pairs, self.qt)
                else:
                    self.k_scales = stored(pairs, self.qt)
            self.k, self.v = caches
        elif kv != "i8":
            nan = np.uint16(0x7FC0) if kv == "bf16" else np.float16(np.nan)
            # NaN keys and infinite values
            inf = np.uint16(0x7F80) if kv == "bf16" else np.float16(np.inf)
            self.k = np.where(hide, nan, self.k).astype(self.k.dtype)
            self.v = np.where(hide, np.where(rng.random(self.v.shape) < 0.5, nan, inf),
                              self.v).astype(self.v.dtype)

    def sequences(self):
        """Per sequence: k, v, k_size, v_size float64 [L, Hkv, D] (hidden rows 0)."""
        ks, vs, kz, vz = [], [], [], []
        for b, length in enumerate(self.lens.tolist()):
            at = [(self.true_tables[b, t // 16], t % 16) for t in range(length)]
            blk = np.array([x[0] for x in at], np.int64)
            row = np.array([x[1] for x in at], np.int64)
            for i, (full, size) in enumerate(((ks, kz), (vs, vz))):
                if self.kv == "u4":
                    codes, pairs = self.pairs[i]
                    c, s = codes[blk, :, row], pairs[blk, :, row]
                    full.append(ow.u4_values(c, s))
                    size.append(c * s[..., :1] + np.abs(s[..., 1:]))
                else:
                    x = _gather_sequence(self.v if i else self.k,
                                         self.v_scales if i else self.k_scales,
                                         self.true_tables, b, length, 16)
                    x = np.where(self.seen[blk, row][:, None, None], x, 0.0)
                    full.append(x)
                    size.append(np.abs(x))
        return ks, vs, kz, vz

    def expect(self, one_part=False):
        """(exact output, its tolerance), rows by query (decode: by sequence, empty ones zero)."""
        k, v, kz, vz = self.sequences()
        q = self.q
        if len(q) != sum(self.counts):      # decode: a row for every sequence
            q = q[[b for b, n in enumerate(self.counts) if n]]
        want, size, dots, most = ow.window_attention(q, k, v, self.counts, self.lens.tolist(),
                                                     self.scale, self.window, self.sinks, kz, vz)
        tol = tolerance(self, want, size, dots, most, one_part)
        if len(q) != len(self.q):
            full = np.zeros(self.q.shape), np.full(self.q.shape, 1e-30)
            live = [b for b, n in enumerate(self.counts) if n]
            full[0][live], full[1][live] = want, tol
            return full
        return want, tol

    def gpu(self):
        import torch
        from _pkv_helpers import to_dev
        names = ("k", "v", "q", "tables", "lens", "k_scales", "v_scales", "cu")
        t = {n: None if getattr(self, n) is None else to_dev(getattr(self, n)) for n in names}
        t["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        t["out"] = torch.full(self.q.shape, float("nan"), device="cuda").to(t["q"].dtype)
        return t


def tolerance(case, want, size, dots, tokens, one_part=False):
    """Bound of |kernel - exact| by counting roundings, as in ``_longctx.attention_tolerance``.

    4-bit rows: ``size`` and ``dots`` are sums of the parts' magnitudes, c s and |lo|, since both
    parts are summed apart. A score takes a chain of at most 4 products of 16 terms, the sum of a
    head's q (at most 40 fp32 additions) and 5 more roundings; the sum of P lo over the tokens
    adds a rounding per token and lane, within `steps`. fp16 parts of P s 2^-e, 2^-e >= 2^12 /
    max s, are off by up to 2^-25 below 2^-14: 2^-37 15 max s a token.
    ``one_part``: weights in one fp16 part (2^-11) where bf16 caches usually have two, and values
    in fp16: off by 2^-25, or, where the largest is below 2^-8, by 2^-39 of it."""
    codes = case.kv in ("i8", "u4")
    p = {"bf16": 2.0 ** -16, "f16": 2.0 ** -21}[case.kv] if not codes else (
        2.0 ** -21 if case.qt == "f16" else 2.0 ** -11)
    if one_part:
        p = 2.0 ** -11
    score = abs(case.scale) * dots * (4 * 17 + 3 + (25 if case.kv == "u4" else 0)) * 2.0 ** -23
    steps = 2 * (tokens / 16 + 4) * 17 * 2.0 ** -23
    weight = 2 * score + 2.0 ** -20 + p + steps
    tiny = 0.0
    if one_part and case.kv == "bf16":
        top = float(np.abs(case.sequences()[1][0]).max()) if hasattr(case, "sequences") else 1.0
        tiny = min(2.0 ** -25, 2.0 ** -17 * top)
    if case.kv == "f16":
        tiny = tokens * 2.0 ** -25 * float(np.nanmax(np.abs(np.where(
            np.isinf(case.v), 0, case.v).astype(np.float64))))
    elif case.kv == "i8":
        tiny = tokens * 2.0 ** -37 * 127 * float(np.nanmax(case.v_scales))
    elif case.kv == "u4":
        tiny = tokens * 2.0 ** -37 * 15 * float(case.pairs[1][1][..., 0].max())
    return HALF_STEP[case.qt] * np.abs(want) + weight[..., None] * size * 1.01 + tiny + 1e-30


def close(got, want, tol):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], got[bad][:4], want[bad][:4],
                           tol[bad][:4])


__all__ = ["Windowed", "close", "tolerance", "decode_kv"]
