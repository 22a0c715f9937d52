"""Oracle of the long-context operators, in float64 from their definitions.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

* ``qk_norm_rope``   y = x w / sqrt(mean x^2 + eps), then pairs of y turn by
  their axis's angle.
* ``block_bounds``, ``block_scores``   channel-wise min / max of a block's
  valid keys; max over the group's heads of sum_d max(q lo, q hi).
* ``choose``   the first, the last and the largest of a row, ascending, equal
  values to the lowest index, NaN lowest.
* ``listed_attention``, ``attention_mass``   softmax attention over listed
  blocks; the softmax weight of every token summed over a group's heads.
* ``evict``   the chosen rows of every (sequence, kv head) compacted; INT8
  codes are re-expressed under the largest scale of the rows of a tile, in
  float32 as the append rule does.
"""

from __future__ import annotations

import numpy as np

from .append import requantize_int8
from .paged_attention import _gather_sequence, decode_kv


def qk_norm_rope(x, weight, eps, cos_sin, positions, pair_axis, interleaved):
    """x [N, H, D] (stored bits) -> float64 rows. ``weight`` None: no norm; ``cos_sin`` None: no
    rotation. positions [axes, N]; pair_axis [rot / 2] or None."""
    y = decode_kv(x)
    D = y.shape[-1]
    if weight is not None:
        y = y / np.sqrt((y * y).sum(-1, keepdims=True) / D + eps) * decode_kv(weight)
    if cos_sin is None:
        return y
    rot = cos_sin.shape[1]
    out = y.copy()
    for j in range(rot // 2):
        axis = 0 if pair_axis is None else pair_axis[j]
        rows = cos_sin[positions[axis]].astype(np.float64)
        c, s = rows[:, j, None], rows[:, rot // 2 + j, None]
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)
        u, v = y[..., a], y[..., b]
        out[..., a], out[..., b] = u * c - v * s, u * s + v * c
    return out


def block_bounds(k_cache, block, valid):
    """(min, max) of rows [0, valid) of a block, per kv head: float64 [Hkv, 2, D]."""
    rows = decode_kv(k_cache[block, :, :valid, :])
    return np.stack([rows.min(1), rows.max(1)], 1)


def block_scores(q, bounds, block_tables, context_lens, k_scales=None):
    """float64 [B, Hkv, MB], -inf past a sequence's end, and the sums of absolute terms."""
    B, Hq, D = q.shape
    Hkv, MB = bounds.shape[1], block_tables.shape[1]
    g = Hq // Hkv
    out = np.full((B, Hkv, MB), -np.inf)
    size = np.zeros((B, Hkv, MB))
    for b in range(B):
        n = -(-int(context_lens[b]) // 16)
        box = decode_kv(bounds[block_tables[b, :n]])               # [n, Hkv, 2, D]
        qb = decode_kv(q[b]).reshape(Hkv, g, D)
        for h in range(Hkv):
            s = np.ones(n) if k_scales is None else k_scales[block_tables[b, :n],
                    h].astype(np.float64)
            for i in range(g):
                terms = np.maximum(qb[h, i] * box[:, h, 0], qb[h, i] * box[:, h, 1])
                out[b, h, :n] = np.maximum(out[b, h, :n], terms.sum(-1) * s)
                size[b, h, :n] = np.maximum(size[b, h, :n], np.abs(terms).sum(-1) * s)
    return out, size


def choose(row, keep_first, keep_last, budget):
    """Ascending indices of the min(len(row), budget) kept values of a float32 row."""
    n = len(row)
    if n <= budget:
        return np.arange(n)
    forced = np.zeros(n, bool)
    forced[:keep_first] = True
    forced[n - keep_last:] = True
    rest = [i for i in range(n) if not forced[i]]
    # NaN below everything; sorted() is stable, so equal values keep their order
    rank = sorted(rest, key=lambda i: (bool(np.isnan(row[i])), -row[i] if not np.isnan(row[i])
                                       else 0.0))
    kept = [i for i in range(n) if forced[i]] + rank[:budget - int(forced.sum())]
    return np.array(sorted(kept))


def _softmax(scores):
    if scores.shape[0] == 0:
        return scores
    w = np.exp(scores - scores.max(0))
    return w / w.sum(0)


def listed_attention(q, k_cache, v_cache, block_tables, context_lens, lists, list_lens, scale,
                     k_scales=None, v_scales=None):
    """Attention of each query head over the listed blocks of its kv head (a block listed twice
    counts twice). Returns (out, sum_t p_t |v_t|, max_t sum_d |q_d k_td|) in float64."""
    B, Hq, D = q.shape
    Hkv = k_cache.shape[1]
    g = Hq // Hkv
    out, size, dots = np.zeros((B, Hq, D)), np.zeros((B, Hq, D)), np.zeros((B, Hq))
    for b in range(B):
        L = int(context_lens[b])
        K = _gather_sequence(k_cache, k_scales, block_tables, b, L, 16)
        V = _gather_sequence(v_cache, v_scales, block_tables, b, L, 16)
        qb = decode_kv(q[b])
        for h in range(Hkv):
            at = np.array([t for e in lists[b, h, :list_lens[b]]
                           for t in range(16 * e, min(16 * e + 16, L))], np.int64)
            if at.size == 0:
                continue
            k, v = K[at, h], V[at, h]
            for i in range(h * g, h * g + g):
                w = _softmax(float(scale) * (k @ qb[i]))
                out[b, i], size[b, i] = w @ v, w @ np.abs(v)
                dots[b, i] = (np.abs(k) @ np.abs(qb[i])).max()
    return out, size, dots


def attention_mass(q, k_cache, block_tables, context_lens, scale, k_scales=None):
    """Softmax weights summed over each kv head's query heads: float64 [B, Hkv, MB * 16]."""
    B, Hq, _ = q.shape
    Hkv, MB = k_cache.shape[1], block_tables.shape[1]
    g = Hq // Hkv
    mass = np.zeros((B, Hkv, MB * 16))
    for b in range(B):
        L = int(context_lens[b])
        K = _gather_sequence(k_cache, k_scales, block_tables, b, L, 16)
        qb = decode_kv(q[b]).reshape(Hkv, g, -1)
        for h in range(Hkv):
            mass[b, h, :L] = _softmax(float(scale) * (K[:, h] @ qb[h].T)).sum(1) if L else 0.0
    return mass


def evict(k_cache, v_cache, block_tables, context_lens, mass, keep_first, keep_last, budget,
          new_tables, k_scales=None, v_scales=None):
    """New (k, v, k_scales, v_scales, kept, new_lens, new_mass); the inputs are left alone."""
    B, Hkv = mass.shape[:2]
    caches = [k_cache.copy(), v_cache.copy()]
    scales = [None if s is None else s.copy() for s in (k_scales, v_scales)]
    kept = np.full((B, Hkv, budget), -1, np.int32)
    new_mass = np.zeros((B, Hkv, new_tables.shape[1] * 16), np.float32)
    new_lens = np.minimum(context_lens, budget).astype(np.int32)
    for b in range(B):
        for h in range(Hkv):
            at = choose(mass[b, h, :context_lens[b]], keep_first, keep_last, budget)
            kept[b, h, :len(at)] = at
            new_mass[b, h, :len(at)] = mass[b, h, at]
            src = block_tables[b, at // 16]
            for r0 in range(0, len(at), 16):
                dst, rows = new_tables[b, r0 // 16], np.arange(r0, min(r0 + 16, len(at)))
                if all(src[r] == dst and at[r] % 16 == r % 16 for r in rows):
                    continue
                for new, old, s_new, s_old in zip(caches, (k_cache, v_cache), scales,
                                                  (k_scales, v_scales)):
                    x = old[src[rows], h, at[rows] % 16]
                    if s_old is not None:
                        s = s_old[src[rows], h]
                        top = s.max()
                        if top > 0:
                            x = np.stack([requantize_int8(c, a, top) if a != top else c
                                          for c, a in zip(x, s)])
                        s_new[dst, h] = top
                    new[dst, h, rows % 16] = x
    return caches[0], caches[1], scales[0], scales[1], kept, new_lens, new_mass
