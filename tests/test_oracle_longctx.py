"""Pins of the long-context oracle (``oracle/longctx.py``), CPU only."""

import numpy as np
import pytest

import oracle
from oracle import longctx as lc


def test_rotation_keeps_length_and_relative_angle():
    """<R(a) x, R(b) y> depends on a - b alone, and |R(a) x| = |x|."""
    rng = np.random.default_rng(0)
    D, half = 16, 8
    ang = np.arange(64)[:, None] * 10.0 ** (-np.arange(half) / half)
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    x, y = rng.standard_normal((2, 1, 1, D))
    for inter in (False, True):
        def turn(v, p):
            return lc.qk_norm_rope(v, None, 0.0, table, np.array([[p]]), None, inter)
        assert np.allclose((turn(x, 5) ** 2).sum(), (x ** 2).sum())
        a = (turn(x, 7) * turn(y, 3)).sum()
        assert np.allclose(a, (turn(x, 44) * turn(y, 40)).sum())
        assert not np.allclose(a, (turn(x, 7) * turn(y, 4)).sum())


def test_axes_turn_their_own_pairs():
    D, half = 8, 2                              # pairs (0, 2) and (1, 3); dims 4..7 stay
    table = np.array([[1.0, 1.0, 0.0, 0.0], [0.0, 0.0, 1.0, 1.0]])   # angles 0 and 90 degrees
    x = np.arange(1.0, 9.0).reshape(1, 1, D)
    y = lc.qk_norm_rope(x, None, 0.0, table, np.array([[0], [1]]), [0, 1], False)[0, 0]
    assert np.allclose(y, [1, -4, 3, 2, 5, 6, 7, 8])
    y = lc.qk_norm_rope(x, None, 0.0, table, np.array([[1], [0]]), [0, 1], True)[0, 0]
    assert np.allclose(y, [-2, 1, 3, 4, 5, 6, 7, 8])
    assert half == 2


def test_norm_of_a_constant_row():
    y = lc.qk_norm_rope(np.full((1, 1, 4), 3.0), np.array([1.0, 2.0, 0.0, -1.0]), 0.0, None, None,
                        None, False)
    assert np.allclose(y[0, 0], [1, 2, 0, -1])


def test_scores_bound_every_key():
    rng = np.random.default_rng(1)
    k = rng.standard_normal((5, 2, 16, 64))
    q = rng.standard_normal((1, 4, 64))
    tables = np.array([[3, 0, 4, 1]], np.int32)
    bounds = np.stack([lc.block_bounds(k, i, 16) for i in range(5)])
    s, size = lc.block_scores(q, bounds, tables, [50])
    best = np.einsum("hd,jhtd->hjt", np.zeros((2, 64)), k)
    for h in range(2):
        for j, blk in enumerate(tables[0]):
            best = max((q[0, i] @ k[blk, h].T).max() for i in (2 * h, 2 * h + 1))
            assert s[0, h, j] >= best - 1e-12
            assert size[0, h, j] >= abs(s[0, h, j]) - 1e-12
    assert np.isneginf(lc.block_scores(q, bounds, tables, [32])[0][0, :, 2:]).all()


@pytest.mark.parametrize("row, first, last, budget, want", [
    ([5, 1, 4, 3, 2], 0, 0, 2, [0, 2]),
    ([5, 1, 4, 3, 2], 0, 1, 2, [0, 4]),
    ([1, 1, 1, 1], 0, 0, 2, [0, 1]),                     # ties to the lowest index
    ([1, 2, 2, 2, 0], 1, 1, 4, [0, 1, 2, 4]),
    ([np.nan, -np.inf, np.inf, 0], 0, 0, 3, [1, 2, 3]),  # NaN lowest
    ([0.0, -0.0, 1.0], 0, 0, 2, [0, 2]),                 # -0 equals +0
    ([3, 2], 1, 1, 5, [0, 1]),
    ([], 0, 0, 1, []),
])
def test_choose(row, first, last, budget, want):
    assert lc.choose(np.array(row, np.float32), first, last, budget).tolist() == want


def test_listed_attention_over_all_blocks_is_decode_attention():
    rng = np.random.default_rng(2)
    k, v = rng.standard_normal((2, 6, 2, 16, 64))
    q = rng.standard_normal((2, 4, 64))
    tables = np.array([[3, 0, 4], [1, 5, 2]], np.int32)
    lens = np.array([40, 17], np.int32)
    lists = np.broadcast_to(np.array([2, 0, 1]), (2, 2, 3)).copy()
    lists[1] = [1, 0, 0]
    out, size, _ = lc.listed_attention(q, k, v, tables, lens, lists, [3, 2], 0.125)
    want = oracle.paged_decode_attention(q, k, v, tables, lens, 0.125)
    assert np.allclose(out, want, atol=1e-12) and (size >= np.abs(out) - 1e-12).all()


def test_mass_sums_to_the_group_size():
    rng = np.random.default_rng(3)
    k = rng.standard_normal((6, 2, 16, 64))
    q = rng.standard_normal((2, 8, 64))
    tables = np.array([[3, 0, 4], [1, 5, 2]], np.int32)
    mass = lc.attention_mass(q, k, tables, [33, 0], 0.125)
    assert np.allclose(mass[0].sum(-1), 4) and (mass[1] == 0).all()
    assert (mass[0, :, 33:] == 0).all()


def test_evict_compacts_rows_and_settles_scales():
    k = np.zeros((4, 1, 16, 64), np.int8)
    k[0, 0] = np.arange(16)[:, None]
    k[1, 0] = 100 + np.arange(16)[:, None]
    ks = np.array([[2.0], [1.0], [0.0], [0.0]], np.float32)
    mass = np.zeros((1, 1, 32), np.float32)
    mass[0, 0, [3, 20]] = 1
    k2, _, ks2, _, kept, lens, nm = lc.evict(k, k, np.array([[0, 1]]), np.array([30]), mass, 1, 1,
                                             4,
                                             np.array([[2]]), ks, ks)
    assert kept[0, 0].tolist() == [0, 3, 20, 29] and lens.tolist() == [4]
    assert ks2[2, 0] == 2.0
    assert k2[2, 0, :4, 0].tolist() == [0, 3, 52, 56]      # 104 / 2, 113 / 2 to even
    assert nm[0, 0, :5].tolist() == [0, 1, 1, 0, 0]
    assert (k2[:2] == k[:2]).all()


def test_evict_in_place_leaves_tiles_that_stay():
    k = np.random.default_rng(4).integers(-127, 128, (3, 1, 16, 64)).astype(np.int8)
    ks = np.array([[1.0], [3.0], [2.0]], np.float32)
    mass = np.zeros((1, 1, 48), np.float32)
    mass[0, 0, :16] = 2
    mass[0, 0, 40] = 1
    t = np.array([[0, 1, 2]])
    k2, _, ks2, _, kept, _, _ = lc.evict(k, k, t, np.array([48]), mass, 0, 1, 18, t, ks, ks)
    assert kept[0, 0].tolist() == list(range(16)) + [40, 47]
    assert (k2[0] == k[0]).all() and ks2[:, 0].tolist() == [1.0, 2.0, 2.0]
    assert (k2[1, 0, :2] == k[2, 0, [8, 15]]).all()
