"""Pins of the oracle of windowed attention and of the 4-bit cache."""

import numpy as np
import pytest

from _longctx import stored
from oracle import decode_kv, paged_multiquery_attention
from oracle import window as ow


def test_visible_by_hand():
    assert ow.visible(5, 6, 0, 0) == [0, 1, 2, 3, 4, 5]
    assert ow.visible(5, 6, 2, 0) == [4, 5]
    assert ow.visible(5, 6, 2, 1) == [0, 4, 5]
    assert ow.visible(5, 9, 3, 4) == [0, 1, 2, 3, 4, 5]
    assert ow.visible(0, 1, 1, 0) == [0]
    assert ow.visible(7, 8, 100, 0) == list(range(8))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_row_by_hand(dtype):
    """0 .. 15 in steps of one: s = 1, the codes are the values; ties go to even."""
    x = stored(np.array([[0, 1, 2, 3, 7.5, 8.5, 14.5, 15]]), dtype)
    codes, pairs = ow.u4_quantise(x)
    assert pairs.tolist() == [[1.0, 0.0]]
    assert codes.tolist() == [[0, 1, 2, 3, 8, 8, 14, 15]]
    assert ow.u4_pack(codes).tolist() == [[0x10, 0x32, 0x88, 0xFE]]
    assert ow.u4_values(codes, pairs).tolist() == [[0, 1, 2, 3, 8, 8, 14, 15]]
    same, pairs = ow.u4_quantise(stored(np.full((1, 4), -2.5), dtype))
    assert same.tolist() == [[0] * 4] and pairs.tolist() == [[0.0, -2.5]]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("size", [1e-7, 1e-2, 1.0, 1e4])
def test_values_lie_within_half_a_step(dtype, size):
    rng = np.random.default_rng(0)
    x = stored(rng.standard_normal((200, 64)) * size + rng.standard_normal((200, 1)) * size, dtype)
    codes, pairs = ow.u4_quantise(x)
    f = decode_kv(x)
    s, lo = pairs[:, 0], pairs[:, 1]
    assert codes.max() <= 15 and (lo == f.min(1)).all()
    # the scale is the type's, not below a 15th of the range and less than a step above it
    assert (decode_kv(stored(s, dtype)) == s).all()
    want = (f.max(1) - f.min(1)) / 15
    step = {"bf16": 2.0 ** -7, "f16": 2.0 ** -10}[dtype]
    assert (s >= want * (1 - 1e-6)).all()
    assert (s <= want * (1 + step) + 2.0 ** -24 * (dtype == "f16")).all()
    # x - lo is rounded to fp32
    assert (np.abs(ow.u4_values(codes, pairs) - f) <= s[:, None] / 2 + np.abs(f).max() * 2e-7).all()


def test_without_a_window_it_is_multiquery_attention():
    rng = np.random.default_rng(1)
    hkv, g, d, lens, counts = 2, 2, 16, [9, 20], [3, 20]
    k, v = (rng.standard_normal((4, hkv, 16, d)).astype(np.float16) for _ in range(2))
    tables = np.array([[2, 0], [1, 3]], np.int32)
    q = rng.standard_normal((23, hkv * g, d)).astype(np.float16)
    cu = np.array([0, 3, 23], np.int32)
    want = paged_multiquery_attention(q, cu, k, v, tables, np.array(lens, np.int32), 0.3)

    def rows(x):
        return [decode_kv(x)[tables[b]].transpose(0, 2, 1, 3).reshape(32, hkv, d)[:n]
                for b, n in enumerate(lens)]
    got, size, dots, most = ow.window_attention(q, rows(k), rows(v), counts, lens, 0.3, 0, 0)
    assert np.abs(got - want).max() < 1e-12 and most == 20
    # a window as long as the sequence, and sinks that cover it, change nothing
    for window, sinks in ((20, 0), (1, 20)):
        same = ow.window_attention(q, rows(k), rows(v), counts, lens, 0.3, window, sinks)[0]
        assert np.abs(same - want).max() < 1e-12
    # a window of one is the token's own value
    own = ow.window_attention(q, rows(k), rows(v), counts, lens, 0.3, 1, 0)[0]
    at = rows(v)[1]
    assert np.abs(own[3:] - np.repeat(at, g, 1)).max() < 1e-12
