"""Sparse decode attention on the GPU: bounds, scores, choice, attention over lists."""

import numpy as np
import pytest

from _longctx import Paged, attention_tolerance
from _pkv_helpers import out_to_f64, to_dev, to_host_bits
from oracle import decode_kv
from oracle import longctx as lc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_decode_05_gb300.build import build
    build()


# ----------------------------------------------------------------- bounds ---
@pytest.mark.parametrize("kv, hkv, d", [("bf16", 8, 128), ("f16", 3, 64), ("i8", 2, 128),
                                        ("i8", 5, 64), ("f16", 1, 128), ("bf16", 2, 64)])
def test_bounds_after_a_step_and_of_everything(kv, hkv, d):
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    c = Paged([1, 0, 15, 16, 17, 33, 300], hkv, d, kv, seed=3)
    t = c.gpu()
    want = c.bounds()
    got = torch.full((len(c.k), hkv, 2, d), 5, device="cuda").to(t["k"].dtype)
    B.pkv_block_bounds(t["k"], t["tables"], t["lens"], got, dev_status=t["status"])
    newest = [int(c.tables[b, (n - 1) // 16]) for b, n in enumerate(c.lens) if n]
    g = decode_kv(to_host_bits(got))
    for blk in range(len(c.k)):
        assert (g[blk] == (decode_kv(want[blk]) if blk in newest else 5)).all()
    # the last n tokens of each sequence
    for n_new in ([1, 0, 15, 16, 17, 33, 300], [1, 0, 2, 1, 2, 18, 33], [0, 0, 0, 0, 0, 0, 0]):
        got.fill_(5)
        num = to_dev(np.array(n_new, np.int32))
        B.pkv_block_bounds(t["k"], t["tables"], t["lens"], got, num, 300, dev_status=t["status"])
        touched = {int(c.tables[b, j]) for b, (n, L) in enumerate(zip(n_new, c.lens)) if n
                   for j in range((L - n) // 16, (L - 1) // 16 + 1)}
        g = decode_kv(to_host_bits(got))
        for blk in range(len(c.k)):
            assert (g[blk] == (decode_kv(want[blk]) if blk in touched else 5)).all(), blk
    assert int(t["status"].item()) == 0


def test_bounds_flags_and_skips_bad_sequences():
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    c = Paged([40, 40, 40, 40], 2, 64, "bf16", seed=4)
    t = c.gpu()
    t["lens"].copy_(torch.tensor([40, 16 * c.mb + 1, -1, 40]))
    t["tables"][3, 2] = len(c.k)
    got = torch.full((len(c.k), 2, 2, 64), 5, device="cuda").to(t["k"].dtype)
    B.pkv_block_bounds(t["k"], t["tables"], t["lens"], got, dev_status=t["status"])
    assert int(t["status"].item()) == B.DEV_BAD_LENGTH | B.DEV_BAD_BLOCK
    g = decode_kv(to_host_bits(got))
    changed = [blk for blk in range(len(c.k)) if (g[blk] != 5).any()]
    assert changed == [c.tables[0, 2]]
    t["status"].zero_()
    t["lens"].copy_(torch.tensor([40, 40, 40, 0]))
    num = torch.tensor([41, 3, -1, 0], dtype=torch.int32, device="cuda")
    B.pkv_block_bounds(t["k"], t["tables"], t["lens"], got.fill_(5), num, 41,
                       dev_status=t["status"])
    assert int(t["status"].item()) == B.DEV_BAD_LENGTH
    g = decode_kv(to_host_bits(got))
    assert [blk for blk in range(len(c.k)) if (g[blk] != 5).any()] == [c.tables[1, 2]]


# ----------------------------------------------------------------- scores ---
@pytest.mark.parametrize("kv, q", [("bf16", "bf16"), ("f16", "f16"), ("i8", "bf16"), ("i8", "f16")])
@pytest.mark.parametrize("g", [1, 2, 4, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_scores(kv, q, g, d):
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    c = Paged([1, 0, 255, 257, 700], 3, d, kv, seed=g, q=q, g=g, cols=g)
    t = c.gpu()
    bounds = c.bounds()
    got = torch.full((5, 3, c.mb), 7.0, device="cuda")
    B.pkv_block_scores(t["q"], to_dev(bounds), t["k"], t["tables"], t["lens"], got, t["k_scales"],
                       t["status"])
    want, size = lc.block_scores(c.q, bounds, c.tables, c.lens, c.k_scales)
    got = got.cpu().numpy().astype(np.float64)
    assert (np.isneginf(got) == np.isneginf(want)).all()
    fin = np.isfinite(want)
    # at most 2 D / 64 products of 16 terms per accumulator, each cut off within
    # 17 units of 2^-23 of the terms' absolute sum; 3 additions, one scale; an
    # INT8 call's bf16 q below 2^-14 rounds to fp16 by at most 2^-25
    tol = (2 * d / 64 * 17 + 4) * 2.0 ** -23 * size[fin]
    if kv == "i8" and q == "bf16":
        tol = tol + d * 127 * 0.03 * 2.0 ** -25
    assert (np.abs(got[fin] - want[fin]) <= tol).all()
    assert int(t["status"].item()) == 0


def test_scores_flag_bad_blocks_and_lengths():
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    c = Paged([90, 40, 64], 2, 128, "bf16", seed=1, g=4)
    t = c.gpu()
    bounds = c.bounds()
    t["tables"][0, 3] = -1
    t["lens"][1] = -5
    got = torch.empty((3, 2, c.mb), device="cuda")
    B.pkv_block_scores(t["q"], to_dev(bounds), t["k"], t["tables"], t["lens"], got,
                       dev_status=t["status"])
    assert int(t["status"].item()) == B.DEV_BAD_LENGTH | B.DEV_BAD_BLOCK
    got = got.cpu().numpy()
    assert np.isneginf(got[0, :, 3]).all() and np.isfinite(got[0, :, [0, 1, 2, 4, 5]]).all()
    assert np.isneginf(got[1]).all() and np.isfinite(got[2, :, :4]).all()


# ----------------------------------------------------------------- choice ---
def _select(scores, lens, first, last, budget):
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    Bn, H, _ = scores.shape
    lists = torch.full((Bn, H, budget), 99, dtype=torch.int32, device="cuda")
    n = torch.full((Bn,), 99, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.pkv_block_select(to_dev(scores), to_dev(np.asarray(lens, np.int32)), first, last, lists, n,
                       st)
    return lists.cpu().numpy(), n.cpu().numpy(), int(st.item())


def _check_select(scores, lens, first, last, budget):
    lists, n, st = _select(scores, lens, first, last, budget)
    assert st == 0
    for b, L in enumerate(lens):
        nb = -(-int(L) // 16)
        assert n[b] == min(nb, budget)
        for h in range(scores.shape[1]):
            want = lc.choose(scores[b, h, :nb], first, last, budget)
            assert lists[b, h, :len(want)].tolist() == want.tolist(), (b, h)
            assert (lists[b, h, len(want):] == -1).all()


@pytest.mark.parametrize("first, last, budget", [(0, 0, 1), (1, 2, 8), (0, 1, 32), (5, 7, 12),
                                                 (0, 0, 200), (3, 0, 64), (1, 1, 77)])
@pytest.mark.parametrize("kind", ["normal", "few_values", "special", "one_value", "wide"])
def test_select(first, last, budget, kind):
    rng = np.random.default_rng(budget)
    lens = [0, 1, 16, 17, 16 * budget, 16 * budget + 1, 1999, 2100]
    mb = max(-(-n // 16) for n in lens) + 3
    x = rng.standard_normal((len(lens), 3, mb)).astype(np.float32)
    if kind == "few_values":
        x = rng.integers(-2, 3, x.shape).astype(np.float32) * np.float32(0.0)  + rng.integers(0, 3,
                x.shape).astype(np.float32)
    elif kind == "special":
        pick = rng.integers(0, 8, x.shape)
        for i, v in enumerate([np.nan, np.inf, -np.inf, 0.0, -0.0]):
            x[pick == i] = v
    elif kind == "one_value":
        x[:] = -3.5
    elif kind == "wide":
        x = (np.sign(x) * 10.0 ** rng.uniform(-44, 38, x.shape)).astype(np.float32)
    _check_select(x, lens, first, last, budget)


@pytest.mark.parametrize("blocks, budget", [(5000, 256), (32768, 700), (40001, 1000),
                                            (33000, 32999)])
def test_select_long_rows(blocks, budget):
    """More blocks than one thread block of 256 handles well, and than shared memory keeps."""
    rng = np.random.default_rng(blocks)
    x = rng.standard_normal((2, 1, blocks)).astype(np.float32)
    x[1, 0, :] = np.round(x[1, 0, :], 1)
    lists, n, st = _select(x, [16 * blocks, 16 * blocks - 40], 1, 4, budget)
    assert st == 0 and n.tolist() == [budget, min(budget, blocks - 2)]
    for b, nb in enumerate((blocks, blocks - 2)):
        row = x[b, 0, :nb]
        keep = np.zeros(nb, bool)
        keep[:1] = keep[nb - 4:] = True
        rest = np.flatnonzero(~keep)
        keep[rest[np.argsort(-row[rest], kind="stable")[:max(0, budget - 5)]]] = True
        assert (lists[b, 0, :n[b]] == np.flatnonzero(keep)).all()


def test_select_flags_bad_lengths():
    from paged_kv_decode_05_gb300 import binding as B
    x = np.arange(24, dtype=np.float32).reshape(2, 1, 12)
    lists, n, st = _select(x, [-1, 16 * 12 + 1], 0, 1, 3)
    assert st == B.DEV_BAD_LENGTH and n.tolist() == [0, 3]
    assert lists[0, 0].tolist() == [-1, -1, -1] and lists[1, 0].tolist() == [9, 10, 11]


# -------------------------------------------------------------- attention ---
def _lists(c, budget, seed=0, shuffle=False, counts=None):
    rng = np.random.default_rng(seed)
    nb = -(-c.lens // 16)
    n = np.minimum(nb, budget).astype(np.int32) if counts is None else np.asarray(counts, np.int32)
    lists = np.full((len(c.lens), c.hkv, budget), -1, np.int32)
    for b in range(len(c.lens)):
        for h in range(c.hkv):
            pick = rng.permutation(nb[b])[:n[b]]
            lists[b, h, :len(pick)] = pick if shuffle else np.sort(pick)
    return lists, n


def _attend(c, lists, n, num_parts=0, t=None):
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    t = t or c.gpu()
    ws = torch.empty(B.pkv_sparse_decode_workspace_size(len(c.lens), c.q.shape[1], t["k"],
                                                        num_parts),
                     dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)
    B.pkv_sparse_decode_attn(t["q"], t["k"], t["v"], t["tables"], t["lens"], to_dev(lists),
                             to_dev(n),
                             c.scale, t["out"], ws, t["k_scales"], t["v_scales"], num_parts,
                             t["status"])
    return out_to_f64(t["out"]), int(t["status"].item())


def _check_attend(c, lists, n, num_parts=0):
    got, st = _attend(c, lists, n, num_parts)
    assert st == 0
    want, size, dots = lc.listed_attention(c.q, c.k, c.v, c.tables, c.lens, lists, n, c.scale,
                                           c.k_scales, c.v_scales)
    tol = attention_tolerance(c, want, size, dots, 16 * max(1, int(n.max(initial=0))))
    err = np.abs(got - want)
    assert (err <= tol).all(), (float(err.max()), float((err / tol).max()))


@pytest.mark.parametrize("kv, q", [("bf16", "bf16"), ("f16", "f16"), ("i8", "bf16"), ("i8", "f16")])
@pytest.mark.parametrize("g", [1, 2, 4, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_sparse_attention(kv, q, g, d):
    c = Paged([1, 0, 16, 17, 130, 699, 1024], 3, d, kv, seed=10 * g + d, q=q, g=g)
    lists, n = _lists(c, 9, seed=g)
    _check_attend(c, lists, n)
    _check_attend(c, lists, n, num_parts=1)


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("num_parts", [0, 1, 3, 7, 64, 1000])
def test_sparse_attention_over_parts(kv, num_parts):
    """Lists in any order, long enough that several workers share a (sequence, kv head)."""
    c = Paged([5000, 33, 2047, 1], 2, 128, kv, seed=num_parts, g=4)
    lists, n = _lists(c, 301, seed=3, shuffle=True, counts=[301, 2, 77, 1])
    _check_attend(c, lists, n, num_parts)


@pytest.mark.parametrize("kv, d", [("bf16", 128), ("f16", 64), ("i8", 128), ("i8", 64)])
@pytest.mark.parametrize("hkv, g", [(2, 8), (5, 4), (13, 1), (40, 2), (77, 1)])
def test_sparse_attention_of_few_segments(kv, d, hkv, g):
    """From 8 to 308 (sequence, kv head) pairs: several thread blocks to a pair, one, waves of
    them; with lists shorter than the warps that share them."""
    c = Paged([2900, 0, 31, 1500], hkv, d, kv, seed=hkv, g=g)
    lists, n = _lists(c, 150, seed=2, shuffle=True, counts=[150, 0, 1, 77])
    _check_attend(c, lists, n)


@pytest.mark.parametrize("kv", ["f16", "i8"])
def test_sparse_attention_of_many_sequences(kv):
    """More sequences than the exact prefix in shared memory holds."""
    rng = np.random.default_rng(5)
    c = Paged(rng.integers(0, 90, 601), 1, 64, kv, seed=6, g=2)
    lists, n = _lists(c, 4)
    _check_attend(c, lists, n)


@pytest.mark.parametrize("batch, hkv", [(467, 3), (5003, 4)])
def test_sparse_attention_of_thousands_of_segments(batch, hkv):
    """More (sequence, kv head) pairs than thread blocks that merge them: runs of a few and
    of more than a warp has lanes."""
    rng = np.random.default_rng(batch)
    c = Paged(rng.integers(0, 24, batch), hkv, 64, "f16", seed=7, g=1)
    lists, n = _lists(c, 2)
    _check_attend(c, lists, n)


def test_sparse_attention_empty_lists_and_repeats():
    c = Paged([100, 100, 100], 2, 128, "bf16", seed=8, g=4)
    lists = np.array([[[6, 6, 0], [1, 1, 1]], [[0, 0, 0], [0, 0, 0]], [[2, 3, 9], [4, 0, 9]]],
                     np.int32)
    n = np.array([3, 0, 2], np.int32)
    _check_attend(c, lists, n)
    got, st = _attend(c, np.zeros((3, 2, 0), np.int32), np.zeros(3, np.int32))
    assert st == 0 and (got == 0).all()


@pytest.mark.parametrize("kv", ["bf16", "i8"])
def test_sparse_attention_skips_and_flags_bad_entries(kv):
    from paged_kv_decode_05_gb300 import binding as B
    c = Paged([100, 80, 60], 2, 64, kv, seed=9, g=2)
    lists = np.array([[[0, 7, 3], [-1, 2, 5]], [[1, 2, 4], [0, 1, 4]], [[0, 1, 2], [3, 2, 1]]],
                     np.int32)
    n = np.array([3, 3, 7], np.int32)
    t = c.gpu()
    t["tables"][1, 2] = len(c.k)
    got, st = _attend(c, lists, n, t=t)
    assert st == B.DEV_BAD_INDEX | B.DEV_BAD_BLOCK | B.DEV_BAD_LENGTH
    good = np.array([[[0, 3, 0], [2, 5, 0]], [[1, 4, 0], [0, 1, 4]], [[0, 1, 2], [3, 2, 1]]],
                    np.int32)
    for b, h, m in [(0, 0, 2), (0, 1, 2), (1, 0, 2), (1, 1, 3), (2, 0, 3), (2, 1, 3)]:
        want, size, dots = lc.listed_attention(c.q, c.k, c.v, c.tables, c.lens, good,
                                               np.full(3, m), c.scale, c.k_scales, c.v_scales)
        tol = attention_tolerance(c, want, size, dots, 48)
        hs = slice(2 * h, 2 * h + 2)
        assert (np.abs(got - want)[b, hs] <= tol[b, hs]).all(), (b, h)


@pytest.mark.parametrize("kv", ["bf16", "f16", "i8"])
@pytest.mark.parametrize("scale, std", [(4.0, 3.0), (0.0, 1.0), (-0.3, 1.0), (0.125, 1e-3)])
def test_sparse_attention_scales(kv, scale, std):
    """Weights on one token, equal weights, a negative scale, small values and scales."""
    c = Paged([700, 333], 2, 128, kv, seed=12, g=4, std=std)
    c.scale = scale
    lists, n = _lists(c, 21)
    _check_attend(c, lists, n)
