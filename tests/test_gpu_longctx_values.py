"""The long-context operators on values at the ends of their ranges: infinities
and NaN that a query does see, queries and scales far from one."""

import numpy as np
import pytest

from _longctx import Paged, attention_tolerance, stored
from _pkv_helpers import out_to_f64, to_dev
from oracle import decode_kv
from oracle import longctx as lc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_decode_05_gb300.build import build
    build()


def _scores(c, q, bounds):
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    t = c.gpu()
    got = torch.full((len(c.lens), c.hkv, c.mb), 7.0, device="cuda")
    B.pkv_block_scores(to_dev(q), to_dev(bounds), t["k"], t["tables"], t["lens"], got,
                       t["k_scales"], t["status"])
    assert int(t["status"].item()) == 0
    return got.cpu().numpy().astype(np.float64)


def _times(a, b):
    """a b, where nothing times infinity is nothing."""
    with np.errstate(invalid="ignore"):
        x = a * b
    return np.where(np.isnan(x) & ~np.isnan(a) & ~np.isnan(b), 0.0, x)


def _want(c, q, bounds):
    """(score, sum of absolute terms) of every block, sums that are not a number left out."""
    g, want = c.g, np.full((len(c.lens), c.hkv, c.mb), -np.inf)
    size = np.zeros_like(want)
    x, box = decode_kv(q), decode_kv(bounds)
    for b, L in enumerate(c.lens):
        for j in range(-(-int(L) // 16)):
            for h in range(c.hkv):
                lo, hi = box[c.tables[b, j], h]
                s = 1.0 if c.k_scales is None else float(c.k_scales[c.tables[b, j], h])
                for i in range(h * g, h * g + g):
                    terms = np.maximum(_times(x[b, i], lo), _times(x[b, i], hi))
                    with np.errstate(invalid="ignore"):
                        total = terms.sum() * s
                    if not np.isnan(total):
                        want[b, h, j] = max(want[b, h, j], total)
                        size[b, h, j] = max(size[b, h, j], np.abs(terms).sum() * s)
    return want, size


@pytest.mark.parametrize("kv, d, g", [("bf16", 128, 4), ("f16", 64, 1), ("f16", 128, 8),
                                      ("bf16", 64, 2)])
def test_scores_of_infinite_bounds(kv, d, g):
    """Keys that overflowed leave infinite bounds. A channel whose other end is the larger
    product, or whose query is zero, keeps its finite value."""
    c = Paged([1, 0, 300, 700], 2, d, kv, seed=g, g=g)
    rng = np.random.default_rng(d + g)
    bounds = c.bounds().copy()
    lo, hi = bounds[:, :, 0], bounds[:, :, 1]
    pick = rng.random(lo.shape)
    ninf, pinf = stored([-np.inf], kv)[0], stored([np.inf], kv)[0]
    lo[pick < 0.01] = ninf
    hi[(pick > 0.005) & (pick < 0.015)] = pinf
    lo[pick > 0.999] = pinf
    hi[pick > 0.999] = pinf
    lo[(pick > 0.997) & (pick < 0.998)] = ninf
    hi[(pick > 0.997) & (pick < 0.998)] = ninf
    # few queries per channel with the sign that makes such a bound infinite
    x = rng.standard_normal(c.q.shape)
    x[..., rng.random(d) < 0.5] = 0.0
    q = stored(x, kv)
    got, (want, size) = _scores(c, q, bounds), _want(c, q, bounds)
    assert np.isfinite(want).any() and np.isposinf(want).any() and np.isneginf(want).any()
    fin = np.isfinite(want)
    assert (got[~fin] == want[~fin]).all()
    # sums of 2 D products of one head, at worst one after the other, in fp32
    assert (np.abs(got[fin] - want[fin]) <= (2 * d / 64 * 17 + 4 + d) * 2.0 ** -23 * size[fin]).all()


@pytest.mark.parametrize("kv, q", [("bf16", "bf16"), ("f16", "f16"), ("i8", "bf16"), ("i8", "f16")])
def test_scores_of_infinite_queries(kv, q):
    c = Paged([40, 500], 2, 128, kv, seed=3, q=q, g=2)
    rng = np.random.default_rng(3)
    x = rng.standard_normal(c.q.shape)
    x[0, 0, 5], x[0, 3, 7], x[1, 0, 9], x[1, 1, 100] = np.inf, -np.inf, np.nan, np.nan
    qs, bounds = stored(x, c.qt), c.bounds()
    got, (want, size) = _scores(c, qs, bounds), _want(c, qs, bounds)
    fin = np.isfinite(want)
    assert np.isneginf(want[1, 0]).all() and np.isfinite(want[1, 1, :32]).all()
    assert (got[~fin] == want[~fin]).all()
    assert (np.abs(got[fin] - want[fin]) <= (2 * 2 * 17 + 4 + 128) * 2.0 ** -23 * size[fin]).all()


def _attend(c, t, num_parts=0, mass_in=None):
    """Attention over all blocks through a list, attention with weights, and the weights."""
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    n, hq = c.q.shape[:2]
    lists = torch.arange(c.mb, dtype=torch.int32, device="cuda").expand(n, c.hkv, c.mb).contiguous()
    counts = to_dev((-(-c.lens // 16)).astype(np.int32))
    out, full = (torch.full_like(t["q"], 3.0) for _ in range(2))
    mass = torch.zeros((n, c.hkv, 16 * c.mb), device="cuda")
    ws = torch.empty(max(B.pkv_sparse_decode_workspace_size(n, hq, t["k"], num_parts),
                         B.pkv_decode_mass_workspace_size(n, hq, c.mb, t["k"], num_parts)),
                     dtype=torch.uint8, device="cuda").fill_(0xFF)
    B.pkv_sparse_decode_attn(t["q"], t["k"], t["v"], t["tables"], t["lens"], lists, counts, c.scale,
                             out, ws, t["k_scales"], t["v_scales"], num_parts, t["status"])
    B.pkv_decode_attn_mass(t["q"], t["k"], t["v"], t["tables"], t["lens"], c.scale, full, None,
                           mass, ws, t["k_scales"], t["v_scales"], num_parts, t["status"])
    assert int(t["status"].item()) == 0
    return out, full, mass


def _exact(c):
    lists = np.broadcast_to(np.arange(c.mb), (len(c.lens), c.hkv, c.mb))
    with np.errstate(invalid="ignore"):
        return lc.listed_attention(c.q, c.k, c.v, c.tables, c.lens, lists, -(-c.lens // 16),
                                   c.scale, c.k_scales, c.v_scales)


@pytest.mark.parametrize("power", [-100, -30, -15, 17, 60, 100])
@pytest.mark.parametrize("num_parts", [0, 40])
def test_int8_takes_bf16_queries_of_any_size(power, num_parts):
    """A query 2^power times as large under a softmax scale 2^power times as small: the same
    products, so the same bits. Scores grow by the factor."""
    import torch
    c = Paged([700, 0, 17, 333], 2, 128, "i8", seed=2, g=4)
    t = c.gpu()
    want = _attend(c, t, num_parts)
    plain = _scores(c, c.q, c.bounds())
    c.q = stored(decode_kv(c.q) * 2.0 ** power, "bf16")
    c.scale *= 2.0 ** -power
    t["q"] = to_dev(c.q)
    for got, x in zip(_attend(c, t, num_parts), want):
        assert torch.equal(got, x)
    assert (_scores(c, c.q, c.bounds()) == plain * 2.0 ** power).all()


@pytest.mark.parametrize("g", [1, 8])
def test_int8_takes_bf16_queries_with_one_large_channel(g):
    """A channel beyond fp16's range, which the keys do not use, beside ordinary ones."""
    c = Paged([300, 90], 3, 64, "i8", seed=g, g=g)
    c.k[..., 3] = 0
    x = decode_kv(c.q)
    x[..., 3] = 3e5
    c.q = stored(x, "bf16")
    want, size, dots = _exact(c)
    tol = attention_tolerance(c, want, size, dots, 300)
    for got in _attend(c, c.gpu())[:2]:
        assert (np.abs(out_to_f64(got) - want) <= tol).all()
    got, (want, size) = _scores(c, c.q, c.bounds()), _want(c, c.q, c.bounds())
    fin = np.isfinite(want)
    # q in units of 2^4: values below 2^-10 round by 2^-21 at most
    tol = (2 * 2 * 17 + 4) * 2.0 ** -23 * size[fin] + 64 * 127 * 0.03 * 2.0 ** -21
    assert (np.abs(got[fin] - want[fin]) <= tol).all() and (got[~fin] == want[~fin]).all()


@pytest.mark.parametrize("power", [-108, -110, -116])
@pytest.mark.parametrize("num_parts", [0, 1, 40])
def test_int8_value_scales_down_to_the_smallest(power, num_parts):
    """Value scales near the end of fp32's normal range: rows as small, not NaN."""
    c = Paged([700, 0, 17, 333], 2, 128, "i8", seed=3, g=4)
    c.v_scales = (c.v_scales * 2.0 ** power).astype(np.float32)
    want, size, dots = _exact(c)
    tol = attention_tolerance(c, want, size, dots, 700)
    # V's scales enter the products times 2^126 at most: below 2^-113, fp16 parts of P v_scale
    # keep less (attention_tolerance counts 2^-37 of the largest scale per token); a bf16 output
    # below 2^-126 rounds by 2^-134, a piece in fp32 by 2^-150
    top = float(np.nanmax(c.v_scales))
    less = max(1.0, 2.0 ** -113 / top)
    tol = tol + less * 700 * 2.0 ** -37 * 127 * top + 2.0 ** -134 + 50 * 2.0 ** -150
    for got in _attend(c, c.gpu(), num_parts)[:2]:
        err = np.abs(out_to_f64(got) - want)
        assert (err <= tol).all(), float(np.nanmax(err / tol))


@pytest.mark.parametrize("kv", ["bf16", "f16", "i8"])
@pytest.mark.parametrize("num_parts", [0, 1, 5, 64])
def test_nan_scores_are_not_lost(kv, num_parts):
    """A NaN or +inf score makes its head's row and weights NaN, and no other's; a score of
    -inf has no weight."""
    c = Paged([700, 333, 40, 64], 2, 128, kv, seed=4, g=2)
    x = decode_kv(c.q)
    x[1, 0, 7] = np.nan                                   # sequence 1, head 0
    x[3, 3] = np.nan                                      # sequence 3, head 3: no score is a number
    x[2, 0, 4], x[2, 1, 4] = 1.0, -1.0
    c.q = stored(x, c.qt)
    if kv == "i8":
        c.k_scales[c.tables[0, 10], 1] = np.nan           # sequence 0, heads 2 and 3
        bad = [(0, 2), (0, 3), (1, 0), (3, 3)]
    else:
        c.k[c.tables[0, 10], 1, 5, 3] = stored([np.nan], kv)[0]
        c.k[c.tables[2, 0], 0, 2, 4] = stored([np.inf], kv)[0]    # sequence 2: head 0, not head 1
        bad = [(0, 2), (0, 3), (1, 0), (2, 0), (3, 3)]
    want, size, dots = _exact(c)
    nan = np.zeros(want.shape[:2], bool)
    for b, h in bad:
        nan[b, h] = True
    assert (np.isnan(want).all(-1) == nan).all()
    with np.errstate(invalid="ignore"):
        tol = attention_tolerance(c, want, size, dots, 700)
        weights = lc.attention_mass(c.q, c.k, c.tables, c.lens, c.scale, c.k_scales)
    out, full, mass = _attend(c, c.gpu(), num_parts)
    for got in (out_to_f64(out), out_to_f64(full)):
        assert (np.isnan(got).all(-1) == nan).all() and not np.isnan(got[~nan]).any()
        assert (np.abs(got - want)[~nan] <= tol[~nan]).all()
    mass = mass.cpu().numpy()
    for b, L in enumerate(c.lens):
        got, w = mass[b, :, :L], weights[b, :, :L]
        assert (np.isnan(got) == np.isnan(w)).all()
        assert np.allclose(got[~np.isnan(w)], w[~np.isnan(w)], rtol=1e-3, atol=1e-30)


@pytest.mark.parametrize("kv", ["bf16", "f16"])
def test_bounds_pass_over_nan_keys(kv):
    """A channel's bounds are those of its numbers, infinities among them; NaN if it has none."""
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    c = Paged([48, 21], 2, 64, kv, seed=6)
    rng = np.random.default_rng(6)
    pick = rng.random(c.k.shape)
    for lo, hi, x in ((0, 0.2, np.nan), (0.2, 0.22, np.inf), (0.22, 0.24, -np.inf)):
        c.k[(pick >= lo) & (pick < hi)] = stored([x], kv)[0]
    c.k[c.tables[0, 1], 1, :, 5] = stored([np.nan], kv)[0]
    t = c.gpu()
    bounds = torch.zeros((len(c.k), 2, 2, 64), device="cuda").to(t["k"].dtype)
    B.pkv_block_bounds(t["k"], t["tables"], t["lens"], bounds, t["lens"], 48)
    got = out_to_f64(bounds)
    for b, L in enumerate(c.lens):
        for j in range(-(-int(L) // 16)):
            rows = decode_kv(c.k[c.tables[b, j]])[:, :min(16, L - 16 * j)]
            want = np.stack([np.fmin.reduce(rows, 1), np.fmax.reduce(rows, 1)], 1)
            assert np.array_equal(got[c.tables[b, j]], want, equal_nan=True)
    assert np.isnan(got[c.tables[0, 1], 1, :, 5]).all()
