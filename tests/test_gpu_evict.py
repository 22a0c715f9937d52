"""Eviction by accumulated weight, on the GPU: every output equal to the oracle's."""

import numpy as np
import pytest

from _longctx import Paged
from _pkv_helpers import to_dev, to_host_bits
from oracle import longctx as lc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_decode_05_gb300.build import build
    build()


def _evict(c, mass, first, last, budget, in_place=False, t=None):
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    t = t or c.gpu()
    new_tables = t["tables"] if in_place else t["new_tables"]
    n = len(c.lens)
    o = dict(lens=torch.full((n,), 99, dtype=torch.int32, device="cuda"),
             mass=torch.full((n, c.hkv, 16 * new_tables.shape[1]), 9.0, device="cuda"),
             kept=torch.full((n, c.hkv, budget), 99, dtype=torch.int32, device="cuda"))
    B.pkv_evict_tokens(t["k"], t["v"], t["tables"], t["lens"], to_dev(mass), first, last,
                       new_tables,
                       o["lens"], o["mass"], o["kept"], t["k_scales"], t["v_scales"], t["status"])
    return t, {k: v.cpu().numpy() for k, v in o.items()}, int(t["status"].item())


def _same(a, b):
    """Equal bit for bit (NaN rows of unused blocks among them)."""
    a, b = np.ascontiguousarray(a), np.ascontiguousarray(b)
    return a.shape == b.shape and a.tobytes() == b.tobytes()


def _mass(c, kind="lognormal"):
    shape = (len(c.lens), c.hkv, 16 * c.mb)
    if kind == "lognormal":
        return np.exp(2 * c.rng.standard_normal(shape)).astype(np.float32)
    if kind == "ties":
        return c.rng.integers(0, 3, shape).astype(np.float32)
    m = c.rng.standard_normal(shape).astype(np.float32)
    pick = c.rng.integers(0, 9, shape)
    for i, v in enumerate([np.nan, np.inf, -np.inf, 0.0, -0.0]):
        m[pick == i] = v
    return m


def _check(c, mass, first, last, budget, in_place=False):
    t, got, st = _evict(c, mass, first, last, budget, in_place)
    assert st == 0
    k, v, ks, vs, kept, lens, nm = lc.evict(c.k, c.v, c.tables, c.lens, mass, first, last, budget,
                                            c.tables if in_place else c.new_tables, c.k_scales,
                                            c.v_scales)
    assert (got["kept"] == kept).all() and (got["lens"] == lens).all()
    assert _same(got["mass"], nm)
    assert _same(to_host_bits(t["k"]), k) and _same(to_host_bits(t["v"]), v)
    if ks is not None:
        assert _same(t["k_scales"].cpu().numpy(), ks) and _same(t["v_scales"].cpu().numpy(), vs)


@pytest.mark.parametrize("kv, hkv, d", [("bf16", 2, 128), ("f16", 3, 64), ("i8", 2, 128),
                                        ("i8", 3, 64)])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("first, last, budget", [(0, 0, 1), (4, 16, 64), (0, 33, 100), (2, 3, 5),
                                                 (1, 0, 129), (10, 90, 400)])
def test_evict(kv, hkv, d, in_place, first, last, budget):
    c = Paged([0, 1, 15, 64, 65, 129, 400, 777], hkv, d, kv, seed=budget, more=-(-budget // 16) + 1,
              cols=26)
    _check(c, _mass(c), first, last, budget, in_place)


@pytest.mark.parametrize("kind", ["ties", "special"])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_order(kind, in_place):
    c = Paged([300, 500, 1000], 2, 64, "bf16", seed=4, more=7)
    _check(c, _mass(c, kind), 3, 20, 100, in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n, budget", [(5000, 1024), (40000, 3000)])
def test_evict_long_rows(n, budget, in_place):
    """More tokens than 4096, and than shared memory keeps."""
    c = Paged([n, 100], 1, 64, "i8", seed=4, more=-(-budget // 16))
    mass = _mass(c)
    if n > 32768:      # the oracle's choice, from numpy's stable order
        t, got, st = _evict(c, mass, 4, 64, budget, in_place)
        row = mass[0, 0, :n]
        keep = np.zeros(n, bool)
        keep[:4] = keep[n - 64:] = True
        rest = np.flatnonzero(~keep)
        keep[rest[np.argsort(-row[rest], kind="stable")[:budget - 68]]] = True
        assert st == 0 and (got["kept"][0, 0] == np.flatnonzero(keep)).all()
        assert (got["mass"][0, 0, :budget] == row[keep]).all()
        return
    _check(c, mass, 4, 64, budget, in_place)


def test_evict_nothing_in_place_changes_nothing():
    c = Paged([64, 100, 3], 2, 128, "i8", seed=5)
    _check(c, _mass(c), 0, 0, 100, in_place=True)


def test_evict_flags_bad_tables_and_lengths():
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    c = Paged([64, 64, 64], 2, 128, "bf16", seed=6, more=2)
    mass = _mass(c)
    t = c.gpu()
    t["lens"].copy_(torch.tensor([64, -2, 64]))
    t["tables"][0, 1] = len(c.k)
    t["new_tables"][2, 0] = -1
    t, got, st = _evict(c, mass, 0, 8, 32, t=t)
    assert st == B.DEV_BAD_BLOCK | B.DEV_BAD_LENGTH
    assert got["lens"].tolist() == [32, 0, 32]
    assert (got["kept"][1] == -1).all() and (got["mass"][1] == 0).all()
    k, _, _, _, kept, _, _ = lc.evict(c.k, c.v, c.tables, c.lens, mass, 0, 8, 32, c.new_tables)
    gk = to_host_bits(t["k"])
    assert (got["kept"][[0, 2]] == kept[[0, 2]]).all()
    for h in range(2):
        for r in range(32):
            blk = c.new_tables[0, r // 16]
            want = 0 if kept[0, h, r] // 16 == 1 else k[blk, h, r % 16]
            assert (gk[blk, h, r % 16] == want).all()
    assert (gk[c.new_tables[2, 1]] == k[c.new_tables[2, 1]]).all()
    assert _same(gk[c.new_tables[2, 0]], c.k[c.new_tables[2, 0]])     # not written
    assert _same(gk[c.new_tables[1]], c.k[c.new_tables[1]])
