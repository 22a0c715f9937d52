"""Eviction into tables that repeat the old ones without being the same array."""

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


def _same(a, b):
    return a.shape == b.shape and a.tobytes() == np.ascontiguousarray(b).tobytes()


@pytest.mark.parametrize("kv, hkv, d", [("bf16", 2, 128), ("f16", 3, 64), ("i8", 2, 128),
                                        ("i8", 1, 64)])
@pytest.mark.parametrize("kind", ["copy", "first_columns", "some_places", "some_sequences"])
def test_evict_into_a_table_that_repeats_the_old_one(kv, hkv, d, kind):
    """Rows that move within their own blocks, many groups of tiles of them: the result of a
    compaction whose every source is read before it is overwritten."""
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    budget = 4000
    nb = budget // 16
    c = Paged([5000, 4100, 300, 0, 4500], hkv, d, kv, seed=d, more=nb)
    new = c.tables.copy() if kind == "copy" else c.tables[:, :nb].copy()
    if kind == "some_places":
        new[:, 5::7] = c.new_tables[:, 5::7]
    elif kind == "some_sequences":
        new[[0, 2]] = c.new_tables[[0, 2]]
    mass = np.exp(2 * c.rng.standard_normal((5, hkv, 16 * c.mb))).astype(np.float32)
    t = c.gpu()
    n, width = len(c.lens), new.shape[1]
    lens = torch.full((n,), 99, dtype=torch.int32, device="cuda")
    got_mass = torch.full((n, hkv, 16 * width), 9.0, device="cuda")
    kept = torch.full((n, hkv, budget), 99, dtype=torch.int32, device="cuda")
    B.pkv_evict_tokens(t["k"], t["v"], t["tables"], t["lens"], to_dev(mass), 4, 64, to_dev(new),
                       lens, got_mass, kept, t["k_scales"], t["v_scales"], t["status"])
    assert int(t["status"].item()) == 0
    k, v, ks, vs, want_kept, want_lens, want_mass = lc.evict(
        c.k, c.v, c.tables, c.lens, mass, 4, 64, budget, new, c.k_scales, c.v_scales)
    assert (kept.cpu().numpy() == want_kept).all() and (lens.cpu().numpy() == want_lens).all()
    assert _same(got_mass.cpu().numpy(), want_mass)
    assert _same(to_host_bits(t["k"]), k) and _same(to_host_bits(t["v"]), v)
    if ks is not None:
        assert _same(t["k_scales"].cpu().numpy(), ks) and _same(t["v_scales"].cpu().numpy(), vs)
