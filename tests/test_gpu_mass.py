"""Decode attention with accumulated weights, on the GPU."""

import numpy as np
import pytest

from _longctx import Paged, attention_tolerance
from _pkv_helpers import out_to_f64, to_dev
from oracle import longctx as lc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_decode_05_gb300.build import build
    build()


def _run(c, mass_in, num_parts=0, t=None, alias=False):
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    t = t or c.gpu()
    ws = torch.empty(B.pkv_decode_mass_workspace_size(len(c.lens), c.q.shape[1], c.mb, t["k"],
                                                      num_parts),
                     dtype=torch.uint8, device="cuda").fill_(0xFF)
    m_in = None if mass_in is None else to_dev(mass_in)
    m_out = m_in if alias else torch.full((len(c.lens), c.hkv, 16 * c.mb), 9.0, device="cuda")
    B.pkv_decode_attn_mass(t["q"], t["k"], t["v"], t["tables"], t["lens"], c.scale, t["out"], m_in,
                           m_out, ws, t["k_scales"], t["v_scales"], num_parts, t["status"])
    return out_to_f64(t["out"]), m_out.cpu().numpy(), int(t["status"].item())


def _check(c, num_parts=0, with_old=True, alias=False):
    old = c.rng.random((len(c.lens), c.hkv, 16 * c.mb)).astype(np.float32) if with_old else None
    out, mass, st = _run(c, old, num_parts, alias=alias)
    assert st == 0
    nb = -(-c.lens // 16)
    lists = np.broadcast_to(np.arange(c.mb, dtype=np.int32), (len(c.lens), c.hkv, c.mb))
    want, size, dots = lc.listed_attention(c.q, c.k, c.v, c.tables, c.lens, lists, nb, c.scale,
                                           c.k_scales, c.v_scales)
    tol = attention_tolerance(c, want, size, dots, int(c.lens.max(initial=1)))
    err = np.abs(out - want)
    assert (err <= tol).all(), float((err / tol).max())
    w = lc.attention_mass(c.q, c.k, c.tables, c.lens, c.scale, c.k_scales)
    # a weight's relative error: its score and the largest one (as in
    # attention_tolerance), exp2 (2^-21 each, and once more for the rescalings
    # of l), a sum over the tokens of fp32 terms, the quotient; then one
    # addition per head and one to the old value
    steps = (c.lens.max(initial=1) / 16 + 40) * 2.0 ** -23
    rel = (4 * abs(c.scale) * dots.reshape(len(c.lens), c.hkv, c.g).max(2) * 71 * 2.0 ** -23
           + 2.0 ** -19 + steps)[..., None]
    full = w + (0 if old is None else old)
    for b, L in enumerate(c.lens):
        got = mass[b, :, :L].astype(np.float64)
        bound = rel[b] * w[b, :, :L] + (c.g + 1) * 2.0 ** -24 * np.abs(full[b, :, :L]) + 1e-37
        assert (np.abs(got - full[b, :, :L]) <= bound).all(), b
        assert (mass[b, :, L:] == (9.0 if not alias else old[b, :, L:])).all()     # left alone


@pytest.mark.parametrize("kv, q", [("bf16", "bf16"), ("f16", "f16"), ("i8", "bf16"), ("i8", "f16")])
@pytest.mark.parametrize("g", [1, 2, 4, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_mass(kv, q, g, d):
    c = Paged([1, 0, 16, 17, 130, 699, 1024], 3, d, kv, seed=g + d, q=q, g=g)
    _check(c)
    _check(c, num_parts=1, with_old=False)


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("num_parts", [0, 2, 5, 64, 999])
def test_mass_over_parts_in_place(kv, num_parts):
    _check(Paged([5003, 33, 2047, 0, 1], 2, 128, kv, seed=num_parts, g=4), num_parts, alias=True)


@pytest.mark.parametrize("kv, d", [("bf16", 128), ("f16", 64), ("i8", 128), ("i8", 64)])
@pytest.mark.parametrize("hkv, g", [(2, 8), (5, 4), (13, 1), (40, 2), (77, 1)])
def test_mass_of_few_segments(kv, d, hkv, g):
    """From 8 to 308 (sequence, kv head) pairs: several thread blocks to a pair, one, waves of
    them; with sequences shorter than the warps that share them."""
    _check(Paged([1500, 0, 31, 777], hkv, d, kv, seed=hkv, g=g), alias=True)


@pytest.mark.parametrize("kv, d, g", [("bf16", 128, 4), ("f16", 64, 1), ("i8", 128, 8),
                                      ("i8", 64, 2)])
def test_mass_of_short_sequences(kv, d, g):
    """A thread block per (sequence, kv head), more of them than the device holds at once."""
    _check(Paged([40, 0, 7, 130], 40, d, kv, seed=g, g=g))


@pytest.mark.parametrize("kv", ["f16", "i8"])
def test_mass_of_many_sequences(kv):
    rng = np.random.default_rng(5)
    _check(Paged(rng.integers(0, 60, 700), 1, 64, kv, seed=6, g=2))


@pytest.mark.parametrize("batch, hkv", [(467, 3), (5003, 4)])
def test_mass_of_thousands_of_segments(batch, hkv):
    """More (sequence, kv head) pairs than thread blocks that merge them: runs of a few and
    of more than a warp has lanes."""
    rng = np.random.default_rng(batch)
    c = Paged(rng.integers(0, 24, batch), hkv, 64, "f16", seed=7, g=1)
    _check(c)


def test_mass_of_nothing():
    c = Paged([0, 0], 2, 64, "bf16", g=2)
    out, mass, st = _run(c, None)
    assert st == 0 and (out == 0).all() and (mass == 9).all()


@pytest.mark.parametrize("kv", ["bf16", "f16", "i8"])
@pytest.mark.parametrize("scale, std", [(4.0, 3.0), (0.0, 1.0), (-0.3, 1.0), (0.125, 1e-3)])
def test_mass_scales(kv, scale, std):
    c = Paged([700, 333], 2, 128, kv, seed=12, g=4, std=std)
    c.scale = scale
    _check(c)


@pytest.mark.parametrize("kv", ["bf16", "i8"])
def test_mass_gives_bad_blocks_no_weight(kv):
    from paged_kv_decode_05_gb300 import binding as B
    c = Paged([100, 80, 70], 2, 64, kv, seed=9, g=2)
    t = c.gpu()
    t["tables"][1, 2] = -3
    t["lens"][2] = -1
    out, mass, st = _run(c, None, t=t)
    assert st == B.DEV_BAD_BLOCK | B.DEV_BAD_LENGTH
    lists = np.array([[[0, 1, 2, 3, 4, 5, 6]] * 2, [[0, 1, 3, 4, 0, 0, 0]] * 2, [[0] * 7] * 2])
    want, size, dots = lc.listed_attention(c.q, c.k, c.v, c.tables, c.lens, lists, [7, 4, 0],
                                           c.scale,
                                           c.k_scales, c.v_scales)
    tol = attention_tolerance(c, want, size, dots, 112)
    assert (np.abs(out - want) <= tol).all()
    assert (mass[1, :, 32:48] == 0).all() and (mass[2] == 9).all()
    assert np.allclose(mass[1, :, :80].sum(-1), c.g, rtol=1e-4)


@pytest.mark.parametrize("kv", ["bf16", "i8"])
def test_mass_attention_equals_decode_attention(kv):
    """The same attention as pkv_decode_attn, within both kernels' tolerance."""
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    c = Paged([900, 64, 1], 4, 128, kv, seed=2, g=8)
    t = c.gpu()
    out, _, _ = _run(c, None, t=t)
    ws = torch.empty(B.pkv_decode_workspace_size(3, 32, t["k"]), dtype=torch.uint8, device="cuda")
    ref = torch.empty_like(t["q"])
    B.pkv_decode_attn(t["q"], t["k"], t["v"], t["tables"], t["lens"], c.scale, ref, ws,
                      t["k_scales"],
                      t["v_scales"])
    lists = np.broadcast_to(np.arange(c.mb, dtype=np.int32), (3, 4, c.mb))
    want, size, dots = lc.listed_attention(c.q, c.k, c.v, c.tables, c.lens, lists, -(-c.lens // 16),
                                           c.scale, c.k_scales, c.v_scales)
    tol = attention_tolerance(c, want, size, dots, 900)
    assert (np.abs(out - out_to_f64(ref)) <= 2 * tol + (2e-2 if kv == "i8" else 0)).all()
