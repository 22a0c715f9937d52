"""Norms, rotation and cache write in one pass, on the GPU."""

import numpy as np
import pytest

from _longctx import HALF_STEP, stored
from _pkv_helpers import out_to_f64, to_dev, to_host_bits
from oracle import decode_kv
from oracle import longctx as lc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_decode_05_gb300.build import build
    build()


def _table(rows, rot):
    half = rot // 2
    ang = np.arange(rows)[:, None] * 10000.0 ** (-np.arange(half) / max(half, 1))
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def _tolerance(x, w, eps, want, dtype):
    """Half a step of the type, and fp32: 8 + 4 additions of squares, the mean, rsqrt (2 units),
    three products: within 2^-20 of |y|; the two products and the sum of the rotation, with table
    values as given: within 2^-22 of |u| + |v|, which a row's largest |y| bounds twice."""
    y = lc.qk_norm_rope(x, w, eps, None, None, None, False)
    top = np.abs(y).max(-1, keepdims=True)
    return HALF_STEP[dtype] * np.abs(want) + 2 * top * (2.0 ** -20 + 2.0 ** -22) + (
        2.0 ** -25 if dtype == "f16" else 0)


class Case:
    def __init__(self, n, hq, hkv, d, dtype, rot, axes=1, norm=True, seed=0, split="even",
                 pool=None):
        rng = np.random.default_rng(seed)
        self.n, self.hq, self.hkv, self.d, self.dtype = n, hq, hkv, d, dtype
        self.qkv = stored(rng.standard_normal((n, hq + 2 * hkv, d)) * 3, dtype)
        self.q, self.k, self.v = np.split(self.qkv, [hq, hq + hkv], 1)
        self.w = [stored(rng.uniform(-2, 2, d), dtype) if norm else None for _ in range(2)]
        self.table = _table(300, rot) if rot else None
        self.pos = rng.integers(0, 300, (axes, n)).astype(np.int32)
        self.axis = None
        if axes > 1:
            self.axis = (rng.integers(0, axes, rot // 2) if split == "mixed"
                         else np.arange(rot // 2) * axes // max(1, rot // 2)).tolist()
        self.nb = pool or -(-n // 16) + 2
        self.slots = rng.permutation(self.nb * 16)[:n].astype(np.int64)

    def wants(self, inter, eps=1e-6):
        return [lc.qk_norm_rope(x, w, eps, self.table, self.pos, self.axis, inter)
                for x, w in ((self.q, self.w[0]), (self.k, self.w[1]))]

    def dev(self):
        t = to_dev(self.qkv)
        q, k, v = t[:, :self.hq], t[:, self.hq:self.hq + self.hkv], t[:, self.hq + self.hkv:]
        return q, k, v, [None if w is None else to_dev(w) for w in self.w], (
            None if self.table is None else to_dev(self.table)), to_dev(self.pos)


SHAPES = [  # n, hq, hkv, d, rot
    (1, 32, 8, 128, 128), (1, 1, 1, 64, 64), (3, 7, 5, 64, 32), (17, 8, 1, 128, 96),
          (130, 5, 2, 128, 16),
    (33, 16, 16, 64, 48), (5, 4, 4, 128, 0), (2049, 3, 1, 64, 64),
]


@pytest.mark.parametrize("n, hq, hkv, d, rot", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_norm_rope(n, hq, hkv, d, rot, dtype, inter, norm):
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    c = Case(n, hq, hkv, d, dtype, rot, norm=norm, seed=n + d)
    q, k, v, w, table, pos = c.dev()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out, k_out = (torch.full((n, h, d), 9.0, device="cuda").to(q.dtype) for h in (hq, hkv))
    B.pkv_qk_norm_rope(q, k, pos, table, q_out, k_out, *w, interleaved=inter, dev_status=st)
    wants = c.wants(inter)
    for got, want, x, wt in zip((q_out, k_out), wants, (c.q, c.k), c.w):
        err = np.abs(out_to_f64(got) - want)
        assert (err <= _tolerance(x, wt, 1e-6, want, dtype)).all()
    # the same rows through the cache
    kc, vc = (torch.full((c.nb, hkv, 16, d), 9.0, device="cuda").to(q.dtype) for _ in range(2))
    q2 = torch.empty_like(q_out)
    B.pkv_qk_norm_rope_append(q, k, v, pos, table, to_dev(c.slots), kc, vc, q2, *w,
                              interleaved=inter,
                              dev_status=st)
    assert torch.equal(q2.view(torch.int16), q_out.view(torch.int16)) and int(st.item()) == 0
    s = to_dev(c.slots)
    for cache, rows in ((kc, k_out), (vc, v)):
        want = torch.full((c.nb * 16, hkv, d), 9.0, device="cuda").to(q.dtype)
        want[s] = rows
        got = cache.transpose(1, 2).reshape(c.nb * 16, hkv, d)
        assert torch.equal(got.contiguous().view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("split", ["even", "mixed"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d, rot", [(128, 128), (128, 96), (64, 64)])
def test_position_axes(axes, split, inter, d, rot):
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    c = Case(21, 6, 2, d, "bf16", rot, axes=axes, seed=axes, split=split)
    q, k, _, w, table, pos = c.dev()
    q_out, k_out = torch.empty((21, 6, d), dtype=q.dtype, device="cuda"), torch.empty((21, 2, d),
            dtype=q.dtype, device="cuda")
    B.pkv_qk_norm_rope(q, k, pos, table, q_out, k_out, *w, pair_axis=c.axis, interleaved=inter)
    for got, want, x, wt in zip((q_out, k_out), c.wants(inter), (c.q, c.k), c.w):
        assert (np.abs(out_to_f64(got) - want) <= _tolerance(x, wt, 1e-6, want, "bf16")).all()


@pytest.mark.parametrize("inter", [False, True])
def test_in_place(inter):
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    c = Case(40, 4, 2, 128, "f16", 96, seed=1)
    q, k, _, w, table, pos = c.dev()
    q, k = q.contiguous(), k.contiguous()
    q_out, k_out = torch.empty_like(q), torch.empty_like(k)
    B.pkv_qk_norm_rope(q, k, pos, table, q_out, k_out, *w, interleaved=inter)
    B.pkv_qk_norm_rope(q, k, pos, table, q, k, *w, interleaved=inter)
    assert torch.equal(q, q_out) and torch.equal(k, k_out)


def test_zero_rows_and_large_values():
    """eps keeps a zero row finite; squares near fp32's range are summed in fp32."""
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    c = Case(4, 2, 2, 64, "bf16", 64, seed=2)
    c.q[1] = c.k[1] = 0
    c.q[2] = c.k[2] = stored(np.full((2, 64), 1e18), "bf16")
    c.qkv = np.concatenate([c.q, c.k, c.v], 1)
    q, k, _, w, table, pos = c.dev()
    q_out, k_out = torch.empty((4, 2, 64), dtype=q.dtype, device="cuda"), torch.empty((4, 2, 64),
            dtype=q.dtype, device="cuda")
    B.pkv_qk_norm_rope(q, k, pos, table, q_out, k_out, *w, eps=1e-5)
    for got, want, x, wt in zip((q_out, k_out), c.wants(False, 1e-5), (c.q, c.k), c.w):
        assert (np.abs(out_to_f64(got) - want) <= _tolerance(x, wt, 1e-5, want, "bf16")).all()
    assert (out_to_f64(q_out)[1] == 0).all()


def test_slots_and_positions_outside():
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    c = Case(6, 2, 1, 128, "bf16", 128, axes=2, seed=3)
    c.slots[1], c.slots[2] = -1, c.nb * 16
    c.pos[1, 4] = 300
    c.pos[0, 5] = -1
    q, k, v, w, table, pos = c.dev()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kc, vc = (torch.full((c.nb, 1, 16, 128), 9.0, device="cuda").to(q.dtype) for _ in range(2))
    q_out = torch.full((6, 2, 128), 9.0, device="cuda").to(q.dtype)
    B.pkv_qk_norm_rope_append(q, k, v, pos, table, to_dev(c.slots), kc, vc, q_out, *w,
                              pair_axis=c.axis,
                              dev_status=st)
    assert int(st.item()) == B.DEV_BAD_SLOT | B.DEV_BAD_INDEX
    c.pos[:, 4:] = 0
    want = c.wants(False)[0]
    got = out_to_f64(q_out)
    tol = _tolerance(c.q, c.w[0], 1e-6, want, "bf16")
    assert (np.abs(got - want) <= tol)[:4].all() and (got[4:] == 9).all()
    flat = decode_kv(to_host_bits(vc)).transpose(0, 2, 1, 3).reshape(-1, 1, 128)
    written = np.flatnonzero((flat != 9).any((1, 2)))
    assert sorted(written) == sorted(c.slots[[0, 3]])
