"""Runs of queries over INT8 values of very different sizes."""

import numpy as np
import pytest

from _longctx import HALF_STEP
from _pkv_helpers import out_to_f64
from _window import Windowed, close
from oracle import window as ow

pytestmark = pytest.mark.gpu

I8 = [("i8", "bf16"), ("i8", "f16")]
# queries, heads per group: every kernel that the sizes choose
SHORT, TILE, LONG = ([5, 4], 2), ([13, 9], 2), ([400, 300], 2)


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_decode_05_gb300.build import build
    build()


def kernel(c, max_q=None):
    from paged_kv_decode_05_gb300 import binding as B
    code = {"bf16": B.PKV_BF16, "f16": B.PKV_F16, "i8": B.PKV_I8}
    nb, hkv, _, d = c.k.shape
    return B.pkv_testing_window_multiquery_kernel(
        len(c.lens), c.q.shape[1], max(c.counts), B.CacheDesc(nb, 16, hkv, d, code[c.kv]),
        code[c.qt], c.tables.shape[1], c.window, c.sinks)[0]


def run(c, parts=0, split=False):
    """``split``: an out that is not 16-byte aligned keeps long runs off the kernel of whole tiles."""
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    t = c.gpu()
    if split:
        t["out"] = torch.empty(t["out"].numel() + 2, dtype=t["out"].dtype,
                               device="cuda")[2:].view(t["out"].shape)
    ws = torch.empty(B.pkv_window_multiquery_workspace_size(len(c.lens), c.q.shape[1],
                                                            max(c.counts), t["k"], parts),
                     dtype=torch.uint8, device="cuda")
    B.pkv_window_multiquery_attn(t["q"], t["cu"], max(c.counts), t["k"], t["v"], t["tables"],
                                 t["lens"], c.scale, c.window, c.sinks, t["out"], ws,
                                 t["k_scales"], t["v_scales"], parts, t["status"])
    assert int(t["status"].item()) == 0
    return out_to_f64(t["out"])


def expect(c):
    """(exact, tolerance) by counting roundings, as in ``_window.tolerance``, but by what a row
    itself sees: sizes are sums over its own tokens, and the one absolute term, weights in fp16
    below 2^-14, goes with the largest V scale among them. Over INT8 a weight times its scale
    enters by 2^7 or more of the row's largest such product, off by 2^-25: 2^-32 127 of that
    scale a token. Weights over 16-bit caches come in two parts: 2^-16 (bf16), 2^-21 (fp16);
    over INT8 in one (2^-11), under an fp16 q in two. An fp16 output has no step below 2^-24."""
    k, v, kz, vz = c.sequences()
    lens, top = c.lens.tolist(), 0.0
    args = (c.q, k, v, c.counts, lens, c.scale, c.window, c.sinks)
    big = 0.0
    if c.kv == "i8":
        blk = [c.true_tables[b, np.arange(n) // 16] for b, n in enumerate(lens)]
        vs = [np.nan_to_num(c.v_scales[x]) for x in blk]
        # codes may enter the products as 1152 + c, whose 1152 comes off the sums
        kz = [np.abs(x) + 1152.0 * np.nan_to_num(c.k_scales[y])[..., None] for x, y in zip(k, blk)]
        vb = [np.abs(x) + 1152.0 * y[..., None] for x, y in zip(v, vs)]
        big = ow.window_attention(*args, None, vb)[1]
        top, at, g = np.zeros(c.q.shape[:2]), 0, c.q.shape[1] // c.hkv
        for b, (n, length) in enumerate(zip(c.counts, lens)):
            for i in range(n):
                t = ow.visible(length - n + i, length, c.window, c.sinks)
                top[at + i] = np.repeat(vs[b][t].max(0), g)
            at += n
    want, size, dots, most = ow.window_attention(*args, kz, None)
    p = {"bf16": 2.0 ** -16, "f16": 2.0 ** -21,
         "i8": 2.0 ** -11 if c.qt == "bf16" else 2.0 ** -21}[c.kv]
    steps = 2 * (most / 16 + 4) * 17 * 2.0 ** -23
    weight = 2 * abs(c.scale) * dots * (4 * 17 + 3) * 2.0 ** -23 + 2.0 ** -20 + p + steps
    tiny = most * 2.0 ** -31 * 127 * top
    if c.kv == "f16":
        tiny = most * 2.0 ** -25 * np.nanmax(np.abs(np.concatenate(v)))
    return want, (HALF_STEP[c.qt] * np.abs(want) + weight[..., None] * size * 1.01 + steps * big
                  + np.asarray(tiny)[..., None] + 2.0 ** -25 * (c.qt == "f16") + 1e-40)


def check(c, parts=(0, 7)):
    want, tol = expect(c)
    for n in parts if kernel(c) != "mq_wide_kernel" else ():
        close(run(c, n), want, tol)
    close(run(c, split=True), want, tol)


@pytest.mark.parametrize("kv, q", I8)
@pytest.mark.parametrize("counts, g", [SHORT, TILE, LONG])
@pytest.mark.parametrize("window, sinks, d", [(1, 0, 128), (1, 0, 64), (40, 3, 128), (0, 0, 64)])
def test_int8_scales_of_every_size(kv, q, counts, g, window, sinks, d):
    """V scales over 12 orders of magnitude, zero ones among them, by block and head."""
    c = Windowed([600, 700], 2, d, kv, window, sinks, seed=8, q=q, g=g, counts=counts)
    rng = np.random.default_rng(2)
    used = np.isfinite(c.v_scales)
    lo, hi = (-9, 3) if q == "bf16" else (-10, 2)
    s = 10.0 ** rng.uniform(lo, hi, c.v_scales.shape) * (rng.random(c.v_scales.shape) > 0.1)
    c.v_scales = np.where(used, s, np.nan).astype(np.float32)
    check(c)


@pytest.mark.parametrize("kv, q", I8)
@pytest.mark.parametrize("counts, g", [SHORT, TILE, LONG])
@pytest.mark.parametrize("size", [1e-3, 1e-4, 1e-6, 1e-9, 1e-30, 1e30])
def test_int8_scales_of_one_size(kv, q, counts, g, size):
    if q == "f16" and not 1e-7 < size < 1e2:
        pytest.skip("outputs beyond fp16's range")
    c = Windowed([600, 700], 2, 128, kv, 300, 3, seed=9, q=q, g=g, counts=counts)
    c.v_scales = (np.float32(size) * np.abs(c.v_scales)).astype(np.float32)
    check(c)


@pytest.mark.parametrize("counts, g", [SHORT, TILE, LONG])
def test_int8_blocks_of_two_sizes(counts, g):
    """A block of scale 1e6 that the last rows do not see, theirs are 1e-6."""
    c = Windowed([600, 700], 1, 128, "i8", 40, 0, seed=3, q="bf16", g=g, counts=counts)
    for b, length in enumerate(c.lens.tolist()):
        for j in range(-(-length // 16)):
            near = 16 * j >= length - max(1, counts[b] // 2) - 20
            c.v_scales[c.true_tables[b, j]] *= 1e-6 if near else 1e6
    check(c)
