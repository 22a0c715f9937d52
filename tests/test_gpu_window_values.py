"""Runs of queries over values of very different sizes: what a row does not see does not touch it,
and a row keeps its bits whatever size its values have."""

import numpy as np
import pytest

from _longctx import HALF_STEP, stored
from _pkv_helpers import out_to_f64
from _window import Windowed, close
from oracle import decode_kv
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
    for n in parts:
        close(run(c, n), want, tol)
    close(run(c, split=True), want, tol)


def values(c, factor):
    """The visible rows of a 16-bit V times ``factor`` [blocks, 1, 16 or 1, 1]."""
    live = c.seen[:, None, :, None]
    c.v = np.where(live, stored(np.where(live, decode_kv(c.v), 0.0) * factor, c.kv), c.v).astype(
        c.v.dtype)


@pytest.mark.parametrize("counts, g", [SHORT, TILE, LONG, ([200, 90], 1)])
def test_one_token_among_values_of_every_size(counts, g):
    """A window of 1: out is the token's own value, its neighbours 2^-100 to 2^100 of it."""
    c = Windowed([600, 700], 1, 128, "bf16", 1, 0, seed=5, g=g, counts=counts)
    assert (kernel(c) == "mq_wide_kernel") == (max(counts) * g > 32)
    rng = np.random.default_rng(1)
    values(c, 2.0 ** rng.uniform(-100, 100, (len(c.v), 1, 16, 1)))
    check(c)


@pytest.mark.parametrize("counts, g", [SHORT, TILE, LONG])
@pytest.mark.parametrize("far, near", [(2.0 ** 41, 1.0), (2.0 ** 48, 1.0), (2.0 ** 60, 2.0 ** -60),
                                       (1.0, 2.0 ** -20), (2.0 ** -30, 2.0 ** 30)])
def test_values_of_two_sizes(counts, g, far, near):
    """The tokens of the last rows are ``near``, those before them, which only others see, ``far``:
    by blocks that share a chunk of 128 tokens and by chunks."""
    c = Windowed([600, 700], 1, 128, "bf16", 40, 0, seed=6, g=g, counts=counts)
    factor = np.full((len(c.v), 1, 1, 1), far)
    for b, length in enumerate(c.lens.tolist()):
        for j in range(-(-length // 16)):
            if 16 * j >= length - max(1, counts[b] // 2) - 20:
                factor[c.true_tables[b, j]] = near
    values(c, factor)
    check(c)


def test_small_channels_beside_ordinary_ones():
    """Channels of 1e-6 and 1e-12 in rows of ordinary size keep the bits of their own."""
    for counts, g in (SHORT, TILE, LONG):
        c = Windowed([600, 700], 1, 64, "bf16", 200, 3, seed=7, g=g, counts=counts)
        values(c, 10.0 ** -(np.arange(64) % 3 * 6.0))
        check(c)


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


@pytest.mark.parametrize("counts, g", [SHORT, TILE, LONG])
@pytest.mark.parametrize("size, q", [(1e-3, "bf16"), (1e-4, "bf16"), (1e-6, "bf16"),
                                     (1e-9, "bf16"), (1e-30, "bf16"), (1e30, "bf16"),
                                     (1e-3, "f16"), (1e-4, "f16"), (1e-6, "f16")])
def test_int8_scales_of_one_size(q, counts, g, size):
    c = Windowed([600, 700], 2, 128, "i8", 300, 3, seed=9, q=q, g=g, counts=counts)
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
