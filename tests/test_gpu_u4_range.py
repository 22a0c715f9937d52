"""4-bit rows that reach the largest value of their type: what they stand for stays finite."""

import numpy as np
import pytest

from _longctx import HALF_STEP, stored
from _pkv_helpers import out_to_f64, to_dev, to_host_bits
from oracle import decode_kv
from oracle import window as ow

MOST = {"bf16": 255 * 2.0 ** 120, "f16": 65504.0}


def rows(dtype, n, d, seed=0):
    """Rows whose range is the type's, or ends at its largest or smallest value, as clamping leaves
    them. (max - min is finite in fp32.)"""
    rng = np.random.default_rng(seed)
    m = MOST[dtype]
    low = -m if dtype == "f16" else -1e36
    ends = [(0.0, m), (low, m), (-1.0, m), (m / 3, m), (0.99 * m, m), (m, m), (-m, 0.0),
            (-m, -m / 7), (-m, -m), (2.0 ** -24, m)]
    x = np.empty((n, d))
    for i in range(n):
        lo, hi = ends[i % len(ends)] if i < 4 * len(ends) else (
            (rng.uniform(low, m), m) if i % 2 else (-m, rng.uniform(-m, -low)))
        x[i] = rng.uniform(lo, hi, d) if i % 3 else np.where(rng.random(d) < 0.5, lo, hi)
        x[i, :2] = lo, hi
    return stored(np.clip(x, -m, m), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_the_oracle_keeps_its_type(dtype):
    x = rows(dtype, 200, 64)
    codes, pairs = ow.u4_quantise(x)
    f, s = decode_kv(x), pairs[:, :1]
    values = ow.u4_values(codes, pairs)
    assert codes.max() == 15 and (np.abs(values) <= MOST[dtype] * (1 + 2.0 ** -24)).all()
    assert np.isfinite(decode_kv(stored(values, dtype))).all()
    assert (np.abs(values - f) <= s / 2 + np.abs(f).max(1, keepdims=True) * 2.0 ** -22).all()
    # the scale is the rounded-up one, or the value next below it
    step = {"bf16": 2.0 ** -7, "f16": 2.0 ** -10}[dtype]
    want = (f.max(1) - f.min(1)) / 15
    assert (np.abs(s[:, 0] - want) <= want * step * 1.001).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hkv, d", [(2, 64), (3, 128)])
def test_written_read_back_and_attended_to(dtype, hkv, d):
    """Codes and pairs bit for bit, every value read back finite and within half a step of what
    was written; fp16: attention over such values of V too."""
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    n, dt = 160, {"bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    x = rows(dtype, n * hkv, d).reshape(n, hkv, d)
    k = stored(np.random.default_rng(1).standard_normal((n, hkv, d)), dtype)
    codes = [torch.zeros((n // 16, hkv, 16, d // 2), dtype=torch.uint8, device="cuda")
             for _ in range(2)]
    pairs = [torch.zeros((n // 16, hkv, 16, 2), dtype=dt, device="cuda") for _ in range(2)]
    slots = torch.arange(n, device="cuda")
    B.pkv_u4_append(to_dev(k), to_dev(x), slots, *codes, *pairs)
    c, p = ow.u4_quantise(x)
    got_p = decode_kv(to_host_bits(pairs[1])).transpose(0, 2, 1, 3).reshape(n, hkv, 2)
    assert (got_p == p).all()
    assert (codes[1].cpu().numpy().transpose(0, 2, 1, 3).reshape(n, hkv, -1) == ow.u4_pack(c)).all()
    out = [torch.empty((n // 16, hkv, 16, d), dtype=dt, device="cuda") for _ in range(2)]
    blocks = torch.arange(n // 16, dtype=torch.int32, device="cuda")
    B.pkv_u4_read_blocks(*codes, *pairs, blocks, *out, blocks)
    back = decode_kv(to_host_bits(out[1])).transpose(0, 2, 1, 3).reshape(n, hkv, d)
    f = decode_kv(x)
    assert np.isfinite(back).all()
    # half a step, x - lo rounded to fp32, the value rounded to its type
    assert (np.abs(back - f) <= p[..., :1] / 2 + np.abs(f).max(-1, keepdims=True) * 2.0 ** -22
            + HALF_STEP[dtype] * np.abs(back) * 1.01).all()
    if dtype == "bf16":
        return          # sums of such values pass fp32
    g = 2
    q = stored(np.random.default_rng(2).standard_normal((1, hkv * g, d)), dtype)
    ws = torch.empty(B.pkv_window_decode_workspace_size(1, hkv * g, codes[0]), dtype=torch.uint8,
                     device="cuda")
    kc, kp = ow.u4_quantise(k)
    for window in (0, 1, 2, 3, 7):
        for length in range(1, n + 1, 1 if window == 1 else 31):
            res = torch.empty((1, hkv * g, d), dtype=dt, device="cuda")
            lens = torch.tensor([length], dtype=torch.int32, device="cuda")
            B.pkv_window_decode_attn(to_dev(q), *codes, blocks[None], lens, d ** -0.5, window, 0,
                                     res, ws, *pairs)
            kv, vv = ow.u4_values(kc, kp)[:length], ow.u4_values(c, p)[:length]
            want, size, dots, most = ow.window_attention(
                q, [kv], [vv], [1], [length], d ** -0.5, window, 0,
                [(kc * kp[..., :1] + np.abs(kp[..., 1:]))[:length]],
                [(c * p[..., :1] + np.abs(p[..., 1:]))[:length]])
            # roundings as _window.tolerance counts them for 4-bit rows under an fp16 q
            score = d ** -0.5 * dots * (4 * 17 + 28) * 2.0 ** -23
            weight = 2 * score + 2.0 ** -20 + 2.0 ** -21 + 2 * (most / 16 + 4) * 17 * 2.0 ** -23
            tol = (HALF_STEP[dtype] * np.abs(want) + weight[..., None] * size * 1.01
                   + most * 2.0 ** -37 * 15 * p[..., 0].max())
            got = out_to_f64(res)
            assert np.isfinite(got).all()
            assert (np.abs(got - want) <= tol).all(), (window, length)


@pytest.mark.gpu
def test_a_destination_named_twice_holds_values_of_its_sources():
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    nb, hkv, d, m = 64, 4, 128, 40
    rng = np.random.default_rng(0)
    codes = [torch.from_numpy(rng.integers(0, 256, (nb, hkv, 16, d // 2)).astype(np.uint8)).cuda()
             for _ in range(2)]
    pairs = [torch.from_numpy(rng.random((nb, hkv, 16, 2))).cuda().half() for _ in range(2)]

    def read(src, dst):
        out = [torch.full((3, hkv, 16, d), 9.0, device="cuda").half() for _ in range(2)]
        B.pkv_u4_read_blocks(*codes, *pairs, src, *out, dst)
        return out

    src = torch.from_numpy(rng.permutation(nb)[:m].astype(np.int32)).cuda()
    once = [read(src[i:i + 1], torch.zeros_like(src[:1])) for i in range(m)]
    twice = read(src, (torch.arange(m, device="cuda") % 2).int())
    for x in range(2):
        for to in range(2):
            some = torch.stack([once[i][x][0] == twice[x][to] for i in range(to, m, 2)]).any(0)
            assert bool(some.all())
        assert bool((twice[x][2] == 9).all())
