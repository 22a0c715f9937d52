"""The 4-bit cache on the GPU: rows quantised as they are written, blocks read back."""

import numpy as np
import pytest

from _longctx import stored
from _pkv_helpers import to_dev, to_host_bits
from oracle import decode_kv
from oracle import window as ow

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_decode_05_gb300.build import build
    build()


def cache(nb, hkv, d, dtype, fill=0xA5):
    """Codes and pairs of an empty cache, filled with a pattern that calls must leave alone."""
    import torch
    dt = {"bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    codes = [torch.full((nb, hkv, 16, d // 2), fill, dtype=torch.uint8, device="cuda")
             for _ in range(2)]
    pairs = [torch.full((nb, hkv, 16, 2), -3.5, dtype=dt, device="cuda") for _ in range(2)]
    return codes, pairs


def hard_rows(rng, n, hkv, d, dtype):
    """Normal rows, and rows where a decision is near: constant ones, ties, far offsets, the
    type's largest and smallest values, signed zeros."""
    x = rng.standard_normal((n, hkv, d))
    kinds = [lambda: np.full(d, 1.5), lambda: np.zeros(d) * -1.0,
             lambda: np.arange(d) % 31 * 0.5 - 3.0,           # multiples of s / 2: ties
             lambda: 200.0 + rng.integers(0, 3, d), lambda: rng.standard_normal(d) * 1e-6,
             lambda: rng.standard_normal(d) * 2.0 ** -23,
             lambda: np.where(np.arange(d) == 5, 60000.0, rng.standard_normal(d)),
             lambda: np.where(rng.random(d) < 0.5, -65504.0, 65504.0),
             lambda: rng.integers(-8, 8, d) * 0.0625]
    if dtype == "bf16":
        kinds += [lambda: rng.standard_normal(d) * 1e30, lambda: rng.standard_normal(d) * 1e-33,
                  lambda: rng.standard_normal(d) * 1e-39, lambda: np.where(np.arange(d) == 0, 1.5e38,
                                                                           -1.5e38)]
    for i, make in enumerate(kinds * 2):
        x[(3 * i + 1) % n, i % hkv] = make()
    return stored(x, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hkv, d, n", [(1, 64, 1), (3, 128, 37), (8, 128, 200), (5, 64, 333),
                                       (2, 128, 4001)])
def test_write_and_read(dtype, hkv, d, n):
    """Codes and pairs bit for bit; rows and blocks that no slot names stay as they were; the
    values read back to the last bit."""
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    rng = np.random.default_rng(n + d)
    k, v = (hard_rows(rng, n, hkv, d, dtype) for _ in range(2))
    nb = n // 8 + 4
    slots = rng.permutation(nb * 16)[:n].astype(np.int64)
    slots[rng.random(n) < 0.1] = -1
    codes, pairs = cache(nb, hkv, d, dtype)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    # both are parts of one projection's rows
    rows = torch.zeros((n, 3 * hkv, d), dtype=pairs[0].dtype, device="cuda")
    rows[:, hkv:2 * hkv], rows[:, 2 * hkv:] = to_dev(k), to_dev(v)
    B.pkv_u4_append(rows[:, hkv:2 * hkv], rows[:, 2 * hkv:], to_dev(slots), *codes, *pairs,
                    dev_status=status)
    assert int(status.item()) == 0
    values = []
    for x, c, p in zip((k, v), codes, pairs):
        want_c = np.full((nb * 16, hkv, d // 2), 0xA5, np.uint8)
        want_p = np.full((nb * 16, hkv, 2), -3.5)
        live = slots >= 0
        q, s = ow.u4_quantise(x[live])
        want_c[slots[live]], want_p[slots[live]] = ow.u4_pack(q), s
        want_c = want_c.reshape(nb, 16, hkv, -1).transpose(0, 2, 1, 3)
        want_p = want_p.reshape(nb, 16, hkv, 2).transpose(0, 2, 1, 3)
        got_p = decode_kv(to_host_bits(p))
        assert (got_p == want_p).all(), np.argwhere(got_p != want_p)[:3]
        assert (c.cpu().numpy() == want_c).all()
        # what a row stands for is at most half a step from what was written
        off = np.abs(ow.u4_values(q, s) - decode_kv(x[live]))
        assert (off <= s[..., :1] / 2 + 2.0 ** -22 * np.abs(decode_kv(x[live])).max(
            -1, keepdims=True)).all()
        full = np.stack([want_c & 15, want_c >> 4], -1).reshape(nb, hkv, 16, d)
        exact = full.astype(np.float32) * want_p[..., :1].astype(np.float32)     # exact products
        values.append(stored(exact + want_p[..., 1:].astype(np.float32), dtype))
    # read every second block, one of them twice, to scattered places
    src = np.concatenate([np.arange(0, nb, 2), [0]]).astype(np.int32)
    out_nb = len(src) + 2
    dst = rng.permutation(out_nb)[:len(src)].astype(np.int32)
    outs = [torch.full((out_nb, hkv, 16, d), 7.0, dtype=p.dtype, device="cuda") for p in pairs]
    B.pkv_u4_read_blocks(*codes, *pairs, to_dev(src), *outs, to_dev(dst), dev_status=status)
    assert int(status.item()) == 0
    for out, val in zip(outs, values):
        want = np.full(out.shape, stored(np.array(7.0), dtype), val.dtype)
        want[dst] = val[src]
        assert (decode_kv(to_host_bits(out)) == decode_kv(want)).all()


def test_write_skips_and_flags_slots():
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    codes, pairs = cache(3, 2, 64, "bf16")
    x = torch.randn((5, 2, 64), device="cuda").bfloat16()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.tensor([-1, 48, 5, 1 << 40, -(1 << 40)], device="cuda")
    B.pkv_u4_append(x, x, slots, *codes, *pairs, dev_status=status)
    assert int(status.item()) == B.DEV_BAD_SLOT
    assert int((pairs[0] != -3.5).any(-1).sum()) == 2      # the two heads' rows of slot 5
    assert bool((pairs[1][0, :, 5] != -3.5).any(-1).all())
    B.pkv_u4_append(x, x, slots, *codes, *pairs)           # no status word
    B.pkv_u4_append(x[:0], x[:0], slots[:0], *codes, *pairs)
    torch.cuda.synchronize()


def test_read_skips_and_flags_blocks():
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    codes, pairs = cache(3, 1, 64, "f16")
    for p in pairs:
        p[..., 0], p[..., 1] = 1.0, 0.0
    outs = [torch.full((4, 1, 16, 64), 9.0, device="cuda").half() for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    src = torch.tensor([3, -1, 1, 2, 0], dtype=torch.int32, device="cuda")
    dst = torch.tensor([0, 1, 4, -1, 3], dtype=torch.int32, device="cuda")
    B.pkv_u4_read_blocks(*codes, *pairs, src, *outs, dst, dev_status=status)
    assert int(status.item()) == B.DEV_BAD_BLOCK
    for out in outs:
        assert bool((out[:3] == 9).all())
        assert bool((out[3, 0, :, 0::2] == 5).all()) and bool((out[3, 0, :, 1::2] == 10).all())


def test_rows_with_no_finite_range_stay_their_own():
    """Infinite and NaN inputs are a caller error; they spoil their own rows only."""
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    x = torch.randn((16, 2, 128), device="cuda").half()
    bad = x.clone()
    bad[3, 1, 7], bad[9, 0, 0] = float("inf"), float("nan")
    slots = torch.arange(16, device="cuda")
    a, b = cache(1, 2, 128, "f16"), cache(1, 2, 128, "f16")
    B.pkv_u4_append(x, x, slots, *a[0], *a[1])
    B.pkv_u4_append(bad, bad, slots, *b[0], *b[1])
    same = (a[0][0] == b[0][0]).all(-1) & (a[1][0] == b[1][0]).all(-1)
    want = torch.ones_like(same)
    want[0, 1, 3] = want[0, 0, 9] = False
    assert bool((same | ~want).all())
