"""Decode attention over a sliding window and sinks on the GPU, every cache type."""

import numpy as np
import pytest

from _pkv_helpers import out_to_f64, to_dev
from _window import Windowed, close

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16"), ("f16", "f16"), ("i8", "bf16"), ("i8", "f16"), ("u4", "bf16"),
         ("u4", "f16")]


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_decode_05_gb300.build import build
    build()


def run(c, t, parts=0):
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    ws = torch.empty(B.pkv_window_decode_workspace_size(len(c.lens), c.q.shape[1], t["k"], parts),
                     dtype=torch.uint8, device="cuda")
    B.pkv_window_decode_attn(t["q"], t["k"], t["v"], t["tables"], t["lens"], c.scale, c.window,
                             c.sinks, t["out"], ws, t["k_scales"], t["v_scales"], parts,
                             t["status"])
    return out_to_f64(t["out"])


@pytest.mark.parametrize("kv, q", TYPES)
@pytest.mark.parametrize("g", [1, 2, 4, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_types_and_groups(kv, q, g, d):
    c = Windowed([1, 0, 40, 257, 700], 3, d, kv, 100, 5, seed=g, q=q, g=g)
    t = c.gpu()
    want, tol = c.expect()
    for parts in (0, 1, 7, 64):
        t["out"].fill_(float("nan"))
        close(run(c, t, parts), want, tol)
    assert int(t["status"].item()) == 0


@pytest.mark.parametrize("kv, q", TYPES)
@pytest.mark.parametrize("window, sinks", [(1, 0), (1, 1), (16, 0), (17, 16), (15, 17), (64, 3),
                                           (100, 40), (333, 0), (700, 9), (5000, 2), (0, 0),
                                           (0, 7), (2, 600), (2**31 - 1, 2**31 - 1)])
def test_windows_and_sinks(kv, q, window, sinks):
    """Windows and sinks that end at, before and behind a block's border, meet, cover everything."""
    c = Windowed([0, 1, 2, 16, 17, 31, 48, 64, 65, 200, 333, 334, 600], 2, 128, kv, window, sinks,
                 seed=window % 97, q=q, g=4, cols=2)
    t = c.gpu()
    want, tol = c.expect()
    for parts in (0, 5, 40):
        t["out"].fill_(float("nan"))
        close(run(c, t, parts), want, tol)
    assert int(t["status"].item()) == 0


@pytest.mark.parametrize("kv, q", TYPES)
def test_long_sequences_and_many(kv, q):
    """Long contexts, more sequences than the exact prefix holds, all forms of the split."""
    for lens, window, sinks, g in (([9000], 2000, 100, 4), ([5, 4100, 2500, 0, 3001], 0, 0, 2),
                                   ([37 * i % 200 for i in range(300)], 50, 4, 1)):
        c = Windowed(lens, 1, 64 if len(lens) > 5 else 128, kv, window, sinks, seed=len(lens), q=q,
                     g=g)
        t = c.gpu()
        want, tol = c.expect()
        for parts in (0, 33, 1216):
            t["out"].fill_(float("nan"))
            close(run(c, t, parts), want, tol)
        assert int(t["status"].item()) == 0


@pytest.mark.parametrize("kv, q", TYPES)
def test_bad_lengths_and_blocks_are_flagged(kv, q):
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    c = Windowed([90, 40, 64, 80], 2, 64, kv, 30, 3, seed=1, q=q, g=2)
    t = c.gpu()
    want, tol = c.expect()
    t["tables"][0, 5] = len(c.k)               # a visible block outside the pool
    t["lens"][1] = -5
    t["tables"][2, 0] = -1                     # the sinks' block
    for parts in (0, 9):
        t["status"].zero_()
        got = run(c, t, parts)
        assert int(t["status"].item()) == B.DEV_BAD_LENGTH | B.DEV_BAD_BLOCK
        close(got[3], want[3], tol[3])
        assert (got[1] == 0).all() and np.isfinite(got).all()
    t["lens"][1] = 16 * c.mb + 1               # clamped to the table, flagged
    t["tables"].clamp_(0, len(c.k) - 1)
    t["status"].zero_()
    got = run(c, t, 9)
    assert int(t["status"].item()) == B.DEV_BAD_LENGTH
    close(got[3], want[3], tol[3])
    torch.cuda.synchronize()


def test_sizes_of_4_bit_scales():
    """Values from 1e-30 to 1e30 within one sequence and between sequences: P carries the scale
    into fp16 at an exponent of its own."""
    import torch
    for e in (-30, -10, 0, 10, 30):
        c = Windowed([100, 300], 2, 128, "u4", 0, 0, seed=e + 50, q="bf16", g=4, std=10.0 ** e)
        c.scale = c.scale * 10.0 ** -e
        t = c.gpu()
        want, tol = c.expect()
        for parts in (0, 6):
            close(run(c, t, parts), want, tol)
    # a scale that grows a millionfold on the way
    c = Windowed([500], 1, 128, "u4", 0, 0, seed=9, q="bf16", g=2)
    for i in range(2):
        codes, pairs = c.pairs[i]
        at = [(c.true_tables[0, t // 16], t % 16) for t in range(500)]
        for n, (blk, row) in enumerate(at):
            if i:
                pairs[blk, 0, row] *= 2.0 ** (n // 25 - 10)
        from _longctx import stored
        if i:
            c.v_scales = stored(np.where(c.seen[:, None, :, None], pairs, np.nan), "bf16")
    t = c.gpu()
    want, tol = c.expect()
    for parts in (0, 3):
        close(run(c, t, parts), want, tol)
    torch.cuda.synchronize()


@pytest.mark.parametrize("kv, q", TYPES)
def test_visible_nan_and_infinite_scores_reach_the_row(kv, q):
    c = Windowed([300, 300], 1, 128, kv, 64, 2, seed=3, q=q, g=4)
    t = c.gpu()
    want, tol = c.expect()
    t["q"][0, 1, 5] = float("nan")
    for parts in (0, 4):
        got = run(c, t, parts)
        assert np.isnan(got[0, 1]).all()
        close(got[0, [0, 2, 3]], want[0, [0, 2, 3]], tol[0, [0, 2, 3]])
        close(got[1], want[1], tol[1])


def test_window_zero_is_decode_attention():
    """Without a window, the same rows as pkv_decode_attn within both calls' tolerance."""
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    c = Windowed([700, 33, 1], 2, 128, "bf16", 0, 0, seed=8, g=4)
    t = c.gpu()
    want, tol = c.expect()
    got = run(c, t)
    ws = torch.empty(B.pkv_decode_workspace_size(3, 8, t["k"]), dtype=torch.uint8, device="cuda")
    other = torch.empty_like(t["out"])
    B.pkv_decode_attn(t["q"], t["k"], t["v"], t["tables"], t["lens"], c.scale, other, ws)
    close(got, want, tol)
    close(out_to_f64(other), got, 2 * tol + 2e-3)


def test_repeatable():
    """The same call gives the same bits."""
    import torch
    for kv, q in TYPES:
        c = Windowed([2000, 700, 1500], 2, 128, kv, 900, 10, seed=5, q=q, g=4)
        t = c.gpu()
        for parts in (0, 50):
            run(c, t, parts)
            first = t["out"].clone()
            for _ in range(5):
                t["out"].zero_()
                run(c, t, parts)
                assert torch.equal(first, t["out"])


def test_pool_beyond_32_bits():
    """Element offsets past 2^32 in a 4-bit pool: pairs and codes at both ends."""
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    hkv, d, nb = 8, 128, 600000                # 4.9e9 bytes of codes for K
    codes = [torch.zeros((nb, hkv, 16, d // 2), dtype=torch.uint8, device="cuda") for _ in range(2)]
    pairs = [torch.full((nb, hkv, 16, 2), float("nan"), device="cuda").bfloat16() for _ in range(2)]
    blocks = torch.tensor([nb - 1, 0, nb - 2], dtype=torch.int32, device="cuda")
    slots = (blocks.long()[:, None] * 16 + torch.arange(16, device="cuda")).flatten()[:40]
    k, v = (torch.randn((40, hkv, d), device="cuda").bfloat16() for _ in range(2))
    B.pkv_u4_append(k, v, slots.contiguous(), *codes, *pairs)
    outs = [torch.zeros((3, hkv, 16, d), device="cuda").bfloat16() for _ in range(2)]
    B.pkv_u4_read_blocks(*codes, *pairs, blocks, *outs,
                         torch.arange(3, dtype=torch.int32, device="cuda"))
    q = torch.randn((1, 32, d), device="cuda").bfloat16()
    lens = torch.tensor([40], dtype=torch.int32, device="cuda")
    got, want = torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty(B.pkv_window_decode_workspace_size(1, 32, codes[0]), dtype=torch.uint8,
                     device="cuda")
    B.pkv_window_decode_attn(q, *codes, blocks[None], lens, d ** -0.5, 0, 0, got, ws, *pairs)
    B.pkv_window_decode_attn(q, *outs, torch.arange(3, dtype=torch.int32, device="cuda")[None],
                             lens, d ** -0.5, 0, 0, want, ws)
    # the values read back are off by their own rounding, 2^-8, in k (scores to about 6) and v
    assert float((got.float() - want.float()).abs().max()) < 0.1
    assert bool(torch.isfinite(got).all())


def test_the_stall_hook_refuses_4_bit_caches():
    """Nothing there waits on a barrier."""
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    c = Windowed([20], 1, 64, "u4", 0, 0, q="bf16")
    t = c.gpu()
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    with pytest.raises(B.PkvError):
        B.pkv_testing_window_decode_attn_stall(t["q"], t["k"], t["v"], t["tables"], t["lens"],
                                               c.scale, 0, 0, t["out"], ws, wait_limit_ns=1000,
                                               stall_worker=0, k_scales=t["k_scales"],
                                               v_scales=t["v_scales"])


@pytest.mark.parametrize("kv, q", TYPES[:4])
def test_a_wait_that_runs_out_is_reported(kv, q):
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    c = Windowed([2000, 1900, 2000], 2, 128, kv, 1500, 4, seed=2, q=q, g=4)
    t = c.gpu()
    want, tol = c.expect()
    ws = torch.empty(B.pkv_window_decode_workspace_size(3, 8, t["k"], 48), dtype=torch.uint8,
                     device="cuda")
    args = (t["q"], t["k"], t["v"], t["tables"], t["lens"], c.scale, c.window, c.sinks, t["out"],
            ws)
    B.pkv_testing_window_decode_attn_stall(*args, wait_limit_ns=20_000_000, stall_worker=3,
                                           num_parts=48, k_scales=t["k_scales"],
                                           v_scales=t["v_scales"], dev_status=t["status"])
    torch.cuda.synchronize()
    assert int(t["status"].item()) == B.DEV_TIMEOUT
    t["status"].zero_()
    close(run(c, t, 48), want, tol)
    assert int(t["status"].item()) == 0


@pytest.mark.parametrize("kv, q", TYPES)
@pytest.mark.parametrize("scale", [0.0, -0.2, 30.0])
def test_any_softmax_scale(kv, q, scale):
    c = Windowed([200, 150], 3, 64, kv, 90, 2, seed=6, q=q, g=4)
    c.scale = scale
    t = c.gpu()
    want, tol = c.expect()
    for parts in (0, 5):
        close(run(c, t, parts), want, tol)


@pytest.mark.parametrize("kv, q", TYPES)
def test_many_kv_heads(kv, q):
    """More kv heads than workers asked for, and numbers of them that divide nothing."""
    for hkv, parts in ((40, 7), (5, 33), (13, 0)):
        c = Windowed([300, 17, 90], hkv, 64, kv, 70, 5, seed=hkv, q=q, g=1)
        t = c.gpu()
        want, tol = c.expect()
        close(run(c, t, parts), want, tol)
