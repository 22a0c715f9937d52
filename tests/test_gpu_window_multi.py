"""Runs of queries over a sliding window and sinks on the GPU, 16-bit and INT8 caches."""

import numpy as np
import pytest

from _longctx import HALF_STEP
from _pkv_helpers import out_to_f64, to_dev
from _window import Windowed, close, tolerance
from oracle import window as ow

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16"), ("f16", "f16"), ("i8", "bf16"), ("i8", "f16")]


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_decode_05_gb300.build import build
    build()


def expect(c):
    """(exact, tolerance). Runs of more than 32 rows over bf16 caches take P in one fp16 part.
    INT8 codes may enter the products as 1152 + c, whose 1152 comes off the sums: what the sums
    round by goes with that size (`steps`, scores), what a weight is off by with the values';
    weights are one fp16 part (2^-11) there, two under an fp16 output."""
    long = max(c.counts) * (c.q.shape[1] // c.hkv) > 32
    if c.kv != "i8":
        return c.expect(c.kv == "bf16" and long)
    k, v, _, _ = c.sequences()
    kb, vb = [], []
    for b, length in enumerate(c.lens.tolist()):
        blk = c.true_tables[b, np.arange(length) // 16]
        kb.append(np.abs(k[b]) + 1152.0 * np.nan_to_num(c.k_scales[blk])[..., None])
        vb.append(np.abs(v[b]) + 1152.0 * np.nan_to_num(c.v_scales[blk])[..., None])
    args = (c.q, k, v, c.counts, c.lens.tolist(), c.scale, c.window, c.sinks)
    want, size, dots, most = ow.window_attention(*args, kb, None)
    _, big, _, _ = ow.window_attention(*args, None, vb)
    steps = 2 * (most / 16 + 4) * 17 * 2.0 ** -23
    return want, tolerance(c, want, size, dots, most, c.qt == "bf16") + steps * big


def run(c, t, parts=0, max_q=None):
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    max_q = max(c.counts) if max_q is None else max_q
    ws = torch.empty(B.pkv_window_multiquery_workspace_size(len(c.lens), c.q.shape[1], max_q,
                                                            t["k"], parts),
                     dtype=torch.uint8, device="cuda")
    B.pkv_window_multiquery_attn(t["q"], t["cu"], max_q, t["k"], t["v"], t["tables"], t["lens"],
                                 c.scale, c.window, c.sinks, t["out"], ws, t["k_scales"],
                                 t["v_scales"], parts, t["status"])
    return out_to_f64(t["out"])


@pytest.mark.parametrize("kv, q", TYPES)
@pytest.mark.parametrize("g", [1, 2, 4, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_types_and_groups(kv, q, g, d):
    """Short and long runs: every kernel that the sizes choose."""
    for counts, lens in (([1, 3, 2], [60, 3, 230]), ([5, 0, 7, 4], [5, 9, 200, 99]),
                         ([28 // g, 1], [77, 40]), ([32 // g, 1], [99, 40]), ([33, 20], [90, 70]),
                         ([140, 1, 37], [200, 170, 37])):
        c = Windowed(lens, 2, d, kv, 40, 5, seed=g, q=q, g=g, counts=counts)
        t = c.gpu()
        want, tol = expect(c)
        for parts in (0, 1, 9):
            t["out"].fill_(float("nan"))
            close(run(c, t, parts), want, tol)
        assert int(t["status"].item()) == 0


@pytest.mark.parametrize("kv, q", TYPES)
@pytest.mark.parametrize("window, sinks", [(1, 0), (1, 1), (16, 0), (17, 16), (15, 17), (64, 3),
                                           (100, 40), (333, 0), (5000, 2), (0, 0), (0, 7), (2, 300),
                                           (2**31 - 1, 2**31 - 1), (40, 64), (30, 33)])
def test_windows_and_sinks(kv, q, window, sinks):
    for counts, lens, g in (([1, 4, 5, 3, 2, 6], [1, 300, 64, 65, 17, 33], 4),
                            ([70, 1, 130, 33], [333, 200, 140, 33], 2)):
        c = Windowed(lens, 1, 128, kv, window, sinks, seed=window % 97, q=q, g=g, counts=counts,
                     cols=2)
        t = c.gpu()
        want, tol = expect(c)
        for parts in (0, 5):
            t["out"].fill_(float("nan"))
            close(run(c, t, parts), want, tol)
        assert int(t["status"].item()) == 0


@pytest.mark.parametrize("kv, q", TYPES)
def test_long_runs(kv, q):
    """Prompt chunks whose later queries no longer see what the first ones do; a row spread that
    rescales."""
    for counts, lens, window, sinks, g, d in (([300, 257], [1500, 257], 200, 20, 1, 64),
                                              ([260], [3900], 1000, 70, 2, 128),
                                              ([513], [600], 64, 0, 1, 128)):
        c = Windowed(lens, 1, d, kv, window, sinks, seed=counts[0], q=q, g=g, counts=counts)
        c.scale *= 3
        t = c.gpu()
        want, tol = expect(c)
        for parts in (0, 21):
            t["out"].fill_(float("nan"))
            close(run(c, t, parts), want, tol)
        assert int(t["status"].item()) == 0


@pytest.mark.parametrize("kv, q", TYPES)
def test_one_query_each_is_window_decode(kv, q):
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    c = Windowed([90, 700, 1, 33], 2, 128, kv, 64, 3, seed=4, q=q, g=4, counts=[1] * 4)
    t = c.gpu()
    want, tol = expect(c)
    got = run(c, t)
    ws = torch.empty(B.pkv_window_decode_workspace_size(4, 8, t["k"]), dtype=torch.uint8,
                     device="cuda")
    other = torch.empty_like(t["out"])
    B.pkv_window_decode_attn(t["q"], t["k"], t["v"], t["tables"], t["lens"], c.scale, c.window,
                             c.sinks, other, ws, t["k_scales"], t["v_scales"])
    close(got, want, tol)
    close(out_to_f64(other), got, 2 * tol + HALF_STEP[c.qt] * np.abs(got))


@pytest.mark.parametrize("counts, g", [([3, 4, 2], 2), ([150, 160, 140], 1)])
@pytest.mark.parametrize("kv, q", TYPES)
def test_bad_shapes_and_blocks_are_flagged(kv, q, counts, g):
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    c = Windowed([300, 310, 170], 2, 64, kv, 100, 3, seed=1, q=q, g=g, counts=counts)
    t = c.gpu()
    want, tol = expect(c)
    t["lens"][0] = counts[0] - 1               # more queries than tokens: rows not written
    t["tables"][1, 18] = len(c.k)              # a visible block outside the pool: not seen
    for parts in (0, 9):
        t["status"].zero_()
        t["out"].fill_(77.0)
        got = run(c, t, parts)
        assert int(t["status"].item()) == B.DEV_BAD_LENGTH | B.DEV_BAD_BLOCK
        at = sum(counts[:2])
        assert (got[:counts[0]] == 77).all() and np.isfinite(got).all()
        close(got[at:], want[at:], tol[at:])
    t["lens"][0] = 300
    t["tables"].clamp_(0, len(c.k) - 1)
    t["status"].zero_()
    t["out"].fill_(77.0)
    got = run(c, t, 9, max(counts) - 1)         # a run longer than max_q_len
    assert int(t["status"].item()) == B.DEV_BAD_LENGTH
    assert (got[counts[0]:counts[0] + counts[1]] == 77).all()
    close(got[:counts[0]], want[:counts[0]], tol[:counts[0]])
    torch.cuda.synchronize()


def test_a_prompt_over_a_4_bit_cache():
    """Chunk by chunk: rows written in 4 bits, the prefix read back into a 16-bit scratch cache,
    the chunk's attention there; then single tokens over the 4-bit cache itself. The oracle
    attends to the oracle's own quantised rows."""
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    rng = np.random.default_rng(3)
    hkv, g, d, total, chunk, nb = 2, 4, 128, 300, 128, 24
    from _longctx import stored
    rows = [stored(rng.standard_normal((total, hkv, d)), "bf16") for _ in range(2)]
    q = stored(rng.standard_normal((total, hkv * g, d)), "bf16")
    table = rng.permutation(nb)[:19].astype(np.int32)
    slots = (table[np.arange(total) // 16].astype(np.int64) * 16 + np.arange(total) % 16)
    dev = "cuda"
    codes = [torch.zeros((nb, hkv, 16, d // 2), dtype=torch.uint8, device=dev) for _ in range(2)]
    pairs = [torch.zeros((nb, hkv, 16, 2), device=dev).bfloat16() for _ in range(2)]
    scratch = [torch.full((nb, hkv, 16, d), float("nan"), device=dev).bfloat16() for _ in range(2)]
    tab, k, v, qd = to_dev(table), to_dev(rows[0]), to_dev(rows[1]), to_dev(q)
    out = torch.empty_like(qd)
    parts = [ow.u4_quantise(x) for x in rows]
    vals = [stored(ow.u4_values(*p), "bf16") for p in parts]     # what the scratch cache holds
    from oracle import decode_kv
    ref = [decode_kv(x) for x in vals]
    for at in range(0, total - 44, chunk):
        n = min(chunk, total - 44 - at)
        B.pkv_u4_append(k[at:at + n], v[at:at + n], to_dev(slots[at:at + n]), *codes, *pairs)
        used = tab[:-(-(at + n) // 16)].contiguous()
        B.pkv_u4_read_blocks(*codes, *pairs, used, *scratch, used)
        cu = torch.tensor([0, n], dtype=torch.int32, device=dev)
        lens = torch.tensor([at + n], dtype=torch.int32, device=dev)
        for window, sinks in ((0, 0), (100, 4)):
            ws = torch.empty(B.pkv_window_multiquery_workspace_size(1, hkv * g, n, scratch[0]),
                             dtype=torch.uint8, device=dev)
            B.pkv_window_multiquery_attn(qd[at:at + n], cu, n, *scratch, tab[None], lens,
                                         d ** -0.5, window, sinks, out[at:at + n], ws)
            want, size, dots, most = ow.window_attention(
                q[at:at + n], [ref[0][:at + n]], [ref[1][:at + n]], [n], [at + n], d ** -0.5, window,
                sinks)
            case = type("C", (), dict(kv="bf16", qt="bf16", scale=d ** -0.5))
            close(out_to_f64(out[at:at + n]), want,
                  tolerance(case, want, size, dots, most, n * g > 32))
    for at in range(total - 44, total):
        B.pkv_u4_append(k[at:at + 1], v[at:at + 1], to_dev(slots[at:at + 1]), *codes, *pairs)
        lens = torch.tensor([at + 1], dtype=torch.int32, device=dev)
        ws = torch.empty(B.pkv_window_decode_workspace_size(1, hkv * g, codes[0]),
                         dtype=torch.uint8, device=dev)
        B.pkv_window_decode_attn(qd[at:at + 1], *codes, tab[None], lens, d ** -0.5, 0, 0,
                                 out[at:at + 1], ws, *pairs)
        if at % 11 == 0 or at == total - 1:
            full = [ow.u4_values(c[:at + 1], s[:at + 1]) for c, s in parts]
            sizes = [c[:at + 1] * s[:at + 1, :, :1] + np.abs(s[:at + 1, :, 1:]) for c, s in parts]
            want, size, dots, most = ow.window_attention(q[at:at + 1], full[:1], full[1:], [1],
                                                         [at + 1], d ** -0.5, 0, 0, sizes[:1],
                                                         sizes[1:])
            case = type("C", (), dict(kv="u4", qt="bf16", scale=d ** -0.5, pairs=[None, parts[1]]))
            close(out_to_f64(out[at:at + 1]), want, tolerance(case, want, size, dots, most))


@pytest.mark.parametrize("kv, q", TYPES)
@pytest.mark.parametrize("counts, g", [([3, 2], 2), ([9, 8], 4), ([40, 70], 4)])
def test_a_wait_that_runs_out_is_reported(kv, q, counts, g):
    """Every kernel that the sizes choose: the call returns, says so, and the next one is right."""
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    c = Windowed([900, 700], 2, 128, kv, 500, 4, seed=2, q=q, g=g, counts=counts)
    t = c.gpu()
    want, tol = expect(c)
    ws = torch.empty(B.pkv_window_multiquery_workspace_size(2, 2 * g, max(counts), t["k"], 16),
                     dtype=torch.uint8, device="cuda")
    B.pkv_testing_window_multiquery_attn_stall(
        t["q"], t["cu"], max(counts), t["k"], t["v"], t["tables"], t["lens"], c.scale, c.window,
        c.sinks, t["out"], ws, wait_limit_ns=20_000_000, stall_cta=1, num_parts=16,
        k_scales=t["k_scales"], v_scales=t["v_scales"], dev_status=t["status"])
    torch.cuda.synchronize()
    assert int(t["status"].item()) & B.DEV_TIMEOUT
    t["status"].zero_()
    close(run(c, t, 16), want, tol)
    assert int(t["status"].item()) == 0


@pytest.mark.parametrize("kv, q", TYPES)
@pytest.mark.parametrize("scale", [0.0, -0.2, 30.0])
def test_any_softmax_scale(kv, q, scale):
    for counts, g in (([2, 3], 2), ([70, 60], 4)):
        c = Windowed([200, 150], 3, 64, kv, 90, 2, seed=6, q=q, g=g, counts=counts)
        c.scale = scale
        t = c.gpu()
        want, tol = expect(c)
        close(run(c, t), want, tol)


@pytest.mark.parametrize("g", [1, 4])
def test_values_of_any_size_in_bf16_and_int8(g):
    """bf16 values from 2^15 on meet P in units of a power of two that grows on the way; INT8
    scales of any size, zero ones among them; queries over INT8 beyond fp16's range."""
    for std in (1e4, 3e6, 1e30, 1e-6, 1e-30):
        c = Windowed([600, 400], 1, 128, "bf16", 300, 4, seed=3, g=g, counts=[200, 150])
        from _longctx import stored
        from oracle import decode_kv
        v = decode_kv(c.v)
        live = c.seen[:, None, :, None]
        grow = 10.0 ** np.linspace(-3, 3, len(c.v))[:, None, None, None]
        c.v = np.where(live, stored(np.where(live, v, 0.0) * std * grow, "bf16"), c.v).astype(
            c.v.dtype)
        t = c.gpu()
        want, tol = expect(c)
        # beside larger values O's unit grows: P of a chunk is off by 2^-25 in units that meet
        # values of 2^15 of 2^-7 of that unit, whose 2^15 is at most the largest value
        top = max(np.abs(x).max() for x in c.sequences()[1])
        close(run(c, t), want, tol + 400 * 2.0 ** -32 * top)
    c = Windowed([600, 400], 1, 128, "i8", 300, 4, seed=3, q="bf16", g=g, counts=[200, 150])
    used = np.isfinite(c.v_scales)
    rng = np.random.default_rng(0)
    c.v_scales = np.where(used, 10.0 ** rng.uniform(-6, 6, c.v_scales.shape), np.nan).astype(
        np.float32)
    zero = rng.random(c.k_scales.shape) < 0.2
    c.k_scales = np.where(zero & used, 0.0, c.k_scales).astype(np.float32)
    t = c.gpu()
    want, tol = expect(c)
    # weights below 2^-14 of a unit of the largest scale: 2^-25 2^-7 127 max scale a token
    close(run(c, t), want, tol + 400 * 2.0 ** -32 * 127 * 1e6)
    c = Windowed([600, 400], 1, 128, "i8", 300, 4, seed=4, q="bf16", g=g, counts=[200, 150])
    c.q = stored(decode_kv(c.q) * 1e20, "bf16")
    c.scale *= 1e-20
    t = c.gpu()
    want, tol = expect(c)
    close(run(c, t), want, tol)


@pytest.mark.parametrize("kv, q", TYPES)
@pytest.mark.parametrize("batch, pad", [(30, 20000), (30, 400), (700, 400), (700, 130)])
def test_padded_and_mixed_batches(kv, q, batch, pad):
    """A few long runs among single tokens and empty ones, under any max_q_len: more tile pairs
    than CTAs (two kv heads, 64 or 128 queries a tile), and more than one unit for a CTA."""
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    rng = np.random.default_rng(batch)
    counts = [int(x) for x in rng.integers(0, 4, batch)]
    counts[batch // 2], counts[-1], counts[3] = min(pad, 400), 130, 70
    lens = [n + int(x) for n, x in zip(counts, rng.integers(0, 60, batch))]
    c = Windowed(lens, 2, 64, kv, 40, 3, seed=batch, q=q, g=2, counts=counts)
    t = c.gpu()
    want, tol = expect(c)
    close(run(c, t, max_q=pad), want, tol)
    assert int(t["status"].item()) == 0
    # a sequence with more queries than tokens
    t["lens"][batch // 2] = counts[batch // 2] - 1
    t["out"].fill_(77.0)
    got = run(c, t, max_q=pad)
    assert int(t["status"].item()) == B.DEV_BAD_LENGTH
    a, b = c.cu[batch // 2], c.cu[batch // 2 + 1]
    keep = np.ones(len(got), bool)
    keep[a:b] = False
    assert (got[a:b] == 77).all()
    close(got[keep], want[keep], tol[keep])
    # a wait that runs out ends one CTA's work, not the next call's
    t["lens"].copy_(torch.from_numpy(c.lens))
    ws = torch.empty(B.pkv_window_multiquery_workspace_size(batch, 4, pad, t["k"]),
                     dtype=torch.uint8, device="cuda")
    B.pkv_testing_window_multiquery_attn_stall(
        t["q"], t["cu"], pad, t["k"], t["v"], t["tables"], t["lens"], c.scale, c.window, c.sinks,
        t["out"], ws, wait_limit_ns=20_000_000, stall_cta=0, k_scales=t["k_scales"],
        v_scales=t["v_scales"], dev_status=t["status"])
    torch.cuda.synchronize()
    if counts[0]:
        assert int(t["status"].item()) & B.DEV_TIMEOUT
    t["status"].zero_()
    close(run(c, t, max_q=pad), want, tol)
    assert int(t["status"].item()) == 0


@pytest.mark.parametrize("kv, q", TYPES)
@pytest.mark.parametrize("window", [0, 1800])
def test_long_runs_behind_long_contexts(kv, q, window):
    """Many rows and many chunks of 128 tokens: the kernel of whole tiles, its last pair of them with
    one tile only."""
    c = Windowed([2500, 2050], 2, 128, kv, window, 20, seed=9, q=q, g=8, counts=[300, 260])
    t = c.gpu()
    want, tol = expect(c)
    close(run(c, t), want, tol)
    assert int(t["status"].item()) == 0


def test_thousands_of_sequences_in_long_runs():
    """More sequences than threads: a thread counts the pairs of a run of them."""
    rng = np.random.default_rng(6)
    counts = [int(x) for x in rng.integers(0, 3, 3000)]
    counts[1500] = 140
    lens = [n + int(x) for n, x in zip(counts, rng.integers(0, 20, 3000))]
    c = Windowed(lens, 1, 64, "bf16", 10, 2, seed=6, g=1, counts=counts)
    t = c.gpu()
    want, tol = expect(c)
    close(run(c, t), want, tol)
    close(run(c, t, max_q=1000), want, tol)
    assert int(t["status"].item()) == 0


@pytest.mark.parametrize("far, near, unit", [(1.0, 2.0 ** -16, 1.0), (1.0, 2.0 ** -9, 1.0),
                                             (0.0, 2.0 ** -40, 2.0 ** -35),
                                             (2.0 ** -30, 1.0, 1.0), (2.0 ** 20, 1.0, 2.0 ** 14)])
def test_small_values_beside_large_ones(far, near, unit):
    """Rows that see only the small values among those of their run: a long run's first rows see
    values of one size, its last rows only those of another."""
    from _longctx import stored
    from oracle import decode_kv
    c = Windowed([600, 700], 1, 128, "bf16", 64, 0, seed=5, g=2, counts=[400, 300])
    v = np.where(c.seen[:, None, :, None], decode_kv(c.v), 0.0)
    for b, length in enumerate(c.lens.tolist()):
        for j in range(-(-length // 16)):
            v[c.true_tables[b, j]] *= far if 16 * j < length - 150 else near
    c.v = np.where(c.seen[:, None, :, None], stored(v, "bf16"), c.v).astype(c.v.dtype)
    t = c.gpu()
    want, tol = expect(c)
    # P is off by 2^-25 of 2^7 P 2^(e' - e), O's unit being 2^e and the small values at most
    # 2^(e' - 3) where e' < e: 2^(e - 35) a token, of 64. `unit` is 2^e or more: 1 where the
    # largest values lie in [2^-8, 2^15), else a 2^14th of them.
    close(run(c, t), want, tol + 64 * 2.0 ** -35 * unit)


@pytest.mark.parametrize("kv, q", TYPES)
def test_rows_that_are_not_16_byte_aligned(kv, q):
    """q (16-bit caches) and out may begin at any 4 bytes: long runs then take another kernel."""
    import torch
    for counts in ([60, 35], [130, 20]):
        c = Windowed([300, 200], 2, 128, kv, 100, 3, seed=8, q=q, g=2, counts=counts)
        t = c.gpu()
        for name in ("out",) + (("q",) if kv != "i8" else ()):
            x = t[name]
            t[name] = torch.empty(x.numel() + 2, dtype=x.dtype, device="cuda")[2:].view(x.shape)
            t[name].copy_(x)
        want, tol = expect(c)
        for parts in (0, 7):
            close(run(c, t, parts), want, tol)


def test_rows_behind_the_last_query_stay():
    import torch
    for counts, g in (([3, 2], 2), ([150, 60], 2)):
        c = Windowed([300, 200], 2, 64, "bf16", 100, 3, seed=1, g=g, counts=counts)
        t = c.gpu()
        want, tol = expect(c)
        n = sum(counts)
        t["q"] = torch.cat([t["q"], t["q"][:5] * float("nan")])
        t["out"] = torch.full(t["q"].shape, 5.0, device="cuda").bfloat16()
        got = run(c, t)
        close(got[:n], want, tol)
        assert (got[n:] == 5).all()


def test_repeatable_and_many_heads():
    import torch
    for kv, q in TYPES:
        for counts, g, hkv in (([5, 4], 1, 7), ([90, 131], 4, 3)):
            c = Windowed([500, 300], hkv, 64, kv, 200, 10, seed=5, q=q, g=g, counts=counts)
            t = c.gpu()
            want, tol = expect(c)
            close(run(c, t, 40), want, tol)
            first = t["out"].clone()
            for _ in range(4):
                t["out"].zero_()
                run(c, t, 40)
                assert torch.equal(first, t["out"])
