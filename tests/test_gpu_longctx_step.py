"""The long-context operators as a serving loop uses them: together, step after
step, in captured graphs, on other streams, over pools beyond 32-bit offsets,
and when an in-kernel wait runs out."""

import os
import subprocess
import sys

import numpy as np
import pytest

from _longctx import Paged, attention_tolerance, stored
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
    ang = np.arange(rows)[:, None] * 10000.0 ** (-np.arange(half) / half)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


class View:
    """What attention_tolerance wants to know of a case, read back from the GPU."""

    def __init__(self, kv, scale, v, v_scales=None):
        self.kv, self.qt, self.scale, self.v, self.v_scales = kv, kv, scale, v, v_scales


@pytest.mark.parametrize("kv, hkv, g, d", [("bf16", 2, 4, 128), ("f16", 3, 2, 64)])
def test_serving_loop(kv, hkv, g, d):
    """A prompt is written, then tokens are decoded with sparse attention over a growing cache;
    the weights add up and the cache is cut in place whenever it outgrows its budget. Every
    output is checked against the oracle on the cache as it is stored."""
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    rng = np.random.default_rng(7)
    dt = torch.bfloat16 if kv == "bf16" else torch.float16
    lens = np.array([70, 1, 131], np.int32)
    n, hq, mb, budget, keep = 3, hkv * g, 13, 6, 150
    tables = rng.permutation(n * mb + 2)[:n * mb].reshape(n, mb).astype(np.int32)
    dev = dict(device="cuda")
    kc, vc = (torch.full((n * mb + 2, hkv, 16, d), float("nan"), dtype=dt, **dev) for _ in range(2))
    bounds = torch.zeros((n * mb + 2, hkv, 2, d), dtype=dt, **dev)
    st = torch.zeros(1, dtype=torch.int32, **dev)
    table, rot = to_dev(_table(400, d)), d
    w = [stored(rng.uniform(0.5, 1.5, d), kv) for _ in range(2)]
    axis = [j % 2 for j in range(rot // 2)]
    t_tab = to_dev(tables)
    mass = torch.zeros((n, hkv, 16 * mb), **dev)
    ws_m = torch.empty(B.pkv_decode_mass_workspace_size(n, hq, mb, kc), dtype=torch.uint8, **dev)
    ws_s = torch.empty(B.pkv_sparse_decode_workspace_size(n, hq, kc), dtype=torch.uint8, **dev)
    scale = d ** -0.5

    def write(tokens, pos, slots):
        x = to_dev(stored(rng.standard_normal((tokens, hq + 2 * hkv, d)), kv))
        q = torch.empty((tokens, hq, d), dtype=dt, **dev)
        B.pkv_qk_norm_rope_append(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], to_dev(pos), table,
                                  to_dev(slots), kc, vc, q, to_dev(w[0]), to_dev(w[1]),
                                  pair_axis=axis,
                                  dev_status=st)
        want = lc.qk_norm_rope(to_host_bits(x[:, :hq].contiguous()), w[0], 1e-6,
                               table.cpu().numpy(), pos, axis, False)
        tol = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}[kv] * np.abs(want) + 1e-5 * np.abs(want).max()
        assert (np.abs(out_to_f64(q) - want) <= tol).all()
        return q

    where = [(b, p) for b in range(n) for p in range(lens[b])]
    slots = np.array([tables[b, p // 16] * 16 + p % 16 for b, p in where], np.int64)
    pos = np.array([[p, p // 7] for _, p in where], np.int32).T.copy()
    write(len(where), pos, slots)
    B.pkv_block_bounds(kc, t_tab, to_dev(lens), bounds, to_dev(lens), int(lens.max()), st)
    positions = lens.copy()                     # rotary positions go on when the cache is cut
    cut = 0
    for step in range(40):
        lens = lens + 1
        slots = np.array([tables[b, (L - 1) // 16] * 16 + (L - 1) % 16 for b, L in enumerate(lens)],
                         np.int64)
        q = write(n, np.stack([positions, positions // 7]).astype(np.int32), slots)
        positions = positions + 1
        t_len = to_dev(lens)
        B.pkv_block_bounds(kc, t_tab, t_len, bounds, dev_status=st)
        scores = torch.empty((n, hkv, mb), **dev)
        B.pkv_block_scores(q, bounds, kc, t_tab, t_len, scores, dev_status=st)
        lists = torch.empty((n, hkv, budget), dtype=torch.int32, **dev)
        counts = torch.empty(n, dtype=torch.int32, **dev)
        B.pkv_block_select(scores, t_len, 1, 2, lists, counts, st)
        out = torch.empty_like(q)
        B.pkv_sparse_decode_attn(q, kc, vc, t_tab, t_len, lists, counts, scale, out, ws_s,
                                 dev_status=st)
        before = mass.cpu().numpy()
        full = torch.empty_like(q)
        B.pkv_decode_attn_mass(q, kc, vc, t_tab, t_len, scale, full, mass, mass, ws_m,
                               dev_status=st)
        if step % 8 and lens.max() <= keep:
            continue
        k, v, qh = to_host_bits(kc), to_host_bits(vc), to_host_bits(q)
        s, size = lc.block_scores(qh, to_host_bits(bounds), tables, lens)
        sc = scores.cpu().numpy()
        ok = np.isfinite(s)
        assert (np.isneginf(sc) == ~ok).all()
        assert (np.abs(sc[ok] - s[ok]) <= 1e-5 * size[ok]).all()
        for b in range(n):
            for blk in range(-(-int(lens[b]) // 16)):
                want = lc.block_bounds(k, tables[b, blk], min(16, lens[b] - 16 * blk))
                assert (decode_kv(to_host_bits(bounds))[tables[b, blk]] == want).all()
            for h in range(hkv):
                want = lc.choose(sc[b, h, :-(-int(lens[b]) // 16)], 1, 2, budget)
                assert lists[b, h, :len(want)].tolist() == want.tolist()
        case = View(kv, scale, v)
        for got, li, cnt in ((out, lists.cpu().numpy(), counts.cpu().numpy()),
                             (full, np.broadcast_to(np.arange(mb), (n, hkv, mb)), -(-lens // 16))):
            want, size, dots = lc.listed_attention(qh, k, v, tables, lens, li, cnt, scale)
            assert (np.abs(out_to_f64(got) - want) <= attention_tolerance(case, want, size, dots,
                    256)).all()
        add = mass.cpu().numpy() - before
        want = lc.attention_mass(qh, k, tables, lens, scale)
        for b, L in enumerate(lens):
            assert np.allclose(add[b, :, :L], want[b, :, :L], rtol=1e-4, atol=1e-5)
            assert np.allclose(add[b, :, :L].sum(-1), g, rtol=1e-5)
        if lens.max() > keep:
            cut += 1
            new_lens = torch.empty(n, dtype=torch.int32, **dev)
            new_mass = torch.empty_like(mass)
            kept = torch.empty((n, hkv, 100), dtype=torch.int32, **dev)
            m = mass.cpu().numpy()
            k, v = to_host_bits(kc), to_host_bits(vc)
            B.pkv_evict_tokens(kc, vc, t_tab, t_len, mass, 4, 16, t_tab, new_lens, new_mass, kept,
                               dev_status=st)
            k2, v2, _, _, kept2, lens2, m2 = lc.evict(k, v, tables, lens, m, 4, 16, 100, tables)
            assert (kept.cpu().numpy() == kept2).all() and (new_mass.cpu().numpy() == m2).all()
            assert to_host_bits(kc).tobytes() == k2.tobytes()
            assert to_host_bits(vc).tobytes() == v2.tobytes()
            lens, mass = lens2, new_mass
            # rows moved, so every block's bounds are made anew
            B.pkv_block_bounds(kc, t_tab, to_dev(lens), bounds, to_dev(lens), int(lens.max()), st)
    assert cut >= 1 and int(st.item()) == 0


def _everything(c, t, ws=None):
    """One call of each operator over case c; returns (call, its outputs)."""
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    n, hq = len(c.lens), c.q.shape[1]
    dev = dict(device="cuda")
    bounds = to_dev(c.bounds())
    scores = torch.full((n, c.hkv, c.mb), 5.0, **dev)
    lists = torch.full((n, c.hkv, 7), 99, dtype=torch.int32, **dev)
    counts = torch.full((n,), 99, dtype=torch.int32, **dev)
    sparse, full = torch.zeros_like(t["q"]), torch.zeros_like(t["q"])
    mass_in = torch.rand((n, c.hkv, 16 * c.mb), generator=torch.Generator("cuda").manual_seed(3),
                         **dev)
    mass = torch.zeros_like(mass_in)
    ws_s = torch.empty(B.pkv_sparse_decode_workspace_size(n, hq, t["k"]), dtype=torch.uint8, **dev)
    ws_m = torch.empty(B.pkv_decode_mass_workspace_size(n, hq, c.mb, t["k"]), dtype=torch.uint8,
                       **dev)
    new_lens = torch.zeros(n, dtype=torch.int32, **dev)
    new_mass = torch.zeros((n, c.hkv, 16 * t["new_tables"].shape[1]), **dev)
    kept = torch.zeros((n, c.hkv, 60), dtype=torch.int32, **dev)

    def call(stream=None):
        B.pkv_block_bounds(t["k"], t["tables"], t["lens"], bounds, dev_status=t["status"],
                           stream=stream)
        B.pkv_block_scores(t["q"], bounds, t["k"], t["tables"], t["lens"], scores, t["k_scales"],
                           t["status"], stream)
        B.pkv_block_select(scores, t["lens"], 1, 2, lists, counts, t["status"], stream)
        B.pkv_sparse_decode_attn(t["q"], t["k"], t["v"], t["tables"], t["lens"], lists, counts,
                                 c.scale,
                                 sparse, ws_s, t["k_scales"], t["v_scales"], 0, t["status"], stream)
        B.pkv_decode_attn_mass(t["q"], t["k"], t["v"], t["tables"], t["lens"], c.scale, full,
                               mass_in,
                               mass, ws_m, t["k_scales"], t["v_scales"], 0, t["status"], stream)
        B.pkv_evict_tokens(t["k"], t["v"], t["tables"], t["lens"], mass, 2, 8, t["new_tables"],
                           new_lens,
                           new_mass, kept, t["k_scales"], t["v_scales"], t["status"], stream)
    outs = [bounds, scores, lists, counts, sparse, full, mass, new_lens, new_mass, kept, t["k"],
            t["v"]]
    return call, outs + [t[s] for s in ("k_scales", "v_scales") if t[s] is not None]


def _bits(t):
    return t.contiguous().view(-1).view(t.dtype).cpu().reshape(-1).contiguous().view(
        {1: __import__("torch").int8, 2: __import__("torch").int16, 4: __import__("torch").int32}[
            t.element_size()]).clone()


def _case(kv, seed=0):
    return Paged([500, 0, 17, 1203, 64, 333], 2, 128, kv, seed=seed, more=4, g=4)


@pytest.mark.parametrize("kv", ["bf16", "i8"])
def test_graph_replays_equal_eager(kv):
    """Two captured graphs, replayed in turn with other calls between them."""
    import torch
    runs = []
    for seed in (1, 2):
        c = _case(kv, seed)
        call, outs = _everything(c, c.gpu())
        call()
        torch.cuda.synchronize()
        want = [_bits(o) for o in outs]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        runs.append((graph, call, outs, want))
    for turn in range(3):
        for graph, call, outs, want in runs:
            for o in outs[1:10]:
                o.zero_()
            graph.replay()
            if turn == 1:
                runs[0][1]()
        torch.cuda.synchronize()
        for graph, call, outs, want in runs:
            for i, (o, x) in enumerate(zip(outs, want)):
                assert torch.equal(_bits(o), x), i


COLD = """
import sys
sys.path[:0] = [sys.argv[1], sys.argv[1] + "/tests"]
import torch
import test_gpu_longctx_step as m
torch.zeros(1, device="cuda")
for kv in ("bf16", "i8"):
    c = m._case(kv, 5)
    call, outs = m._everything(c, c.gpu())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    graph.replay()
    torch.cuda.synchronize()
    got = [m._bits(o) for o in outs]
    c = m._case(kv, 5)
    call, outs = m._everything(c, c.gpu())
    call()
    torch.cuda.synchronize()
    assert all(torch.equal(x, m._bits(o)) for x, o in zip(got, outs))
print("same")
"""


def test_first_call_may_be_captured():
    """A process whose first call of every operator is a capture."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", COLD, root], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.split() == ["same"], r.stderr[-2000:]


@pytest.mark.parametrize("kv", ["f16", "i8"])
def test_other_streams_side_by_side(kv):
    """Calls on two side streams at once, each with its own workspaces, give what the default
    stream gives."""
    import torch
    runs = []
    for seed in (3, 4):
        c = _case(kv, seed)
        call, outs = _everything(c, c.gpu())
        call()
        torch.cuda.synchronize()
        runs.append((call, outs, [_bits(o) for o in outs], torch.cuda.Stream()))
    for call, outs, want, s in runs:
        for o in outs[1:10]:
            o.zero_()
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for call, outs, want, s in runs:
            call(s)
    torch.cuda.synchronize()
    for call, outs, want, s in runs:
        for i, (o, x) in enumerate(zip(outs, want)):
            assert torch.equal(_bits(o), x), i


@pytest.mark.parametrize("kv", ["bf16", "i8"])
def test_pool_beyond_32_bit_offsets(kv):
    """The same sequences in the last blocks of a pool of more than 2^32 bytes (16-bit) or 2^31
    (INT8): the same bits as in a small pool."""
    import torch
    c = _case(kv, 5)
    n, big_n = len(c.k), 140000
    shift = big_n - n
    # 8 kv heads make the pool large; the sequences' heads are repeated over them
    rep = 4
    c8 = _case(kv, 5)
    c8.hkv, c8.k, c8.v = c.hkv * rep, np.tile(c.k, (1, rep, 1, 1)), np.tile(c.v, (1, rep, 1, 1))
    c8.q = np.tile(c.q, (1, rep, 1))
    if kv == "i8":
        c8.k_scales, c8.v_scales = np.tile(c.k_scales, (1, rep)), np.tile(c.v_scales, (1, rep))
    ts, tb = c8.gpu(), c8.gpu()
    for name in ("k", "v", "k_scales", "v_scales"):
        if ts[name] is None:
            continue
        x = torch.zeros((big_n,) + tuple(ts[name].shape[1:]), dtype=ts[name].dtype, device="cuda")
        assert name[2:] or x.numel() * x.element_size() > (2 ** 31 if kv == "i8" else 2 ** 32)
        x[shift:] = ts[name]
        tb[name] = x
    tb["tables"], tb["new_tables"] = ts["tables"] + shift, ts["new_tables"] + shift
    small_call, small_outs = _everything(c8, ts)
    x = torch.zeros((big_n,) + tuple(small_outs[0].shape[1:]), dtype=small_outs[0].dtype,
                    device="cuda")
    x[shift:] = small_outs[0]
    # the bounds of the large pool
    import paged_kv_decode_05_gb300.binding as B
    small_call()
    hq = c8.q.shape[1]
    B.pkv_block_bounds(tb["k"], tb["tables"], tb["lens"], x, dev_status=tb["status"])
    scores = torch.full_like(small_outs[1], 5.0)
    B.pkv_block_scores(tb["q"], x, tb["k"], tb["tables"], tb["lens"], scores, tb["k_scales"],
                       tb["status"])
    out, full = torch.empty_like(tb["q"]), torch.empty_like(tb["q"])
    ws = torch.empty(B.pkv_sparse_decode_workspace_size(6, hq, tb["k"]), dtype=torch.uint8,
                     device="cuda")
    B.pkv_sparse_decode_attn(tb["q"], tb["k"], tb["v"], tb["tables"], tb["lens"], small_outs[2],
                             small_outs[3], c8.scale, out, ws, tb["k_scales"], tb["v_scales"], 0,
                             tb["status"])
    ws = torch.empty(B.pkv_decode_mass_workspace_size(6, hq, c8.mb, tb["k"]), dtype=torch.uint8,
                     device="cuda")
    mass = torch.zeros_like(small_outs[6])
    mass_in = torch.rand(mass.shape, generator=torch.Generator("cuda").manual_seed(3),
                         device="cuda")
    B.pkv_decode_attn_mass(tb["q"], tb["k"], tb["v"], tb["tables"], tb["lens"], c8.scale, full,
                           mass_in, mass,
                           ws, tb["k_scales"], tb["v_scales"], 0, tb["status"])
    new_lens, new_mass, kept = (torch.zeros_like(o) for o in small_outs[7:10])
    B.pkv_evict_tokens(tb["k"], tb["v"], tb["tables"], tb["lens"], mass, 2, 8, tb["new_tables"],
                       new_lens,
                       new_mass, kept, tb["k_scales"], tb["v_scales"], tb["status"])
    assert int(tb["status"].item()) == 0
    for a, b in ((x[shift:], small_outs[0]), (scores, small_outs[1]), (out, small_outs[4]),
                 (full, small_outs[5]), (mass, small_outs[6]), (kept, small_outs[9]),
                 (tb["k"][shift:], ts["k"]), (tb["v"][shift:], ts["v"])):
        assert torch.equal(_bits(a), _bits(b))
    if kv == "i8":
        assert torch.equal(_bits(tb["k_scales"][shift:]), _bits(ts["k_scales"]))
        return
    # the write path: the last slots of the large pool
    q, k = tb["q"][:, :hq], tb["q"][:, :c8.hkv]
    slots = torch.arange(6, device="cuda") + (big_n * 16 - 6)
    q_out = torch.empty_like(tb["q"])
    B.pkv_qk_norm_rope_append(q, k, k, None, None, slots, tb["k"], tb["v"], q_out,
                              dev_status=tb["status"])
    assert torch.equal(tb["k"][-1, :, 10:].transpose(0, 1), k) and int(tb["status"].item()) == 0


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("which", ["sparse", "mass"])
def test_stalled_wait_times_out(kv, which):
    """A wait that runs out sets the timeout bit; other sequences are right, the context lives."""
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    c = Paged([400, 400, 400, 400], 2, 128, kv, seed=11, g=4)
    t = c.gpu()
    nb = c.mb - 1
    lists = torch.arange(nb, dtype=torch.int32, device="cuda").expand(4, 2, nb).contiguous()
    counts = torch.full((4,), nb, dtype=torch.int32, device="cuda")
    mass = torch.zeros((4, 2, 16 * c.mb), device="cuda")
    parts = 8                                   # one worker per (sequence, kv head)
    ws = torch.zeros(B.pkv_decode_mass_workspace_size(4, 8, c.mb, t["k"], parts), dtype=torch.uint8,
                     device="cuda")
    head = (t["q"], t["k"], t["v"], t["tables"], t["lens"])
    args = head + ((lists, counts, c.scale, t["out"], ws) if which == "sparse"
                   else (c.scale, t["out"], None, mass, ws))
    fn = (B.pkv_testing_sparse_decode_attn_stall if which == "sparse"
          else B.pkv_testing_decode_attn_mass_stall)
    kw = dict(num_parts=parts, k_scales=t["k_scales"], v_scales=t["v_scales"],
              dev_status=t["status"])
    fn(*args, wait_limit_ns=50_000_000, stall_worker=-1, **kw)
    good = out_to_f64(t["out"])
    assert int(t["status"].item()) == 0
    fn(*args, wait_limit_ns=50_000_000, stall_worker=3, **kw)      # sequence 1, kv head 1
    assert int(t["status"].item()) == B.DEV_TIMEOUT
    got = out_to_f64(t["out"])
    same = (got == good).all(-1)
    assert same[[0, 2, 3]].all() and same[1, :4].all()
    t["status"].zero_()
    fn(*args, wait_limit_ns=50_000_000, stall_worker=-1, **kw)
    assert int(t["status"].item()) == 0 and (out_to_f64(t["out"]) == good).all()
    with pytest.raises(B.PkvError):
        fn(*args, wait_limit_ns=5_000_000_000, stall_worker=0, **kw)


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("which", ["sparse", "mass"])
def test_stalled_wait_times_out_where_blocks_finish_alone(kv, which):
    """As above with the library's own split: few pairs, each finished by the blocks that have
    it. Every warp of the first pair has work, so worker 3 is one of them."""
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    c = Paged([2100, 2100, 2100, 2100], 2, 128, kv, seed=11, g=4)
    t = c.gpu()
    nb = c.mb - 1
    lists = torch.arange(nb, dtype=torch.int32, device="cuda").expand(4, 2, nb).contiguous()
    counts = torch.full((4,), nb, dtype=torch.int32, device="cuda")
    mass = torch.zeros((4, 2, 16 * c.mb), device="cuda")
    ws = torch.zeros(B.pkv_decode_mass_workspace_size(4, 8, c.mb, t["k"]), dtype=torch.uint8,
                     device="cuda")
    head = (t["q"], t["k"], t["v"], t["tables"], t["lens"])
    args = head + ((lists, counts, c.scale, t["out"], ws) if which == "sparse"
                   else (c.scale, t["out"], None, mass, ws))
    fn = (B.pkv_testing_sparse_decode_attn_stall if which == "sparse"
          else B.pkv_testing_decode_attn_mass_stall)
    kw = dict(num_parts=0, k_scales=t["k_scales"], v_scales=t["v_scales"], dev_status=t["status"])
    fn(*args, wait_limit_ns=50_000_000, stall_worker=-1, **kw)
    good = out_to_f64(t["out"])
    assert int(t["status"].item()) == 0
    fn(*args, wait_limit_ns=50_000_000, stall_worker=3, **kw)
    assert int(t["status"].item()) == B.DEV_TIMEOUT
    got = out_to_f64(t["out"])
    assert (got[0, 4:] == good[0, 4:]).all() and (got[1:] == good[1:]).all()
    t["status"].zero_()
    fn(*args, wait_limit_ns=50_000_000, stall_worker=-1, **kw)
    assert int(t["status"].item()) == 0 and (out_to_f64(t["out"]) == good).all()


def test_results_repeat_bit_for_bit():
    import torch
    c = _case("bf16", 9)
    call, outs = _everything(c, c.gpu())
    call()
    torch.cuda.synchronize()
    want = [_bits(o) for o in outs]
    for _ in range(4):
        call()
    torch.cuda.synchronize()
    for o, x in zip(outs, want):
        assert torch.equal(_bits(o), x)
