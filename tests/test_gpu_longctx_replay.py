"""Captured graphs, side streams and long evictions, with every buffer that the calls
write spoilt beforehand: what they leave must be theirs."""

import numpy as np
import pytest

from _longctx import Paged
from _pkv_helpers import to_dev, to_host_bits
from oracle import longctx as lc
from test_gpu_longctx_step import _bits, _case, _everything

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_decode_05_gb300.build import build
    build()


def _spoil(c, t, outs):
    """Junk in all outputs, the newest blocks' bounds and the blocks that eviction fills."""
    for o in outs[1:10]:
        o.view(-1)[:] = 77
    newest = [int(c.tables[b, (n - 1) // 16]) for b, n in enumerate(c.lens) if n]
    outs[0][newest] = 55
    new = t["new_tables"].reshape(-1).long()
    for name in ("k", "v", "k_scales", "v_scales"):
        if t[name] is not None:
            t[name][new] = 33


def _expect(seed, kv):
    """The case, its call and outputs, and what one eager call makes of spoilt outputs."""
    import torch
    c = _case(kv, seed)
    t = c.gpu()
    call, outs = _everything(c, t)
    _spoil(c, t, outs)
    call()
    torch.cuda.synchronize()
    want = [_bits(o) for o in outs]
    _spoil(c, t, outs)
    torch.cuda.synchronize()
    spoilt = [_bits(o) for o in outs]
    assert all(not torch.equal(x, y) for x, y in zip(want, spoilt))
    return c, t, call, outs, want


@pytest.mark.parametrize("kv", ["bf16", "i8"])
def test_graph_replays_write_everything(kv):
    import torch
    runs = []
    for seed in (1, 2):
        c, t, call, outs, want = _expect(seed, kv)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        runs.append((c, t, outs, want, call, graph))    # the call owns its workspaces
    for _ in range(3):
        for c, t, outs, _, _, _ in runs:
            _spoil(c, t, outs)
        for run in runs:
            run[-1].replay()
        torch.cuda.synchronize()
        for _, _, outs, want, _, _ in runs:
            for i, (o, x) in enumerate(zip(outs, want)):
                assert torch.equal(_bits(o), x), i


@pytest.mark.parametrize("kv", ["f16", "i8"])
def test_side_streams_write_everything(kv):
    import torch
    runs = [_expect(seed, kv) + (torch.cuda.Stream(),) for seed in (3, 4)]
    for _ in range(3):
        for c, t, _, outs, _, s in runs:
            _spoil(c, t, outs)
            s.wait_stream(torch.cuda.current_stream())
        for _, _, call, _, _, s in runs:
            call(s)
        torch.cuda.synchronize()
        for _, _, _, outs, want, _ in runs:
            for i, (o, x) in enumerate(zip(outs, want)):
                assert torch.equal(_bits(o), x), i


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_rows_beyond_shared_memory(kv, in_place, monkeypatch):
    """40000 and 100 tokens cut to 3000: every output, the choice taken from numpy's order."""
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    n, budget, first, last = 40000, 3000, 4, 64
    c = Paged([n, 100], 1, 64, kv, seed=4, more=-(-budget // 16))
    mass = np.exp(2 * c.rng.standard_normal((2, 1, 16 * c.mb))).astype(np.float32)

    def choose(row, first, last, budget):
        if len(row) <= budget:
            return np.arange(len(row))
        keep = np.zeros(len(row), bool)
        keep[:first] = keep[len(row) - last:] = True
        rest = np.flatnonzero(~keep)
        keep[rest[np.argsort(-row[rest], kind="stable")[:budget - first - last]]] = True
        return np.flatnonzero(keep)

    small = np.round(mass[0, 0, :500], 1)
    assert (choose(small, 3, 9, 80) == lc.choose(small, 3, 9, 80)).all()
    monkeypatch.setattr(lc, "choose", choose)
    new = c.tables if in_place else c.new_tables
    k, v, ks, vs, want_kept, want_lens, want_mass = lc.evict(
        c.k, c.v, c.tables, c.lens, mass, first, last, budget, new, c.k_scales, c.v_scales)
    t = c.gpu()
    lens = torch.full((2,), 99, dtype=torch.int32, device="cuda")
    got_mass = torch.full(want_mass.shape, 9.0, device="cuda")
    kept = torch.full((2, 1, budget), 99, dtype=torch.int32, device="cuda")
    B.pkv_evict_tokens(t["k"], t["v"], t["tables"], t["lens"], to_dev(mass), first, last,
                       t["tables"] if in_place else t["new_tables"], lens, got_mass, kept,
                       t["k_scales"], t["v_scales"], t["status"])
    assert int(t["status"].item()) == 0
    assert (kept.cpu().numpy() == want_kept).all() and (lens.cpu().numpy() == want_lens).all()
    assert got_mass.cpu().numpy().tobytes() == want_mass.tobytes()
    assert to_host_bits(t["k"]).tobytes() == k.tobytes()
    assert to_host_bits(t["v"]).tobytes() == v.tobytes()
    if ks is not None:
        assert t["k_scales"].cpu().numpy().tobytes() == ks.tobytes()
        assert t["v_scales"].cpu().numpy().tobytes() == vs.tobytes()


@pytest.mark.parametrize("kv", ["bf16", "i8"])
def test_lengths_that_the_call_before_wrote(kv):
    """An eviction's lengths, in the same cache line as the ones that it reads, with launches
    that overlap: every call after it sees the new ones, and the weights that it wrote."""
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    n, hkv, g, d, budget = 8, 4, 4, 64, 64
    c = Paged([700 + 31 * b for b in range(n)], hkv, d, kv, seed=8, g=g, more=budget // 16)
    t = c.gpu()
    mb, nb = c.mb, budget // 16
    buf = torch.zeros((3, n), dtype=torch.int32, device="cuda")       # 96 bytes
    mass = torch.rand((n, hkv, 16 * mb), device="cuda")
    new_mass = torch.zeros((n, hkv, 16 * nb), device="cuda")
    kept = torch.zeros((n, hkv, budget), dtype=torch.int32, device="cuda")
    bounds = to_dev(c.bounds())
    scores = torch.zeros((2, n, hkv, nb), device="cuda")
    lists = torch.zeros((2, n, hkv, 2), dtype=torch.int32, device="cuda")
    counts = torch.zeros((2, n), dtype=torch.int32, device="cuda")
    outs = torch.zeros((2,) + tuple(t["q"].shape), dtype=t["q"].dtype, device="cuda")
    total = torch.zeros((2, n, hkv, 16 * nb), device="cuda")
    ws = torch.empty(max(B.pkv_decode_mass_workspace_size(n, hkv * g, nb, t["k"]),
                         B.pkv_sparse_decode_workspace_size(n, hkv * g, t["k"])),
                     dtype=torch.uint8, device="cuda")

    def read(i):
        args = (t["k"], t["v"], t["new_tables"], buf[1])
        B.pkv_block_bounds(t["k"], t["new_tables"], buf[1], bounds, buf[1], budget)
        B.pkv_block_scores(t["q"], bounds, t["k"], t["new_tables"], buf[1], scores[i],
                           t["k_scales"])
        B.pkv_block_select(scores[i], buf[1], 0, 1, lists[i], counts[i])
        B.pkv_sparse_decode_attn(t["q"], *args, lists[i], counts[i], c.scale, outs[i], ws,
                                 t["k_scales"], t["v_scales"])
        B.pkv_decode_attn_mass(t["q"], *args, c.scale, outs[i], new_mass, total[i], ws,
                               t["k_scales"], t["v_scales"])

    def step():
        buf[1].copy_(buf[2])
        read(0)                                # lengths of buf[2]
        B.pkv_evict_tokens(t["k"], t["v"], t["tables"], buf[0], mass, 2, 4, t["new_tables"],
                           buf[1], new_mass, kept, t["k_scales"], t["v_scales"], t["status"])
        read(1)                                # lengths that the eviction wrote

    lens = [[1] * n, [40, 64, 3, 64, 17, 64, 33, 64]]
    buf[2] = 20
    graphs, wants = [], []
    for x in (0, 1):
        buf[0].copy_(torch.tensor(lens[x]))
        step()
        torch.cuda.synchronize()
        wants.append([_bits(o) for o in (scores[1], lists[1], counts[1], outs[1], total[1])])
        assert counts[1].tolist() == [min(2, -(-v // 16)) for v in lens[x]]
        total.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for turn in range(400):
        x = turn % 2
        buf[0].copy_(torch.tensor(lens[x]))
        total.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [_bits(o) for o in (scores[1], lists[1], counts[1], outs[1], total[1])]
        for i, (o, w) in enumerate(zip(got, wants[x])):
            assert torch.equal(o, w), (turn, i)
