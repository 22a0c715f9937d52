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
