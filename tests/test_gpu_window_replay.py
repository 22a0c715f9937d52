"""Windowed attention and the 4-bit cache in captured graphs, on side streams and from two host
threads."""

import subprocess
import sys
import threading

import numpy as np
import pytest

from _pkv_helpers import out_to_f64
from _window import Windowed, close

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16"), ("f16", "f16"), ("i8", "bf16"), ("u4", "bf16"), ("u4", "f16")]


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_decode_05_gb300.build import build
    build()


def decode(c, t, ws):
    from paged_kv_decode_05_gb300 import binding as B
    B.pkv_window_decode_attn(t["q"], t["k"], t["v"], t["tables"], t["lens"], c.scale, c.window,
                             c.sinks, t["out"], ws, t["k_scales"], t["v_scales"])


def multi(c, t, ws):
    from paged_kv_decode_05_gb300 import binding as B
    B.pkv_window_multiquery_attn(t["q"], t["cu"], max(c.counts), t["k"], t["v"], t["tables"],
                                 t["lens"], c.scale, c.window, c.sinks, t["out"], ws,
                                 t["k_scales"], t["v_scales"])


def workspace(c, t, name):
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    if name == "decode":
        n = B.pkv_window_decode_workspace_size(len(c.lens), c.q.shape[1], t["k"])
    else:
        n = B.pkv_window_multiquery_workspace_size(len(c.lens), c.q.shape[1], max(c.counts),
                                                   t["k"])
    return torch.full((n,), 0xEE, dtype=torch.uint8, device="cuda")


def cases():
    for kv, q in TYPES:
        yield "decode", Windowed([2000, 1, 700, 0, 40], 2, 128, kv, 600, 7, seed=1, q=q, g=4)
    for kv, q in TYPES[:3]:
        yield "multi", Windowed([900, 200], 2, 128, kv, 300, 7, seed=2, q=q, g=4, counts=[5, 3])
        yield "multi", Windowed([900, 200], 2, 128, kv, 300, 7, seed=3, q=q, g=4, counts=[60, 90])


def expect(c, name):
    if name == "decode":
        return c.expect()
    from test_gpu_window_multi import expect as e
    return e(c)


def test_graphs_that_share_a_workspace_replay_in_turn():
    """Two graphs of one call each over the same workspace, replayed in turn from spoilt outputs
    and workspaces, with other queries and lengths in between; eager calls between them."""
    import torch
    for name, c in cases():
        fn = decode if name == "decode" else multi
        want, tol = expect(c, name)
        ts = [c.gpu(), c.gpu()]
        ws = workspace(c, ts[0], name)
        graphs = []
        for t in ts:
            fn(c, t, ws)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                fn(c, t, ws)
            graphs.append(g)
        q, lens = ts[0]["q"].clone(), ts[0]["lens"].clone()
        for _ in range(3):
            for t, g in zip(ts, graphs):
                t["out"].fill_(float("nan"))
                ws.fill_(0x7F)
                t["q"].zero_()
                g.replay()
                t["q"].copy_(q)
                t["lens"].zero_()
                if name == "decode":
                    g.replay()
                    assert bool((t["out"] == 0).all())
                t["lens"].copy_(lens)
                g.replay()
                close(out_to_f64(t["out"]), want, tol)
                fn(c, t, ws)
                close(out_to_f64(t["out"]), want, tol)


def test_side_streams():
    """Inputs written, the call and its readers on one side stream while the default stream is
    busy; the stream may also be named."""
    import torch
    for name, c in cases():
        fn = decode if name == "decode" else multi
        want, tol = expect(c, name)
        t = c.gpu()
        ws = workspace(c, t, name)
        q = t["q"].clone()
        t["q"].fill_(1.0)
        busy = torch.randn(4096, 4096, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(10):
            busy = busy @ busy * 1e-3
        with torch.cuda.stream(side):
            t["q"].copy_(q)
            fn(c, t, ws)
            got = t["out"].clone()
        side.synchronize()
        close(out_to_f64(got), want, tol)
        torch.cuda.synchronize()


def test_4_bit_writes_and_reads_replay():
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    k, v = (torch.randn((70, 3, 128), device="cuda").half() for _ in range(2))
    slots = torch.randperm(96, device="cuda")[:70].contiguous()
    codes = [torch.zeros((6, 3, 16, 64), dtype=torch.uint8, device="cuda") for _ in range(2)]
    pairs = [torch.zeros((6, 3, 16, 2), device="cuda").half() for _ in range(2)]
    outs = [torch.zeros((6, 3, 16, 128), device="cuda").half() for _ in range(2)]
    ids = torch.arange(6, dtype=torch.int32, device="cuda")

    def both():
        B.pkv_u4_append(k, v, slots, *codes, *pairs)
        B.pkv_u4_read_blocks(*codes, *pairs, ids, *outs, ids)
    both()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    for seed in range(3):
        torch.manual_seed(seed)
        k.copy_(torch.randn(k.shape, device="cuda") * 10.0 ** seed)
        v.copy_(torch.randn(v.shape, device="cuda"))
        slots.copy_(torch.randperm(96, device="cuda")[:70])
        for x in codes + pairs + outs:
            x.zero_()
        both()
        want = [x.clone() for x in codes + pairs + outs]
        for x in codes + pairs + outs:
            x.zero_()
        g.replay()
        for x, y in zip(codes + pairs + outs, want):
            assert torch.equal(x, y)


def test_two_host_threads():
    """Calls of different sizes from two threads, streams and workspaces of their own."""
    import torch
    todo = [(n, c, expect(c, n)) for n, c in cases()]
    errors = []

    def work(items):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for name, c, (want, tol) in items:
                    t = c.gpu()
                    ws = workspace(c, t, name)
                    for _ in range(20):
                        (decode if name == "decode" else multi)(c, t, ws)
                    close(out_to_f64(t["out"]), want, tol)
        except Exception as e:      # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(x,)) for x in (todo, todo[::-1])]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors, errors


FIRST = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import test_gpu_window_replay as m
for name, c in m.cases():
    t = c.gpu()
    ws = m.workspace(c, t, name)
    fn = m.decode if name == "decode" else m.multi
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):       # the process's first call of this form is captured
        fn(c, t, ws)
    g.replay()
    m.close(m.out_to_f64(t["out"]), *m.expect(c, name))
print("fine")
"""


def test_first_calls_may_be_captured():
    import os
    tests = os.path.dirname(os.path.abspath(__file__))
    code = FIRST.format(root=os.path.dirname(tests), tests=tests)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


def test_another_device_or_stream_is_refused():
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    name, c = next(iter(cases()))
    t = c.gpu()
    ws = workspace(c, t, name)
    t["lens"] = t["lens"].cpu()
    with pytest.raises(ValueError):
        decode(c, t, ws)
    x = torch.zeros((2, 1, 64), device="cuda").half()
    codes = torch.zeros((1, 1, 16, 32), dtype=torch.uint8, device="cuda")
    pairs = torch.zeros((1, 1, 16, 2), device="cuda").half()
    slots = torch.zeros(2, dtype=torch.int64, device="cuda")
    with pytest.raises((TypeError, ValueError)):
        B.pkv_u4_append(x, x, slots, codes, codes, pairs.float(), pairs)
    with pytest.raises((TypeError, ValueError)):
        B.pkv_u4_append(x, x.bfloat16(), slots, codes, codes, pairs, pairs)
    with pytest.raises((TypeError, ValueError)):
        B.pkv_u4_append(x, x, slots.int(), codes, codes, pairs, pairs)
    with pytest.raises((TypeError, ValueError)):
        B.pkv_u4_append(x.transpose(0, 2), x, slots, codes, codes, pairs, pairs)
    with pytest.raises((TypeError, ValueError)):
        B.pkv_u4_read_blocks(codes, codes, pairs, pairs, slots.int()[:1], x, x, slots.int()[:1])
