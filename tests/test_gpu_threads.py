"""Decode and multi-query attention called by two host threads at once, each on a stream of
its own, with batches that take different amounts of shared memory."""

import ctypes
import threading

import pytest

pytestmark = pytest.mark.gpu

CALLS = 3000


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_decode_05_gb300.build import build
    build()


def _state(batch, seed, kv):
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    gen = torch.Generator("cuda").manual_seed(seed)
    shape = (2 * batch, 2, 16, 128)
    s = dict(B=B, batch=batch, stream=torch.cuda.Stream())
    if kv == "i8":
        s["k"], s["v"] = (torch.randint(-127, 128, shape, generator=gen, device="cuda",
                                        dtype=torch.int8) for _ in range(2))
        s["ks"], s["vs"] = (torch.full(shape[:2], 0.02, device="cuda") for _ in range(2))
    else:
        s["k"], s["v"] = (torch.randn(shape, generator=gen, device="cuda").bfloat16()
                          for _ in range(2))
        s["ks"] = s["vs"] = None
    s["tables"] = torch.arange(2 * batch, dtype=torch.int32, device="cuda").view(batch, 2)
    s["lens"] = torch.full((batch,), 29, dtype=torch.int32, device="cuda")
    s["q"] = torch.randn((batch, 8, 128), generator=gen, device="cuda").bfloat16()
    s["out"] = torch.zeros_like(s["q"])
    s["desc"] = B.cache_desc(s["k"])
    return s


def _ptr(t):
    return None if t is None else t.data_ptr()


def _decode(batch, seed, kv):
    import torch
    s = _state(batch, seed, kv)
    B = s["B"]
    s["ws"] = torch.empty(B.pkv_decode_workspace_size(batch, 8, s["k"]), dtype=torch.uint8,
                          device="cuda")
    args = (_ptr(s["q"]), B.PKV_BF16, _ptr(s["k"]), _ptr(s["v"]), _ptr(s["ks"]), _ptr(s["vs"]),
            ctypes.byref(s["desc"]), _ptr(s["tables"]), 2, _ptr(s["lens"]), batch, 8, 0.088,
            _ptr(s["out"]), _ptr(s["ws"]), s["ws"].numel(), 0, None,
            ctypes.c_void_p(s["stream"].cuda_stream))
    fn = B.lib().pkv_decode_attn
    return (lambda: fn(*args)), s


def _multiquery(batch, seed, kv, heads_and_rows=(8, 1)):
    import torch
    s = _state(batch, seed, kv)
    B = s["B"]
    hq, rows = heads_and_rows
    s["q"] = torch.randn((batch * rows, hq, 128), device="cuda").bfloat16()
    s["out"] = torch.zeros_like(s["q"])
    s["cu"] = torch.arange(batch + 1, dtype=torch.int32, device="cuda") * rows
    s["ws"] = torch.empty(B.pkv_multiquery_workspace_size(batch, hq, rows, s["k"]),
                          dtype=torch.uint8, device="cuda")
    args = (_ptr(s["q"]), B.PKV_BF16, _ptr(s["cu"]), rows, _ptr(s["k"]), _ptr(s["v"]),
            _ptr(s["ks"]), _ptr(s["vs"]), ctypes.byref(s["desc"]), _ptr(s["tables"]), 2,
            _ptr(s["lens"]), batch, hq, 0.088, _ptr(s["out"]), _ptr(s["ws"]), s["ws"].numel(), 0,
            None, ctypes.c_void_p(s["stream"].cuda_stream))
    fn = B.lib().pkv_multiquery_attn
    return (lambda: fn(*args)), s


def _multiquery_rows(batch, seed, kv):
    return _multiquery(batch, seed, kv, (8, 7))      # 28 rows: 16 rows per warp


@pytest.mark.parametrize("kv", ["bf16", "i8"])
@pytest.mark.parametrize("make, batches", [(_decode, (256, 1)), (_multiquery, (1000, 1)),
                                           (_multiquery_rows, (1000, 1))])
def test_batches_of_two_sizes(make, batches, kv):
    """No thread's call fails because of the other's, and both get what they get alone."""
    import torch
    runs = [make(b, i, kv) for i, b in enumerate(batches)]
    wants = []
    for call, s in runs:
        assert call() == 0
        torch.cuda.synchronize()
        wants.append(s["out"].clone())
        assert torch.isfinite(s["out"].float()).all() and (s["out"] != 0).any()
    codes = [set(), set()]
    start = threading.Barrier(2)

    def loop(i):
        call, s = runs[i]
        start.wait()
        for n in range(CALLS):
            codes[i].add(call())
            if n % 200 == 199:
                s["stream"].synchronize()

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [{0}, {0}]
    for (_, s), want in zip(runs, wants):
        assert torch.equal(s["out"], want)
