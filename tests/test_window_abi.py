"""Refusals of the windowed-attention and 4-bit cache entry points: turned away by host-side checks
before any CUDA call, so no GPU is needed."""

import ctypes

import pytest
import torch

from paged_kv_decode_05_gb300 import binding as B
from paged_kv_decode_05_gb300.build import build

FAKE = 0x100000          # never dereferenced
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    build()
    return B.lib()


def desc(nb=8, bs=16, h=2, d=128, dt=B.PKV_U4):
    return B.CacheDesc(nb, bs, h, d, dt)


def _call(lib, fn, names, base, **over):
    args = dict(base, **over)
    return getattr(lib, fn)(*[ctypes.byref(a) if isinstance(a, B.CacheDesc) else a
                              for a in (args[n] for n in names)])


@pytest.mark.parametrize("over, want", [
    (dict(n=0), 0), (dict(n=-1), INVALID), (dict(cache=None), INVALID),
    (dict(cache=desc(dt=B.PKV_BF16)), INVALID), (dict(cache=desc(dt=B.PKV_I8)), INVALID),
    (dict(cache=desc(bs=32)), UNSUPPORTED), (dict(cache=desc(d=96)), UNSUPPORTED),
    (dict(cache=desc(nb=0)), INVALID), (dict(cache=desc(h=0)), INVALID),
    (dict(cache=desc(h=70000)), UNSUPPORTED), (dict(dt=B.PKV_I8), INVALID),
    (dict(dt=B.PKV_U4), INVALID), (dict(ks=248), INVALID), (dict(vs=260), INVALID),
    (dict(ks=255), INVALID), (dict(k=None), INVALID), (dict(v=FAKE + 8), INVALID),
    (dict(slots=None), INVALID), (dict(slots=FAKE + 4), INVALID), (dict(kc=FAKE + 8), INVALID),
    (dict(vc=None), INVALID), (dict(kp=FAKE + 4), INVALID), (dict(vp=None), INVALID),
    (dict(st=FAKE + 2), INVALID),
])
def test_append(lib, over, want):
    names = "k ks v vs dt n slots kc vc kp vp cache st stream".split()
    base = dict(k=FAKE, ks=256, v=FAKE, vs=256, dt=B.PKV_F16, n=3, slots=FAKE, kc=FAKE, vc=FAKE,
                kp=FAKE, vp=FAKE, cache=desc(), st=None, stream=None)
    assert _call(lib, "pkv_u4_append", names, base, **over) == want


@pytest.mark.parametrize("over, want", [
    (dict(n=0), 0), (dict(n=-1), INVALID), (dict(cache=None), INVALID),
    (dict(cache=desc(dt=B.PKV_F16)), INVALID), (dict(cache=desc(d=32)), UNSUPPORTED),
    (dict(dt=B.PKV_I8), INVALID), (dict(onb=0), INVALID), (dict(k=None), INVALID),
    (dict(v=FAKE + 8), INVALID), (dict(kp=FAKE + 8), INVALID), (dict(vp=None), INVALID),
    (dict(src=None), INVALID), (dict(src=FAKE + 2), INVALID), (dict(dst=FAKE + 1), INVALID),
    (dict(ko=None), INVALID), (dict(vo=FAKE + 8), INVALID), (dict(st=FAKE + 1), INVALID),
])
def test_read_blocks(lib, over, want):
    names = "k v kp vp cache src dt ko vo onb dst n st stream".split()
    base = dict(k=FAKE, v=FAKE, kp=FAKE, vp=FAKE, cache=desc(), src=FAKE, dt=B.PKV_BF16, ko=FAKE,
                vo=FAKE, onb=4, dst=FAKE, n=2, st=None, stream=None)
    assert _call(lib, "pkv_u4_read_blocks", names, base, **over) == want


@pytest.mark.parametrize("over, want", [
    (dict(b=0), 0), (dict(cache=None), INVALID), (dict(hq=7), INVALID), (dict(hq=32), UNSUPPORTED),
    (dict(cache=desc(d=80)), UNSUPPORTED), (dict(cache=desc(bs=32)), UNSUPPORTED),
    (dict(qt=B.PKV_I8), INVALID), (dict(qt=B.PKV_U4), INVALID),
    (dict(cache=desc(dt=B.PKV_BF16), qt=B.PKV_F16), INVALID), (dict(cache=desc(dt=7)), INVALID),
    (dict(b=9000), UNSUPPORTED), (dict(b=-1), INVALID), (dict(window=-1), INVALID),
    (dict(sinks=-1), INVALID), (dict(q=None), INVALID), (dict(q=FAKE + 8), INVALID),
    (dict(out=FAKE + 8), INVALID), (dict(k=None), INVALID), (dict(ks=None), INVALID),
    (dict(vs=FAKE + 8), INVALID), (dict(cache=desc(dt=B.PKV_I8), ks=None), INVALID),
    (dict(cache=desc(dt=B.PKV_I8), ks=FAKE + 2), INVALID), (dict(tables=None), INVALID),
    (dict(lens=FAKE + 1), INVALID), (dict(mb=0), INVALID), (dict(mb=1 << 28), INVALID),
    (dict(b=8192, mb=1 << 20), UNSUPPORTED), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(parts=-1), INVALID), (dict(ws_bytes=16), WORKSPACE),
    (dict(ws=None), WORKSPACE), (dict(ws=FAKE + 128), WORKSPACE), (dict(st=FAKE + 1), INVALID),
])
def test_decode(lib, over, want):
    names = ("q qt k v ks vs cache tables mb lens b hq scale window sinks out ws ws_bytes parts st "
             "stream").split()
    base = dict(q=FAKE, qt=B.PKV_BF16, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, cache=desc(), tables=FAKE,
                mb=4, lens=FAKE, b=4, hq=8, scale=0.125, window=5, sinks=1, out=FAKE, ws=FAKE,
                ws_bytes=1 << 40, parts=64, st=None, stream=None)
    assert _call(lib, "pkv_window_decode_attn", names, base, **over) == want


@pytest.mark.parametrize("over, want", [
    (dict(b=0), 0), (dict(cache=None), INVALID), (dict(cache=desc()), INVALID),
    (dict(hq=7), INVALID), (dict(hq=32), UNSUPPORTED), (dict(window=-1), INVALID),
    (dict(sinks=-1), INVALID), (dict(max_q=0), INVALID), (dict(qt=B.PKV_F16), INVALID),
    (dict(cache=desc(dt=B.PKV_BF16, d=80)), UNSUPPORTED), (dict(b=5000), UNSUPPORTED),
    (dict(cache=desc(dt=B.PKV_BF16, nb=1 << 27)), UNSUPPORTED), (dict(q=None), INVALID),
    (dict(cu=None), INVALID), (dict(k=FAKE + 8), INVALID), (dict(out=None), INVALID),
    (dict(cache=desc(dt=B.PKV_I8)), INVALID), (dict(mb=0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(ws=None), WORKSPACE), (dict(ws_bytes=16), WORKSPACE),
    (dict(st=FAKE + 2), INVALID),
])
def test_multi(lib, over, want):
    names = ("q qt cu max_q k v ks vs cache tables mb lens b hq scale window sinks out ws ws_bytes "
             "parts st stream").split()
    base = dict(q=FAKE, qt=B.PKV_BF16, cu=FAKE, max_q=5, k=FAKE, v=FAKE, ks=None, vs=None,
                cache=desc(dt=B.PKV_BF16), tables=FAKE, mb=4, lens=FAKE, b=4, hq=8, scale=0.125,
                window=5, sinks=1, out=FAKE, ws=FAKE, ws_bytes=1 << 40, parts=64, st=None,
                stream=None)
    assert _call(lib, "pkv_window_multiquery_attn", names, base, **over) == want


def test_other_calls_refuse_4_bit_caches(lib):
    """No call that does not name them takes a cache of 4-bit codes."""
    d = ctypes.byref(desc())
    assert lib.pkv_append_workspace_size(d) == 0
    assert lib.pkv_decode_workspace_size(4, 8, d, 16) == 0
    assert lib.pkv_sparse_decode_workspace_size(4, 8, d, 16) == 0
    assert lib.pkv_decode_mass_workspace_size(4, 8, 4, d, 16) == 0
    assert lib.pkv_multiquery_workspace_size(4, 8, 5, d, 16) == 0
    assert lib.pkv_window_multiquery_workspace_size(4, 8, 5, d, 16) == 0
    assert lib.pkv_append(FAKE, FAKE, B.PKV_BF16, 1, FAKE, FAKE, FAKE, FAKE, FAKE, d, FAKE, 1 << 40,
                          None, None) == INVALID
    assert lib.pkv_copy_blocks(FAKE, FAKE, FAKE, FAKE, d, FAKE, FAKE, 1, None, None) == INVALID
    assert lib.pkv_block_bounds(FAKE, d, FAKE, 4, FAKE, None, 1, 2, FAKE, None, None) == INVALID


def test_workspace_sizes(lib):
    def a(x):
        return (x + 255) // 256 * 256
    slots = 32 * 8 + 640
    base = a(4 * 33) + a(slots * 4 * 2 * 4) + a(slots * 4 * 128 * 4)
    for dt in (B.PKV_U4, B.PKV_I8, B.PKV_BF16):
        d = ctypes.byref(desc(nb=100, h=8, dt=dt))
        assert lib.pkv_window_decode_workspace_size(32, 32, d, 640) == base
        assert lib.pkv_window_decode_workspace_size(32, 32, d, 647) == base    # whole ranges
        assert lib.pkv_window_decode_workspace_size(32, 12, d, 640) == 0
        assert lib.pkv_window_decode_workspace_size(32, 32, d, -1) == 0
        assert lib.pkv_window_decode_workspace_size(9000, 32, d, 640) == 0
    d = ctypes.byref(desc(nb=100, h=8))
    assert lib.pkv_window_decode_workspace_size(32, 32, d, 3) > 0              # fewer than kv heads


def test_binding_checks_types_and_shapes():
    """The Python layer names what is wrong before it takes a pointer."""
    bf, i32 = torch.bfloat16, torch.int32
    codes = torch.zeros(8, 2, 16, 64, dtype=torch.uint8)
    pairs = torch.zeros(8, 2, 16, 2, dtype=bf)
    rows, slots = torch.zeros(3, 2, 128, dtype=bf), torch.zeros(3, dtype=torch.int64)
    for bad in (dict(), dict(rows=rows[:, :1]), dict(rows=rows[:, :, :64]), dict(codes=codes.char()),
                dict(slots=slots.int()), dict(pairs=pairs.half())):      # {}: not on a CUDA device
        a = dict(dict(rows=rows, codes=codes, slots=slots, pairs=pairs), **bad)
        with pytest.raises((TypeError, ValueError)):
            B.pkv_u4_append(a["rows"], a["rows"], a["slots"], a["codes"], a["codes"], a["pairs"],
                            a["pairs"])
    out = torch.zeros(4, 2, 16, 128, dtype=bf)
    ids = torch.zeros(2, dtype=i32)
    for bad in (dict(), dict(out=out[:, :1]), dict(out=out.float()), dict(ids=ids.long())):
        a = dict(dict(out=out, ids=ids), **bad)
        with pytest.raises((TypeError, ValueError)):
            B.pkv_u4_read_blocks(codes, codes, pairs, pairs, a["ids"], a["out"], a["out"], a["ids"])
    q, tables, lens = torch.zeros(3, 8, 128, dtype=bf), torch.zeros(3, 4, dtype=i32), ids.new_zeros(3)
    ws = torch.zeros(16, dtype=torch.uint8)
    for bad in (dict(), dict(q=q[:, :, :64]), dict(lens=lens.long()), dict(tables=tables[:2]),
                dict(pairs=None), dict(out=q.half())):
        a = dict(dict(q=q, lens=lens, tables=tables, pairs=pairs, out=q), **bad)
        with pytest.raises((TypeError, ValueError)):
            B.pkv_window_decode_attn(a["q"], codes, codes, a["tables"], a["lens"], 0.1, 4, 0,
                                     a["out"], ws, a["pairs"], a["pairs"])
    k, cu = torch.zeros(8, 2, 16, 128, dtype=bf), torch.zeros(4, dtype=i32)
    for bad in (dict(), dict(cu=cu[:3]), dict(cu=cu.long()), dict(q=q[:, :, :64]), dict(k=k.half())):
        a = dict(dict(q=q, cu=cu, k=k), **bad)
        with pytest.raises((TypeError, ValueError)):
            B.pkv_window_multiquery_attn(a["q"], a["cu"], 5, a["k"], k, tables, lens, 0.1, 4, 0, q,
                                         ws)
