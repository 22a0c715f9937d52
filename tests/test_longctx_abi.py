"""Refusals of the long-context entry points: every call here is turned away by
host-side checks before any CUDA call, so no GPU is needed."""

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


def desc(nb=8, bs=16, h=2, d=128, dt=B.PKV_BF16):
    return B.CacheDesc(nb, bs, h, d, dt)


def _call(lib, fn, names, base, **over):
    args = dict(base, **over)
    return getattr(lib, fn)(*[ctypes.byref(a) if isinstance(a, B.CacheDesc) else a
                              for a in (args[n] for n in names)])


ROPE = ("q qs k ks dtype n hq hkv d qw kw eps table rows rot inter pos axes axis q_out k_out st "
        "stream").split()
ROPE_BASE = dict(q=FAKE, qs=1024, k=FAKE * 2, ks=256, dtype=B.PKV_BF16, n=4, hq=8, hkv=2, d=128,
                 qw=None,
                 kw=None, eps=1e-6, table=FAKE, rows=100, rot=128, inter=0, pos=FAKE, axes=1,
                 axis=None,
                 q_out=FAKE * 3, k_out=FAKE * 4, st=None, stream=None)


@pytest.mark.parametrize("over, want", [
    (dict(n=0), 0), (dict(n=-1), INVALID), (dict(dtype=B.PKV_I8), INVALID), (dict(hq=0), INVALID),
    (dict(hkv=0), INVALID), (dict(d=96), UNSUPPORTED), (dict(rot=130), INVALID),
    (dict(rot=-16), INVALID),
    (dict(rot=24), UNSUPPORTED), (dict(inter=2), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(qs=1016), INVALID), (dict(qs=1028), INVALID),
    (dict(ks=250), INVALID), (dict(axes=0), INVALID), (dict(axes=5), INVALID),
    (dict(rows=0), INVALID),
    (dict(axis=(ctypes.c_int32 * 64)(*[1] * 64)), INVALID),
    (dict(axis=(ctypes.c_int32 * 64)(*[-1] * 64), axes=2), INVALID), (dict(q=None), INVALID),
    (dict(k=None), INVALID), (dict(q_out=None), INVALID), (dict(k_out=None), INVALID),
    (dict(table=None), INVALID), (dict(pos=None), INVALID), (dict(table=FAKE + 4), INVALID),
    (dict(q=FAKE + 8), INVALID), (dict(qw=FAKE + 2), INVALID), (dict(pos=FAKE + 1), INVALID),
    (dict(q_out=FAKE, qs=2048), INVALID), (dict(k_out=FAKE * 2, ks=512), INVALID),
    (dict(st=FAKE + 2), INVALID),
])
def test_rope(lib, over, want):
    assert _call(lib, "pkv_qk_norm_rope", ROPE, ROPE_BASE, **over) == want


@pytest.mark.parametrize("over, want", [
    (dict(n=0), 0), (dict(cache=None), INVALID), (dict(cache=desc(dt=B.PKV_I8)), UNSUPPORTED),
    (dict(cache=desc(bs=32)), UNSUPPORTED), (dict(cache=desc(d=80)), UNSUPPORTED),
    (dict(cache=desc(nb=0)), INVALID), (dict(dtype=B.PKV_F16), INVALID), (dict(v=None), INVALID),
    (dict(vs=200), INVALID), (dict(vs=260), INVALID), (dict(slots=None), INVALID),
    (dict(slots=FAKE + 4), INVALID), (dict(kc=None), INVALID), (dict(vc=FAKE + 8), INVALID),
])
def test_rope_append(lib, over, want):
    names = ("q qs k ks v vs dtype n hq qw kw eps table rows rot inter pos axes axis q_out slots "
             "kc vc cache st stream").split()
    base = dict(ROPE_BASE, v=FAKE, vs=256, slots=FAKE, kc=FAKE * 5, vc=FAKE * 6, cache=desc())
    assert _call(lib, "pkv_qk_norm_rope_append", names, base, **over) == want


@pytest.mark.parametrize("over, want", [
    (dict(b=0), 0), (dict(max_new=0, num=FAKE), 0), (dict(max_new=0), INVALID),
    (dict(max_new=2), INVALID),
    (dict(b=-1), INVALID), (dict(mb=0), INVALID), (dict(cache=None), INVALID),
    (dict(cache=desc(d=96)), UNSUPPORTED), (dict(cache=desc(bs=8)), UNSUPPORTED),
    (dict(k=None), INVALID),
    (dict(k=FAKE + 8), INVALID), (dict(bounds=None), INVALID), (dict(lens=None), INVALID),
    (dict(tables=None), INVALID), (dict(mb=1 << 28), INVALID),
])
def test_bounds(lib, over, want):
    names = "k cache tables mb lens num max_new b bounds st stream".split()
    base = dict(k=FAKE, cache=desc(), tables=FAKE, mb=4, lens=FAKE, num=None, max_new=1, b=3,
                bounds=FAKE,
                st=None, stream=None)
    assert _call(lib, "pkv_block_bounds", names, base, **over) == want


@pytest.mark.parametrize("over, want", [
    (dict(b=0), 0), (dict(qt=B.PKV_F16), INVALID), (dict(qt=B.PKV_I8), INVALID),
    (dict(hq=7), INVALID),
    (dict(hq=32), UNSUPPORTED), (dict(hq=6), UNSUPPORTED), (dict(cache=desc(dt=B.PKV_I8)), INVALID),
    (dict(cache=desc(d=32)), UNSUPPORTED), (dict(q=FAKE + 2), INVALID),
    (dict(scores=None), INVALID),
    (dict(bounds=FAKE + 8), INVALID), (dict(mb=0), INVALID),
])
def test_scores(lib, over, want):
    names = "q qt bounds ks cache tables mb lens b hq scores st stream".split()
    base = dict(q=FAKE, qt=B.PKV_BF16, bounds=FAKE, ks=None, cache=desc(), tables=FAKE, mb=4,
                lens=FAKE,
                b=3, hq=8, scores=FAKE, st=None, stream=None)
    assert _call(lib, "pkv_block_scores", names, base, **over) == want


@pytest.mark.parametrize("over, want", [
    (dict(b=0), 0), (dict(b=-1), INVALID), (dict(h=0), INVALID), (dict(mb=0), INVALID),
    (dict(budget=0), INVALID), (dict(first=-1), INVALID), (dict(last=-1), INVALID),
    (dict(first=5, last=4), INVALID), (dict(first=2**31 - 1, last=2**31 - 1), INVALID),
    (dict(scores=None), INVALID), (dict(lists=None), INVALID), (dict(n=None), INVALID),
    (dict(lens=FAKE + 2), INVALID),
])
def test_select(lib, over, want):
    names = "scores b h mb lens first last budget lists n st stream".split()
    base = dict(scores=FAKE, b=3, h=2, mb=40, lens=FAKE, first=1, last=2, budget=8, lists=FAKE,
                n=FAKE,
                st=None, stream=None)
    assert _call(lib, "pkv_block_select", names, base, **over) == want


ATTN = [
    (dict(b=0), 0), (dict(cache=None), INVALID), (dict(hq=7), INVALID), (dict(hq=32), UNSUPPORTED),
    (dict(cache=desc(d=80)), UNSUPPORTED), (dict(cache=desc(bs=32)), UNSUPPORTED),
    (dict(qt=B.PKV_F16), INVALID), (dict(qt=B.PKV_I8), INVALID), (dict(b=9000), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(q=FAKE + 8), INVALID), (dict(out=FAKE + 8), INVALID),
    (dict(k=None), INVALID), (dict(cache=desc(dt=B.PKV_I8)), INVALID), (dict(mb=0), INVALID),
    (dict(mb=1 << 28), INVALID), (dict(b=8192, mb=1 << 20), UNSUPPORTED),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(parts=-1), INVALID),
    (dict(ws_bytes=16), WORKSPACE), (dict(ws=None), WORKSPACE), (dict(ws=FAKE + 128), WORKSPACE),
    (dict(st=FAKE + 1), INVALID),
]
ATTN_BASE = dict(q=FAKE, qt=B.PKV_BF16, k=FAKE, v=FAKE, ks=None, vs=None, cache=desc(),
                 tables=FAKE, mb=4,
                 lens=FAKE, b=4, hq=8, scale=0.125, out=FAKE, ws=FAKE, ws_bytes=1 << 40, parts=64,
                 st=None,
                 stream=None)


@pytest.mark.parametrize("over, want", ATTN + [
    (dict(max_list=-1), INVALID), (dict(lists=None), INVALID), (dict(list_lens=None), INVALID),
    (dict(list_lens=FAKE + 2), INVALID), (dict(b=8192, max_list=1 << 20), UNSUPPORTED),
    (dict(max_list=0, lists=None, ws_bytes=16), WORKSPACE)])
def test_sparse_attn(lib, over, want):
    names = ("q qt k v ks vs cache tables mb lens lists max_list list_lens b hq scale out ws "
             "ws_bytes parts st stream").split()
    base = dict(ATTN_BASE, lists=FAKE, max_list=3, list_lens=FAKE)
    assert _call(lib, "pkv_sparse_decode_attn", names, base, **over) == want


@pytest.mark.parametrize("over, want", ATTN + [(dict(m_out=None), INVALID),
                                               (dict(m_out=FAKE + 2), INVALID),
                                               (dict(m_in=FAKE + 2), INVALID),
                                               (dict(m_in=FAKE + 4), INVALID),
                                               (dict(m_in=FAKE + 4 * 4 * 2 * 64 - 4), INVALID),
                                               (dict(m_out=FAKE * 2, m_in=FAKE * 2 - 4), INVALID),
                                               (dict(m_in=FAKE, ws=None), WORKSPACE),
                                               (dict(m_in=FAKE + 4 * 4 * 2 * 64, ws=None),
                                                WORKSPACE)])
def test_mass_attn(lib, over, want):
    names = ("q qt k v ks vs cache tables mb lens b hq scale out m_in m_out ws ws_bytes parts st "
             "stream").split()
    assert _call(lib, "pkv_decode_attn_mass", names, dict(ATTN_BASE, m_in=None, m_out=FAKE),
                 **over) == want


def test_workspace_sizes(lib):
    def a(x):
        return (x + 255) // 256 * 256
    d = ctypes.byref(desc(nb=100, h=8))
    slots = 32 * 8 + 640
    base = a(4 * 33) + a(slots * 4 * 2 * 4) + a(slots * 4 * 128 * 4)
    assert lib.pkv_sparse_decode_workspace_size(32, 32, d, 640) == base
    assert lib.pkv_decode_mass_workspace_size(32, 32, 50, d, 640) == base + a(32 * 8 * 800 * 4 * 4)
    assert lib.pkv_sparse_decode_workspace_size(32, 12, d, 640) == 0
    assert lib.pkv_sparse_decode_workspace_size(32, 32, d, -1) == 0
    assert lib.pkv_decode_mass_workspace_size(32, 32, 0, d, 640) == 0
    assert lib.pkv_decode_mass_workspace_size(9000, 32, 5, d, 640) == 0


@pytest.mark.parametrize("over, want", [
    (dict(b=0), 0), (dict(b=-1), INVALID), (dict(cache=None), INVALID),
    (dict(cache=desc(d=96)), UNSUPPORTED),
    (dict(cache=desc(bs=32)), UNSUPPORTED), (dict(cache=desc(dt=B.PKV_I8)), INVALID),
    (dict(budget=0), INVALID), (dict(budget=65), INVALID), (dict(first=-1), INVALID),
    (dict(first=20, last=13), INVALID), (dict(mb=0), INVALID), (dict(new_mb=0), INVALID),
    (dict(mass=None), INVALID), (dict(kept=None), INVALID), (dict(new_lens=FAKE), INVALID),
    (dict(new_mass=FAKE * 2), INVALID), (dict(new_tables=FAKE * 3, new_mb=3), INVALID),
    (dict(new_mass=FAKE * 2 + 4 * 6 * 16 * 9 - 4), INVALID), (dict(new_mass=FAKE * 2 - 4), INVALID),
    (dict(new_lens=FAKE + 8), INVALID), (dict(new_lens=FAKE - 8), INVALID),
    (dict(k=FAKE + 8), INVALID), (dict(new_mass=FAKE + 2), INVALID),
    (dict(new_tables=None), INVALID),
])
def test_evict(lib, over, want):
    names = ("k v ks vs cache tables mb lens mass b budget first last new_tables new_mb new_lens "
             "new_mass kept st stream").split()
    base = dict(k=FAKE, v=FAKE, ks=None, vs=None, cache=desc(), tables=FAKE * 3, mb=9, lens=FAKE,
                mass=FAKE * 2, b=3, budget=32, first=1, last=2, new_tables=FAKE * 4, new_mb=4,
                new_lens=FAKE * 5, new_mass=FAKE * 6, kept=FAKE * 7, st=None, stream=None)
    assert _call(lib, "pkv_evict_tokens", names, base, **over) == want


def test_binding_checks_types_and_shapes():
    """The Python layer names what is wrong before it takes a pointer."""
    bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    k = torch.zeros(8, 2, 16, 128, dtype=bf)
    tables, lens = torch.zeros(3, 4, dtype=i32), torch.zeros(3, dtype=i32)
    q = torch.zeros(3, 8, 128, dtype=bf)
    bounds, scores = torch.zeros(8, 2, 2, 128, dtype=bf), torch.zeros(3, 2, 4)
    lists, n = torch.zeros(3, 2, 5, dtype=i32), torch.zeros(3, dtype=i32)
    mass, ws = torch.zeros(3, 2, 64), torch.zeros(16, dtype=torch.uint8)
    for bad in (dict(bounds=bounds[:7]), dict(bounds=bounds.half()), dict(lens=lens.long()),
                dict(tables=tables[:2]), dict(num=lens.long()),
                dict()):      # {}: not on a CUDA device
        a = dict(dict(bounds=bounds, lens=lens, tables=tables, num=None), **bad)
        with pytest.raises((TypeError, ValueError)):
            B.pkv_block_bounds(k, a["tables"], a["lens"], a["bounds"], a["num"])
    for bad in (dict(q=q[:, :, :64]), dict(q=q[:2]), dict(scores=scores.double()),
                dict(scores=scores[:, :, :3]), dict(ks=torch.zeros(8, 3))):
        a = dict(dict(q=q, scores=scores, ks=None), **bad)
        with pytest.raises((TypeError, ValueError)):
            B.pkv_block_scores(a["q"], bounds, k, tables, lens, a["scores"], a["ks"])
    for bad in (dict(lists=lists.long()), dict(lists=lists[:, :1]), dict(n=n[:2]),
                dict(lens=lens[:2])):
        a = dict(dict(lists=lists, n=n, lens=lens), **bad)
        with pytest.raises((TypeError, ValueError)):
            B.pkv_block_select(scores, a["lens"], 1, 1, a["lists"], a["n"])
        with pytest.raises((TypeError, ValueError)):
            B.pkv_sparse_decode_attn(q, k, k, tables, a["lens"], a["lists"], a["n"], 0.1, q, ws)
    for bad in (dict(m=mass[:, :, :63]), dict(m=mass.half()), dict(out=q.half()), dict(v=k[:4])):
        a = dict(dict(m=mass, out=q, v=k), **bad)
        with pytest.raises((TypeError, ValueError)):
            B.pkv_decode_attn_mass(q, k, a["v"], tables, lens, 0.1, a["out"], None, a["m"], ws)
    for bad in (dict(nm=mass[:, :, :32]), dict(kept=lists.long()), dict(new=tables.long()),
                dict(m=mass[:2])):
        a = dict(dict(nm=mass, kept=lists, new=tables, m=mass), **bad)
        with pytest.raises((TypeError, ValueError)):
            B.pkv_evict_tokens(k, k, tables, lens, a["m"], 0, 0, a["new"], n, a["nm"], a["kept"])
    pos, table = torch.zeros(3, dtype=i32), torch.zeros(9, 128, dtype=f32)
    kk = torch.zeros(3, 2, 128, dtype=bf)
    for bad in (dict(pos=pos.long()), dict(pos=pos[:2]), dict(axis=[0] * 63),
                dict(qw=torch.zeros(64, dtype=bf)),
                dict(k=kk[:2]), dict(table=table.double()), dict(q_out=q.half())):
        a = dict(dict(pos=pos, axis=None, qw=None, k=kk, table=table, q_out=q), **bad)
        with pytest.raises((TypeError, ValueError)):
            B.pkv_qk_norm_rope(q, a["k"], a["pos"], a["table"], a["q_out"], kk, a["qw"],
                               pair_axis=a["axis"])
        with pytest.raises((TypeError, ValueError)):
            B.pkv_qk_norm_rope_append(q, a["k"], a["k"], a["pos"], a["table"],
                                      torch.zeros(3).long(), k, k,
                                      a["q_out"], a["qw"], pair_axis=a["axis"])
