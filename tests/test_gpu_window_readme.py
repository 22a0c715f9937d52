"""The README's calls of windowed attention and of the 4-bit cache, run as they stand."""

import os
import re

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_decode_05_gb300.build import build
    build()


def _example():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    return next(b for b in blocks if "pkv_u4_append" in b)


def test_the_readme_runs_as_it_stands():
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    batch, hkv, g, d, mb, n = 2, 2, 4, 64, 330, 70
    dev, bf, i32 = "cuda", torch.bfloat16, torch.int32
    gen = torch.Generator(dev).manual_seed(3)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev).to(bf)

    nb = batch * mb
    tables = torch.randperm(nb, generator=gen, device=dev).to(i32).view(batch, mb)
    lens = torch.tensor([300, 5000], dtype=i32, device=dev)
    k_cache, v_cache = normal(nb, hkv, 16, d), normal(nb, hkv, 16, d)
    old = k_cache.clone(), v_cache.clone()
    rows = [(b, t) for b in range(batch) for t in range(lens[b].item())]
    slots = torch.tensor([tables[b, t // 16].item() * 16 + t % 16 for b, t in rows], device=dev)
    k_new, v_new = normal(len(rows), hkv, d), normal(len(rows), hkv, d)
    ns = dict(
        B=B, torch=torch, batch=batch, num_q_heads=hkv * g, head_dim=d, q=normal(batch, hkv * g, d),
        k_cache=k_cache, v_cache=v_cache, block_tables=tables, context_lens=lens,
        out=torch.empty((batch, hkv * g, d), dtype=bf, device=dev), k_new=k_new, v_new=v_new,
        slot_mapping=slots, src_blocks=tables.flatten(), dst_blocks=tables.flatten(), max_q_len=n,
        cu_q=torch.tensor([0, n, 2 * n], dtype=i32, device=dev), q_runs=normal(2 * n, hkv * g, d),
        out_runs=torch.empty((2 * n, hkv * g, d), dtype=bf, device=dev))
    for x in "kv":
        ns[x + "_codes"] = torch.zeros((nb, hkv, 16, d // 2), dtype=torch.uint8, device=dev)
        ns[x + "_pairs"] = torch.zeros((nb, hkv, 16, 2), dtype=bf, device=dev)
    code = _example()
    outs = []

    # the first call's output is overwritten by the 4-bit one: keep both
    class Calls:
        def __getattr__(self, name):
            fn = getattr(B, name)
            if name != "pkv_window_decode_attn":
                return fn

            def call(*args, **kw):
                fn(*args, **kw)
                outs.append(ns["out"].clone())
            return call
    ns["B"] = Calls()
    exec(code, ns)

    def values(codes, pairs):
        c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double()
        return c * pairs[..., :1].double() + pairs[..., 1:].double()

    def attend(q, kc, vc, k_size, v_size, b, p, window, sinks):
        """The output in 64 bits, and the bound of an error: half a step of bf16, and of the sum of
        the weighted sizes of V 2^-11 (weights in one fp16 part), 2^-20 (exponentials), twice a
        score's error (chains of 4 products of 16 terms and 25 more roundings over 4 bits: 96
        2^-23 of the sum of |q| by K's sizes) and the roundings of sums in 16s, 17 each, twice."""
        ks, vs, kz, vz = (x[tables[b].long()].transpose(0, 1).reshape(hkv, mb * 16, d).double()
                          for x in (kc, vc, k_size, v_size))
        t = torch.arange(mb * 16, device=dev)
        seen = (t <= p) & ((t > p - window) | (t < sinks) if window else t >= 0)
        qs = q.view(hkv, g, d).double() * d ** -0.5
        dots = (qs.abs() @ kz.transpose(1, 2))[..., seen].amax()
        w = (qs @ ks.transpose(1, 2)).masked_fill(~seen, -float("inf")).softmax(-1)
        off = 2.0 ** -11 + 2.0 ** -20 + 2 * 96 * 2.0 ** -23 * dots + (
            2 * (int(seen.sum()) / 16 + 4) * 17 * 2.0 ** -23)
        want = (w @ vs).reshape(hkv * g, d)
        return want, 2.0 ** -8 * want.abs() + 1.01 * off * (w @ vz).reshape(hkv * g, d) + 2.0 ** -24

    def sizes(codes, pairs):
        return values(codes, torch.stack([pairs[..., 0], pairs[..., 1].abs()], -1))

    k4, v4 = values(ns["k_codes"], ns["k_pairs"]), values(ns["v_codes"], ns["v_pairs"])
    written = torch.zeros((nb, 16), dtype=torch.bool, device=dev)
    written.view(-1)[slots] = True
    for got, want in ((k_cache, k4), (v_cache, v4)):
        m = written[:, None, :, None]
        # one rounding to bf16 of the value, computed in fp32
        err = torch.where(m, (got.double() - want).abs() - (2.0 ** -8 + 2.0 ** -22) * want.abs(), 0.0)
        assert err.max() <= 2.0 ** -20
    z4 = sizes(ns["k_codes"], ns["k_pairs"]), sizes(ns["v_codes"], ns["v_pairs"])
    for b in range(batch):
        p = lens[b].item() - 1
        for got, kv, size, w, s in ((outs[0], old, [x.abs() for x in old], 4096, 4),
                                    (outs[1], (k4, v4), z4, 0, 0)):
            want, tol = attend(ns["q"][b], *kv, *size, b, p, w, s)
            assert ((got[b].double() - want).abs() <= tol).all(), b
        for i in range(n):
            want, tol = attend(ns["q_runs"][b * n + i], k_cache, v_cache, k_cache.abs(),
                               v_cache.abs(), b, p - (n - 1 - i), 4096, 4)
            assert ((ns["out_runs"][b * n + i].double() - want).abs() <= tol).all(), (b, i)
