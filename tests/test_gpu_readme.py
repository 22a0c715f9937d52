"""The README's decode step over a long context, run as it stands, step after step."""

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
    return next(b for b in blocks if "pkv_evict_tokens" in b)


def test_scores_stay_upper_bounds_after_an_eviction():
    """After the example's eviction every block's score is at least its keys' largest product."""
    import torch
    from paged_kv_decode_05_gb300 import binding as B
    batch, hkv, g, d, mb, budget = 2, 2, 4, 64, 200, 1000
    dev, bf, i32 = "cuda", torch.bfloat16, torch.int32
    gen = torch.Generator(dev).manual_seed(1)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev).to(bf)

    nb = batch * mb
    k_cache, v_cache = normal(nb, hkv, 16, d), normal(nb, hkv, 16, d)
    tables = torch.randperm(nb, generator=gen, device=dev).to(i32).view(batch, mb)
    lens = torch.tensor([2500, 3100], dtype=i32, device=dev)
    ang = torch.arange(4000, device=dev)[:, None] * 10000.0 ** (-torch.arange(32, device=dev) / 32)
    ns = dict(
        B=B, torch=torch, batch=batch, num_q_heads=hkv * g, head_dim=d, k_cache=k_cache,
        v_cache=v_cache, block_tables=tables, context_lens=lens,
        cos_sin=torch.cat([ang.cos(), ang.sin()], 1), q_weight=torch.ones(d, dtype=bf, device=dev),
        k_weight=torch.ones(d, dtype=bf, device=dev), q_rot=normal(batch, hkv * g, d),
        bounds=torch.empty((nb, hkv, 2, d), dtype=bf, device=dev),
        scores=torch.empty((batch, hkv, mb), device=dev),
        block_lists=torch.empty((batch, hkv, 128), dtype=i32, device=dev),
        list_lens=torch.empty(batch, dtype=i32, device=dev), out=normal(batch, hkv * g, d),
        mass=torch.zeros((batch, hkv, 16 * mb), device=dev), new_lens=torch.empty_like(lens),
        new_mass=torch.empty((batch, hkv, 16 * mb), device=dev),
        kept=torch.empty((batch, hkv, budget), dtype=i32, device=dev),
        ws_mass=torch.empty(B.pkv_decode_mass_workspace_size(batch, hkv * g, mb, k_cache),
                            dtype=torch.uint8, device=dev))
    B.pkv_block_bounds(k_cache, tables, lens, ns["bounds"], lens, 3200)
    for step in range(3):
        ns["context_lens"] = L = ns["context_lens"] + 1
        ns["positions"] = torch.tensor([2500, 3100], dtype=i32, device=dev) + step
        last = tables[torch.arange(batch, device=dev), (L.long() - 1) // 16].long()
        ns["slot_mapping"] = last * 16 + (L.long() - 1) % 16
        ns["q"], ns["k"], ns["v"] = (normal(batch, h, d) for h in (hkv * g, hkv, hkv))
        exec(_example(), ns)
        assert (ns["mass"][:, :, :budget] > 0).all()
        # the next step's scores, over the cache as it is now
        lens, scores = ns["context_lens"], torch.empty_like(ns["scores"])
        assert lens.tolist() == [budget, budget]
        B.pkv_block_scores(ns["q_rot"], ns["bounds"], k_cache, tables, lens, scores)
        for b, n in enumerate(lens.tolist()):
            keys = k_cache[tables[b].long()].transpose(0, 1).reshape(hkv, mb * 16, d).double()
            q = ns["q_rot"][b].view(hkv, g, d).double()
            top = (q @ keys.transpose(1, 2)).amax(1)
            top[:, n:] = -float("inf")
            blocks = -(-n // 16)
            top = top.view(hkv, mb, 16).amax(-1)[:, :blocks]
            # 2 d products summed in fp32 by products of 16 terms, as the scores' own test counts
            size = (q.abs() @ keys.abs().transpose(1, 2)).amax()
            assert (scores[b, :, :blocks] >= top - 1e-5 * size).all(), (step, b)
