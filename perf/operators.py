"""Workloads of the long-context operators, in plain torch and through the library.

Five operators of a decode step over a long paged KV cache:

* ``rope``    per-head norms of q and k, the position rotation, and the write
              of K and V into the paged cache;
* ``score``   the channel bounds of the blocks that got new keys, and the
              upper bound of every block's scores against the new queries;
* ``sparse``  the choice of blocks by score, and attention over the chosen ones;
* ``mass``    decode attention that adds each token's weights to an accumulator;
* ``evict``   the cut of every sequence to a budget of tokens by accumulated
              weight, compacted into new blocks.

``run`` computes them with elementary torch operations, or, where ``own`` is
true, through the library. The cache layout is the library's: blocks of 16
tokens, ``[num_blocks, num_kv_heads, 16, head_dim]``.
"""

import math

import torch

own = False

BS = 16
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "i8": torch.int8}
BYTES = {"bf16": 2, "f16": 2, "i8": 1}


# ------------------------------------------------------------------ cases ---
def listed():
    return [
        # one sequence's new token: latency of the write path
        dict(name="rope_one_token", op="rope", tokens=1, hq=32, hkv=8, d=128, dt="bf16", axes=1,
             rot=128, inter=False, norm=True),
        # a prefill chunk of an image-text batch: three position axes, part of
        # the head rotated, an odd token count
        dict(name="rope_chunk_3axes", op="rope", tokens=8191, hq=32, hkv=8, d=128, dt="bf16",
             axes=3, rot=96, inter=False, norm=True),
        # a handful of short sequences, odd lengths
        dict(name="score_few", op="score", batch=3, hq=32, hkv=8, d=128, kv="f16", lo=333, hi=3001),
        # a long-context batch
        dict(name="score_long", op="score", batch=32, hq=32, hkv=8, d=128, kv="bf16", lo=8192,
             hi=32768),
        # two chats, a small budget: latency of choice and attention
        dict(name="sparse_two", op="sparse", batch=2, hq=32, hkv=8, d=128, kv="bf16", q="bf16",
             lo=1000, hi=5001, budget=32, first=1, last=2),
        # a long-context batch, 2048 tokens of each head's context read
        dict(name="sparse_long", op="sparse", batch=64, hq=32, hkv=8, d=128, kv="bf16", q="bf16",
             lo=8192, hi=32768, budget=128, first=1, last=4),
        # the same choice over an INT8 cache, one group size up
        dict(name="sparse_int8", op="sparse", batch=48, hq=32, hkv=4, d=128, kv="i8", q="bf16",
             lo=4096, hi=32768, budget=256, first=4, last=8),
        # one sequence: latency
        dict(name="mass_one", op="mass", batch=1, hq=32, hkv=8, d=128, kv="bf16", q="bf16", lo=1023,
             hi=1023),
        # the benchmark's decode batch
        dict(name="mass_batch", op="mass", batch=256, hq=32, hkv=8, d=128, kv="bf16", q="bf16",
             lo=128, hi=4096),
        # an INT8 cache without head groups, head_dim 64
        dict(name="mass_int8", op="mass", batch=64, hq=16, hkv=16, d=64, kv="i8", q="f16", lo=100,
             hi=8000),
        # two sequences outgrow their budget
        dict(name="evict_two", op="evict", batch=2, hkv=8, d=128, kv="f16", lo=1500, hi=2500,
             budget=1000, first=4, last=128),
        # a whole batch is cut under memory pressure
        dict(name="evict_batch", op="evict", batch=48, hkv=8, d=128, kv="bf16", lo=2048, hi=12288,
             budget=2048, first=4, last=512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "score", "sparse", "mass", "evict"])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128])
    dt = rng.choice(["bf16", "f16"])
    if op == "rope":
        rot = rng.choice([d, d, d // 2, d - 16])
        return dict(op=op, tokens=_log(rng, 1, min(30000, 48000000 // ((g + 2) * hkv * d))),
                    hq=hkv * g, hkv=hkv, d=d, dt=dt, axes=rng.choice([1, 2, 3]), rot=rot,
                    inter=rng.random() < 0.4, norm=rng.random() < 0.8)
    if op == "score":
        batch = _log(rng, 1, 32)
        hi = _log(rng, 20, 32768)
        return dict(op=op, batch=batch, hq=hkv * g, hkv=hkv, d=d, kv=dt, lo=rng.randint(1, hi),
                    hi=hi)
    if op == "sparse":
        batch = _log(rng, 1, 48)
        hi = _log(rng, 40, 32768)
        first, last = rng.randint(0, 4), rng.randint(1, 8)
        kv = rng.choice([dt, dt, "i8"])
        return dict(op=op, batch=batch, hq=hkv * g, hkv=hkv, d=d, kv=kv, q=dt,
                    lo=rng.randint(1, hi), hi=hi, budget=max(first + last, _log(rng, 4, 128)),
                    first=first, last=last)
    if op == "mass":
        batch = _log(rng, 1, 200)
        hi = _log(rng, 30, min(32768, 540000 // batch))
        kv = rng.choice([dt, dt, "i8"])
        return dict(op=op, batch=batch, hq=hkv * g, hkv=hkv, d=d, kv=kv, q=dt,
                    lo=rng.randint(1, hi), hi=hi)
    batch = _log(rng, 1, 40)
    hi = _log(rng, 40, min(12288, 300000 // batch))
    budget = max(16, min(90000 // batch, int(hi * rng.uniform(0.05, 0.5))))
    return dict(op=op, batch=batch, hkv=hkv, d=d, kv=dt, lo=rng.randint(1, hi), hi=hi,
                budget=budget, first=rng.randint(0, 4), last=rng.randint(1, 12))


def _lens(case):
    """Lengths spread over [lo, hi] by the golden ratio, the same for every seed."""
    lo, hi, n = case["lo"], case["hi"], case["batch"]
    return [lo + int((hi - lo + 1) * ((i * 0.6180339887498949 + 0.999) % 1.0)) for i in range(n)]


# ----------------------------------------------------------------- inputs ---
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, dtype, gen, scale=1.0):
    x = torch.empty(shape, dtype=dtype, device="cuda")
    flat, step = x.view(-1), 1 << 26
    for i in range(0, flat.numel(), step):   # in pieces: no fp32 copy of a large cache
        part = flat[i:i + step]
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda") * scale)
    return x


def _codes(shape, gen):
    x = torch.empty(shape, dtype=torch.int8, device="cuda")
    flat, step = x.view(-1), 1 << 26
    for i in range(0, flat.numel(), step):
        part = flat[i:i + step]
        y = torch.randn(part.shape, generator=gen, device="cuda") * 42.0
        part.copy_(y.round_().clamp_(-127, 127))
    return x


def _tables(lens, gen, extra_cols=1, extra_blocks=5, more=0):
    """Block tables over a shuffled pool; `more` further blocks per sequence in a second table."""
    nb = [-(-n // BS) for n in lens]
    mb = max(nb) + extra_cols
    total = sum(nb) + len(lens) * more + extra_blocks
    perm = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    t = torch.zeros((len(lens), mb), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(nb):
        t[b, :n] = perm[at:at + n]
        at += n
    second = perm[at:at + len(lens) * more].reshape(len(lens), more).contiguous()
    return t, second, total, mb


def _cache(case, total, gen, values=True):
    shape = (total, case["hkv"], BS, case["d"])
    if case["kv"] == "i8":
        s = [torch.rand(shape[:2], generator=gen, device="cuda") * 0.02 + 0.01 for _ in range(2)]
        return _codes(shape, gen), _codes(shape, gen) if values else None, s[0], s[1]
    dt = DT[case["kv"]]
    # keys: channels of different size, as a trained projection gives
    k = _normal(shape, dt, gen)
    k *= (0.5 + torch.rand((case["hkv"], 1, case["d"]), generator=gen, device="cuda")).to(dt)
    return k, _normal(shape, dt, gen) if values else None, None, None


def prepare(case, seed):
    gen = _gen(seed)
    s = dict(case=case)
    if case["op"] == "rope":
        n, hq, hkv, d, dt = case["tokens"], case["hq"], case["hkv"], case["d"], DT[case["dt"]]
        # q, k and v are parts of one projection's rows
        qkv = _normal((n, hq + 2 * hkv, d), dt, gen)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["qw"] = s["kw"] = None
        if case["norm"]:
            s["qw"], s["kw"] = ((1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(dt)
                                for _ in range(2))
        rows, half = 16384, case["rot"] // 2
        freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        ang = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * freq
        s["table"] = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
        s["pos"] = torch.randint(0, rows, (case["axes"], n), generator=gen, device="cuda",
                                 dtype=torch.int32)
        # consecutive runs of pairs, one for each axis
        s["pair_axis"] = [min(case["axes"] - 1, j * case["axes"] // half) for j in range(half)]
        s["pair_axis_dev"] = torch.tensor(s["pair_axis"], device="cuda")
        nb = -(-n // BS) + 3
        s["slots"] = torch.randperm(nb * BS, generator=gen, device="cuda")[:n].contiguous()
        s["k_cache"], s["v_cache"] = (torch.zeros((nb, hkv, BS, d), dtype=dt, device="cuda")
                                      for _ in range(2))
        return s
    lens = _lens(case)
    s["max_len"] = max(lens)
    if case["op"] == "evict":
        new_mb = -(-case["budget"] // BS) + 1
        s["tables"], s["new_tables"], total, mb = _tables(lens, gen, more=new_mb)
        s["mass"] = torch.exp(2 * torch.randn((case["batch"], case["hkv"], mb * BS), generator=gen,
                                              device="cuda")) * 0.01
        s["new_mass"] = torch.zeros((case["batch"], case["hkv"], new_mb * BS), device="cuda")
        s["kept"] = torch.empty((case["batch"], case["hkv"], case["budget"]), dtype=torch.int32,
                                device="cuda")
        s["new_lens"] = torch.empty(case["batch"], dtype=torch.int32, device="cuda")
    else:
        s["tables"], _, total, mb = _tables(lens, gen)
        s["q"] = _normal((case["batch"], case["hq"], case["d"]), DT[case.get("q", case["kv"])], gen)
        s["scale"] = case["d"] ** -0.5
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"] = _cache(case, total, gen,
                                                                      case["op"] != "score")
    if case["op"] == "score":
        # bounds of all older blocks are in hand; the newest block's are stale
        k = s["k_cache"]
        s["bounds"] = torch.stack([k.amin(2), k.amax(2)], 2).contiguous()
        last = s["tables"][torch.arange(case["batch"], device="cuda"), (s["lens"].long() - 1) // BS]
        s["bounds"][last.long()] = 0
        s["scores"] = torch.empty((case["batch"], case["hkv"], mb), device="cuda")
    if case["op"] == "sparse":
        s["scores"] = 12 + 4 * torch.randn((case["batch"], case["hkv"], mb), generator=gen,
                                           device="cuda")
    if case["op"] == "mass":
        # weights of earlier steps, nothing yet for the newest token
        m = torch.rand((case["batch"], case["hkv"], mb * BS), generator=gen, device="cuda") * 0.1
        at = torch.arange(mb * BS, device="cuda")
        s["mass"] = torch.where(at < s["lens"][:, None, None] - 1, m, torch.zeros_like(m))
        s["mass_out"] = torch.zeros_like(s["mass"])
    return s


# --------------------------------------------------------------- the work ---
def work(case):
    op = case["op"]
    if op == "rope":
        n, d, rows = case["tokens"], case["d"], case["hq"] + 2 * case["hkv"]
        return {"bytes": n * (rows * d * 4 + case["rot"] * 4 + 4 * case["axes"] + 8),
                "flops": n * (case["hq"] + case["hkv"]) * d * 7}
    lens, hkv, d, e = _lens(case), case["hkv"], case["d"], BYTES[case["kv"]]
    blocks = [-(-n // BS) for n in lens]
    if op == "evict":
        kept = [min(n, case["budget"]) for n in lens]
        return {"bytes": hkv * (4 * sum(lens) + sum(kept) * (4 * d * e + 8)), "flops": 0}
    g = case["hq"] // hkv
    io = case["batch"] * case["hq"] * d * 2
    if op == "score":
        newest = sum((n - 1) % BS + 1 for n in lens)
        return {"bytes": hkv * (sum(blocks) * (2 * d * e + 4) + newest * d * e
                                + len(lens) * 2 * d * e) + io,
                "flops": sum(blocks) * hkv * g * 4 * d}
    if op == "sparse":
        chosen = [min(n, case["budget"]) for n in blocks]
        return {"bytes": hkv * (4 * sum(blocks) + sum(chosen) * (4 + 2 * BS * d * e)) + 2 * io,
                "flops": sum(chosen) * BS * hkv * g * 4 * d}
    return {"bytes": hkv * sum(lens) * (2 * d * e + 8) + 2 * io,
            "flops": sum(lens) * hkv * g * 4 * d}


# ------------------------------------------------------------- plain form ---
def _rms(x, w, eps=1e-6):
    x = x.float()
    if w is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()


def _rotate(x, cos, sin, rot, inter):
    """x [n, heads, d] fp32; cos, sin [n, 1, rot / 2]."""
    r = x[..., :rot]
    if inter:
        u, v = r[..., 0::2], r[..., 1::2]
        y = torch.stack([u * cos - v * sin, u * sin + v * cos], -1).flatten(-2)
    else:
        u, v = r[..., :rot // 2], r[..., rot // 2:]
        y = torch.cat([u * cos - v * sin, u * sin + v * cos], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _rope(s):
    c = s["case"]
    half = c["rot"] // 2
    rows = s["table"][s["pos"].long()]                       # [axes, n, rot]
    pick = s["pair_axis_dev"][None, None].expand(1, c["tokens"], half)
    cos = torch.gather(rows[..., :half], 0, pick)[0][:, None]
    sin = torch.gather(rows[..., half:], 0, pick)[0][:, None]
    q = _rotate(_rms(s["q"], s["qw"]), cos, sin, c["rot"], c["inter"]).to(s["q"].dtype)
    k = _rotate(_rms(s["k"], s["kw"]), cos, sin, c["rot"], c["inter"]).to(s["q"].dtype)
    blk, row = s["slots"] // BS, s["slots"] % BS
    s["k_cache"][blk, :, row] = k
    s["v_cache"][blk, :, row] = s["v"]
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _score(s):
    c, mb = s["case"], s["tables"].shape[1]
    # the newest block of each sequence
    at = (s["lens"].long() - 1) // BS
    blk = s["tables"].long().gather(1, at[:, None])[:, 0]
    tile = s["k_cache"][blk].float()                          # [B, hkv, 16, d]
    live = torch.arange(BS, device="cuda") < (s["lens"].long() - at * BS)[:, None]
    live = live[:, None, :, None]
    lo = torch.where(live, tile, torch.full_like(tile, math.inf)).amin(2)
    hi = torch.where(live, tile, torch.full_like(tile, -math.inf)).amax(2)
    s["bounds"][blk] = torch.stack([lo, hi], 2).to(s["bounds"].dtype)
    b = s["bounds"][s["tables"].long()].float().transpose(1, 2)   # [B, hkv, mb, 2, d]
    q = s["q"].float().view(c["batch"], c["hkv"], -1, c["d"])
    up = torch.matmul(b[..., 1, :], q.clamp(min=0).transpose(-1, -2))
    up = up + torch.matmul(b[..., 0, :], q.clamp(max=0).transpose(-1, -2))
    up = up.amax(-1)
    live = torch.arange(mb, device="cuda") * BS < s["lens"][:, None]
    return {"bounds": s["bounds"],
            "scores": torch.where(live[:, None], up, torch.full_like(up, -math.inf))}


def _choose(score, n, first, last, budget):
    """Ascending indices of the chosen of n[b] entries of score [B, hkv, m]; -1 behind them."""
    m = score.shape[-1]
    at = torch.arange(m, device=score.device)
    n = n.long()[:, None, None]
    forced = ((at < first) | (at >= n - last)) & (at < n)
    key = torch.where(forced, torch.full_like(score, math.inf), score)
    key = torch.where(at < n, key, torch.full_like(score, -math.inf))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    width = min(budget, m)
    rank = torch.arange(width, device=score.device)
    idx = torch.where(rank < n, order[..., :width], torch.full_like(order[..., :width], m))
    idx = torch.sort(idx, dim=-1).values
    idx = torch.where(idx == m, torch.full_like(idx, -1), idx)
    return torch.nn.functional.pad(idx, (0, budget - width), value=-1)


def _rows(cache, scales, blk, head):
    """Tiles of the cache as fp32: blk, head broadcast to [..., 16, d]."""
    x = cache[blk, head].float()
    return x if scales is None else x * scales[blk, head][..., None, None]


def _weights(q, k, live, scale):
    """softmax over the last axis of scale q k^T, 0 where not live (all, for an empty row)."""
    x = torch.matmul(q, k.transpose(-1, -2)) * scale
    x = torch.where(live, x, torch.full_like(x, -math.inf))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    return p, p.sum(-1, keepdim=True)


def _attend(s, tiles, blk):
    """Attention over the 16-token tiles of physical blocks blk [B, hkv, n]; tiles [B, hkv, n]:
    their place in the sequence, -1 where there is none."""
    c = s["case"]
    head = torch.arange(c["hkv"], device="cuda")[None, :, None]
    k = _rows(s["k_cache"], s["k_scales"], blk, head).flatten(2, 3)
    v = _rows(s["v_cache"], s["v_scales"], blk, head).flatten(2, 3)
    pos = (tiles[..., None] * BS + torch.arange(BS, device="cuda")).flatten(2)
    live = (pos < s["lens"][:, None, None]) & (tiles >= 0).repeat_interleave(BS, -1)
    q = s["q"].float().view(c["batch"], c["hkv"], -1, c["d"])
    p, l = _weights(q, k, live[:, :, None], s["scale"])
    p = p / torch.where(l == 0, torch.ones_like(l), l)
    out = torch.matmul(p, v * live[..., None])
    return out.reshape(s["q"].shape).to(s["q"].dtype), p, live


def _sparse(s):
    c = s["case"]
    n = (s["lens"] + BS - 1) // BS
    lists = _choose(s["scores"], n, c["first"], c["last"], c["budget"])
    blk = torch.gather(s["tables"].long()[:, None].expand(-1, c["hkv"], -1), 2,
                       lists.clamp(min=0))
    out, _, _ = _attend(s, lists, blk)
    return {"lists": lists.to(torch.int32), "list_lens": n.clamp(max=c["budget"]), "out": out}


def _mass(s):
    c, mb = s["case"], s["tables"].shape[1]
    blk = s["tables"].long()[:, None].expand(-1, c["hkv"], -1)
    out, p, live = _attend(s, torch.arange(mb, device="cuda").expand(blk.shape), blk)
    s["mass_out"].copy_(torch.where(live, s["mass"] + p.sum(2), s["mass_out"]))
    return {"out": out, "mass": s["mass_out"]}


def _evict(s):
    c = s["case"]
    kept = _choose(s["mass"], s["lens"], c["first"], c["last"], c["budget"])
    at = kept.clamp(min=0)
    b = torch.arange(c["batch"], device="cuda")[:, None, None]
    h = torch.arange(c["hkv"], device="cuda")[None, :, None]
    src = s["tables"].long()[b, at // BS]
    rank = torch.arange(c["budget"], device="cuda")
    dst = s["new_tables"].long()[b, (rank // BS)[None, None]]
    live = kept >= 0
    hh, row = h.expand(kept.shape)[live], (rank % BS).expand(kept.shape)[live]
    dst, src, at_row = dst.expand(kept.shape)[live], src[live], (at % BS)[live]
    s["k_cache"][dst, hh, row] = s["k_cache"][src, hh, at_row]
    s["v_cache"][dst, hh, row] = s["v_cache"][src, hh, at_row]
    s["new_mass"].zero_()
    s["new_mass"][..., :c["budget"]] = torch.where(live, torch.gather(s["mass"], 2, at), 0.0)
    return {"kept": kept.to(torch.int32), "lens": s["lens"].clamp(max=c["budget"]),
            "mass": s["new_mass"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


# ------------------------------------------------------------ the library ---
def _own_rope(s, B):
    if "q_out" not in s:
        s["q_out"] = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
    B.pkv_qk_norm_rope_append(s["q"], s["k"], s["v"], s["pos"], s["table"], s["slots"],
                              s["k_cache"], s["v_cache"], s["q_out"], q_weight=s["qw"],
                              k_weight=s["kw"], eps=1e-6, pair_axis=s["pair_axis"],
                              interleaved=s["case"]["inter"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_score(s, B):
    B.pkv_block_bounds(s["k_cache"], s["tables"], s["lens"], s["bounds"])
    B.pkv_block_scores(s["q"], s["bounds"], s["k_cache"], s["tables"], s["lens"], s["scores"])
    return {"bounds": s["bounds"], "scores": s["scores"]}


def _own_sparse(s, B):
    c = s["case"]
    if "ws" not in s:
        s["lists"] = torch.empty((c["batch"], c["hkv"], c["budget"]), dtype=torch.int32,
                                 device="cuda")
        s["list_lens"] = torch.empty(c["batch"], dtype=torch.int32, device="cuda")
        s["out"] = torch.empty_like(s["q"])
        s["ws"] = torch.empty(B.pkv_sparse_decode_workspace_size(c["batch"], c["hq"], s["k_cache"]),
                              dtype=torch.uint8, device="cuda")
    B.pkv_block_select(s["scores"], s["lens"], c["first"], c["last"], s["lists"], s["list_lens"])
    B.pkv_sparse_decode_attn(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["lists"],
                             s["list_lens"], s["scale"], s["out"], s["ws"], s["k_scales"],
                             s["v_scales"])
    return {"lists": s["lists"], "list_lens": s["list_lens"], "out": s["out"]}


def _own_mass(s, B):
    c = s["case"]
    if "ws" not in s:
        s["out"] = torch.empty_like(s["q"])
        s["ws"] = torch.empty(B.pkv_decode_mass_workspace_size(c["batch"], c["hq"],
                                                               s["tables"].shape[1], s["k_cache"]),
                              dtype=torch.uint8, device="cuda")
    B.pkv_decode_attn_mass(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["scale"],
                           s["out"], s["mass"], s["mass_out"], s["ws"], s["k_scales"],
                           s["v_scales"])
    return {"out": s["out"], "mass": s["mass_out"]}


def _own_evict(s, B):
    c = s["case"]
    B.pkv_evict_tokens(s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["mass"], c["first"],
                       c["last"], s["new_tables"], s["new_lens"], s["new_mass"], s["kept"])
    return {"kept": s["kept"], "lens": s["new_lens"], "mass": s["new_mass"],
            "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


PLAIN = {"rope": _rope, "score": _score, "sparse": _sparse, "mass": _mass, "evict": _evict}
OWN = {"rope": _own_rope, "score": _own_score, "sparse": _own_sparse, "mass": _own_mass,
       "evict": _own_evict}


def run(state):
    if own:
        from paged_kv_decode_05_gb300 import binding
        return OWN[state["case"]["op"]](state, binding)
    return PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- 64 bits ---
def _exact_rope(s):
    c = s["case"]
    n, half = c["tokens"], c["rot"] // 2

    def turn(x, w):
        x = x.double()
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / c["d"] + 1e-6).sqrt() * w.double()
        y = x.clone()
        for j in range(half):
            i0, i1 = (2 * j, 2 * j + 1) if c["inter"] else (j, j + half)
            t = s["table"][s["pos"][s["pair_axis"][j]].long()].double()
            z = torch.complex(x[..., i0], x[..., i1])
            z = z * torch.complex(t[:, j], t[:, j + half])[:, None]
            y[..., i0], y[..., i1] = z.real, z.imag
        return y

    caches = []
    for new in (turn(s["k"], s["kw"]), s["v"].double()):
        flat = torch.zeros((s["k_cache"].shape[0] * BS, c["hkv"], c["d"]), dtype=torch.float64,
                           device="cuda")
        flat[s["slots"]] = new
        caches.append(flat.view(-1, BS, c["hkv"], c["d"]).transpose(1, 2).contiguous())
    assert n == s["q"].shape[0]
    return {"q": turn(s["q"], s["qw"]), "k_cache": caches[0], "v_cache": caches[1]}


def _sequence(s, name, b, h, length):
    """The first `length` rows of sequence b, head h, in 64 bits."""
    blk = s["tables"][b, :-(-length // BS)].long()
    x = s[name + "_cache"][blk, h].double()
    if s[name + "_scales"] is not None:
        x = x * s[name + "_scales"][blk, h].double()[:, None, None]
    return x.reshape(-1, x.shape[-1])[:length]


def _exact_score(s):
    c, mb = s["case"], s["tables"].shape[1]
    bounds = s["bounds"].clone()
    scores = torch.full((c["batch"], c["hkv"], mb), -math.inf, dtype=torch.float64, device="cuda")
    for b, length in enumerate(s["lens"].tolist()):
        n = -(-length // BS)
        blk = s["tables"][b, :n].long()
        rows = s["k_cache"][blk[-1], :, :length - (n - 1) * BS]
        bounds[blk[-1], :, 0], bounds[blk[-1], :, 1] = rows.min(1).values, rows.max(1).values
        box = bounds[blk].double()                                # [n, hkv, 2, d]
        q = s["q"][b].double().view(c["hkv"], -1, c["d"])
        for g in range(q.shape[1]):
            per = torch.maximum(box[:, :, 0] * q[:, g], box[:, :, 1] * q[:, g]).sum(-1)
            scores[b, :, :n] = torch.maximum(scores[b, :, :n], per.t())
    return {"bounds": bounds, "scores": scores}


def _exact_choice(row, n, first, last, budget):
    """The chosen of row[:n], ascending, from (value, index) pairs in numpy's stable order."""
    import numpy as np
    x = row[:n].double().cpu().numpy()
    keep = np.zeros(n, bool)
    keep[:first] = True
    keep[max(0, n - last):] = True
    rest = np.flatnonzero(~keep)
    room = max(0, min(n, budget) - int(keep.sum()))
    keep[rest[np.argsort(-x[rest], kind="stable")[:room]]] = True
    return torch.from_numpy(np.flatnonzero(keep)[:budget])


def _exact_attention(q, k, v, scale):
    e = (k @ q.double().t()) * scale                              # [tokens, heads]
    w = torch.softmax(e, 0)
    return w.t() @ v, w.sum(1)


def _exact_sparse(s):
    c = s["case"]
    lists = torch.full((c["batch"], c["hkv"], c["budget"]), -1, dtype=torch.int32)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lens, g, scores = s["lens"].tolist(), c["hq"] // c["hkv"], s["scores"].cpu()
    for b, length in enumerate(lens):
        for h in range(c["hkv"]):
            pick = _exact_choice(scores[b, h], -(-length // BS), c["first"], c["last"], c["budget"])
            lists[b, h, :len(pick)] = pick.int()
            at = (pick[:, None] * BS + torch.arange(BS)).flatten().cuda()
            at = at[at < length]
            k, v = (_sequence(s, n, b, h, length)[at] for n in ("k", "v"))
            hs = slice(h * g, h * g + g)
            out[b, hs] = _exact_attention(s["q"][b, hs], k, v, s["scale"])[0]
    counts = torch.tensor([min(c["budget"], -(-n // BS)) for n in lens], dtype=torch.int32)
    return {"lists": lists, "list_lens": counts, "out": out}


def _exact_mass(s):
    c = s["case"]
    g = c["hq"] // c["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    mass = s["mass_out"].double()
    for b, length in enumerate(s["lens"].tolist()):
        for h in range(c["hkv"]):
            k, v = (_sequence(s, n, b, h, length) for n in ("k", "v"))
            hs = slice(h * g, h * g + g)
            out[b, hs], w = _exact_attention(s["q"][b, hs], k, v, s["scale"])
            mass[b, h, :length] = s["mass"][b, h, :length].double() + w
    return {"out": out, "mass": mass}


def _exact_evict(s):
    c = s["case"]
    shape = (c["batch"], c["hkv"], c["budget"])
    kept = torch.full(shape, -1, dtype=torch.int32)
    new_mass = torch.zeros(s["new_mass"].shape, dtype=torch.float64)
    caches = {n: s[n].clone() for n in ("k_cache", "v_cache")}
    mass, lens = s["mass"].cpu(), s["lens"].tolist()
    tables, new_tables = s["tables"].cpu().long(), s["new_tables"].cpu().long()
    for b, length in enumerate(lens):
        for h in range(c["hkv"]):
            pick = _exact_choice(mass[b, h], length, c["first"], c["last"], c["budget"])
            n = len(pick)
            kept[b, h, :n] = pick.int()
            new_mass[b, h, :n] = mass[b, h, pick].double()
            to = torch.arange(n)
            src, dst = tables[b, pick // BS].cuda(), new_tables[b, to // BS].cuda()
            for name, cache in caches.items():
                cache[dst, h, (to % BS).cuda()] = s[name][src, h, (pick % BS).cuda()]
    return {"kept": kept, "mass": new_mass,
            "lens": torch.tensor([min(c["budget"], n) for n in lens], dtype=torch.int32), **caches}


EXACT = {"rope": _exact_rope, "score": _exact_score, "sparse": _exact_sparse, "mass": _exact_mass,
         "evict": _exact_evict}


def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))
