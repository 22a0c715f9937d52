"""Workloads of windowed attention and of the 4-bit cache, in plain torch and through the library.

Four operators of layers with a sliding window, and of caches held in 4 bits:

* ``decode``  one query token per sequence attends to the last ``window`` tokens and to the first
              ``sinks`` (window 0: to all), over 16-bit, INT8 and 4-bit caches;
* ``multi``   the same for runs of queries: prompt chunks and speculative verification;
* ``write``   new K and V rows quantised into a 4-bit cache, and the blocks they went to read back;
* ``read``    blocks of a 4-bit cache read back into a 16-bit one.

``run`` computes them with elementary torch operations, or, where ``own`` is true, through the
library. Caches are ``[num_blocks, num_kv_heads, 16, head_dim]``; 4-bit ones hold two codes per byte
(the even channel low) and, per row, a scale and a lowest value of the model's type.
"""

import math

import torch

own = False

BS = 16
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases ---
def listed():
    return [
        # one sequence's token in a window layer: latency
        dict(name="decode_one", op="decode", batch=1, hq=32, hkv=8, d=128, kv="bf16", q="bf16",
             lo=1000, hi=1000, window=512, sinks=4),
        # a long-context batch through a window layer
        dict(name="decode_window", op="decode", batch=64, hq=32, hkv=8, d=128, kv="bf16", q="bf16",
             lo=8192, hi=32768, window=4096, sinks=4),
        # groups of 8 heads over an INT8 cache, window and sinks that end inside blocks
        dict(name="decode_window_int8", op="decode", batch=48, hq=64, hkv=8, d=128, kv="i8",
             q="f16", lo=500, hi=12000, window=2000, sinks=5),
        # the benchmark's batch with its cache in 4 bits, full attention
        dict(name="decode_u4", op="decode", batch=256, hq=32, hkv=8, d=128, kv="u4", q="bf16",
             lo=128, hi=4096, window=0, sinks=0),
        # a handful of sequences over a 4-bit cache, odd lengths, head_dim 64
        dict(name="decode_u4_few", op="decode", batch=3, hq=16, hkv=8, d=64, kv="u4", q="f16",
             lo=333, hi=3001, window=0, sinks=0),
        # speculative verification: four drafts and one more token each
        dict(name="multi_verify", op="multi", batch=64, hq=32, hkv=8, d=128, kv="bf16", q="bf16",
             qlo=5, qhi=5, lo=1000, hi=16000, window=4096, sinks=0),
        # prompt chunks of 512 tokens
        dict(name="multi_chunk", op="multi", batch=8, hq=32, hkv=8, d=128, kv="bf16", q="bf16",
             qlo=512, qhi=512, lo=2048, hi=8192, window=2048, sinks=4),
        # ragged runs over an INT8 cache
        dict(name="multi_ragged_int8", op="multi", batch=6, hq=16, hkv=8, d=128, kv="i8", q="bf16",
             qlo=3, qhi=301, lo=301, hi=5000, window=1000, sinks=20),
        # a decode step's rows
        dict(name="write_step", op="write", tokens=256, each=1, hkv=8, d=128, q="bf16"),
        # a long prompt's rows, an odd count
        dict(name="write_chunk", op="write", tokens=8191, each=8191, hkv=8, d=128, q="bf16"),
        # a short prefix
        dict(name="read_few", op="read", blocks=3, hkv=8, d=64, q="f16"),
        # the prefixes of a batch, for its next prompt chunks
        dict(name="read_prefix", op="read", blocks=8192, hkv=8, d=128, q="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "multi", "multi", "write", "read"])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128])
    q = rng.choice(["bf16", "f16"])
    if op == "write":
        tokens = _log(rng, 1, 8191 * 8 // hkv)
        each = rng.choice([1, tokens, _log(rng, 1, tokens)])
        return dict(op=op, tokens=tokens, each=each, hkv=hkv, d=d, q=q)
    if op == "read":
        return dict(op=op, blocks=_log(rng, 1, 8192), hkv=hkv, d=d, q=q)
    sinks = rng.choice([0, rng.randint(1, 8), rng.randint(9, 80)])
    if op == "decode":
        batch = _log(rng, 1, 200)
        kv = rng.choice([q, "i8", "u4"])
        hi = _log(rng, 30, min(32768, (540000 if kv == "u4" else 260000) // batch))
        return dict(op=op, batch=batch, hq=hkv * g, hkv=hkv, d=d, kv=kv, q=q,
                    lo=rng.randint(0, hi), hi=hi,
                    window=rng.choice([0, _log(rng, 1, hi), _log(rng, 16, 4096)]), sinks=sinks)
    qhi = _log(rng, 1, 512)
    batch = _log(rng, 1, max(1, min(64, 131072 // (qhi * hkv * g))))
    hi = _log(rng, qhi, 8192)
    return dict(op=op, batch=batch, hq=hkv * g, hkv=hkv, d=d, q=q, kv=rng.choice([q, q, "i8"]),
                qlo=rng.randint(1, qhi), qhi=qhi, lo=rng.randint(qhi, hi), hi=hi,
                window=_log(rng, 1, 2048), sinks=sinks)


def _spread(lo, hi, n, phase=0.999):
    """n sizes over [lo, hi] by the golden ratio, the same for every seed."""
    return [lo + int((hi - lo + 1) * ((i * 0.6180339887498949 + phase) % 1.0)) for i in range(n)]


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


def _int8(shape, gen):
    x = torch.empty(shape, dtype=torch.int8, device="cuda")
    flat, step = x.view(-1), 1 << 26
    for i in range(0, flat.numel(), step):
        part = flat[i:i + step]
        y = torch.randn(part.shape, generator=gen, device="cuda") * 42.0
        part.copy_(y.round_().clamp_(-127, 127))
    return x


def _u4(total, hkv, d, dtype, gen):
    """A 4-bit cache of normal rows: packed codes and (scale, lowest value) per row."""
    codes = torch.empty((total, hkv, BS, d // 2), dtype=torch.uint8, device="cuda")
    params = torch.empty((total, hkv, BS, 2), dtype=dtype, device="cuda")
    step = max(1, (1 << 25) // (hkv * BS * d))
    for i in range(0, total, step):
        x = torch.randn(codes[i:i + step].shape[:-1] + (d,), generator=gen, device="cuda")
        lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
        scale = (hi - lo) / 15.0
        c = ((x - lo) / scale).round_().clamp_(0, 15).to(torch.uint8)
        codes[i:i + step] = c[..., 0::2] | (c[..., 1::2] << 4)
        params[i:i + step, ..., 0] = scale[..., 0].to(dtype)
        params[i:i + step, ..., 1] = lo[..., 0].to(dtype)
    return codes, params


def _tables(lens, gen):
    """Block tables over a shuffled pool."""
    nb = [-(-n // BS) for n in lens]
    mb, total = max(nb) + 1, sum(nb) + 5
    perm = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    t = torch.zeros((len(lens), mb), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(nb):
        t[b, :n] = perm[at:at + n]
        at += n
    return t, total


def prepare(case, seed):
    gen = _gen(seed)
    s = dict(case=case)
    hkv, d, dt = case["hkv"], case["d"], DT[case["q"]]
    if case["op"] == "write":
        n, each = case["tokens"], case["each"]
        # k and v are parts of one projection's rows; a few channels are larger
        rows = _normal((n, 6 * hkv, d), dt, gen)
        rows *= (0.5 + 2 * torch.rand((6 * hkv, d), generator=gen, device="cuda") ** 4).to(dt)
        s["k"], s["v"] = rows[:, 4 * hkv:5 * hkv], rows[:, 5 * hkv:]
        # runs of `each` tokens, every run from the start of a block of its own
        per = -(-each // BS)
        runs = -(-n // each)
        perm = torch.randperm(runs * per + 3, generator=gen, device="cuda")
        at = torch.arange(n, device="cuda")
        run, off = at // each, at % each
        s["slots"] = perm[run * per + off // BS] * BS + off % BS
        total = runs * per + 3
        s["k_codes"], s["v_codes"] = (torch.zeros((total, hkv, BS, d // 2), dtype=torch.uint8,
                                                  device="cuda") for _ in range(2))
        s["k_params"], s["v_params"] = (torch.zeros((total, hkv, BS, 2), dtype=dt, device="cuda")
                                        for _ in range(2))
        s["src"] = torch.unique(s["slots"] // BS).to(torch.int32)
        nb = s["src"].numel()
    elif case["op"] == "read":
        nb = case["blocks"]
        total = nb + nb // 4 + 1
        s["k_codes"], s["k_params"] = _u4(total, hkv, d, dt, gen)
        s["v_codes"], s["v_params"] = _u4(total, hkv, d, dt, gen)
        s["src"] = torch.randperm(total, generator=gen, device="cuda")[:nb].to(torch.int32)
    if case["op"] in ("write", "read"):
        s["dst"] = torch.randperm(nb, generator=gen, device="cuda").to(torch.int32)
        s["k_out"], s["v_out"] = (torch.zeros((nb, hkv, BS, d), dtype=dt, device="cuda")
                                  for _ in range(2))
        return s
    lens = _spread(case["lo"], case["hi"], case["batch"])
    s["host_lens"] = lens
    s["tables"], total = _tables(lens, gen)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["scale"] = d ** -0.5
    rows = case["batch"]
    if case["op"] == "multi":
        s["host_n"] = _spread(case["qlo"], case["qhi"], case["batch"], 0.3)
        cu = [0]
        for n in s["host_n"]:
            cu.append(cu[-1] + n)
        s["cu_q"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        rows = cu[-1]
    s["q"] = _normal((rows, case["hq"], d), dt, gen)
    shape = (total, hkv, BS, d)
    s["k_scales"] = s["v_scales"] = None
    if case["kv"] == "u4":
        s["k_cache"], s["k_scales"] = _u4(total, hkv, d, dt, gen)
        s["v_cache"], s["v_scales"] = _u4(total, hkv, d, dt, gen)
    elif case["kv"] == "i8":
        s["k_cache"], s["v_cache"] = _int8(shape, gen), _int8(shape, gen)
        s["k_scales"], s["v_scales"] = (torch.rand(shape[:2], generator=gen, device="cuda") * 0.02
                                        + 0.01 for _ in range(2))
    else:
        # keys: channels of different size, as a trained projection gives
        s["k_cache"], s["v_cache"] = _normal(shape, dt, gen), _normal(shape, dt, gen)
        s["k_cache"] *= (0.5 + torch.rand((hkv, 1, d), generator=gen, device="cuda")).to(dt)
    return s


# --------------------------------------------------------------- the work ---
def _visible(p, window, sinks):
    """How many tokens the query at position p sees."""
    if window == 0 or p + 1 <= window:
        return p + 1
    return window + min(sinks, p + 1 - window)


def work(case):
    hkv, d = case["hkv"], case["d"]
    if case["op"] == "write":
        n, each = case["tokens"], case["each"]
        blocks = sum(-(-min(each, n - i) // BS) for i in range(0, n, each))
        return {"bytes": n * (hkv * 2 * (2 * d + d // 2 + 4) + 8)
                + blocks * BS * hkv * 2 * (d // 2 + 4 + 2 * d), "flops": n * hkv * 2 * d * 5}
    if case["op"] == "read":
        return {"bytes": case["blocks"] * BS * hkv * 2 * (d // 2 + 4 + 2 * d),
                "flops": case["blocks"] * BS * hkv * 2 * d * 2}
    row = {"i8": d, "u4": d // 2 + 4}.get(case["kv"], 2 * d)
    lens = _spread(case["lo"], case["hi"], case["batch"])
    w, sinks = case["window"], case["sinks"]
    if case["op"] == "decode":
        ns = [min(n, 1) for n in lens]
    else:
        ns = _spread(case["qlo"], case["qhi"], case["batch"], 0.3)
    tokens = pairs = 0
    for n, length in zip(ns, lens):
        if length:
            # what the run's queries see together, and one by one
            tokens += min(length, _visible(length - 1, w, sinks) + n - 1)
            pairs += sum(_visible(p, w, sinks) for p in range(length - n, length))
    rows = case["batch"] if case["op"] == "decode" else sum(ns)
    return {"bytes": tokens * hkv * 2 * row + 2 * rows * case["hq"] * d * 2,
            "flops": pairs * case["hq"] * 4 * d}


# ------------------------------------------------------------- plain form ---
def _unpack(codes, params):
    """Values of 4-bit rows, fp32: codes [..., d / 2], params [..., 2]."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    return c * params[..., :1].float() + params[..., 1:].float()


def _rows(s, name, blk, row):
    """Rows `row` of blocks `blk` (broadcast [..., 1]) of all heads, fp32 [..., hkv, d]."""
    c = s["case"]
    h = torch.arange(c["hkv"], device="cuda")
    x, scales = s[name + "_cache"][blk, h, row], s[name + "_scales"]
    if c["kv"] == "u4":
        return _unpack(x, scales[blk, h, row])
    return x.float() if scales is None else x.float() * scales[blk, h][..., None]


def _softmax(x, live):
    """Weights over the last axis, 0 where not live (everywhere, for an empty row)."""
    x = torch.where(live, x, torch.full_like(x, -math.inf))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    return p / torch.where(l == 0, torch.ones_like(l), l)


def _decode(s):
    c = s["case"]
    lens = s["lens"].long()[:, None]
    first = (lens - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(lens)
    # the sinks before the window, then the window
    lead = torch.minimum(first, torch.full_like(first, c["sinks"]))
    width = max(1, max(s["host_lens"]))
    if c["window"]:
        width = min(width, c["window"] + c["sinks"])
    j = torch.arange(width, device="cuda")[None]
    at = torch.where(j < lead, j, j - lead + first)             # [B, width]
    live = at < lens
    at = torch.where(live, at, torch.zeros_like(at))
    blk = torch.gather(s["tables"].long(), 1, at // BS)[..., None]
    row = (at % BS)[..., None]
    q = s["q"].float().view(c["batch"], c["hkv"], -1, c["d"])
    k = _rows(s, "k", blk, row).permute(0, 2, 3, 1)             # [B, hkv, d, width]
    p = _softmax(torch.matmul(q, k) * s["scale"], live[:, None, None])
    del k
    v = _rows(s, "v", blk, row).transpose(1, 2)
    return torch.matmul(p, v).reshape(s["q"].shape).to(s["q"].dtype)


def _multi(s):
    c = s["case"]
    out = torch.empty_like(s["q"])
    at = 0
    for b, (n, length) in enumerate(zip(s["host_n"], s["host_lens"])):
        lo = max(0, length - n - c["window"] + 1)
        t = torch.cat([torch.arange(min(c["sinks"], lo), device="cuda"),
                       torch.arange(lo, length, device="cuda")])
        blk, row = s["tables"][b, t // BS].long()[:, None], (t % BS)[:, None]
        p = torch.arange(length - n, length, device="cuda")[:, None]
        live = (t <= p) & ((t > p - c["window"]) | (t < c["sinks"]))    # [n, tokens]
        q = s["q"][at:at + n].float().view(n, c["hkv"], -1, c["d"]).permute(1, 2, 0, 3)
        k = _rows(s, "k", blk, row).permute(1, 2, 0)[:, None]           # [hkv, 1, d, tokens]
        w = _softmax(torch.matmul(q, k) * s["scale"], live)
        v = _rows(s, "v", blk, row).transpose(0, 1)[:, None]
        o = torch.matmul(w, v)                                          # [hkv, g, n, d]
        out[at:at + n] = o.permute(2, 0, 1, 3).reshape(n, c["hq"], c["d"]).to(out.dtype)
        at += n
    return out


def _quantise(x):
    """16-bit rows [..., d] -> packed codes, (scale, lowest value) of the rows' type. The scale is
    rounded up, so that no code passes 15; codes are decided in 64 bits, next to a border too."""
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    want = (hi.float() - lo.float()) / torch.full_like(lo, 15.0, dtype=torch.float32)
    scale = want.to(x.dtype)
    scale = torch.where(scale.float() < want, (scale.view(torch.int16) + 1).view(x.dtype), scale)
    dist = (x.float() - lo.float()).double()
    step = torch.where(scale == 0, torch.ones_like(scale), scale).double()
    c = torch.round(dist / step).to(torch.uint8)
    c = torch.where(scale == 0, torch.zeros_like(c), c)
    return c[..., 0::2] | (c[..., 1::2] << 4), torch.cat([scale, lo], -1)


def _read(s):
    src, dst = s["src"].long(), s["dst"].long()
    for name in ("k", "v"):
        x = _unpack(s[name + "_codes"][src], s[name + "_params"][src])
        s[name + "_out"][dst] = x.to(s[name + "_out"].dtype)
    return {"k": s["k_out"], "v": s["v_out"]}


def _write(s):
    blk, row = s["slots"] // BS, s["slots"] % BS
    for name in ("k", "v"):
        codes, params = _quantise(s[name])
        s[name + "_codes"][blk, :, row] = codes
        s[name + "_params"][blk, :, row] = params
    return {**_read(s), "k_params": s["k_params"], "v_params": s["v_params"]}


# ------------------------------------------------------------ the library ---
def _own_decode(s, B):
    c = s["case"]
    if "ws" not in s:
        s["out"] = torch.empty_like(s["q"])
        s["ws"] = torch.empty(B.pkv_window_decode_workspace_size(c["batch"], c["hq"], s["k_cache"]),
                              dtype=torch.uint8, device="cuda")
    B.pkv_window_decode_attn(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["scale"],
                             c["window"], c["sinks"], s["out"], s["ws"], s["k_scales"],
                             s["v_scales"])
    return s["out"]


def _own_multi(s, B):
    c = s["case"]
    if "ws" not in s:
        s["out"] = torch.empty_like(s["q"])
        s["ws"] = torch.empty(B.pkv_window_multiquery_workspace_size(c["batch"], c["hq"],
                                                                     c["qhi"], s["k_cache"]),
                              dtype=torch.uint8, device="cuda")
    B.pkv_window_multiquery_attn(s["q"], s["cu_q"], c["qhi"], s["k_cache"], s["v_cache"],
                                 s["tables"], s["lens"], s["scale"], c["window"], c["sinks"],
                                 s["out"], s["ws"], s["k_scales"], s["v_scales"])
    return s["out"]


def _own_read(s, B):
    B.pkv_u4_read_blocks(s["k_codes"], s["v_codes"], s["k_params"], s["v_params"], s["src"],
                         s["k_out"], s["v_out"], s["dst"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _own_write(s, B):
    B.pkv_u4_append(s["k"], s["v"], s["slots"], s["k_codes"], s["v_codes"], s["k_params"],
                    s["v_params"])
    return {**_own_read(s, B), "k_params": s["k_params"], "v_params": s["v_params"]}


PLAIN = {"decode": _decode, "multi": _multi, "write": _write, "read": _read}
OWN = {"decode": _own_decode, "multi": _own_multi, "write": _own_write, "read": _own_read}


def run(state):
    if own:
        from paged_kv_decode_05_gb300 import binding
        return OWN[state["case"]["op"]](state, binding)
    return PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- 64 bits ---
def _exact_tile(codes, params):
    """One head's 4-bit rows [..., d / 2] in 64 bits."""
    out = torch.empty(codes.shape[:-1] + (2 * codes.shape[-1],), dtype=torch.float64,
                      device=codes.device)
    scale, low = params[..., 0].double(), params[..., 1].double()
    out[..., 0::2] = (codes % 16).double() * scale[..., None] + low[..., None]
    out[..., 1::2] = (codes // 16).double() * scale[..., None] + low[..., None]
    return out


def _sequence(s, name, b, length):
    """The first `length` rows of sequence b in 64 bits, [hkv, length, d]."""
    blk = s["tables"][b, :-(-length // BS)].long()
    x, scales = s[name + "_cache"][blk], s[name + "_scales"]
    if s["case"]["kv"] == "u4":
        x = _exact_tile(x, scales[blk])
    elif scales is not None:
        x = x.double() * scales[blk].double()[:, :, None, None]
    return x.double().transpose(0, 1).flatten(1, 2)[:, :length]


def _exact_decode(s):
    c = s["case"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, length in enumerate(s["host_lens"]):
        if length == 0:
            continue
        keep = [t for t in range(length)
                if c["window"] == 0 or t >= length - c["window"] or t < c["sinks"]]
        keep = torch.tensor(keep, device="cuda")
        k, v = (_sequence(s, n, b, length)[:, keep] for n in ("k", "v"))
        q = s["q"][b].double().view(c["hkv"], -1, c["d"])
        w = torch.softmax(torch.einsum("hgd,htd->hgt", q, k) * s["scale"], -1)
        out[b] = torch.einsum("hgt,htd->hgd", w, v).reshape(c["hq"], c["d"])
    return out


def _exact_multi(s):
    c = s["case"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    g, at = c["hq"] // c["hkv"], 0
    for b, (n, length) in enumerate(zip(s["host_n"], s["host_lens"])):
        k, v = (_sequence(s, name, b, length) for name in ("k", "v"))
        # in runs of queries, each over the tokens that its first one's window begins with
        for i0 in range(0, n, 128):
            i1 = min(n, i0 + 128)
            low = max(0, length - n + i0 - c["window"] + 1)
            keep = [t for t in range(length - n + i1) if t >= low or t < c["sinks"]]
            keep = torch.tensor(keep, device="cuda")
            pos = torch.arange(length - n + i0, length - n + i1, device="cuda")
            gap = pos[:, None] - keep[None]
            hidden = (gap < 0) | ((gap >= c["window"]) & (keep[None] >= c["sinks"]))
            for h in range(c["hq"]):
                e = s["q"][at + i0:at + i1, h].double() @ k[h // g, keep].t() * s["scale"]
                w = torch.softmax(e.masked_fill(hidden, -math.inf), -1)
                out[at + i0:at + i1, h] = w @ v[h // g, keep]
        at += n
    return out


def _exact_read(s):
    outs = {}
    for name in ("k", "v"):
        x = torch.zeros(s["k_out"].shape, dtype=torch.float64, device="cuda")
        for src, dst in zip(s["src"].split(256), s["dst"].split(256)):
            x[dst.long()] = _exact_tile(s[name + "_codes"][src.long()],
                                        s[name + "_params"][src.long()])
        outs[name] = x
    return outs


def _round_up(x, dtype):
    """The smallest value of a 16-bit type that is not below x >= 0 (fp32 numpy)."""
    import numpy as np
    drop, lowest = (16, 0) if dtype == torch.bfloat16 else (13, -24)
    if dtype == torch.bfloat16:
        bits = x.view(np.uint32).astype(np.uint64)
        up = ((bits + (1 << drop) - 1) >> drop << drop).astype(np.uint32)
        return up.view(np.float32).astype(np.float64)
    m, e = np.frexp(x.astype(np.float64))
    ulp = np.ldexp(1.0, np.maximum(e - 11, lowest))
    return np.where(x == 0, 0.0, np.ceil(x.astype(np.float64) / ulp) * ulp)


def _exact_write(s):
    """Rows quantised and put back to values in numpy, the divisions in 64 bits."""
    import numpy as np
    outs = {}
    slots = s["slots"].cpu().numpy()
    place = np.full(s["k_codes"].shape[0], -1)
    place[s["src"].cpu().numpy()] = s["dst"].cpu().numpy()
    for name in ("k", "v"):
        x = s[name].float().cpu().numpy()
        low, high = x.min(-1), x.max(-1)
        scale = _round_up((high - low) / np.float32(15), s[name].dtype)
        dist = (x - low[..., None]).astype(np.float64)
        step = np.where(scale == 0, 1.0, scale)[..., None]
        code = np.where(scale[..., None] == 0, 0.0, np.rint(dist / step))
        values = code * scale[..., None] + low[..., None].astype(np.float64)
        out = np.zeros(s["k_out"].shape)
        out[place[slots // BS], :, slots % BS] = values
        params = np.zeros(s["k_params"].shape)
        params[slots // BS, :, slots % BS, 0] = scale
        params[slots // BS, :, slots % BS, 1] = low
        outs[name], outs[name + "_params"] = torch.from_numpy(out), torch.from_numpy(params)
    return {n: outs[n] for n in ("k", "v", "k_params", "v_params")}


EXACT = {"decode": _exact_decode, "multi": _exact_multi, "write": _exact_write,
         "read": _exact_read}


def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))
