"""A cache held in 8 or 4 bits, and beam search over a paged cache, as measured cases.

Five operators: ``pkv_quant_write`` (new tokens' keys and values quantised as
they are written), ``pkv_quant_read`` (rows of such a cache as numbers again),
``pkv_quant_decode_attention`` (one new token per sequence over such a cache),
``pkv_beam_select`` (the best continuations over beams and vocabulary) and
``pkv_beam_reorder`` (block tables that follow the chosen beams, last blocks
copied where two beams share one).

``run`` computes each in elementary torch operations, or, with ``own`` set,
through the library.  Lengths are spread evenly over their range and dealt
out by the seed, so a case's work does not depend on the seed.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
ELEM = {"fp32": 4, "bf16": 2, "fp16": 2}
TOP = {"int8": 127.0, "e4m3": 448.0, "int4": 15.0}          # a row's largest code
TINY = 2.0 ** -100                                          # rows smaller than that are zeros


def listed():
    return [
        # one new token of one request: the write's latency
        {"name": "write_one_token", "op": "write", "fmt": "int8", "dtype": "bf16", "T": 1, "pads": 0, "KVH": 8,
         "D": 128, "bs": 16},
        # a long prompt's keys and values, with padding tokens
        {"name": "write_prompt", "op": "write", "fmt": "e4m3", "dtype": "bf16", "T": 16384, "pads": 100, "KVH": 8,
         "D": 128, "bs": 16},
        # cached contexts read back for a chunk of new queries
        {"name": "read_context", "op": "read", "fmt": "int8", "dtype": "bf16", "T": 32768, "pads": 0, "KVH": 8,
         "D": 128, "bs": 16},
        # an odd count, 4 bits, wide head, one KV head
        {"name": "read_odd_4bit", "op": "read", "fmt": "int4", "dtype": "fp16", "T": 5001, "pads": 17, "KVH": 1,
         "D": 256, "bs": 32},
        # one request with a short context: the decode's latency
        {"name": "decode_one", "op": "decode", "fmt": "int8", "dtype": "bf16", "B": 1, "H": 32, "KVH": 8, "D": 128,
         "bs": 16, "n_lo": 300, "n_hi": 300, "softcap": 0.0, "window": 0},
        # the 8B-shaped batch
        {"name": "decode_batch", "op": "decode", "fmt": "int8", "dtype": "bf16", "B": 64, "H": 32, "KVH": 8, "D": 128,
         "bs": 16, "n_lo": 512, "n_hi": 4096, "softcap": 0.0, "window": 0},
        # few long contexts, capped scores
        {"name": "decode_long_capped", "op": "decode", "fmt": "e4m3", "dtype": "bf16", "B": 8, "H": 32, "KVH": 8,
         "D": 128, "bs": 16, "n_lo": 16384, "n_hi": 32768, "softcap": 50.0, "window": 0},
        # one KV head, wide head, 4 bits, log-spread lengths
        {"name": "decode_mqa_4bit", "op": "decode", "fmt": "int4", "dtype": "fp16", "B": 128, "H": 16, "KVH": 1,
         "D": 256, "bs": 32, "n_lo": 1, "n_hi": 8192, "softcap": 0.0, "window": 0},
        # one request's beams
        {"name": "select_one", "op": "select", "dtype": "fp32", "B": 1, "W": 4, "K": 4, "V": 32000, "ended": 1},
        # a batch of wide beams over a large vocabulary
        {"name": "select_batch", "op": "select", "dtype": "bf16", "B": 64, "W": 8, "K": 8, "V": 128256, "ended": 60},
        # one request's beams, one layer
        {"name": "reorder_one", "op": "reorder", "dtype": "bf16", "fmt": "none", "layers": 1, "B": 1, "W": 4, "K": 4,
         "KVH": 8, "D": 128, "bs": 16, "prompt_lo": 200, "prompt_hi": 200, "made": 21},
        # a batch of beams over a quantised cache's layers
        {"name": "reorder_batch", "op": "reorder", "dtype": "bf16", "fmt": "int8", "layers": 16, "B": 32, "W": 8,
         "K": 8, "KVH": 8, "D": 128, "bs": 16, "prompt_lo": 100, "prompt_hi": 1000, "made": 57},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _head_dim(rng, fmt):
    return rng.choice([64, 96, 128, 128, 256] if fmt == "int4" else [64, 80, 96, 128, 128, 192, 256])


def _draw_rows(rng, op):
    fmt = rng.choice(["int8", "e4m3", "int4"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    D, KVH = _head_dim(rng, fmt), rng.choice([1, 2, 4, 8])
    T = _log_int(rng, 1, min(32768, (1 << 25) // (KVH * D)))
    return {"op": op, "fmt": fmt, "dtype": dtype, "T": T, "pads": rng.randint(0, T // 4), "KVH": KVH, "D": D,
            "bs": rng.choice([1, 16, 24, 32])}


def _draw_decode(rng):
    fmt = rng.choice(["int8", "e4m3", "int4"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    KVH = rng.choice([1, 2, 4, 8])
    n_hi = _log_int(rng, 16, 32768)
    return {"op": "decode", "fmt": fmt, "dtype": dtype, "B": _log_int(rng, 1, 128),
            "H": KVH * rng.choice([1, 2, 4, 4, 6, 8, 16]), "KVH": KVH, "D": _head_dim(rng, fmt),
            "bs": rng.choice([1, 16, 16, 24, 32, 64]), "n_lo": rng.randint(0, n_hi), "n_hi": n_hi,
            "softcap": rng.choice([0.0, 0.0, 30.0, 50.0]), "window": rng.choice([0, 0, _log_int(rng, 1, 4096)])}


def _draw_select(rng):
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    V = _log_int(rng, 500, 131072)
    W = rng.choice([1, 2, 4, 4, 8, 16])
    B = _log_int(rng, 1, max(1, min(256, (1 << 25) // (V * W))))
    return {"op": "select", "dtype": dtype, "B": B, "W": W, "K": rng.choice([2, 4, 8, 16]), "V": V,
            "ended": rng.randint(0, B * (W - 1) // 4)}


def _draw_reorder(rng):
    fmt = rng.choice(["none", "int8", "e4m3", "int4"])
    K = rng.choice([2, 4, 8, 16])
    return {"op": "reorder", "dtype": rng.choice(["bf16", "fp16", "fp32"]), "fmt": fmt, "layers": rng.randint(1, 16),
            "B": _log_int(rng, 1, 32), "W": rng.choice([1, K, K]), "K": K, "KVH": rng.choice([1, 2, 4, 8]),
            "D": _head_dim(rng, fmt), "bs": rng.choice([16, 16, 24, 32, 64]), "prompt_lo": rng.randint(1, 100),
            "prompt_hi": rng.randint(100, 1000), "made": rng.randint(0, 70)}


def draw(rng):
    op = rng.choice(["write", "read", "decode", "decode", "decode", "select", "select", "reorder"])
    if op in ("write", "read"):
        return _draw_rows(rng, op)
    big = next(work(c) for c in listed() if c["name"] == "decode_batch")
    while True:
        c = {"decode": _draw_decode, "select": _draw_select, "reorder": _draw_reorder}[op](rng)
        w = work(c)
        if op == "reorder":
            if _pool_bytes(c) <= 3 << 30:
                return c
        elif op == "select":
            return c
        elif (w["bytes"] <= big["bytes"] and w["flops"] <= 2 * big["flops"] and c["B"] * c["n_hi"] * c["H"] <= 1 << 26
              and c["B"] * c["n_hi"] * c["KVH"] * c["D"] <= 1 << 29):
            return c


# ------------------------------------------------------------------- lengths

def _spread(lo, hi, count):
    """`count` whole numbers from lo to hi, evenly spaced (over their logarithm
    where the range spans more than a factor of ten), both ends included."""
    if count == 1:
        return [hi]
    if lo >= 1 and hi > 10 * lo:
        return [min(hi, max(lo, round(math.exp(math.log(lo) + i / (count - 1) * math.log(hi / lo))))) for i in range(count)]
    return [lo + (i * (hi - lo)) // (count - 1) for i in range(count)]


def _ceil(a, b):
    return -(-a // b)


def _pool_blocks(case):
    """(blocks of every prompt, columns of a table) of a reorder case."""
    bs = case["bs"]
    prompts = _spread(case["prompt_lo"], case["prompt_hi"], case["B"])
    return [_ceil(p, bs) for p in prompts], _ceil(max(prompts) + case["made"] + 1, bs) + 1


def _pool_bytes(case):
    own_blocks, cols = _pool_blocks(case)
    lanes = max(case["K"], case["W"])
    blocks = sum(own_blocks) + case["B"] * lanes * (_ceil(case["made"] + 1, case["bs"]) + 3)
    return 2 * case["layers"] * blocks * case["bs"] * case["KVH"] * _row_bytes(case)


def _row_bytes(case):
    """Bytes of one token's row of one KV head in the cache, its numbers for the codes with it."""
    D, fmt = case["D"], case["fmt"]
    return D * ELEM[case["dtype"]] if fmt == "none" else D // 2 + 8 if fmt == "int4" else D + 4


# ----------------------------------------------------------------- quantised

def _quantised(x, fmt):
    """Codes and parameters of x [..., D] (float32): the plain form.

    int8, e4m3: value = scale * code.  int4: value = scale * (code - zero), two
    codes a byte, the even one low.  Products that meet a rounding border are
    taken in 64 bits."""
    if fmt == "int4":
        lo, hi = x.amin(-1).clamp(max=0.0), x.amax(-1).clamp(min=0.0)
        span = hi - lo
    else:
        span = x.abs().amax(-1)
    fine = torch.isfinite(span) & (span >= TINY)
    inv = torch.where(fine, TOP[fmt] / span, 0.0)
    scale = torch.where(fine, span / TOP[fmt], torch.where(torch.isfinite(span), 0.0, math.nan))
    x = torch.where(torch.isfinite(x), x, 0.0)
    if fmt == "e4m3":
        return (x * inv[..., None]).to(torch.float8_e4m3fn), scale
    codes = (x.double() * inv.double()[..., None]).round()
    if fmt == "int8":
        return codes.to(torch.int8), scale
    zero = torch.where(fine, (-lo.double() * inv.double()).round(), 0.0)
    codes = (codes + zero[..., None]).clamp(0, 15).to(torch.uint8)
    return codes[..., 0::2] | (codes[..., 1::2] << 4), torch.stack([scale, zero.float()], -1)


def _values(codes, params, fmt):
    """The numbers that codes [..., D] and their parameters stand for, in 32 bits."""
    if fmt != "int4":
        return codes.float() * params[..., None]
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    return (c - params[..., 1:2]) * params[..., 0:1]


def _cache(case, num_blocks, rand, dev, filled):
    """One cache's codes [num_blocks, bs, KVH, D or D / 2] and parameters
    [num_blocks, KVH, bs(, 2)], written or still zero."""
    bs, KVH, D, fmt = case["bs"], case["KVH"], case["D"], case["fmt"]
    dt = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn, "int4": torch.uint8}[fmt]
    codes = torch.zeros(num_blocks, bs, KVH, D // 2 if fmt == "int4" else D, dtype=dt, device=dev)
    params = torch.zeros((num_blocks, KVH, bs) + ((2,) if fmt == "int4" else ()), device=dev)
    if filled:
        step = max(1, (1 << 26) // (bs * KVH * D))
        channel = torch.exp(0.3 * rand(KVH, D))              # some channels are wider than others
        for at in range(0, num_blocks, step):
            x = rand(min(step, num_blocks - at), bs, KVH, D) * channel
            c, p = _quantised(x, fmt)
            codes[at:at + step], params[at:at + step] = c, p.transpose(1, 2)
    return codes, params


# ------------------------------------------------------------------- prepare

def _generators(seed, dev):
    g = torch.Generator().manual_seed(int(seed))
    dg = torch.Generator(device=dev).manual_seed(int(torch.randint(0, 2 ** 31, (1,), generator=g)))
    return g, lambda *s: torch.randn(s, generator=dg, device=dev)


def _prepare_rows(case, seed, dev):
    g, rand = _generators(seed, dev)
    T, KVH, D, bs = case["T"], case["KVH"], case["D"], case["bs"]
    dt = DTYPES[case["dtype"]]
    num_blocks = _ceil(T + T // 4, bs) + 1
    slots = torch.randperm(num_blocks * bs, generator=g)[:T]
    slots[torch.randperm(T, generator=g)[:case["pads"]]] = -1
    s = {"op": case["op"], "fmt": case["fmt"], "slots": slots.to(torch.int64).to(dev),
         "err": torch.zeros(1, dtype=torch.int32, device=dev)}
    for name in "kv":
        s[name + "_codes"], s[name + "_params"] = _cache(case, num_blocks, rand, dev, case["op"] == "read")
    if case["op"] == "write":
        # k and v lie side by side in one projection's output
        kv = (rand(T, 2 * KVH * D) * torch.exp(rand(2 * KVH * D) * 0.3)).to(dt)
        s["k"], s["v"] = kv[:, :KVH * D].view(T, KVH, D), kv[:, KVH * D:].view(T, KVH, D)
    else:
        s["k_out"], s["v_out"] = (torch.zeros(T, KVH, D, dtype=dt, device=dev) for _ in range(2))
    return s


def _prepare_decode(case, seed, dev):
    g, rand = _generators(seed, dev)
    B, H, KVH, D, bs = (case[k] for k in ("B", "H", "KVH", "D", "bs"))
    dt = DTYPES[case["dtype"]]
    ns = [_spread(case["n_lo"], case["n_hi"], B)[i] for i in torch.randperm(B, generator=g).tolist()]
    need = [_ceil(n, bs) for n in ns]
    num_blocks = sum(need) + sum(need) // 8 + 1
    perm = torch.randperm(num_blocks, generator=g).to(torch.int32)
    tables = torch.full((B, max(need) + 1), 99999, dtype=torch.int32)
    at = 0
    for b in range(B):
        tables[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
    s = {"op": "decode", "fmt": case["fmt"], "q": (rand(B, H, D) * 2.0).to(dt),
         "out": torch.empty(B, H, D, dtype=dt, device=dev), "tables": tables.to(dev),
         "lens": torch.tensor(ns, dtype=torch.int32, device=dev), "scale": 1.0 / math.sqrt(D),
         "softcap": case["softcap"], "window": case["window"], "max_n": max(ns),
         "err": torch.zeros(1, dtype=torch.int32, device=dev)}
    for name in "kv":
        s[name + "_codes"], s[name + "_params"] = _cache(case, num_blocks, rand, dev, True)
    return s


def _prepare_select(case, seed, dev):
    g, rand = _generators(seed, dev)
    B, W, K, V = (case[k] for k in ("B", "W", "K", "V"))
    # logits as a model gives them: a wide bulk and a few likely tokens a beam
    logits = rand(B, W, V) * 2.0
    likely = torch.randint(0, V, (B, W, min(V, 24)), generator=g).to(dev)
    logits.scatter_add_(2, likely, 6.0 + 2.0 * rand(*likely.shape))
    scores = -12.0 - rand(B, W).abs().cumsum(1)
    finished = torch.zeros(B * W, dtype=torch.uint8)
    live = torch.arange(B * W).view(B, W)[:, 1:].reshape(-1)     # every request's first beam goes on
    finished[live[torch.randperm(live.numel(), generator=g)[:case["ended"]]]] = 1
    empty = lambda t: torch.zeros(B, K, dtype=t, device=dev)
    return {"op": "select", "logits": logits.to(DTYPES[case["dtype"]]), "scores": scores,
            "finished": finished.view(B, W).to(dev), "end": 2, "scores_out": empty(torch.float32),
            "parents": empty(torch.int32), "tokens": empty(torch.int32), "finished_out": empty(torch.uint8),
            "err": torch.zeros(1, dtype=torch.int32, device=dev)}


def _prepare_reorder(case, seed, dev):
    g, rand = _generators(seed, dev)
    B, W, K, KVH, D, bs = (case[k] for k in ("B", "W", "K", "KVH", "D", "bs"))
    prompts = _spread(case["prompt_lo"], case["prompt_hi"], B)
    prompts = [prompts[i] for i in torch.randperm(B, generator=g).tolist()]
    need, cols = _pool_blocks(case)
    lanes = max(K, W)
    tail = _ceil(case["made"] + 1, bs) + 3
    num_blocks = sum(need) + B * lanes * tail
    perm = torch.randperm(num_blocks, generator=g).to(torch.int32)
    owned = torch.zeros(B, lanes, cols, dtype=torch.int32)
    tables = torch.zeros(B, W, cols, dtype=torch.int32)
    at = 0
    for b, p in enumerate(prompts):
        full, n = p // bs, p + case["made"]
        shared = perm[at:at + _ceil(p, bs)]
        at += _ceil(p, bs)
        # behind the prompt's full blocks every beam has a block of its own in
        # each column; the prompt's last block, if not full, is the first beam's
        mine = perm[at:at + lanes * tail].view(lanes, tail).clone()
        at += lanes * tail
        if p % bs:
            mine[0, 0] = shared[-1]
        width = min(tail, cols - full)
        owned[b, :, full:full + width] = mine[:, :width]
        owned[b, :, :full] = shared[:full]
        tables[b, :, :] = owned[b, :W]
        for c in range(full, _ceil(n, bs)):                   # beams have crossed before
            pick = torch.randperm(lanes, generator=g)[:W] if c == n // bs else torch.randint(0, lanes, (W,), generator=g)
            tables[b, :, c] = owned[b, pick, c]
    lens = torch.tensor(prompts)[:, None].expand(B, W) + case["made"]
    parents = torch.randint(0, W, (B, K), generator=g)
    parents[:, 0] = 0
    finished = (torch.rand(B, K, generator=g) < 0.1).to(torch.uint8)
    i32 = lambda x: x.to(torch.int32).contiguous().to(dev)
    s = {"op": "reorder", "tables": tables.to(dev), "lens": i32(lens), "parents": i32(parents), "bs": bs,
         "owned": owned[:, :K].contiguous().to(dev), "finished": finished.to(dev),
         "tables_out": torch.zeros(B, K, cols, dtype=torch.int32, device=dev),
         "lens_out": torch.zeros(B, K, dtype=torch.int32, device=dev),
         "slots": torch.zeros(B, K, dtype=torch.int64, device=dev),
         "err": torch.zeros(1, dtype=torch.int32, device=dev), "pools": {}, "block_pools": {}}
    for name in "kv":
        if case["fmt"] == "none":
            x = torch.empty(case["layers"], num_blocks, bs, KVH, D, dtype=DTYPES[case["dtype"]], device=dev)
            for layer in x:
                layer.copy_(rand(num_blocks, bs, KVH, D))
            s["pools"][name] = x
        else:
            both = [_cache(case, num_blocks, rand, dev, True) for _ in range(case["layers"])]
            s["pools"][name] = torch.stack([c for c, _ in both])
            s["block_pools"][name + "_params"] = torch.stack([p for _, p in both])
    return s


def prepare(case, seed):
    dev = torch.device("cuda")
    return {"write": _prepare_rows, "read": _prepare_rows, "decode": _prepare_decode, "select": _prepare_select,
            "reorder": _prepare_reorder}[case["op"]](case, seed, dev)


# --------------------------------------------------------------- plain forms

def _plain_write(s):
    keep = s["slots"] >= 0
    slots = s["slots"][keep]
    for name in "kv":
        codes, params = _quantised(s[name][keep].float(), s["fmt"])
        held, numbers = s[name + "_codes"], s[name + "_params"]
        bs = held.shape[1]
        held.view(torch.uint8).flatten(0, 1)[slots] = codes.view(torch.uint8)
        numbers.transpose(1, 2)[slots // bs, slots % bs] = params
    return {n: s[n] for n in ("k_codes", "v_codes", "k_params", "v_params")}


def _plain_read(s):
    keep = s["slots"] >= 0
    slots = s["slots"][keep]
    bs = s["k_codes"].shape[1]
    for name in "kv":
        codes = s[name + "_codes"].view(torch.uint8).flatten(0, 1)[slots].view(s[name + "_codes"].dtype)
        params = s[name + "_params"].transpose(1, 2)[slots // bs, slots % bs]
        s[name + "_out"][keep] = _values(codes, params, s["fmt"]).to(s[name + "_out"].dtype)
    return {"k_out": s["k_out"], "v_out": s["v_out"]}


def _plain_decode(s):
    B, H, D = s["q"].shape
    num_blocks, bs, KVH, _ = s["k_codes"].shape
    G, N, dev, lens = H // KVH, s["max_n"], s["q"].device, s["lens"].long()
    j = torch.arange(N, device=dev)
    blocks = s["tables"].long()[:, :_ceil(N, bs)].clamp(0, num_blocks - 1)
    real = (j < lens[:, None])[:, None, :, None]
    dense = []
    for name in "kv":                                                  # [B, KVH, N, D], every context padded to the longest
        codes = s[name + "_codes"].view(torch.uint8)[blocks].view(s[name + "_codes"].dtype).flatten(1, 2)[:, :N].permute(0, 2, 1, 3)
        params = s[name + "_params"][blocks].transpose(1, 2).flatten(2, 3)[:, :, :N]
        dense.append(torch.where(real, _values(codes, params, s["fmt"]), 0.0))
    x = (s["q"].float().view(B, KVH, G, D) @ dense[0].transpose(2, 3)) * s["scale"]
    if s["softcap"] > 0:
        x = s["softcap"] * torch.tanh(x / s["softcap"])
    seen = j < lens[:, None]
    if s["window"] > 0:
        seen = seen & (j >= lens[:, None] - s["window"])
    x = torch.where(seen[:, None, None], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    w = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    o = (w @ dense[1]) / w.sum(-1, keepdim=True)
    return torch.where(m == -math.inf, 0.0, o).view(B, H, D).to(s["q"].dtype)


def _plain_select(s):
    # which candidate comes first can hang on the last bits: scores in 64 bits
    B, W, V = s["logits"].shape
    K = s["parents"].shape[1]
    x = s["logits"].float()
    # a beam's candidates by logit, then the lowest token: the logit's bits as a
    # whole number of the same order, the token behind them
    bits = x.view(torch.int32)
    order = torch.where(bits >= 0, bits, bits ^ 0x7fffffff).long()
    v = torch.arange(V, device=x.device)
    top = ((order << 32) | (V - v)).topk(min(K, V), dim=-1).values
    token = V - (top & 0xffffffff)
    x64 = x.double()
    lse = torch.logsumexp(x64, -1, keepdim=True)
    cand = s["scores"].double()[..., None] + (x64.gather(2, token) - lse)
    # a beam that has ended has one candidate: itself
    done = s["finished"][..., None] != 0
    first = torch.arange(cand.shape[2], device=x.device) == 0
    cand = torch.where(done, torch.where(first, s["scores"].double()[..., None], -math.inf), cand)
    token = torch.where(done, s["end"], token)
    parent = torch.arange(W, device=x.device)[None, :, None].expand_as(token)
    best, at = cand.flatten(1).sort(dim=1, descending=True, stable=True)
    best, at = best[:, :K], at[:, :K]
    take = lambda t: t.flatten(1).gather(1, at)
    none = best == -math.inf
    parents, tokens = torch.where(none, -1, take(parent)), torch.where(none, -1, take(token))
    over = ~none & (take(done.expand_as(token)) | (tokens == s["end"]))
    pad = lambda t, value: torch.nn.functional.pad(t, (0, K - t.shape[1]), value=value)
    return {"scores": pad(best, -math.inf).float(), "parents": pad(parents, -1).to(torch.int32),
            "tokens": pad(tokens, -1).to(torch.int32), "finished": pad(over.to(torch.uint8), 0)}


def _plain_reorder(s):
    B, W, C = s["tables"].shape
    K, bs, dev = s["parents"].shape[1], s["bs"], s["tables"].device
    pick = s["parents"].long()
    old = s["tables"].long().gather(1, pick[..., None].expand(B, K, C))
    lens = s["lens"].long().gather(1, pick)
    owned = s["owned"].long()
    col, rest = lens // bs, lens % bs                          # where a child's next token goes
    c = torch.arange(C, device=dev)
    tables = torch.where(c < col[..., None], old, owned)
    here = lambda t, at: t.gather(2, at[:, None, :].expand(B, K, K))    # [B, row, the child whose column it is]
    block = old.gather(2, col[..., None])[..., 0]
    full = here(tables, col).masked_fill(col[:, None, :] >= col[:, :, None], -1)     # blocks that rows use there in full
    k = torch.arange(K, device=dev)
    same = (block[:, :, None] == block[:, None, :]) & (col[:, :, None] == col[:, None, :]) & (rest > 0)[:, :, None]
    keeps = (rest > 0) & ~(same & (k[:, None] < k)).any(1) & ~(full == block[:, None, :]).any(1)
    mine = here(owned, col)                                    # [B, lane, child]
    target = torch.where(keeps, block, -1)
    for i in range(K):                                         # children in order take what is left, their own lane first
        used = torch.cat([full[:, :, i], torch.where(col == col[:, i:i + 1], target, -1)], 1)
        free = ~(mine[:, :, i, None] == used[:, None, :]).any(-1)
        rank = torch.where(free, torch.where(k == i, 0, k + 1), K + 2)
        lane = rank.argmin(1)
        got = mine[:, :, i].gather(1, lane[:, None])[:, 0]
        target[:, i] = torch.where(keeps[:, i], block[:, i], got)
    tables = torch.where(c == col[..., None], target[..., None], tables)
    live = s["finished"] == 0
    slots = torch.where(live, target * bs + rest, -1)
    copy = (rest > 0) & ~keeps
    src, dst, rows = block[copy], target[copy], rest[copy]
    t = torch.arange(bs, device=dev)
    at, row = (t < rows[:, None]).nonzero(as_tuple=True)
    for pool in s["pools"].values():
        flat = pool.view(torch.uint8) if pool.element_size() == 1 else pool
        flat[:, dst[at], row] = flat[:, src[at], row]
    for pool in s["block_pools"].values():
        pool[:, dst] = pool[:, src]
    return {"tables": tables.to(torch.int32), "lens": (lens + live).to(torch.int32), "slots": slots,
            "pools": s["pools"], "block_pools": s["block_pools"]}


# ----------------------------------------------------------------------- own

def _own_write(s):
    import paged_kv_cache_67_gb300 as pkv
    if "call" not in s:  # a serving loop marshals its fixed step buffers once
        s["call"] = pkv.prepare_quant_write(s["k_codes"], s["v_codes"], s["k_params"], s["v_params"], s["k"], s["v"],
                                            s["slots"], err_flags=s["err"])
    s["call"]()
    return {n: s[n] for n in ("k_codes", "v_codes", "k_params", "v_params")}


def _own_read(s):
    import paged_kv_cache_67_gb300 as pkv
    if "call" not in s:
        s["call"] = pkv.prepare_quant_read(s["k_out"], s["v_out"], s["k_codes"], s["v_codes"], s["k_params"],
                                           s["v_params"], s["slots"], err_flags=s["err"])
    s["call"]()
    return {"k_out": s["k_out"], "v_out": s["v_out"]}


def _own_decode(s):
    import paged_kv_cache_67_gb300 as pkv
    if "call" not in s:
        B, H, D = s["q"].shape
        _, bs, KVH, _ = s["k_codes"].shape
        ws = pkv.QuantDecodeWorkspace(B, H, KVH, D, bs, s["tables"].shape[1], s["max_n"])
        s["call"] = pkv.prepare_quant_decode_attention(
            s["out"], s["q"], s["k_codes"], s["v_codes"], s["k_params"], s["v_params"], s["tables"], s["lens"],
            s["scale"], softcap=s["softcap"], window=s["window"], max_context_len=s["max_n"], workspace=ws,
            err_flags=s["err"])
    s["call"]()
    return s["out"]


def _own_select(s):
    import paged_kv_cache_67_gb300 as pkv
    if "call" not in s:
        B, W, V = s["logits"].shape
        ws = pkv.BeamSelectWorkspace(B, W, s["parents"].shape[1], V)
        s["call"] = pkv.prepare_beam_select(s["scores_out"], s["parents"], s["tokens"], s["finished_out"], s["logits"],
                                            s["scores"], s["finished"], end_token=s["end"], workspace=ws,
                                            err_flags=s["err"])
    s["call"]()
    return {"scores": s["scores_out"], "parents": s["parents"], "tokens": s["tokens"], "finished": s["finished_out"]}


def _own_reorder(s):
    import paged_kv_cache_67_gb300 as pkv
    if "call" not in s:
        layers = lambda pools: [layer for pool in pools.values() for layer in pool]
        s["call"] = pkv.prepare_beam_reorder(s["tables_out"], s["lens_out"], s["slots"], s["tables"], s["lens"],
                                             s["parents"], s["owned"], s["bs"], pools=layers(s["pools"]),
                                             block_pools=layers(s["block_pools"]), finished=s["finished"],
                                             err_flags=s["err"])
    s["call"]()
    return {"tables": s["tables_out"], "lens": s["lens_out"], "slots": s["slots"], "pools": s["pools"],
            "block_pools": s["block_pools"]}


def run(state):
    if own:
        return {"write": _own_write, "read": _own_read, "decode": _own_decode, "select": _own_select,
                "reorder": _own_reorder}[state["op"]](state)
    return {"write": _plain_write, "read": _plain_read, "decode": _plain_decode, "select": _plain_select,
            "reorder": _plain_reorder}[state["op"]](state)


# ----------------------------------------------------------------- 64 bits

def _exact_values(codes, params, fmt):
    codes, params = codes, params.double()
    if fmt != "int4":
        return codes.double() * params.unsqueeze(-1)
    x = torch.empty(codes.shape[:-1] + (2 * codes.shape[-1],), dtype=torch.float64, device=codes.device)
    x[..., 0::2], x[..., 1::2] = (codes % 16).double(), (codes // 16).double()
    return (x - params[..., 1].unsqueeze(-1)) * params[..., 0].unsqueeze(-1)


def _exact_write(s):
    out = {"k_codes": None, "v_codes": None}                   # whole numbers, and numbers of 8 bits
    at = (s["slots"] >= 0).nonzero()[:, 0]
    bs = s["k_codes"].shape[1]
    for name in "kv":
        x = s[name][at].double()
        held = s[name + "_params"].double()
        block, row = s["slots"][at] // bs, s["slots"][at] % bs
        if s["fmt"] == "int4":
            low, high = torch.minimum(x.min(-1).values, torch.zeros((), device=x.device, dtype=x.dtype)), x.max(-1).values.clamp(min=0)
            step = (high - low) / 15
            held[block, :, row] = torch.stack([step, torch.round(-low / step)], -1)
        else:
            held[block, :, row] = x.abs().max(-1).values / TOP[s["fmt"]]
        out[name + "_params"] = held
    return out


def _exact_read(s):
    bs, out = s["k_codes"].shape[1], {}
    at = (s["slots"] >= 0).nonzero()[:, 0]
    block, row = s["slots"][at] // bs, s["slots"][at] % bs
    for name in "kv":
        codes = s[name + "_codes"]
        rows = codes.view(torch.int8)[block, row].view(codes.dtype)
        o = s[name + "_out"].double()
        o[at] = _exact_values(rows, s[name + "_params"][block, :, row], s["fmt"])
        out[name + "_out"] = o
    return out


def _exact_decode(s):
    B, H, D = s["q"].shape
    _, bs, KVH, _ = s["k_codes"].shape
    G, out = H // KVH, torch.zeros(B, H, D, dtype=torch.float64, device=s["q"].device)
    for b, n in enumerate(s["lens"].tolist()):
        first = max(0, n - s["window"]) if s["window"] > 0 else 0
        if n == 0:
            continue
        blocks = s["tables"][b, :_ceil(n, bs)].long()
        k, v = (_exact_values(s[c + "_codes"].view(torch.int8)[blocks].view(s[c + "_codes"].dtype).flatten(0, 1)[first:n],
                              s[c + "_params"][blocks].transpose(1, 2).flatten(0, 1)[first:n], s["fmt"]) for c in "kv")
        for h in range(KVH):
            x = s["q"][b, h * G:(h + 1) * G].double() @ k[:, h].T * s["scale"]
            if s["softcap"] > 0:
                x = torch.tanh(x / s["softcap"]) * s["softcap"]
            out[b, h * G:(h + 1) * G] = torch.softmax(x, 1) @ v[:, h]
    return out


def _exact_select(s):
    B, W, V = s["logits"].shape
    K = s["parents"].shape[1]
    scores = torch.full((B, K), -math.inf, dtype=torch.float64, device=s["logits"].device)
    for b in range(B):
        x = torch.log_softmax(s["logits"][b].double(), -1) + s["scores"][b].double()[:, None]
        done = s["finished"][b] != 0
        x = torch.cat([x[~done].flatten(), s["scores"][b].double()[done]]).sort(descending=True).values[:K]
        scores[b, :x.numel()] = x
    return {"scores": scores, "parents": None, "tokens": None, "finished": None}


def exact(case, seed):
    if case["op"] == "reorder":
        return None  # whole numbers, and blocks that are copied
    s = prepare(case, seed)
    return {"write": _exact_write, "read": _exact_read, "decode": _exact_decode, "select": _exact_select}[case["op"]](s)


# ---------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op in ("write", "read"):
        kept = case["T"] - case["pads"]
        return {"bytes": 2 * kept * case["KVH"] * (case["D"] * ELEM[case["dtype"]] + _row_bytes(case)) + 8 * case["T"],
                "flops": 4 * kept * case["KVH"] * case["D"]}
    if op == "decode":
        ns = _spread(case["n_lo"], case["n_hi"], case["B"])
        keys = sum(min(n, case["window"]) if case["window"] else n for n in ns)
        return {"bytes": 2 * case["KVH"] * keys * _row_bytes(case) + 2 * case["B"] * case["H"] * case["D"] * ELEM[case["dtype"]]
                + 4 * sum(_ceil(n, case["bs"]) for n in ns), "flops": 4 * case["D"] * case["H"] * keys}
    if op == "select":
        rows = case["B"] * case["W"] - case["ended"]
        return {"bytes": rows * case["V"] * ELEM[case["dtype"]] + 5 * case["B"] * case["W"] + 13 * case["B"] * case["K"],
                "flops": 4 * rows * case["V"]}
    prompts = _spread(case["prompt_lo"], case["prompt_hi"], case["B"])
    cols = _pool_blocks(case)[1]
    # children chosen evenly: those whose parent has a child before them copy its last rows
    different = case["W"] * (1 - (1 - 1 / case["W"]) ** case["K"])
    rows = sum((p + case["made"]) % case["bs"] for p in prompts) * (case["K"] - different)
    return {"bytes": int(4 * case["layers"] * rows * case["KVH"] * _row_bytes(case)) + 8 * case["B"] * case["K"] * cols
            + 20 * case["B"] * case["K"], "flops": case["B"] * case["K"] * cols}
