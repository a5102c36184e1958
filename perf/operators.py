"""The operators of one serving step over the paged KV cache, as measured cases.

Three operators: ``pkv_build_step`` (block tables, slots, positions and query
offsets of a step from the requests' lengths, blocks taken from and returned
to a free list), ``pkv_rope_write`` (rotary positions over several axes, q
rotated, k rotated and written with v to the cache) and
``pkv_chunk_attention`` (new tokens of each sequence over the paged cache,
with capped scores, a distance bias, a window, a prefix mask or a document
mask; one new token per sequence is its decode form).

``run`` computes each in elementary torch operations in 32 bits, or, with
``own`` set, through the library.  Lengths are spread evenly over their range
and dealt out by the seed, so a case's work does not depend on the seed.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
ELEM = {"fp32": 4, "bf16": 2, "fp16": 2}


def listed():
    return [
        # a decode step's bookkeeping at the padded per-step batch: 180 requests
        # with one new token, 20 that ended (blocks go back), 56 padding entries
        {"name": "step_decode", "op": "step", "B": 256, "live": 180, "ended": 20, "bs": 16, "len_lo": 1,
         "len_hi": 2047, "new_lo": 1, "new_hi": 1, "spare": 0, "prompts": 0, "max_blocks": 132, "max_tokens": 256},
        # chunked prefill beside drafted decode: 64 requests with up to 5 new
        # tokens of which some drafts were turned down before, 32 new prompts
        {"name": "step_mixed", "op": "step", "B": 100, "live": 96, "ended": 4, "bs": 16, "len_lo": 512,
         "len_hi": 4000, "new_lo": 1, "new_hi": 5, "spare": 5, "prompts": 32, "max_blocks": 256, "max_tokens": 65536},
        # a large fleet of requests in chunks of up to 64 tokens
        {"name": "step_fleet", "op": "step", "B": 4096, "live": 4000, "ended": 90, "bs": 32, "len_lo": 1,
         "len_hi": 2000, "new_lo": 1, "new_hi": 64, "spare": 3, "prompts": 0, "max_blocks": 66, "max_tokens": 131072},
        # one new token of one request: the call's latency
        {"name": "rope_one_token", "op": "rope", "dtype": "fp16", "T": 1, "pads": 0, "H": 4, "KVH": 2, "D": 64,
         "rot": 64, "axes": 1, "interleaved": True, "bs": 16, "max_pos": 4096},
        # a decode batch of a vision-language model with 3-axis positions
        {"name": "rope_decode", "op": "rope", "dtype": "bf16", "T": 64, "pads": 5, "H": 32, "KVH": 8, "D": 128,
         "rot": 128, "axes": 3, "interleaved": False, "bs": 16, "max_pos": 32768},
        # a long video prompt: time, height, width positions
        {"name": "rope_video", "op": "rope", "dtype": "bf16", "T": 16384, "pads": 100, "H": 32, "KVH": 8, "D": 128,
         "rot": 128, "axes": 3, "interleaved": False, "bs": 16, "max_pos": 32768},
        # fp32, one KV head, only a part of the head rotated, an odd token count
        {"name": "rope_partial", "op": "rope", "dtype": "fp32", "T": 4099, "pads": 17, "H": 16, "KVH": 1, "D": 256,
         "rot": 64, "axes": 2, "interleaved": True, "bs": 32, "max_pos": 8192},
        # decode with capped scores at the 8B-shaped batch
        {"name": "decode_capped", "op": "chunk", "dtype": "bf16", "B": 64, "H": 32, "KVH": 8, "D": 128, "bs": 16,
         "n_lo": 512, "n_hi": 4096, "q_lo": 1, "q_hi": 1, "softcap": 50.0, "window": 0, "slopes": False,
         "prefix": 0, "doc_lo": 0, "doc_hi": 0},
        # a few drafted tokens per sequence checked against long contexts, distance bias
        {"name": "draft_biased_long", "op": "chunk", "dtype": "bf16", "B": 8, "H": 32, "KVH": 8, "D": 128, "bs": 16,
         "n_lo": 16384, "n_hi": 32768, "q_lo": 2, "q_hi": 6, "softcap": 0.0, "window": 0, "slopes": True,
         "prefix": 0, "doc_lo": 0, "doc_hi": 0},
        # one KV head, wide head, a sliding window over log-spread lengths
        {"name": "decode_window_mqa", "op": "chunk", "dtype": "fp16", "B": 128, "H": 16, "KVH": 1, "D": 256,
         "bs": 32, "n_lo": 1, "n_hi": 8192, "q_lo": 1, "q_hi": 1, "softcap": 0.0, "window": 1024, "slopes": False,
         "prefix": 0, "doc_lo": 0, "doc_hi": 0},
        # chunked prefill: ragged chunks on cached prefixes, capped scores, the
        # prompt's first tokens (an image) seen by every token
        {"name": "prefill_capped_prefix", "op": "chunk", "dtype": "bf16", "B": 4, "H": 32, "KVH": 8, "D": 128,
         "bs": 16, "n_lo": 2048, "n_hi": 4096, "q_lo": 100, "q_hi": 2048, "softcap": 30.0, "window": 0,
         "slopes": False, "prefix": 2500, "doc_lo": 0, "doc_hi": 0},
        # packed documents, whole prompts, distance bias
        {"name": "prefill_documents", "op": "chunk", "dtype": "bf16", "B": 2, "H": 32, "KVH": 8, "D": 128, "bs": 16,
         "n_lo": 6001, "n_hi": 8192, "q_lo": 8192, "q_hi": 8192, "softcap": 0.0, "window": 0, "slopes": True,
         "prefix": 0, "doc_lo": 300, "doc_hi": 3000},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _draw_step(rng):
    bs = rng.choice([1, 8, 16, 32, 64])
    B = _log_int(rng, 1, 4096)
    ended = rng.randint(0, max(0, B // 8))
    live = rng.randint(max(0, (B - ended) // 2), B - ended)
    len_hi = _log_int(rng, 1, max(1, min(4096, (1 << 20) // B)))
    new_hi = _log_int(rng, 1, max(1, min(64, 131072 // B)))
    spare = rng.randint(0, 5)
    prompts = rng.randint(0, live // 3) if rng.random() < 0.5 else 0
    most = live * new_hi + prompts * len_hi
    return {"op": "step", "B": B, "live": live, "ended": ended, "bs": bs, "len_lo": rng.randint(1, len_hi),
            "len_hi": len_hi, "new_lo": rng.randint(0, new_hi), "new_hi": new_hi, "spare": spare,
            "prompts": prompts, "max_blocks": -(-(len_hi + new_hi + spare) // bs) + rng.randint(0, 3),
            "max_tokens": max(1, most + rng.randint(0, most // 4 + 3))}


def _draw_rope(rng):
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    D = rng.choice([64, 80, 96, 128, 128, 192, 256])
    KVH = rng.choice([1, 2, 4, 8])
    H = KVH * rng.choice([1, 2, 4, 7, 8, 16])
    axes = rng.choice([1, 2, 3, 3, 4])
    rot = rng.choice([D, D, D // 2])
    most = max(1, (16384 * 48 * 128 * 2) // ((H + 2 * KVH) * D * ELEM[dtype]))
    T = _log_int(rng, 1, min(16384, most))
    return {"op": "rope", "dtype": dtype, "T": T, "pads": rng.randint(0, T // 4), "H": H, "KVH": KVH, "D": D,
            "rot": rot, "axes": axes, "interleaved": rng.random() < 0.4, "bs": rng.choice([1, 16, 32]),
            "max_pos": _log_int(rng, 64, 32768)}


def _draw_chunk(rng):
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    D = rng.choice([64, 128, 128, 192, 256] if dtype != "fp32" else [64, 80, 128])
    bs = rng.choice([16, 16, 32, 64] if dtype != "fp32" else [1, 16, 24])
    KVH = rng.choice([1, 2, 4, 8])
    H = KVH * rng.choice([1, 2, 4, 4, 6, 8, 16])
    kind = rng.choice(["decode", "draft", "chunk"])
    B = _log_int(rng, 1, 128 if kind == "decode" else 32 if kind == "draft" else 6)
    n_hi = _log_int(rng, 16, 32768 if kind != "chunk" else 8192)
    n_lo = rng.randint(1, n_hi)
    q_hi = {"decode": 1, "draft": rng.randint(2, 16), "chunk": _log_int(rng, 17, 2048)}[kind]
    q_hi = min(q_hi, n_hi)
    q_lo = rng.randint(1, q_hi)
    docs = rng.random() < 0.25
    doc_hi = _log_int(rng, 8, 4096)
    return {"op": "chunk", "dtype": dtype, "B": B, "H": H, "KVH": KVH, "D": D, "bs": bs, "n_lo": n_lo, "n_hi": n_hi,
            "q_lo": q_lo, "q_hi": q_hi, "softcap": rng.choice([0.0, 0.0, 30.0, 50.0]),
            "window": rng.choice([0, 0, _log_int(rng, 1, 4096)]), "slopes": rng.random() < 0.35,
            "prefix": rng.choice([0, 0, _log_int(rng, 1, n_hi)]), "doc_lo": rng.randint(1, doc_hi) if docs else 0,
            "doc_hi": doc_hi if docs else 0}


def draw(rng):
    op = rng.choice(["step", "rope", "rope", "chunk", "chunk", "chunk"])
    if op == "step":
        return _draw_step(rng)
    if op == "rope":
        return _draw_rope(rng)
    big = max((work(c) for c in listed() if c["op"] == "chunk"), key=lambda w: w["flops"])
    while True:
        c = _draw_chunk(rng)
        w, qs, ns = work(c), *_lengths(c)
        scores = c["B"] * c["H"] * max(qs) * max(ns)    # values of the plain form's padded score matrix
        gathered = c["B"] * max(ns) * c["H"] * c["D"]
        limit = big["flops"] if c["dtype"] != "fp32" else big["flops"] / 16
        if w["flops"] <= limit and w["bytes"] <= 1.5e9 and scores <= 2 ** 32 and gathered <= 2 ** 30:
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


def _lengths(case):
    """A chunk case's query counts and context lengths, before they are dealt out."""
    ns = _spread(case["n_lo"], case["n_hi"], case["B"])
    stride = next(s for s in range(3, 3 * case["B"] + 5) if math.gcd(s, case["B"]) == 1)
    qs = _spread(case["q_lo"], case["q_hi"], case["B"])
    qs = [min(qs[(i * stride) % case["B"]], n) for i, n in enumerate(ns)]
    return qs, ns


def _documents(case, n):
    """Lengths of the documents packed into n tokens, before they are dealt out."""
    out, i = [], 0
    sizes = _spread(case["doc_lo"], case["doc_hi"], 7)
    while sum(out) < n:
        out.append(min(sizes[i % 7], n - sum(out)))
        i += 1
    return out


def _step_lengths(case):
    """(cached, new, held tokens) of a step case's requests, before they are dealt out."""
    live, ended, B = case["live"], case["ended"], case["B"]
    cached = _spread(case["len_lo"], case["len_hi"], live) if live else []
    new = [case["new_lo"] + i % (case["new_hi"] - case["new_lo"] + 1) for i in range(live)]
    held = [c + i % (case["spare"] + 1) for i, c in enumerate(cached)]
    for i in range(case["prompts"]):       # prompts: nothing cached yet
        at = (i * 3) % max(live, 1)
        if cached[at]:
            new[at], cached[at], held[at] = cached[at], 0, 0
    held += _spread(case["len_lo"], case["len_hi"], ended) if ended else []
    pad = B - live
    return cached + [0] * pad, new + [0] * pad, held + [0] * (B - len(held))


def _ceil(a, b):
    return -(-a // b)


# ------------------------------------------------------------------- prepare

def _prepare_step(case, g, dev):
    B, bs, MB = case["B"], case["bs"], case["max_blocks"]
    order = torch.randperm(B, generator=g)
    cached, new, held_tokens = (torch.tensor(x, dtype=torch.int64)[order] for x in _step_lengths(case))
    held = (held_tokens + bs - 1) // bs
    want = (cached + new + bs - 1) // bs
    grow = int((want - held).clamp(min=0).sum())
    in_use = int(held.sum())
    num_blocks = in_use + grow + grow // 4 + 8
    perm = torch.randperm(num_blocks, generator=g).to(torch.int32)
    cols = torch.arange(MB)
    tables = torch.full((B, MB), 99999, dtype=torch.int32)
    tables[cols[None, :] < held[:, None]] = perm[:in_use]
    free = torch.full((num_blocks,), -1, dtype=torch.int32)
    free[:num_blocks - in_use] = perm[in_use:]
    i32 = lambda x: x.to(torch.int32).to(dev)
    empty = lambda n, t: torch.zeros(n, dtype=t, device=dev)
    return {"op": "step", "block_tables": tables.to(dev), "held": i32(held), "cached": i32(cached), "new": i32(new),
            "free": free.to(dev), "count": torch.tensor([num_blocks - in_use], dtype=torch.int32, device=dev),
            "num_blocks": num_blocks, "bs": bs, "held_out": empty(B, torch.int32), "count_out": empty(1, torch.int32),
            "lens": empty(B, torch.int32), "cu": empty(B + 1, torch.int32),
            "slots": empty(case["max_tokens"], torch.int64), "positions": empty(case["max_tokens"], torch.int32),
            "err": empty(1, torch.int32)}


def _prepare_rope(case, g, dev):
    T, H, KVH, D, rot, axes, bs = (case[k] for k in ("T", "H", "KVH", "D", "rot", "axes", "bs"))
    dt, max_pos = DTYPES[case["dtype"]], case["max_pos"]
    num_blocks = _ceil(T + T // 4, bs) + 1
    slots = torch.randperm(num_blocks * bs, generator=g)[:T]
    slots[torch.randperm(T, generator=g)[:case["pads"]]] = -1
    # positions as a prompt of text and frames has them: time rises over the
    # tokens, height and width run over a grid inside each frame
    start = int(torch.randint(0, max(1, max_pos - T), (1,), generator=g))
    side = max(2, int(math.sqrt(max(4, T // 8))))
    t = torch.arange(T)
    rows = [start + t, start + t // side % side, start + t % side, start + t // (side * side)]
    positions = torch.stack(rows[:axes]) % max_pos
    # pairs dealt to the axes in sections (time, height, width, ...)
    pairs = rot // 2
    edges = [round(pairs * a / axes) for a in range(axes + 1)]
    pair_axis = [next(a for a in range(axes) if edges[a] <= j < edges[a + 1]) for j in range(pairs)]
    inv = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
    angle = torch.arange(max_pos, dtype=torch.float64)[:, None] * inv[None, :]
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32).to(dev)
    dg = torch.Generator(device=dev).manual_seed(int(torch.randint(0, 2 ** 31, (1,), generator=g)))
    randn = lambda *s: torch.randn(s, generator=dg, device=dev).to(dt)
    # q, k and v lie side by side in one projection's output
    qkv = randn(T, (H + 2 * KVH) * D)
    return {"op": "rope", "q": qkv[:, :H * D].view(T, H, D), "k": qkv[:, H * D:(H + KVH) * D].view(T, KVH, D),
            "v": qkv[:, (H + KVH) * D:].view(T, KVH, D), "k_cache": randn(num_blocks, bs, KVH, D),
            "v_cache": randn(num_blocks, bs, KVH, D), "q_out": torch.zeros(T, H, D, dtype=dt, device=dev),
            "cos_sin": cos_sin, "positions": positions.to(torch.int32).to(dev), "pair_axis": pair_axis,
            "axis_of": torch.tensor(pair_axis, device=dev), "interleaved": case["interleaved"],
            "slots": slots.to(torch.int64).to(dev), "err": torch.zeros(1, dtype=torch.int32, device=dev)}


def _prepare_chunk(case, g, dev):
    B, H, KVH, D, bs = (case[k] for k in ("B", "H", "KVH", "D", "bs"))
    dt = DTYPES[case["dtype"]]
    order = torch.randperm(B, generator=g).tolist()
    qs, ns = _lengths(case)
    qs, ns = [qs[i] for i in order], [ns[i] for i in order]
    need = [_ceil(n, bs) for n in ns]
    num_blocks = sum(need) + sum(need) // 8 + 1
    perm = torch.randperm(num_blocks, generator=g).to(torch.int32)
    MB = max(need) + 1
    tables = torch.full((B, MB), 99999, dtype=torch.int32)
    at = 0
    for b in range(B):
        tables[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
    cu = torch.tensor([0] + qs).cumsum(0)
    total = int(cu[-1])
    starts = None
    if case["doc_hi"]:
        parts = []
        for q, n in zip(qs, ns):
            sizes = torch.tensor(_documents(case, n))
            sizes = sizes[torch.randperm(len(sizes), generator=g)]
            first = (sizes.cumsum(0) - sizes).repeat_interleave(sizes)     # of every position
            parts.append(first[n - q:])
        starts = torch.cat(parts).to(torch.int32).to(dev)
    prefix = None
    if case["prefix"]:
        p = torch.tensor(_spread(0, case["prefix"], B))[torch.randperm(B, generator=g)]
        prefix = p.to(torch.int32).to(dev)
    slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32, device=dev) if case["slopes"] else None
    dg = torch.Generator(device=dev).manual_seed(int(torch.randint(0, 2 ** 31, (1,), generator=g)))
    randn = lambda *s: torch.randn(s, generator=dg, device=dev)
    # queries that give scores of a few units, tens at the most
    return {"op": "chunk", "q": (randn(total, H, D) * 2.5).to(dt), "k_cache": randn(num_blocks, bs, KVH, D).to(dt),
            "v_cache": randn(num_blocks, bs, KVH, D).to(dt), "out": torch.empty(total, H, D, dtype=dt, device=dev),
            "tables": tables.to(dev), "cu": cu.to(torch.int32).to(dev),
            "lens": torch.tensor(ns, dtype=torch.int32, device=dev), "starts": starts, "prefix": prefix,
            "slopes": slopes, "softcap": case["softcap"], "window": case["window"], "scale": 1.0 / math.sqrt(D),
            "max_q": max(qs), "max_n": max(ns), "err": torch.zeros(1, dtype=torch.int32, device=dev)}


def prepare(case, seed):
    g = torch.Generator().manual_seed(int(seed))
    dev = torch.device("cuda")
    return {"step": _prepare_step, "rope": _prepare_rope, "chunk": _prepare_chunk}[case["op"]](case, g, dev)


# --------------------------------------------------------------- plain forms

def _plain_step(s):
    bs, MB, B = s["bs"], s["block_tables"].shape[1], s["held"].shape[0]
    tables, free = s["block_tables"].long(), s["free"].long()
    held, cached, new, count = s["held"].long(), s["cached"].long(), s["new"].long(), s["count"].long()
    dev = held.device
    want = (cached + new + bs - 1) // bs
    need, back = (want - held).clamp(min=0), (held - want).clamp(min=0)
    need_end, back_end, cu_end = need.cumsum(0), back.cumsum(0), new.cumsum(0)
    # the free list with the returned blocks behind it
    r = torch.arange(free.shape[0], device=dev) - count
    rb = torch.searchsorted(back_end, r.clamp(min=0), right=True).clamp(max=B - 1)
    col = (want[rb] + r - (back_end - back)[rb]).clamp(0, MB - 1)
    longer = torch.where((r >= 0) & (r < back_end[-1]), tables[rb, col], free)
    top = count + back_end[-1]
    # new blocks from its end
    cols = torch.arange(MB, device=dev)[None, :]
    k = (need_end - need)[:, None] + cols - held[:, None]
    taken = longer[(top - 1 - k).clamp(0, free.shape[0] - 1)]
    tables = torch.where((cols >= held[:, None]) & (cols < want[:, None]), taken, tables)
    t = torch.arange(s["slots"].shape[0], device=dev)
    live = t < cu_end[-1]
    b = torch.searchsorted(cu_end, t, right=True).clamp(max=B - 1)
    pos = cached[b] + t - (cu_end - new)[b]
    slot = tables[b, (pos // bs).clamp(0, MB - 1)] * bs + pos % bs
    i32 = torch.int32
    return {"block_tables": tables.to(i32), "free": longer.to(i32), "held": want.to(i32),
            "count": (top - need_end[-1]).to(i32), "lens": (cached + new).to(i32),
            "cu": torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), cu_end]).to(i32),
            "slots": torch.where(live, slot, -1), "positions": torch.where(live, pos, 0).to(i32)}


def _rotated(x, c, s, interleaved):
    rot = 2 * c.shape[-1]
    x = x.to(c.dtype)
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_rope(s):
    pairs = s["axis_of"].shape[0]
    row = s["positions"].long()[s["axis_of"]].T                       # [T, pairs]
    j = torch.arange(pairs, device=row.device)
    c, n = s["cos_sin"][row, j][:, None], s["cos_sin"][row, pairs + j][:, None]
    keep = s["slots"] >= 0
    dt, (KVH, D) = s["q"].dtype, s["k"].shape[1:]
    s["q_out"][keep] = _rotated(s["q"], c, n, s["interleaved"]).to(dt)[keep]
    s["k_cache"].view(-1, KVH, D)[s["slots"][keep]] = _rotated(s["k"], c, n, s["interleaved"]).to(dt)[keep]
    s["v_cache"].view(-1, KVH, D)[s["slots"][keep]] = s["v"][keep]
    return {"q_out": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_chunk(s):
    total, H, D = s["q"].shape
    num_blocks, bs, KVH, _ = s["k_cache"].shape
    B, G, Q, N = s["lens"].shape[0], H // KVH, s["max_q"], s["max_n"]
    dev = s["q"].device
    cu, lens = s["cu"].long(), s["lens"].long()
    # every sequence's chunk and context, padded to the longest
    i, j = torch.arange(Q, device=dev), torch.arange(N, device=dev)
    row = (cu[:-1, None] + i).clamp(max=total - 1)                     # [B, Q]
    q = s["q"][row].float().view(B, Q, KVH, G, D).permute(0, 2, 3, 1, 4).reshape(B, KVH, G * Q, D)
    blocks = s["tables"].long()[:, :_ceil(N, bs)].clamp(0, num_blocks - 1)
    real = (j < lens[:, None])[:, None, :, None]                        # [B, 1, N, 1]
    k, v = (torch.where(real, c[blocks].flatten(1, 2)[:, :N].permute(0, 2, 1, 3).float(), 0.0)
            for c in (s["k_cache"], s["v_cache"]))                     # [B, KVH, N, D]
    x = (q @ k.transpose(2, 3)).view(B, KVH, G, Q, N) * s["scale"]
    if s["softcap"] > 0:
        x = s["softcap"] * torch.tanh(x / s["softcap"])
    p = (lens - (cu[1:] - cu[:-1]))[:, None] + i                        # [B, Q] positions
    away = p[:, :, None] - j
    if s["slopes"] is not None:
        x = x - s["slopes"].view(1, KVH, G, 1, 1) * away.abs()[:, None, None].float()
    seen = away >= 0
    if s["prefix"] is not None:
        seen = seen | (j < s["prefix"].long()[:, None, None])
    if s["window"] > 0:
        seen = seen & (away < s["window"])
    if s["starts"] is not None:
        seen = seen & (j >= s["starts"].long()[row][:, :, None])
    seen = seen & (j < lens[:, None, None])
    x = torch.where(seen[:, None, None], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    w = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    o = (w.view(B, KVH, G * Q, N) @ v).view(B, KVH, G, Q, D) / w.sum(-1, keepdim=True)
    o = torch.where(m == -math.inf, 0.0, o).permute(0, 3, 1, 2, 4).reshape(B, Q, H, D)
    t = torch.arange(total, device=dev)
    b = torch.searchsorted(cu[1:], t, right=True)
    return o[b, t - cu[b]].to(s["q"].dtype)


# ----------------------------------------------------------------------- own

def _own_step(s):
    import paged_kv_cache_67_gb300 as pkv
    if "call" not in s:  # a serving loop marshals its fixed step buffers once
        s["call"] = pkv.prepare_build_step(
            s["block_tables"], s["held"], s["held_out"], s["free"], s["count"], s["count_out"], s["cached"], s["new"],
            s["lens"], s["cu"], s["slots"], s["positions"], s["num_blocks"], s["bs"], err_flags=s["err"])
    s["call"]()
    return {"block_tables": s["block_tables"], "free": s["free"], "held": s["held_out"], "count": s["count_out"],
            "lens": s["lens"], "cu": s["cu"], "slots": s["slots"], "positions": s["positions"]}


def _own_rope(s):
    import paged_kv_cache_67_gb300 as pkv
    if "call" not in s:
        s["call"] = pkv.prepare_rope_write(
            s["q_out"], s["k_cache"], s["v_cache"], s["q"], s["k"], s["v"], s["cos_sin"], s["positions"], s["slots"],
            pair_axis=s["pair_axis"], interleaved=s["interleaved"], err_flags=s["err"])
    s["call"]()
    return {"q_out": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_chunk(s):
    import paged_kv_cache_67_gb300 as pkv
    if "call" not in s:
        total, H, D = s["q"].shape
        _, bs, KVH, _ = s["k_cache"].shape
        ws = pkv.ChunkWorkspace(s["lens"].shape[0], total, H, KVH, D, bs, s["tables"].shape[1], s["max_q"], s["max_n"])
        s["call"] = pkv.prepare_chunk_attention(
            s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["cu"], s["lens"], s["scale"],
            softcap=s["softcap"], window=s["window"], slopes=s["slopes"], prefix_lens=s["prefix"],
            kv_starts=s["starts"], max_q_len=s["max_q"], max_context_len=s["max_n"], workspace=ws, err_flags=s["err"])
    s["call"]()
    return s["out"]


def run(state):
    if own:
        return {"step": _own_step, "rope": _own_rope, "chunk": _own_chunk}[state["op"]](state)
    return {"step": _plain_step, "rope": _plain_rope, "chunk": _plain_chunk}[state["op"]](state)


# ----------------------------------------------------------------- 64 bits

def _exact_rope(s):
    T, H, D = s["q"].shape
    KVH, pairs = s["k"].shape[1], len(s["pair_axis"])
    q_out = s["q_out"].double()
    kc, vc = s["k_cache"].double().view(-1, KVH, D), s["v_cache"].double().view(-1, KVH, D)
    keep = (s["slots"] >= 0).nonzero()[:, 0]
    slots = s["slots"][keep]
    q, k = s["q"].double()[keep], s["k"].double()[keep]
    for j in range(pairs):
        at = s["cos_sin"].double()[s["positions"][s["pair_axis"][j]].long()[keep]]
        turn = torch.complex(at[:, j], at[:, pairs + j])[:, None]
        lo, hi = (2 * j, 2 * j + 1) if s["interleaved"] else (j, j + pairs)
        for x in (q, k):
            z = torch.complex(x[..., lo], x[..., hi]) * turn
            x[..., lo], x[..., hi] = z.real, z.imag
    q_out[keep] = q
    kc[slots], vc[slots] = k, s["v"].double()[keep]
    return {"q_out": q_out, "k_cache": kc.view(s["k_cache"].shape), "v_cache": vc.view(s["v_cache"].shape)}


def _exact_chunk(s):
    total, H, D = s["q"].shape
    _, bs, KVH, _ = s["k_cache"].shape
    G, out = H // KVH, torch.zeros(total, H, D, dtype=torch.float64, device=s["q"].device)
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    for b, n in enumerate(lens):
        r0, r1 = cu[b], cu[b + 1]
        if r1 == r0:
            continue
        blocks = s["tables"][b, :_ceil(n, bs)].long()
        kb, vb = (c[blocks].reshape(-1, KVH, D)[:n].double() for c in (s["k_cache"], s["v_cache"]))
        key = torch.arange(n, device=out.device)[None, :]
        pos = torch.arange(n - (r1 - r0), n, device=out.device)[:, None]
        hidden = key > pos
        if s["prefix"] is not None:
            hidden &= key >= s["prefix"][b]
        if s["window"] > 0:
            hidden |= pos - key >= s["window"]
        if s["starts"] is not None:
            hidden |= key < s["starts"][r0:r1, None]
        nothing = hidden.all(1)
        for h in range(H):
            x = s["q"][r0:r1, h].double() @ kb[:, h // G].T * s["scale"]
            if s["softcap"] > 0:
                x = torch.tanh(x / s["softcap"]) * s["softcap"]
            if s["slopes"] is not None:
                x -= s["slopes"][h].double() * (pos - key).abs()
            x = torch.softmax(x.masked_fill(hidden, -math.inf), 1)
            out[r0:r1, h] = (x @ vb[:, h // G]).masked_fill(nothing[:, None], 0.0)
    return out


def exact(case, seed):
    if case["op"] == "step":
        return None  # whole numbers
    s = prepare(case, seed)
    return _exact_rope(s) if case["op"] == "rope" else _exact_chunk(s)


# ---------------------------------------------------------------------- work

def _pairs(case, q, n, prefix):
    """(query, key) pairs of one sequence and head that the masks leave."""
    if case["doc_hi"]:
        # documents are dealt out by the seed: their pairs when all are queries,
        # in proportion to the queries otherwise
        own_pairs = sum(d * (d + 1) // 2 for d in _documents(case, n))
        return max(q, own_pairs * q // n)
    total = 0
    for p in (range(n - q, n) if q <= 64 else range(n - q, n, max(1, q // 64))):
        hi = max(p + 1, min(prefix, n))
        lo = max(0, p - case["window"] + 1) if case["window"] else 0
        total += hi - lo
    return total if q <= 64 else total * q // len(range(n - q, n, max(1, q // 64)))


def work(case):
    if case["op"] == "step":
        cached, new, held = _step_lengths(case)
        bs = case["bs"]
        moved = sum(abs(_ceil(c + n, bs) - _ceil(h, bs)) for c, n, h in zip(cached, new, held))
        return {"bytes": 24 * case["B"] + 12 * case["max_tokens"] + 8 * moved + 4 * sum(1 for n in new if n), "flops": sum(new) * 4}
    el = ELEM[case["dtype"]]
    if case["op"] == "rope":
        kept = case["T"] - case["pads"]
        rows = min(case["max_pos"], case["T"]) * case["rot"] * 4
        return {"bytes": el * kept * case["D"] * (2 * case["H"] + 4 * case["KVH"]) + case["T"] * (8 + 4 * case["axes"]) + rows,
                "flops": 3 * kept * case["rot"] * (case["H"] + case["KVH"])}
    qs, ns = _lengths(case)
    pre = _spread(0, case["prefix"], case["B"]) if case["prefix"] else [0] * case["B"]
    pairs = keys = 0
    for q, n, p in zip(qs, ns, pre):
        pairs += _pairs(case, q, n, p)
        seen = min(n, case["window"] + q - 1) if case["window"] else n
        if case["doc_hi"]:
            seen = min(seen, q + case["doc_hi"])
        keys += seen
    return {"bytes": el * case["D"] * (2 * case["KVH"] * keys + 2 * case["H"] * sum(qs)) + 4 * sum(_ceil(n, case["bs"]) for n in ns),
            "flops": 4 * case["D"] * case["H"] * pairs}
