"""Plain 64-bit restatements of the step operators, on CPU tensors: what the
GPU tests compare pkv_build_step, pkv_rope_write and pkv_chunk_attention with.
Written from the operators' definitions, sequence by sequence."""
from __future__ import annotations

import math

import torch


def build_step(tables, held, free, count, cached, new, bs, max_tokens, num_blocks):
    """Python lists in and out; returns a dict, or None where the call has to
    refuse the step ("invalid" or "blocks" under "why")."""
    tables, free = [list(r) for r in tables], list(free)
    B, MB, cap = len(tables), len(tables[0]) if tables else 0, len(free)
    ceil = lambda x: -(-x // bs)
    bad = not 0 <= count <= cap
    for c, n, h in zip(cached, new, held):
        bad |= c < 0 or n < 0 or not 0 <= h <= MB or c + n > MB * bs or (c >= 0 and ceil(c) > h)
    if bad or sum(new) >= 1 << 30:
        return {"why": "invalid"}
    want = [ceil(c + n) for c, n in zip(cached, new)]
    stack = free[:count]
    for b in range(B):
        stack += tables[b][want[b]:held[b]]
    if len(stack) > cap:
        return {"why": "invalid"}
    if sum(max(0, w - h) for w, h in zip(want, held)) > len(stack):
        return {"why": "blocks"}
    free[:len(stack)] = stack
    for b in range(B):
        for i in range(held[b], want[b]):
            tables[b][i] = stack.pop()
    slots, positions, cu = [], [], [0]
    for b in range(B):
        for p in range(cached[b], cached[b] + new[b]):
            blk = tables[b][p // bs]
            slots.append(blk * bs + p % bs if 0 <= blk < num_blocks else -1)
            positions.append(p)
        cu.append(len(slots))
    del slots[max_tokens:], positions[max_tokens:]      # the lists hold the first max_tokens
    pad = max_tokens - len(slots)
    return {"tables": tables, "held": want, "free": free, "count": len(stack),
            "lens": [c + n for c, n in zip(cached, new)], "cu": cu, "slots": slots + [-1] * pad,
            "positions": positions + [0] * pad}


def rope(x, cos_sin, positions, pair_axis, interleaved):
    """x [T, heads, D] rotated, in float64 (positions [axes, T])."""
    x = x.double().clone()
    pairs = cos_sin.shape[1] // 2
    for j in range(pairs):
        row = cos_sin[positions[pair_axis[j]].long()].double()
        c, s = row[:, j, None], row[:, pairs + j, None]
        lo, hi = (2 * j, 2 * j + 1) if interleaved else (j, j + pairs)
        a, b = x[:, :, lo].clone(), x[:, :, hi].clone()
        x[:, :, lo], x[:, :, hi] = a * c - b * s, b * c + a * s
    return x


def chunk(q, k_cache, v_cache, tables, cu, lens, scale, softcap=0.0, window=0, slopes=None, prefix=None,
          starts=None):
    """Chunk attention in float64; keys and values that a query does not see
    take no part, whatever they hold."""
    total, H, D = q.shape
    _, bs, KVH, _ = k_cache.shape
    G = H // KVH
    out = torch.zeros(total, H, D, dtype=torch.float64)
    for b in range(len(lens)):
        r0, r1, n = int(cu[b]), int(cu[b + 1]), int(lens[b])
        if r1 == r0:
            continue
        nb = -(-n // bs)
        rows = [tables[b, i] for i in range(nb)]
        pool = k_cache.shape[0]
        # blocks that no query sees may have any entry: read block 0 for them
        idx = torch.tensor([int(x) if 0 <= int(x) < pool else 0 for x in rows], dtype=torch.long)
        K = k_cache[idx].reshape(-1, KVH, D)[:n].double()
        V = v_cache[idx].reshape(-1, KVH, D)[:n].double()
        j = torch.arange(n)
        for i in range(r1 - r0):
            p = n - (r1 - r0) + i
            seen = j <= p
            if prefix is not None:
                seen |= j < int(prefix[b])
            if window:
                seen &= p - j < window
            if starts is not None:
                seen &= j >= int(starts[r0 + i])
            at = seen.nonzero()[:, 0]
            if at.numel() == 0:
                continue
            x = torch.einsum("hd,jhd->hj", q[r0 + i].double(), K[at].repeat_interleave(G, 1)) * scale
            if softcap:
                x = softcap * torch.tanh(x / softcap)
            if slopes is not None:
                x = x - slopes.double()[:, None] * (p - at).abs()
            w = torch.softmax(x, 1)
            out[r0 + i] = torch.einsum("hj,jhd->hd", w, V[at].repeat_interleave(G, 1))
    return out
