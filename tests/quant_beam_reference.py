"""Plain restatements of the quantised cache's and beam search's operators, on
CPU tensors, from their definitions: what the GPU tests compare with."""
from __future__ import annotations

import math

import numpy as np
import torch

FORMATS = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn, "int4": torch.uint8}
TINY = 2.0 ** -100


def _e4m3_values():
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    return v


def quantise(x, fmt):
    """x [..., D] -> (codes as numbers [..., D] float64, scale, zero) [...] float64,
    row by row in numpy: float32 where the definition rounds, 64 bits else."""
    shape = x.shape
    rows = x.float().reshape(-1, shape[-1]).numpy()
    codes = np.zeros(rows.shape)
    scale, zero = np.zeros(rows.shape[0]), np.zeros(rows.shape[0])
    f32 = np.float32
    top = {"int8": f32(127), "e4m3": f32(448), "int4": f32(15)}[fmt]
    grid = np.sort(_e4m3_values()[~torch.isnan(_e4m3_values())].numpy())
    for i, r in enumerate(rows):
        if fmt == "int4":
            lo, hi = f32(min(r.min(), 0)), f32(max(r.max(), 0))
            with np.errstate(over="ignore", invalid="ignore"):
                span = f32(hi - lo)
        else:
            span = f32(np.abs(r).max())
        if not np.isfinite(r).all() or not np.isfinite(span):
            scale[i] = math.nan
            continue
        if span < TINY:
            continue
        inv, scale[i] = f32(f32(f32(1) / span) * top), f32(span * f32(f32(1) / top))
        if fmt == "e4m3":
            y = (r * inv).astype(f32).astype(np.float64)
            # nearest value, halves to the even code
            at = np.clip(np.searchsorted(grid, y), 1, len(grid) - 1)
            below, above = grid[at - 1], grid[at]
            pick = np.where(y - below < above - y, below, above)
            tie = (y - below) == (above - y)
            even = (torch.from_numpy(below).to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy() % 2) == 0
            codes[i] = np.where(tie, np.where(even, below, above), pick)
            codes[i] = np.clip(codes[i], -448, 448)
        else:
            q = np.rint(r.astype(np.float64) * np.float64(inv))
            if fmt == "int4":
                zero[i] = np.rint(-np.float64(lo) * np.float64(inv))
                q = np.clip(q + zero[i], 0, 15)
            codes[i] = q
    lead = shape[:-1]
    return (torch.from_numpy(codes).reshape(shape), torch.from_numpy(scale).reshape(lead),
            torch.from_numpy(zero).reshape(lead))


def values(codes, params, fmt):
    """The numbers a cache's codes (as stored, [..., D or D / 2]) and params
    ([...] or [..., 2]) stand for, in 64 bits."""
    p = params.double()
    if fmt != "int4":
        return codes.double() * p[..., None]
    c = torch.empty(codes.shape[:-1] + (2 * codes.shape[-1],), dtype=torch.float64)
    c[..., 0::2], c[..., 1::2] = (codes & 15).double(), (codes >> 4).double()
    return (c - p[..., 1:2]) * p[..., 0:1]


def stored(codes, fmt):
    """Codes as numbers -> as stored."""
    if fmt != "int4":
        return codes.float().to(FORMATS[fmt])
    c = codes.to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def decode(q, k, v, scale, softcap=0.0, window=0):
    """One sequence: q [H, D] over k, v [n, KVH, D] (values), 64 bits."""
    H, D = q.shape
    n, KVH, _ = k.shape
    out = torch.zeros(H, D, dtype=torch.float64)
    if window > 0:
        k, v = k[max(0, n - window):], v[max(0, n - window):]
    if k.shape[0] == 0:
        return out
    for h in range(H):
        x = scale * (k[:, h // (H // KVH)].double() @ q[h].double())
        if softcap > 0:
            x = softcap * torch.tanh(x / softcap)
        w = torch.exp(x - x.max())
        out[h] = (w / w.sum()) @ v[:, h // (H // KVH)].double()
    return out


def beam_select(logits, scores, finished, K, end):
    """logits [B, W, V] (float), scores [B, W], finished [B, W] or None ->
    scores, parents, tokens, finished [B, K]; the order of the definition."""
    B, W, V = logits.shape
    out = (torch.full((B, K), -math.inf, dtype=torch.float64), torch.full((B, K), -1, dtype=torch.int32),
           torch.full((B, K), -1, dtype=torch.int32), torch.zeros(B, K, dtype=torch.uint8))
    for b in range(B):
        s, w_, v_ = [], [], []
        for w in range(W):
            c = float(scores[b, w])
            if not math.isfinite(c):
                continue
            if finished is not None and finished[b, w]:
                s.append(np.array([c])), w_.append(np.array([w])), v_.append(np.array([end]))
                continue
            x = logits[b, w].double().numpy()
            if np.isnan(x).any() or (x == math.inf).any() or (x == -math.inf).all():
                continue
            keep = np.nonzero(x > -math.inf)[0]
            m = x.max()
            # (differences from the largest first: added to a logit of 1e38, c would be lost)
            base = c - math.log(np.exp(x - m).sum())
            s.append(base + (x[keep] - m)), w_.append(np.full(len(keep), w)), v_.append(keep)
        if not s:
            continue
        s, w_, v_ = np.concatenate(s), np.concatenate(w_), np.concatenate(v_)
        order = np.lexsort((v_, w_, -s))[:K]
        for k, i in enumerate(order):
            out[0][b, k], out[1][b, k], out[2][b, k] = s[i], int(w_[i]), int(v_[i])
            out[3][b, k] = int((finished is not None and bool(finished[b, w_[i]])) or v_[i] == end)
    return out


def beam_reorder(tables, lens, parents, owned, finished, bs):
    """Python lists of one request -> (tables, lens, slots, copies (src, dst,
    rows)); every block and length as the definition wants them."""
    K, MB = len(parents), len(owned[0])
    child = []
    for k, p in enumerate(parents):
        n = lens[p] if p >= 0 else 0
        child.append({"p": p, "n": n, "c": n // bs if p >= 0 else -1, "r": n % bs})
    for k, x in enumerate(child):
        x["block"] = tables[x["p"]][x["c"]] if x["p"] >= 0 and x["r"] else None
    for k, x in enumerate(child):
        before = any(y["block"] == x["block"] and y["c"] == x["c"] for y in child[:k])
        whole = any(y["c"] > x["c"] and tables[y["p"]][x["c"]] == x["block"] for y in child if y["p"] >= 0)
        x["keeps"] = x["block"] is not None and not before and not whole
        x["target"] = x["block"] if x["keeps"] else None
    copies = []
    for k, x in enumerate(child):
        if x["p"] < 0 or x["keeps"] or x["c"] >= MB:
            continue
        c = x["c"]
        used = {tables[y["p"]][c] for y in child if y["c"] > c} | {y["target"] for y in child if y["c"] == c}
        lanes = [k] + [i for i in range(K) if i != k]
        x["target"] = next(owned[i][c] for i in lanes if owned[i][c] not in used)
        if x["r"]:
            copies.append((x["block"], x["target"], x["r"]))
    out_t, out_n, out_s = [], [], []
    for k, x in enumerate(child):
        row = list(owned[k])
        if x["p"] >= 0:
            row[:x["c"]] = tables[x["p"]][:x["c"]]
            if x["c"] < MB:
                row[x["c"]] = x["target"]
        out_t.append(row)
        go = x["p"] >= 0 and x["c"] < MB and not (finished is not None and finished[k])
        out_n.append(x["n"] + go)
        out_s.append(x["target"] * bs + x["r"] if go else -1)
    return out_t, out_n, out_s, copies
