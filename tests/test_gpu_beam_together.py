"""Beam search over a quantised paged cache, as a serving loop runs it: the
prompt quantised as it is written, then every step the next tokens' rows written,
attended, turned into logits, the best continuations selected and the cache
reordered, eagerly and as one captured graph.  The model is a toy: a token's
query, key and value are table lookups, logits are the output times a matrix.

Checked each step: the selection on the very logits (beams are told apart by
1e-5, or the step's order is not compared), the attention of every beam over
its own history of tokens in 64 bits, and that reading every beam's table back
gives exactly its history's quantised rows, whatever was shared and copied."""
import math

import pytest
import torch

import paged_kv_cache_67_gb300 as pkv
import quant_beam_reference as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
I32, I64 = torch.int32, torch.int64


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("fmt", ["int8", "e4m3", "int4"])
def test_beam_search_loop(fmt, graph):
    B, W, V, H, KVH, D, bs, MB, steps, end = 2, 4, 500, 8, 2, 64, 4, 10, 18, 3
    dtype = torch.bfloat16
    g = torch.Generator().manual_seed(7)
    rnd = lambda *s: torch.randn(*s, generator=g)
    tq, tk, tv = (rnd(V, H, D) * 1.5).to(dtype), rnd(V, KVH, D).to(dtype), rnd(V, KVH, D).to(dtype)
    unembed = rnd(H * D, V) * 0.35
    prompts = [torch.randint(4, V, (n,), generator=g) for n in (9, 6)]
    lanes = torch.randperm(B * (W * MB + MB), generator=g).to(I32)
    nb = lanes.numel()
    dd = D // 2 if fmt == "int4" else D
    codes = [torch.full((nb, bs, KVH, dd), 0x7f, dtype=torch.uint8).view(ref.FORMATS[fmt]).to(DEV) for _ in range(2)]
    params = [torch.full((nb, KVH, bs) + ((2,) if fmt == "int4" else ()), math.nan, device=DEV) for _ in range(2)]
    cache = codes + params
    owned = lanes[:B * W * MB].view(B, W, MB).clone()
    for b, p in enumerate(prompts):                        # the prompt's full blocks are everybody's
        owned[b, :, :len(p) // bs] = owned[b, :1, :len(p) // bs]
    # the prompt, but for its last token, which is the first step's
    slots = torch.cat([owned[b, 0].long()[torch.arange(len(p) - 1) // bs] * bs + torch.arange(len(p) - 1) % bs
                       for b, p in enumerate(prompts)])
    first = torch.cat([p[:-1] for p in prompts])
    pkv.pkv_quant_write(*cache, tk[first].to(DEV), tv[first].to(DEV), slots.to(DEV))

    d = lambda t: t.to(DEV)
    dq, dk, dv, du, downed = d(tq), d(tk), d(tv), d(unembed), d(owned)
    tables = [downed.clone(), torch.zeros_like(downed)]
    lens0 = torch.tensor([[len(p)] * W for p in prompts], dtype=I32)
    lens = [d(lens0), torch.zeros(B, W, dtype=I32, device=DEV)]
    slot = torch.full((B, W), -1, dtype=I64)
    for b, p in enumerate(prompts):
        n = len(p) - 1
        slot[b, 0] = int(owned[b, 0, n // bs]) * bs + n % bs
    slot = d(slot)
    scores = torch.full((B, W), -math.inf, device=DEV)
    scores[:, 0] = 0
    finished = torch.zeros(B, W, dtype=torch.uint8, device=DEV)
    tokens = torch.zeros(B, W, dtype=I32, device=DEV)
    tokens[:, 0] = d(torch.stack([p[-1] for p in prompts]).to(I32))
    parents = torch.zeros(B, W, dtype=I32, device=DEV)
    out, logits = torch.zeros(B * W, H, D, dtype=dtype, device=DEV), torch.zeros(B, W, V, device=DEV)
    err = torch.zeros(1, dtype=I32, device=DEV)
    wd, wsel = pkv.QuantDecodeWorkspace(B * W, H, KVH, D, bs, MB), pkv.BeamSelectWorkspace(B, W, W, V)
    scale = 1 / math.sqrt(D)

    def step(a, stream=None):
        tok = tokens.view(-1).clamp(min=0).long()
        pkv.pkv_quant_write(*cache, dk[tok], dv[tok], slot.view(-1), err_flags=err, stream=stream)
        pkv.pkv_quant_decode_attention(out, dq[tok], *cache, tables[a].view(B * W, MB), lens[a].view(-1), scale,
                                       workspace=wd, err_flags=err, stream=stream)
        logits.copy_((out.view(B * W, H * D).float() @ du).view(B, W, V))
        pkv.pkv_beam_select(scores, parents, tokens, finished, logits, scores, finished, end_token=end, workspace=wsel,
                            err_flags=err, stream=stream)
        pkv.pkv_beam_reorder(tables[1 - a], lens[1 - a], slot, tables[a], lens[a], parents, downed, bs, pools=codes,
                             block_pools=params, finished=finished, err_flags=err, stream=stream)

    graphs = []
    if graph:
        (out.view(B * W, H * D).float() @ du).sum()         # the library's handle before capture
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        for a in (0, 1):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=side):
                step(a, side)
        torch.cuda.synchronize()
    quant = [[(lambda c, s, z: s[..., None] * (c - z[..., None]))(*ref.quantise(t, fmt)) for t in (tk, tv)]][0]
    history = [[p.tolist() if w == 0 else None for w in range(W)] for p in prompts]     # tokens in the cache after the write
    for i in range(steps):
        a = i & 1
        before = scores.cpu(), finished.cpu(), tokens.cpu()
        if graph:
            graphs[a].replay()
        else:
            step(a)
        torch.cuda.synchronize()
        assert int(err) == 0, i
        o = out.view(B, W, H, D).cpu()
        for b in range(B):
            for w in range(W):
                if history[b][w] is None or before[1][b, w]:
                    continue
                h = torch.tensor(history[b][w])
                want = ref.decode(tq[int(before[2][b, w])], quant[0][h], quant[1][h], scale)
                top = float(quant[1][h].abs().max())
                assert (o[b, w].double() - want).abs().max() <= 1.05 * 2.0 ** -8 * top, (i, b, w)
        want = ref.beam_select(logits.cpu(), before[0], before[1], W + 1, end)
        p, t = parents.cpu(), tokens.cpu()
        for b in range(B):
            s = want[0][b]
            if any(0 < float(s[k] - s[k + 1]) < 1e-5 for k in range(W)):
                continue
            assert torch.equal(p[b], want[1][b, :W]) and torch.equal(t[b], want[2][b, :W]), (i, b)
        f = finished.cpu()
        new = []
        for b in range(B):
            row = []
            for k in range(W):
                parent = int(p[b, k])
                if parent < 0:
                    row.append(None)
                    continue
                done = before[1][b, parent]
                row.append(list(history[b][parent]) + ([] if done or f[b, k] else [int(t[b, k])]))
            new.append(row)
        history = new
        # every beam's rows, but for the next token's, which is not written yet
        tab, n = tables[1 - a].cpu(), lens[1 - a].cpu()
        for b in range(B):
            for k in range(W):
                if history[b][k] is None:
                    continue
                assert int(n[b, k]) == len(history[b][k]), (i, b, k)
                have = len(history[b][k]) - (0 if f[b, k] else 1)
                pos = torch.arange(have)
                where = tab[b, k].long()[pos // bs] * bs + pos % bs
                got = [torch.zeros(have, KVH, D, device=DEV) for _ in range(2)]
                pkv.pkv_quant_read(*got, *cache, where.to(DEV))
                h = torch.tensor(history[b][k][:have])
                for s in range(2):
                    assert torch.equal(got[s].cpu(), quant[s][h].float()), (i, b, k)
        used = [int(x) for x in slot.view(-1) if int(x) >= 0]
        assert len(set(used)) == len(used)                   # no two beams write the same place
