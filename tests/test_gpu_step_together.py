"""The step operators as a serving loop runs them: pkv_build_step lays the step
out, pkv_rope_write rotates and writes it, pkv_chunk_attention attends, with
requests that arrive in chunks, decode, have drafted tokens turned down, end
and hand their blocks on.  Every step's output equals attention over the
request's own history in 64 bits, whatever the cache's blocks went through.

Tolerance: the caches hold rotated keys rounded to the type; the restatement
attends over the same rounded keys and queries, so the bound is the chunk
tests': (eps + 2^-18) max|v| for 16-bit types, 2^-17 max|v| for fp32."""
import math
import random

import pytest
import torch

import paged_kv_cache_67_gb300 as pkv
from step_reference import rope

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
I32, I64 = torch.int32, torch.int64


class Loop:
    """Fixed step buffers on the device, one workspace, one captured graph."""

    def __init__(self, B, H, KVH, D, bs, dtype, max_tokens, max_blocks, nb, softcap, window, axes, graph):
        z = lambda *s, t=I32: torch.zeros(*s, dtype=t, device=DEV)
        self.B, self.H, self.KVH, self.D, self.bs, self.dtype, self.nb = B, H, KVH, D, bs, dtype, nb
        self.tables, self.held, self.cached, self.new = z(B, max_blocks).fill_(99999), z(B), z(B), z(B)
        self.free, self.count = torch.randperm(nb, device=DEV).to(I32), torch.tensor([nb], dtype=I32, device=DEV)
        self.cu, self.slots, self.pos, self.err = z(B + 1), z(max_tokens, t=I64), z(axes, max_tokens), z(1)
        self.k_cache = torch.full((nb, bs, KVH, D), float("nan"), dtype=dtype, device=DEV)
        self.v_cache = self.k_cache.clone()
        self.q, self.out = z(max_tokens, H, D, t=dtype), z(max_tokens, H, D, t=dtype)
        self.k, self.v = z(max_tokens, KVH, D, t=dtype), z(max_tokens, KVH, D, t=dtype)
        pairs = D // 2
        ang = torch.arange(4096, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
        self.cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float().to(DEV)
        self.pair_axis = [j % axes for j in range(pairs)]
        self.scale, self.softcap, self.window, self.axes = 1 / math.sqrt(D), softcap, window, axes
        self.ws = pkv.ChunkWorkspace(B, max_tokens, H, KVH, D, bs, max_blocks, max_tokens, 0)
        self.max_tokens = max_tokens
        self.graph = None
        if graph:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph, stream=side):
                self.enqueue(side)

    def enqueue(self, stream=None):
        pkv.pkv_build_step(self.tables, self.held, self.held, self.free, self.count, self.count, self.cached, self.new,
                           self.cached, self.cu, self.slots, self.pos[0], self.nb, self.bs, err_flags=self.err, stream=stream)
        pkv.pkv_rope_write(self.q, self.k_cache, self.v_cache, self.q, self.k, self.v, self.cos_sin, self.pos, self.slots,
                           pair_axis=self.pair_axis, err_flags=self.err, stream=stream)
        pkv.pkv_chunk_attention(self.out, self.q, self.k_cache, self.v_cache, self.tables, self.cu, self.cached, self.scale,
                                softcap=self.softcap, window=self.window, max_q_len=self.max_tokens, workspace=self.ws,
                                err_flags=self.err, stream=stream)

    def step(self):
        self.graph.replay() if self.graph else self.enqueue()


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("dtype,H,KVH,D,bs,softcap,window,axes", [
    (torch.bfloat16, 4, 2, 128, 16, 20.0, 0, 1), (torch.float16, 2, 1, 256, 32, 0.0, 40, 3),
    (torch.float32, 4, 2, 64, 16, 0.0, 0, 2), (torch.bfloat16, 3, 1, 80, 8, 15.0, 25, 1)])
def test_serving_loop(dtype, H, KVH, D, bs, softcap, window, axes, graph):
    r, g = random.Random(7), torch.Generator().manual_seed(7)
    B, max_tokens = 4, 96
    lp = Loop(B, H, KVH, D, bs, dtype, max_tokens, -(-300 // bs), 4 * -(-300 // bs) // 2 + 8, softcap, window, axes, graph)
    hist = [[torch.zeros(0, KVH, D, dtype=dtype) for _ in range(2)] for _ in range(B)]     # rotated keys, values
    cached = [0] * B
    for step in range(14):
        new, total = [], 0
        for b in range(B):
            if step and r.random() < 0.15:                    # the request ends; another takes its place
                hist[b], cached[b] = [torch.zeros(0, KVH, D, dtype=dtype) for _ in range(2)], 0
            back = min(cached[b], r.randint(0, 2)) if cached[b] else 0      # drafts turned down
            cached[b] -= back
            hist[b] = [h[:cached[b]] for h in hist[b]]
            n = r.choice([0, 1, 1, 4]) if cached[b] else r.randint(1, 40)
            n = min(n, max_tokens - total, 250 - cached[b])
            new.append(n)
            total += n
        q, k, v = (torch.randn(max_tokens, h, D, generator=g).to(dtype) for h in (H, KVH, KVH))
        extra = torch.randint(0, 60, (axes, max_tokens), generator=g, dtype=I32)
        lp.q.copy_(q), lp.k.copy_(k), lp.v.copy_(v), lp.out.fill_(7.0)
        lp.pos.copy_(extra)
        lp.cached.copy_(torch.tensor(cached, dtype=I32)), lp.new.copy_(torch.tensor(new, dtype=I32))
        lp.step()
        torch.cuda.synchronize()
        assert int(lp.err) == 0, hex(int(lp.err))
        assert not lp.ws.buffer[:65536 * 4].any()
        pos = lp.pos.cpu()
        rows = [list(range(sum(new[:b]), sum(new[:b + 1]))) for b in range(B)]
        for b in range(B):                                    # axis 0 is the step's own positions
            assert pos[0, rows[b]].tolist() == list(range(cached[b], cached[b] + new[b]))
        qr = rope(q, lp.cos_sin.cpu(), pos, lp.pair_axis, False).to(dtype)
        kr = rope(k, lp.cos_sin.cpu(), pos, lp.pair_axis, False).to(dtype)
        got, got_q = lp.out.cpu(), lp.q.cpu()
        assert (got[total:] == 7).all()
        table, slots = lp.tables.cpu(), lp.slots.cpu()
        kc, vc = lp.k_cache.cpu().view(-1, KVH, D), lp.v_cache.cpu().view(-1, KVH, D)
        assert (slots[total:] == -1).all()
        for b in range(B):
            # the device's own rounding of the rotation may differ in the last
            # step of the type: its keys and queries are what is attended
            at = slots[rows[b]]
            step_eps = torch.finfo(dtype).eps
            assert ((kc[at].double() - kr[rows[b]].double()).abs() <= step_eps * 6).all()
            assert ((got_q[rows[b]].double() - qr[rows[b]].double()).abs() <= step_eps * 6).all()
            assert torch.equal(vc[at], v[rows[b]])
            hist[b] = [torch.cat([hist[b][0], kc[at]]), torch.cat([hist[b][1], vc[at]])]
            cached[b] += new[b]
            n = cached[b]
            where = torch.tensor([int(table[b, t // bs]) * bs + t % bs for t in range(n)], dtype=torch.long)
            assert torch.equal(kc[where], hist[b][0]) and torch.equal(vc[where], hist[b][1])   # the history is intact
            K, V = (h.double().repeat_interleave(H // KVH, 1) for h in hist[b])
            for i, row in enumerate(rows[b]):
                p = n - new[b] + i
                lo = max(0, p - window + 1) if window else 0
                x = torch.einsum("hd,jhd->hj", got_q[row].double(), K[lo:p + 1]) * lp.scale
                if softcap:
                    x = softcap * torch.tanh(x / softcap)
                want = torch.einsum("hj,jhd->hd", torch.softmax(x, 1), V[lo:p + 1])
                vmax = V.abs().max()
                tol = (2.0 ** -17 if dtype == torch.float32 else step_eps + 2.0 ** -18) * vmax
                assert (got[row].double() - want).abs().max() <= tol, (step, b, i)
