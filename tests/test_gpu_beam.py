"""pkv_beam_select and pkv_beam_reorder against their restatement.

Parents, tokens and flags are whole numbers and have to be equal: the inputs
keep scores of different beams 1e-5 apart or exactly equal, where the sums'
accuracy (some 1e-7) cannot change the order.  Scores are one rounding of a
sum of three: half a step of fp32 at the score's size and of the sum's 2^-22."""
import math

import pytest
import torch

import paged_kv_cache_67_gb300 as pkv
import quant_beam_reference as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
TYPES = [torch.float32, torch.bfloat16, torch.float16]
I32 = torch.int32


def select(logits, scores, finished, K, end=-1, flags=0, ws=None):
    B, W, V = logits.shape
    o = [torch.full((B, K), 7.0, device=DEV), torch.full((B, K), 7, dtype=I32, device=DEV),
         torch.full((B, K), 7, dtype=I32, device=DEV), torch.full((B, K), 7, dtype=torch.uint8, device=DEV)]
    err = torch.zeros(1, dtype=I32, device=DEV)
    ws = ws or pkv.BeamSelectWorkspace(B, W, K, V)
    d = lambda t: None if t is None else t.to(DEV)
    logits = d(logits)
    for _ in range(2):
        pkv.pkv_beam_select(*o, logits, d(scores), d(finished), end_token=end, workspace=ws, err_flags=err)
    torch.cuda.synchronize()
    assert int(err) == flags
    return [t.cpu() for t in o]


def check_select(logits, scores, finished, K, end=-1, flags=0, apart=True, ws=None):
    got = select(logits, scores, finished, K, end, flags, ws)
    want = ref.beam_select(logits.cpu(), scores, finished, K + 1 if apart else K, end)
    if apart:       # the inputs keep what this test compares apart (a fault of the input, not of the kernel)
        for b in range(logits.shape[0]):
            s, p = want[0][b], want[1][b]
            for i in range(K):
                if p[i] >= 0 and p[i + 1] >= 0 and p[i] != p[i + 1]:
                    gap = float(s[i] - s[i + 1])
                    assert gap == 0 or gap > 1e-5, "beams too near"
        want = [t[:, :K] for t in want]
    for g, w, what in zip(got[1:], want[1:], ("parents", "tokens", "finished")):
        assert torch.equal(g, w), (what, g, w)
    fine = want[0] > -math.inf
    assert torch.equal(got[0] > -math.inf, fine)
    off = (got[0].double() - want[0]).abs()[fine]
    assert (off <= (want[0].abs()[fine] + 20) * 2.0 ** -22).all()


def logits_of(B, W, V, dtype, seed, scale=2.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, W, V, generator=g) * scale
    # likely tokens, on a grid of their own for each beam so that beams stay apart
    for b in range(B):
        for w in range(W):
            at = torch.randint(0, V, (min(V, 12),), generator=g)
            x[b, w, at] = (8.0 + 0.25 * torch.randint(0, 20, at.shape, generator=g) + 0.03125 * (w % 8)).float()
    return x.to(dtype)


def scores_of(B, W, seed):
    g = torch.Generator().manual_seed(1000 + seed)
    return -torch.rand(B, W, generator=g).cumsum(1) * 3


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,W,K,V", [(1, 1, 1, 1), (1, 1, 4, 3), (2, 4, 4, 100), (3, 4, 8, 1001), (2, 8, 8, 32000), (1, 32, 32, 777),
                                     (2, 3, 32, 4097), (1, 4, 4, 50257), (5, 2, 3, 8192), (1, 1, 16, 200001), (40, 4, 4, 32001)])
def test_select_shapes(dtype, B, W, K, V):
    check_select(logits_of(B, W, V, dtype, V), scores_of(B, W, V), None, K, end=min(2, V - 1))


@pytest.mark.parametrize("dtype", TYPES)
def test_select_finished_and_unused(dtype):
    x, c = logits_of(4, 6, 999, dtype, 5), scores_of(4, 6, 5)
    f = torch.zeros(4, 6, dtype=torch.uint8)
    f[0, 1] = f[0, 4] = 1
    f[1] = 1                                                   # every beam has ended
    c[2, 1:] = -math.inf                                       # the first step: one beam
    c[3] = -math.inf                                           # a request that is not there
    x[0, 1] = math.nan                                         # rows that are not read
    x[2, 3] = math.nan
    check_select(x, c, f, 8, end=17)
    check_select(x, c, f.bool(), 6, end=17)
    c[1, 2] = -math.inf                                        # ended and unused
    check_select(x, c, f, 6, end=17)


def test_select_end_token():
    x, c = logits_of(2, 3, 500, torch.float32, 6), scores_of(2, 3, 6)
    x[:, :, 44] = 30.0                                         # the end is by far the likeliest
    x[:, 1, 44] += 0.125
    x[:, 2, 44] += 0.5
    got = select(x, c, None, 5, end=44)
    assert (got[3][:, :3] == 1).all() and (got[2][:, :3] == 44).all()
    check_select(x, c, None, 5, end=44)
    check_select(x, c, None, 5, end=-1)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [9, 700, 4099, 20001])
def test_select_ties(dtype, V):
    """Equal logits, equal beams: the lowest beam, then the lowest token, wherever
    the rows start in memory; more ties than a piece ranks at once."""
    row = logits_of(1, 1, V, dtype, V)[0, 0]
    x = row.expand(2, 5, V).contiguous()
    c = torch.tensor([[-1.0] * 5, [-2.0, -1.0, -1.0, -2.0, -1.0]])
    check_select(x, c, None, 12, apart=False)
    check_select(torch.zeros(2, 3, V, dtype=dtype), torch.zeros(2, 3), None, 16, apart=False)
    x = torch.zeros(1, 2, V, dtype=dtype)
    x[..., ::2] = -0.0                                         # equal to 0
    x[..., V // 2:] = -math.inf
    check_select(x, torch.zeros(1, 2), None, 8, apart=False)


@pytest.mark.parametrize("dtype", TYPES)
def test_select_masked_logits(dtype):
    x, c = logits_of(3, 2, 3001, dtype, 8), scores_of(3, 2, 8)
    x[0, :, 5:] = -math.inf                                    # fewer tokens than asked for
    x[1] = -math.inf                                           # none at all
    x[2, 0] = -math.inf
    x[2, 0, 3000] = 1.0
    check_select(x, c, None, 16, apart=False)
    big = torch.finfo(dtype).max                               # the type's ends
    x = torch.full((1, 2, 100), -big, dtype=dtype)
    x[0, 0, 7], x[0, 1, 9] = big, 0.0
    check_select(x, torch.tensor([[-1.0, -2.0]]), None, 4, apart=False)


@pytest.mark.parametrize("dtype", TYPES)
def test_select_flags(dtype):
    x, c = logits_of(3, 4, 5000, dtype, 9), scores_of(3, 4, 9)
    x[0, 1, 4999], x[1, 0, 0] = math.nan, math.inf
    check_select(x, c, None, 6, flags=pkv.FLAG_LOGITS)
    c[2, 3] = math.nan
    c[2, 1] = math.inf
    check_select(x, c, None, 6, flags=pkv.FLAG_LOGITS)


@pytest.mark.parametrize("dtype", TYPES)
def test_select_strided_rows(dtype):
    """Rows inside a wider tensor (a padded vocabulary), at every alignment."""
    for pad, shift in ((1, 0), (3, 1), (8, 3), (5, 7), (16, 8)):
        V, B, W = 1003, 2, 3
        x, c = logits_of(B, W, V, dtype, 10 + pad), scores_of(B, W, 10 + pad)
        buf = torch.full((shift + B * W * (V + pad),), math.nan, dtype=dtype, device=DEV)   # never read
        view = buf[shift:].view(B, W, V + pad)[..., :V]
        view.copy_(x)
        o = [torch.zeros(B, 4, device=DEV), *(torch.zeros(B, 4, dtype=I32, device=DEV) for _ in range(2)),
             torch.zeros(B, 4, dtype=torch.uint8, device=DEV)]
        ws = pkv.BeamSelectWorkspace(B, W, 4, V)
        err = torch.zeros(1, dtype=I32, device=DEV)
        pkv.pkv_beam_select(*o, view, c.to(DEV), end_token=1, workspace=ws, err_flags=err)
        want = ref.beam_select(x, c, None, 4, 1)
        assert int(err) == 0
        for g, w in zip(o[1:], want[1:]):
            assert torch.equal(g.cpu(), w)


def test_select_in_place_one_workspace_and_graph():
    """Scores and flags in place, one workspace for calls of several sizes, a
    captured step replayed."""
    ws = pkv.BeamSelectWorkspace(8, 8, 8, 40000)
    for B, W, K, V in ((8, 8, 8, 40000), (1, 2, 3, 50), (3, 4, 4, 9000)):
        check_select(logits_of(B, W, V, torch.bfloat16, V), scores_of(B, W, V), None, K, ws=ws)
    B, W, V = 2, 4, 3000
    logits = torch.zeros(B, W, V, dtype=torch.bfloat16, device=DEV)
    scores, fin = scores_of(B, W, 1).to(DEV), torch.zeros(B, W, dtype=torch.uint8, device=DEV)
    parents, tokens = (torch.zeros(B, W, dtype=I32, device=DEV) for _ in range(2))
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        pkv.pkv_beam_select(scores, parents, tokens, fin, logits, scores, fin, end_token=5, workspace=ws, stream=side)
    c, f = scores.cpu(), fin.cpu()
    for step in range(4):
        x = logits_of(B, W, V, torch.bfloat16, 60 + step)
        x[0, 0, 5] = 14.0
        logits.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        want = ref.beam_select(x, c, f, W, 5)
        assert torch.equal(parents.cpu(), want[1]) and torch.equal(tokens.cpu(), want[2]) and torch.equal(fin.cpu(), want[3])
        c, f = scores.cpu(), fin.cpu()


# ------------------------------------------------------------------ reorder

def reorder_case(B, W, K, bs, MB, lens, seed, parents=None):
    """Tables whose columns behind a prompt hold blocks of `owned`."""
    g = torch.Generator().manual_seed(seed)
    L = max(W, K)
    nb = B * (MB + L * MB)
    perm = torch.randperm(nb, generator=g).to(I32)
    owned, tables = torch.zeros(B, L, MB, dtype=I32), torch.zeros(B, W, MB, dtype=I32)
    at = 0
    for b in range(B):
        prompt = int(torch.randint(0, max(1, min(min(r) for r in lens) // bs + 1), (1,), generator=g))
        shared = perm[at:at + MB]
        at += MB
        owned[b] = perm[at:at + L * MB].view(L, MB)
        at += L * MB
        owned[b, :, :prompt] = shared[:prompt]
        for c in range(MB):
            tables[b, :, c] = owned[b, torch.randperm(L, generator=g)[:W], c]
            if c < prompt:
                tables[b, :, c] = shared[c]
            elif all((c + 1) * bs <= n for n in lens[b]) and W > 1:    # whole for every beam: may be shared
                tables[b, :, c] = owned[b, torch.randint(0, L, (W,), generator=g), c]
    if parents is None:
        parents = torch.randint(0, W, (B, K), generator=g)
    return tables, owned[:, :K].contiguous(), parents.to(I32), nb


def check_reorder(tables, lens, parents, owned, finished, bs, nb, pools, block_pools, flags=0):
    B, W, MB = tables.shape
    K = parents.shape[1]
    i32 = lambda x: torch.tensor(x, dtype=I32)
    out = [torch.full((B, K, MB), -7, dtype=I32, device=DEV), torch.full((B, K), -7, dtype=I32, device=DEV),
           torch.full((B, K), -7, dtype=torch.int64, device=DEV)]
    err = torch.zeros(1, dtype=I32, device=DEV)
    dp, db = [p.to(DEV) for p in pools], [p.to(DEV) for p in block_pools]
    pkv.pkv_beam_reorder(*out, tables.to(DEV), i32(lens).to(DEV), parents.to(DEV), owned.to(DEV), bs, num_blocks=nb,
                         pools=dp, block_pools=db, finished=None if finished is None else finished.to(DEV), err_flags=err)
    torch.cuda.synchronize()
    assert int(err) == flags
    want_p, want_b = [p.clone() for p in pools], [p.clone() for p in block_pools]
    for b in range(B):
        t, n, s, copies = ref.beam_reorder(tables[b].tolist(), lens[b], parents[b].tolist(), owned[b].tolist(),
                                           None if finished is None else finished[b].tolist(), bs)
        assert out[0][b].tolist() == t, b
        assert out[1][b].tolist() == n and out[2][b].tolist() == s, b
        for src, dst, rows in copies:
            for p, w in zip(pools, want_p):
                w[dst, :rows] = p[src, :rows]
            for p, w in zip(block_pools, want_b):
                w[dst] = p[src]
    for g, w in zip(dp + db, want_p + want_b):
        assert torch.equal(g.cpu().view(torch.uint8), w.view(torch.uint8))


def pools_of(nb, bs, kinds, seed=0):
    g = torch.Generator().manual_seed(seed)
    out = []
    for shape, dtype in kinds:
        x = torch.randint(0, 256, (nb, bs) + shape + (torch.empty(0, dtype=dtype).element_size(),), generator=g, dtype=torch.uint8)
        out.append(x.view(dtype).squeeze(-1))
    return out


@pytest.mark.parametrize("B,W,K,bs,MB", [(1, 1, 1, 16, 3), (2, 4, 4, 16, 6), (3, 1, 8, 4, 5), (2, 8, 3, 1, 7), (4, 4, 4, 5, 9),
                                         (1, 32, 32, 16, 4), (2, 31, 32, 3, 6)])
def test_reorder_shapes(B, W, K, bs, MB):
    for seed in range(4):
        g = torch.Generator().manual_seed(seed)
        n = int(torch.randint(0, (MB - 1) * bs + 1, (1,), generator=g))
        lens = [[n] * W for _ in range(B)]
        tables, owned, parents, nb = reorder_case(B, W, K, bs, MB, lens, seed)
        pools = pools_of(nb, bs, [((2, 8), torch.bfloat16), ((2, 8), torch.bfloat16), ((3,), torch.int8), ((5,), torch.float32)], seed)
        blocks = pools_of(nb, 2, [((bs,), torch.float32), ((3,), torch.uint8)], seed + 1)
        finished = (torch.rand(B, K, generator=g) < 0.3).to(torch.uint8)
        check_reorder(tables, lens, parents, owned, finished if seed % 2 else None, bs, nb, pools, blocks)


def test_reorder_ragged_lengths():
    """Beams that ended earlier, children that are not used, all from one parent."""
    bs, MB, W, K = 4, 8, 5, 6
    for seed in range(8):
        g = torch.Generator().manual_seed(50 + seed)
        top = int(torch.randint(5, MB * bs - 4, (1,), generator=g))
        lens = [[top if i % 2 == 0 else int(torch.randint(1, top + 1, (1,), generator=g)) for i in range(W)] for _ in range(2)]
        # a column of a shorter beam's own: distinct blocks for all beams in every column that is some beam's last
        tables, owned, parents, nb = reorder_case(2, W, K, bs, MB, [[min(r)] * W for r in lens], seed)
        parents[0, 2] = -1
        if seed == 3:
            parents[1] = 1
        if seed == 4:
            parents[:] = -1
        pools = pools_of(nb, bs, [((16,), torch.bfloat16)], seed)
        check_reorder(tables, lens, parents, owned, None, bs, nb, pools, [])


def test_reorder_pool_alignments():
    """Pools that start anywhere and whose rows have any size."""
    bs, MB, W, K = 16, 4, 4, 4
    lens = [[37] * W]
    tables, owned, parents, nb = reorder_case(1, W, K, bs, MB, lens, 3, parents=torch.tensor([[1, 1, 1, 3]]))
    for row in (1, 2, 3, 7, 16, 24, 1000):
        for shift in (0, 1, 4, 8):
            buf = torch.randint(0, 256, (shift + nb * bs * row,), dtype=torch.uint8)
            pool = buf.to(DEV)[shift:].view(nb, bs, row)
            want = pool.clone()
            out = [torch.zeros(1, K, MB, dtype=I32, device=DEV), torch.zeros(1, K, dtype=I32, device=DEV),
                   torch.zeros(1, K, dtype=torch.int64, device=DEV)]
            pkv.pkv_beam_reorder(*out, tables.to(DEV), torch.tensor(lens, dtype=I32, device=DEV), parents.to(DEV), owned.to(DEV),
                                 bs, pools=[pool])
            for src, dst, rows in ref.beam_reorder(tables[0].tolist(), lens[0], parents[0].tolist(), owned[0].tolist(), None, bs)[3]:
                want[dst, :rows] = want[src, :rows]
            assert torch.equal(pool, want), (row, shift)


def test_reorder_flags():
    bs, MB, W, K = 4, 3, 3, 3
    def go(tables, lens, parents, owned, nb=100):
        out = [torch.full((1, K, MB), -7, dtype=I32, device=DEV), torch.full((1, K), -7, dtype=I32, device=DEV),
               torch.full((1, K), -7, dtype=torch.int64, device=DEV)]
        err = torch.zeros(1, dtype=I32, device=DEV)
        pool = torch.arange(100 * bs, dtype=I32, device=DEV).view(100, bs)[:nb].contiguous()
        before = pool.clone()
        t = lambda x: torch.tensor(x, dtype=I32, device=DEV)
        pkv.pkv_beam_reorder(*out, t([tables]), t([lens]), t([parents]), t([owned]), bs, pools=[pool], err_flags=err)
        return out[0][0].tolist(), out[1][0].tolist(), out[2][0].tolist(), int(err), torch.equal(pool, before)
    tables = [[1, 2, 3], [1, 12, 13], [1, 22, 23]]
    owned = [[1, 2, 3], [1, 12, 13], [1, 22, 23]]
    # parents and lengths that cannot be
    t, n, s, f, same = go(tables, [5, 5, -1], [0, 3, 2], owned)
    assert f == pkv.FLAG_BEAM and same and n == [6, 0, 0] and s == [2 * bs + 1, -1, -1] and t[1] == owned[1] and t[2] == owned[2]
    t, n, s, f, same = go(tables, [5, 13, 5], [-2, 1, 0], owned)
    assert f == pkv.FLAG_BEAM and n == [0, 0, 6] and s == [-1, -1, 9]
    # no room for a token
    t, n, s, f, same = go(tables, [12, 5, 5], [0, 0, 1], owned)
    assert f == pkv.FLAG_CONTEXT_TOO_LONG and n == [12, 12, 6] and s == [-1, -1, 49] and t[0] == tables[0] and t[1] == tables[0]
    # a block outside the pool, as the next token's and as a copy's source
    t, n, s, f, same = go([[1, 2, 3], [1, 999, 13], [1, 22, 23]], [5, 5, 5], [0, 1, 1], owned)
    assert f == pkv.FLAG_BLOCK_OUT_OF_RANGE and same and n == [6, 5, 5] and s == [9, -1, -1]
    t, n, s, f, same = go(tables, [5, 5, 5], [0, 0, 2], [[1, 2, 3], [1, -5, 13], [1, 22, 23]])
    assert f == pkv.FLAG_BLOCK_OUT_OF_RANGE and same and n == [6, 5, 6] and s == [9, -1, 89]
    # a request that has no block left
    t, n, s, f, same = go(tables, [5, 5, 5], [0, 0, 0], [[1, 2, 3]] * 3)
    assert f == pkv.FLAG_OUT_OF_BLOCKS and same and n == [6, 5, 5] and s == [9, -1, -1] and t[1] == [1, 2, 3]


def from_largest(logits, scores, K):
    """The selection from differences to each row's largest logit, in 64 bits:
    exact for logits of any size.  Every beam in use, none ended."""
    B, W, V = logits.shape
    x = logits.double()
    d = x - x.amax(2, keepdim=True)
    s = (scores.double()[..., None] + (d - d.exp().sum(2, keepdim=True).log())).flatten(1)
    # best first, of equal ones the lowest (beam, token)
    best, at = s.sort(dim=1, descending=True, stable=True)
    return best[:, :K], (at[:, :K] // V).to(I32), (at[:, :K] % V).to(I32)


def check_from_largest(x, c, K, apart=None):
    got = select(x, c, None, K)
    s, p, t = from_largest(x, c, K)
    if apart:
        s1, p1, _ = from_largest(x, c, K + 1)
        gap = (s1[:, :-1] - s1[:, 1:])[p1[:, :-1] != p1[:, 1:]]
        assert (gap > apart).all(), "beams too near"
    assert torch.equal(got[1], p) and torch.equal(got[2], t), (got[1], p, got[2], t)
    assert ((got[0].double() - s).abs() <= (s.abs() + 20) * 2.0 ** -22).all(), (got[0], s)


LEVELS = [(torch.float32, v) for v in (-6e4, -7e4, -3e8, -1e9, -1e10, -1e12, -1e30, -3.4e38, 1e6, 3e9, 5e9, 1e20, 3.4e38)] + [
    (torch.bfloat16, v) for v in (-1e9, -1e10, -1e12, -1e30, -3.38e38, 3e9, 1e20, 3.38e38)] + [(torch.float16, v) for v in (-65504.0, -3e4, 65504.0)]


@pytest.mark.parametrize("dtype,level", LEVELS)
@pytest.mark.parametrize("V", [50, 5000, 40001])
def test_select_rows_at_one_level(dtype, level, V):
    """A row that is masked throughout with a finite number is an even
    distribution, whatever the number: beside live beams, and alone; and live
    rows whose masked tokens have that number."""
    x = logits_of(3, 4, V, dtype, V + 1)
    c = torch.tensor([[-0.5, -1.0, -1.75, -2.5]]).expand(3, 4).contiguous()
    x[0, 0] = x[0, 2] = level
    x[1] = level
    if level < 0:
        x[2, :, 20:] = level                                   # (whole pieces among them)
        x[2, 1, :30] = level                                   # a live beam among masked ones, and a dead one
    check_from_largest(x, c, 6, apart=1e-5)


@pytest.mark.parametrize("offset", [3e4, 6.4e4, 6.6e4, 1e5, 1e6, 2e7])
@pytest.mark.parametrize("sign", [1, -1])
def test_select_far_logits(offset, sign):
    """Logits far from 0 that differ by little: a row is what it is without the offset."""
    B, W, V = 2, 3, 9001
    unit = 2.0 ** (math.floor(math.log2(offset)) - 23)
    g = torch.Generator().manual_seed(int(offset))
    d = (torch.randn(B, W, V, generator=g).double() * 3 / unit).round() * unit
    x = (sign * math.floor(offset / unit) * unit + d).float()
    assert torch.equal(x.double() - sign * math.floor(offset / unit) * unit, d) or offset > 1e6
    check_from_largest(x, torch.tensor([[-1.0, -1.3, -1.7], [-2.0, -0.1, -0.6]]), 8, apart=1e-6)


def test_select_workspace_of_a_larger_batch():
    """Requests finish: ten, then four, one, with the first's workspace."""
    ws = pkv.BeamSelectWorkspace(10, 4, 4, 128256)
    for B in (10, 4, 1, 10):
        check_select(logits_of(B, 4, 128256, torch.float32, B), scores_of(B, 4, B), None, 4, ws=ws)
