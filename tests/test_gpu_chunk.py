"""pkv_chunk_attention on the GPU against its 64-bit restatement.

Tolerance.  Products of 16-bit inputs are exact in fp32 and summed in fp32;
the weights are rounded to the input type before the second product (relative
eps / 2 each), the result once (eps / 2).  An output is a mean of values with
weights w that sum to 1, so rounding the weights moves it by at most
eps / 2 * sum(w |v|) <= eps / 2 * max|v|, and the output's rounding by
eps / 2 * |o|.  Scores t (log2 units, |t| <= 64 here) carry a few fp32
roundings: 2^-20 covers their effect on a weight.  Hence
|got - want| <= (eps + 2^-18) * max|v| over the values, |o| <= max|v|;
for fp32, where sums run over up to a few thousand terms, 2^-17 * max|v|."""
import math

import pytest
import torch

import paged_kv_cache_67_gb300 as pkv
from step_reference import chunk

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def case(seed, lens, qlens, H, KVH, D, bs, dtype, gain=2.0, poison=True, room=1100):
    """Shuffled blocks, garbage tails (tables of `room` keys or more: small calls,
    up to 1024, may run on another kernel), NaN in every cache row behind a
    context."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // bs) for n in lens]
    nb = sum(need) + 3
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    tables = torch.full((len(lens), max(need + [1, -(-room // bs)]) + 2), 99999, dtype=torch.int32)
    k = torch.randn(nb, bs, KVH, D, generator=g).to(dtype)
    v = torch.randn(nb, bs, KVH, D, generator=g).to(dtype)
    at, used = 0, torch.zeros(nb, bs, dtype=torch.bool)
    for b, n in enumerate(lens):
        tables[b, :need[b]] = perm[at:at + need[b]]
        for t in range(0, n, bs):
            used[int(perm[at + t // bs]), :min(bs, n - t)] = True
        at += need[b]
    if poison:
        k[~used] = float("nan")
        v[~used] = float("nan")
    cu = torch.tensor([0] + qlens).cumsum(0).to(torch.int32)
    q = (torch.randn(int(cu[-1]), H, D, generator=g) * gain).to(dtype)
    return dict(q=q, k=k, v=v, tables=tables, cu=cu, lens=torch.tensor(lens, dtype=torch.int32), scale=1.0 / math.sqrt(D))


def run(c, max_q_len=0, max_context_len=0, partition_size=0, ws=None, stream=None, out=None, **form):
    d = lambda t: None if t is None else t.to(DEV)
    q = d(c["q"])
    total, H, D = q.shape
    B, MB = c["tables"].shape
    _, bs, KVH, _ = c["k"].shape
    if out is None:
        out = torch.full_like(q, 7.0)
    if ws is None:
        ws = pkv.ChunkWorkspace(B, total, H, KVH, D, bs, MB, max_q_len, max_context_len, partition_size)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.pkv_chunk_attention(out, q, d(c["k"]), d(c["v"]), d(c["tables"]), d(c["cu"]), d(c["lens"]), c["scale"],
                            max_q_len=max_q_len, max_context_len=max_context_len, partition_size=partition_size,
                            workspace=ws, err_flags=err, stream=stream, **{k: d(v) if torch.is_tensor(v) else v for k, v in form.items()})
    torch.cuda.synchronize()
    assert not ws.buffer[:65536 * 4].any(), "counters are zero between calls"
    return out.cpu(), int(err)


def reference(c, softcap=0.0, window=0, slopes=None, prefix_lens=None, kv_starts=None):
    return chunk(c["q"], c["k"], c["v"], c["tables"], c["cu"], c["lens"], c["scale"], softcap, window, slopes, prefix_lens, kv_starts)


def close(got, want, c, what=""):
    dt = c["q"].dtype
    vmax = c["v"].double().abs().nan_to_num(0.0, 0.0, 0.0).max()
    tol = (2.0 ** -17 if dt == F32 else torch.finfo(dt).eps + 2.0 ** -18) * vmax
    assert torch.equal(got.isnan(), want.isnan()), f"{what}: NaN at other places"
    off = (got.double() - want).abs().nan_to_num(0.0)
    assert off.max() <= tol, f"{what}: {off.max().item():.3e} > {tol.item():.3e} at {(off == off.max()).nonzero()[0].tolist()}"


def slopes_of(H):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)])


def forms(c, seed=0):
    """Every score form, and all of them at once."""
    g = torch.Generator().manual_seed(seed)
    H, total, B = c["q"].shape[1], c["q"].shape[0], len(c["lens"])
    n = int(c["lens"].max()) if B else 1
    starts = torch.zeros(total, dtype=torch.int32)
    for b in range(B):
        r0, r1 = int(c["cu"][b]), int(c["cu"][b + 1])
        p = torch.arange(int(c["lens"][b]) - (r1 - r0), int(c["lens"][b]))
        size = int(torch.randint(1, max(2, int(c["lens"][b])), (1,), generator=g))
        starts[r0:r1] = (p // size * size).to(torch.int32)
    prefix = torch.randint(0, n + 2, (B,), generator=g, dtype=torch.int32)
    return [{}, {"softcap": 15.0}, {"slopes": slopes_of(H)}, {"window": 1}, {"window": max(1, n // 3)},
            {"prefix_lens": prefix}, {"kv_starts": starts},
            {"softcap": 4.0, "slopes": slopes_of(H), "window": max(1, n // 2), "prefix_lens": prefix, "kv_starts": starts}]


def check(c, what="", partition_size=0, **form):
    got, err = run(c, partition_size=partition_size, **form)
    assert err == 0, f"{what}: flags {err:#x}"
    close(got, reference(c, **form), c, what)


# (dtype, H, KVH, D, block size): each kernel, grouped heads, odd sizes
SHAPES = [(F32, 4, 2, 64, 16), (F32, 7, 1, 80, 5), (F32, 2, 2, 130, 1), (F32, 3, 3, 512, 16), (BF, 5, 1, 72, 16),
          (HF, 4, 2, 64, 24), (BF, 8, 2, 64, 16), (BF, 8, 2, 128, 16), (HF, 4, 1, 128, 32), (BF, 7, 1, 128, 16),
          (HF, 6, 2, 64, 64), (BF, 12, 1, 128, 16), (HF, 4, 4, 192, 16), (BF, 8, 1, 256, 32), (HF, 16, 1, 256, 16),
          (BF, 32, 1, 64, 16), (BF, 40, 2, 128, 16)]


@pytest.mark.parametrize("dtype,H,KVH,D,bs", SHAPES)
def test_decode_forms(dtype, H, KVH, D, bs):
    c = case(D + H, [1, 2, 15, 16, 17, 100, 127, 129, 300], [1] * 9, H, KVH, D, bs, dtype)
    for f in forms(c, 1):
        check(c, f"{sorted(f)}", **f)
        check(c, f"{sorted(f)} split", partition_size=128, **f)


@pytest.mark.parametrize("room", [1, 1100])
@pytest.mark.parametrize("dtype,H,KVH,D,bs", SHAPES)
def test_chunk_forms(dtype, H, KVH, D, bs, room):
    c = case(D * 3 + H, [1, 40, 33, 200, 129, 260], [1, 3, 33, 150, 64, 17], H, KVH, D, bs, dtype, room=room)
    for f in forms(c, 2):
        check(c, f"{sorted(f)}", **f)
        check(c, f"{sorted(f)} split", partition_size=128, **f)


@pytest.mark.parametrize("dtype,H,KVH,D,bs", [(BF, 8, 2, 128, 16), (HF, 4, 4, 64, 16), (BF, 6, 1, 192, 32), (HF, 8, 1, 256, 16),
                                              (BF, 7, 1, 128, 16)])
def test_small_chunks_stay_on_mma(dtype, H, KVH, D, bs):
    """Small calls with many 16-row chunks, more chunks of keys than ring stages, whole and split."""
    c = case(D * 5 + H, [1, 70, 900], [1, 33, 70], H, KVH, D, bs, dtype, room=1)
    total, kw = int(c["cu"][-1]), dict(max_q_len=70, max_context_len=900)
    assert pkv.pkv_chunk_plan(3, total, H, KVH, D, bs, c["tables"].shape[1], 70, 900, dtype=dtype)[2] == 1
    for f in forms(c, 5):
        want = reference(c, **f)
        for part in (0, 128, 1024):
            got, err = run(c, partition_size=part, **kw, **f)
            assert err == 0, f"{sorted(f)} {part}: flags {err:#x}"
            close(got, want, c, f"{sorted(f)} {part}")
            again, _ = run(c, partition_size=part, **kw, **f)
            assert torch.equal(got.view(torch.int16), again.view(torch.int16)), f"{sorted(f)} {part}: bits differ"


def test_each_kernel_is_reached():
    """The plan's kernel by rows, type, shape and the call's size."""
    plan = lambda *a, **k: pkv.pkv_chunk_plan(*a, **k)[2]
    assert plan(4, 4, 8, 2, 128, 16, 200) == 1 and plan(4, 400, 8, 2, 128, 16, 200) == 2
    assert plan(4, 400, 8, 2, 256, 16, 200) == 2 and plan(2, 40, 8, 2, 128, 16, 64, 20) == 1
    assert plan(64, 6400, 8, 2, 128, 16, 64, 100) == 2
    assert plan(4, 400, 8, 2, 128, 8, 200) == 0 and plan(4, 400, 8, 2, 128, 16, 200, dtype=F32) == 0


@pytest.mark.parametrize("dtype,H,KVH,D", [(BF, 8, 2, 128), (BF, 4, 4, 64), (HF, 8, 1, 256), (F32, 4, 2, 64)])
def test_drafts_over_long_contexts_split_automatically(dtype, H, KVH, D):
    lens = [5000, 130, 3001]
    c = case(D, lens, [4, 2, 7], H, KVH, D, 16, dtype)
    assert pkv.pkv_chunk_plan(3, 13, H, KVH, D, 16, c["tables"].shape[1], 0, 0, 0, False, 0, dtype)[1] > 1
    for f in ({"softcap": 20.0}, {"slopes": slopes_of(H)}, {"window": 700}):
        check(c, f"{sorted(f)}", **f)


@pytest.mark.parametrize("dtype,H,KVH,D", [(BF, 4, 2, 128), (HF, 2, 2, 64), (BF, 3, 1, 128)])
def test_long_chunks(dtype, H, KVH, D):
    """Many row tiles and keys per tile edge: whole prompts and chunks on a prefix."""
    c = case(D + 1, [900, 1300, 513], [900, 257, 512], H, KVH, D, 16, dtype)
    for f in forms(c, 3):
        check(c, f"{sorted(f)}", **f)


@pytest.mark.parametrize("dtype,H,KVH,D", [(HF, 2, 2, 192), (BF, 4, 1, 256)])
def test_long_chunks_wide_heads(dtype, H, KVH, D):
    """One row tile an item: several items and key tiles, split and whole."""
    c = case(D + 2, [700, 400, 129], [300, 257, 129], H, KVH, D, 16, dtype)
    for f in forms(c, 4):
        check(c, f"{sorted(f)}", **f)
    check(c, "split", partition_size=128, softcap=15.0)


@pytest.mark.parametrize("H,KVH,D", [(128, 1, 64), (96, 1, 128), (24, 2, 64), (66, 1, 64)])
def test_large_and_odd_groups(H, KVH, D):
    """Up to 128 heads packed in a tile; groups with an odd factor pack fewer."""
    c = case(H, [40, 150, 17], [5, 9, 2], H, KVH, D, 16, BF)
    for f in ({}, {"softcap": 9.0, "window": 50}, {"slopes": slopes_of(H)}):
        check(c, f"{sorted(f)}", **f)
        check(c, f"{sorted(f)} split", partition_size=128, **f)


@pytest.mark.parametrize("bs", [32, 48, 64, 80, 256])
def test_block_sizes(bs):
    for dtype, D, q in ((BF, 128, [3, 1]), (BF, 64, [100, 40]), (HF, 256, [90, 3]), (F32, 64, [40, 3])):
        c = case(bs + D, [333, 500], q, 4, 2, D, bs, dtype)
        check(c, f"{bs} {D}", softcap=12.0, window=170)


@pytest.mark.parametrize("B", [1023, 1100, 2500])
def test_many_sequences(B):
    """More sequences than one scan of the plan covers, and just fewer."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(1, 40, (B,), generator=g).tolist()
    qlens = [min(n, int(torch.randint(0, 12, (1,), generator=g))) for n in lens]
    qlens[5] = lens[5] = 35
    c = case(B, lens, qlens, 4, 2, 64, 16, BF)
    assert pkv.pkv_chunk_plan(B, sum(qlens), 4, 2, 64, 16, c["tables"].shape[1], 35)[2] == 2
    got, err = run(c, max_q_len=35, softcap=9.0)
    assert err == 0
    close(got, reference(c, softcap=9.0), c)


def test_scale_signs():
    """Negative and zero scales, with and without a cap and a bias."""
    for dtype, D, q in ((BF, 128, [3, 2]), (BF, 64, [70, 100]), (HF, 256, [60, 2]), (F32, 64, [3, 50])):
        c = case(31, [200, 300], q, 4, 2, D, 16, dtype)
        for scale in (-0.1, 0.0, 1e-7):
            c["scale"] = scale
            for f in ({}, {"softcap": 8.0}, {"slopes": -slopes_of(4), "window": 90}):
                check(c, f"{scale} {sorted(f)}", **f)


def test_query_offsets_that_overlap():
    """Offsets that go back and forth are flagged; sequences that are fine
    stay right, and nothing outside is touched."""
    for D in (64, 128, 256):
        c = case(33, [60, 60, 60, 60], [50, 50, 50, 50], 4, 2, D, 16, BF)
        want = reference(c)
        c["cu"] = torch.tensor([0, 50, 10, 200, 190], dtype=torch.int32)    # lengths 50, -40, 190, -10
        got, err = run(c)
        assert err & pkv.FLAG_QUERY_LEN
        close(got[:50], want[:50], c)


def test_large_scores_and_cap():
    """Scores far past the cap: tanh saturates, the softmax stays exact."""
    for dtype, D in ((BF, 128), (F32, 64), (HF, 256)):
        c = case(7, [300, 64], [20, 1], 4, 2, D, 16, dtype, gain=12.0)
        for cap in (1.0, 8.0, 30.0):
            check(c, f"cap {cap}", softcap=cap)


@pytest.mark.parametrize("dtype,H,KVH,D", [(HF, 4, 2, 128), (BF, 4, 2, 64), (HF, 4, 1, 256), (HF, 4, 2, 80), (F32, 4, 2, 64)])
@pytest.mark.parametrize("cap", [400.0, 1e3, 1e5, 1e8, 3e38])
def test_caps_far_above_the_scores(dtype, H, KVH, D, cap):
    """A cap that hardly bends the scores leaves them exact, on every kernel:
    its error goes with the score, not with the cap."""
    for qlens in ([3, 5], [100, 90]):
        c = case(51, [260, 400], qlens, H, KVH, D, 16, dtype)
        for f in ({}, {"slopes": slopes_of(H)}):
            check(c, f"{qlens} {sorted(f)}", softcap=cap, **f)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("cap", [300.0, 1000.0])
def test_caps_that_bend_scores_of_hundreds(D, cap):
    """Scores from 0 to 1.2 of a large cap.  The products are exact here (one
    element of q is not 0), so a score t carries the roundings of its cap form
    alone: 8 at most, 2^-24 each, of |t| <= cap log2(e).  A weight is off by
    that of its score and of the row's largest:
    2 ln 2 * 8 * 2^-24 * cap log2(e) = 2^-20 cap, beside what the module's text
    counts."""
    for qlens in ([3, 5], [100, 90]):
        c = case(52, [260, 400], qlens, 4, 2, D, 16, HF)
        g = torch.Generator().manual_seed(53)
        c["q"].zero_()
        rows = c["q"].view(-1, D)
        rows[torch.arange(len(rows)), torch.randint(0, D, (len(rows),), generator=g)] = 8.0
        c["k"] = torch.where(c["k"].isnan(), c["k"], (torch.randint(0, 1001, c["k"].shape, generator=g) / 4).to(HF))
        c["scale"] = 1.2 * cap / 2000
        got, err = run(c, softcap=cap)
        want = reference(c, softcap=cap)
        vmax = c["v"].double().abs().nan_to_num(0.0, 0.0, 0.0).max()
        tol = (torch.finfo(HF).eps + 2.0 ** -18 + 2.0 ** -20 * cap) * vmax
        assert err == 0 and (got.double() - want).abs().max() <= tol, f"{qlens}: {(got.double() - want).abs().max():.3e}"


def test_equal_scores_average_the_values():
    """q = 0: every visible key weighs the same, with and without a cap."""
    c = case(8, [77, 500], [5, 130], 4, 2, 128, 16, BF)
    c["q"].zero_()
    check(c, "zero")
    check(c, "zero, capped", softcap=3.0)
    check(c, "zero, window", window=64)


@pytest.mark.parametrize("dtype,H,KVH,D", [(F32, 4, 2, 64), (BF, 4, 2, 128), (HF, 16, 1, 256), (BF, 4, 1, 64)])
@pytest.mark.parametrize("qlen", [1, 3, 70])
def test_rows_that_see_nothing_are_zero(dtype, H, KVH, D, qlen):
    """Starts behind the query's position: zeros, next to rows that see keys."""
    c = case(9, [90, 300], [qlen, qlen], H, KVH, D, 16, dtype)
    starts = torch.zeros(2 * qlen, dtype=torch.int32)
    starts[::2] = 1000
    for part in (0, 128):
        got, err = run(c, kv_starts=starts, partition_size=part)
        assert err == 0 and not got[::2].any()
        close(got, reference(c, kv_starts=starts), c)
        starts_all = torch.full_like(starts, 2 ** 31 - 1)
        got, err = run(c, kv_starts=starts_all, partition_size=part)
        assert err == 0 and not got.any()


@pytest.mark.parametrize("dtype,H,KVH,D", [(F32, 4, 2, 64), (F32, 4, 2, 512), (BF, 4, 2, 80), (BF, 4, 2, 128), (HF, 16, 1, 256), (BF, 4, 1, 64)])
@pytest.mark.parametrize("qlen", [1, 6, 70])
def test_a_sequence_that_sees_nothing_reads_no_table(dtype, H, KVH, D, qlen):
    """Every table entry is garbage: none is looked at where no query sees a key."""
    c = case(54, [90, 300], [qlen, qlen], H, KVH, D, 16, dtype)
    c["tables"].fill_(99999)
    for start in (1000, 2 ** 31 - 1):
        for part in (0, 128):
            got, err = run(c, kv_starts=torch.full((2 * qlen,), start, dtype=torch.int32), partition_size=part)
            assert err == 0 and not got.any()


@pytest.mark.parametrize("dtype,H,KVH,D", [(F32, 4, 2, 64), (BF, 4, 2, 128), (HF, 16, 1, 256), (BF, 4, 1, 64)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("qlen", [1, 6, 150])
def test_what_a_row_does_not_see_never_reaches_it(dtype, H, KVH, D, bad, qlen):
    """Non-finite keys and values behind a window, in another document or at a
    later position leave every row that does not see them as it was."""
    c = case(10, [260, 400], [qlen, qlen], H, KVH, D, 16, dtype)
    form = {"window": 100, "kv_starts": torch.randint(0, 300, (2 * qlen,), generator=torch.Generator().manual_seed(1), dtype=torch.int32)}
    clean = reference(c, **form)
    for b, n in enumerate((260, 400)):
        for t in (0, 37, n - 140, n - 3, n - 1):
            blk = int(c["tables"][b, t // 16])
            c["k"][blk, t % 16] = bad
            c["v"][blk, t % 16] = bad
    want = reference(c, **form)
    got, err = run(c, **form)
    assert err == 0
    untouched = want.isfinite().all(-1) & (want == clean).all(-1)
    assert untouched.any() or qlen == 1
    g, w = got[untouched], want[untouched]
    vmax = c["v"].double().abs().nan_to_num(0.0, 0.0, 0.0).max()
    tol = (2.0 ** -17 if dtype == F32 else torch.finfo(dtype).eps + 2.0 ** -18) * vmax
    assert (g.double() - w).abs().max() <= tol if g.numel() else True
    # rows that do see one are not finite either
    assert not got[~untouched].isfinite().all(-1).any() if (~untouched).any() and bad != float("-inf") else True


@pytest.mark.parametrize("D,n", [(64, 100_000), (128, 100_000), (256, 40_000)])
@pytest.mark.parametrize("parts", [1, 3])
def test_an_infinity_holds_nobody_up(D, n, parts):
    """The last key of a long sequence has an infinite value: its 255 queries
    that do not see it are done again, over all of their keys, while nothing
    else waits -- no time limit runs out, and another sequence's items, behind
    on the same SM, come out as without it."""
    units, per = 160, 256 if D <= 128 else 128
    g = torch.Generator(device=DEV).manual_seed(D)
    nb = -(-n // 16) + units * per // 16
    k, v = (torch.randn(nb, 16, 1, D, generator=g, device=DEV).to(HF) for _ in range(2))
    q = torch.randn(256 + units * per, 1, D, generator=g, device=DEV).to(HF)
    first = -(-n // 16)
    tables = torch.zeros(2, first + units * per // 16, dtype=torch.int32, device=DEV)
    tables[0, :first] = torch.arange(first, device=DEV)
    tables[1, :units * per // 16] = torch.arange(first, nb, device=DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    cu, lens, err = i32([0, 256, 256 + units * per]), i32([n, units * per]), i32([0])
    part = -(-(-(-n // parts)) // 128) * 128
    ws = pkv.ChunkWorkspace(2, len(q), 1, 1, D, 16, tables.shape[1], units * per, n, part)
    assert pkv.pkv_chunk_plan(2, len(q), 1, 1, D, 16, tables.shape[1], units * per, n, partition_size=part, dtype=HF)[1:] == (parts, 2)
    scale, outs = 1 / math.sqrt(D), []
    for value in (None, float("inf")):
        if value is not None:
            v[(n - 1) // 16, (n - 1) % 16] = value
        out = torch.zeros_like(q)
        pkv.pkv_chunk_attention(out, q, k, v, tables, cu, lens, scale, max_q_len=units * per, max_context_len=n,
                                partition_size=part, workspace=ws, err_flags=err)
        torch.cuda.synchronize()
        assert int(err) == 0
        outs.append(out.cpu())
    assert torch.equal(outs[1][256:], outs[0][256:])
    assert not outs[1][255].isfinite().any()
    keys, vals = k.view(-1, D)[:n - 1].cpu().double(), v.view(-1, D)[:n - 1].cpu().double()
    for i in range(0, 255, 23):
        x = q[i, 0].cpu().double() @ keys[:n - 256 + i + 1].T * scale
        want = torch.softmax(x, 0) @ vals[:n - 256 + i + 1]
        tol = (torch.finfo(HF).eps + 2.0 ** -18) * vals.abs().max()
        assert (outs[1][i, 0].double() - want).abs().max() <= tol
    assert (outs[1][:255].double() - outs[0][:255].double()).abs().max() <= 2 * tol


def test_blocks_outside_the_window_are_not_read():
    """Freed blocks' table entries may be garbage once no query sees them."""
    for dtype, D in ((BF, 128), (F32, 64), (HF, 256)):
        c = case(11, [500, 333], [4, 40], 4, 2, D, 16, dtype)
        want = reference(c, window=64)
        for b, (n, q) in enumerate(((500, 4), (333, 40))):
            first = max(0, n - q - 64 + 1) // 16
            c["tables"][b, :first] = torch.tensor([-5, 123456] * 40, dtype=torch.int32)[:first]
        got, err = run(c, window=64)
        assert err == 0
        close(got, want, c)


def test_prefix_mask_sees_ahead():
    """Whole prompts whose first tokens see one another (an image, a prefix)."""
    for dtype, H, KVH, D in ((BF, 4, 2, 128), (F32, 2, 1, 64), (HF, 4, 1, 256)):
        c = case(12, [300, 70, 140], [300, 70, 5], H, KVH, D, 16, dtype)
        for prefix in ([0, 0, 0], [150, 70, 140], [10 ** 9, -4, 139]):
            pl = torch.tensor(prefix, dtype=torch.int32)
            check(c, f"{prefix}", prefix_lens=pl)
            check(c, f"{prefix} window", prefix_lens=pl, window=33, slopes=slopes_of(H))


def test_rows_behind_the_last_sequence_and_padding():
    """Padded requests (no queries, no context) and rows behind cu[B]."""
    for dtype, D in ((BF, 128), (F32, 64), (BF, 256)):
        c = case(13, [50, 0, 200, 0], [3, 0, 90, 0], 4, 2, D, 16, dtype)
        c["q"] = torch.cat([c["q"], torch.full((5, 4, D), float("nan"), dtype=dtype)])
        got, err = run(c, softcap=9.0)
        assert err == 0 and (got[93:] == 7).all()
        close(got[:93], reference(c, softcap=9.0)[:93], c)
        got, err = run(c, softcap=9.0, max_q_len=90, max_context_len=200)
        assert err == 0
        close(got[:93], reference(c, softcap=9.0)[:93], c)


def test_flags():
    for dtype, D in ((BF, 128), (F32, 64), (HF, 256)):
        c = case(14, [50, 200], [3, 90], 4, 2, D, 16, dtype)
        want = reference(c)
        good = {**c, "lens": torch.tensor([2, 200], dtype=torch.int32)}     # fewer tokens than queries
        got, err = run(good)
        assert err == pkv.FLAG_QUERY_LEN
        close(got[3:], want[3:], c)
        got, err = run({**c, "lens": torch.tensor([50, 10 ** 6], dtype=torch.int32)})
        assert err == pkv.FLAG_QUERY_LEN
        close(got[:3], want[:3], c)
        got, err = run(c, max_q_len=80)
        assert err == pkv.FLAG_QUERY_OVER_HINT
        close(got[:3], want[:3], c)
        got, err = run(c, max_context_len=150)
        assert err == pkv.FLAG_CONTEXT_OVER_HINT
        close(got[:3], want[:3], c)
        t = c["tables"].clone()
        t[0, 1] = 10 ** 6
        got, err = run({**c, "tables": t})
        assert err == pkv.FLAG_BLOCK_OUT_OF_RANGE
        close(got[3:], want[3:], c)


def test_plain_form_agrees_with_decode_and_prefill():
    """Without any score form: decode and causal prefill, as offered already."""
    c = case(15, [300, 17, 129], [1, 1, 1], 8, 2, 128, 16, BF, poison=False)
    d = lambda t: t.to(DEV)
    got, _ = run(c)
    out = torch.empty_like(d(c["q"]))
    ws = pkv.DecodeWorkspace(3, 8, 2, 128, 16, c["tables"].shape[1])
    pkv.pkv_decode_attention(out, d(c["q"]), d(c["k"]), d(c["v"]), d(c["tables"]), d(c["lens"]), c["scale"], workspace=ws)
    close(got, out.cpu().double(), c)
    c = case(16, [300, 17, 129], [300, 5, 129], 8, 2, 128, 16, BF, poison=False)
    got, _ = run(c)
    out = torch.empty_like(d(c["q"]))
    pkv.pkv_prefill_attention(out, d(c["q"]), d(c["k"]), d(c["v"]), d(c["tables"]), d(c["cu"]), d(c["lens"]), c["scale"])
    close(got, out.cpu().double(), c)


def test_one_workspace_for_calls_of_different_shapes():
    """A workspace sized for the largest of a loop's shapes serves them all."""
    cs = [case(17, [3000, 900], [2, 1], 8, 2, 128, 16, BF), case(18, [400] * 3, [100, 1, 64], 8, 2, 128, 16, BF),
          case(19, [2000], [5], 16, 1, 256, 16, HF), case(20, [700, 5], [1, 1], 4, 2, 64, 16, F32)]
    big = max((pkv.ChunkWorkspace(len(c["lens"]), c["q"].shape[0], c["q"].shape[1], c["k"].shape[2], c["q"].shape[2], 16,
                                  c["tables"].shape[1], 0, 0, 128) for c in cs), key=lambda w: w.nbytes)
    for _ in range(2):
        for c in cs:
            got, err = run(c, ws=big, partition_size=128, softcap=20.0)
            assert err == 0
            close(got, reference(c, softcap=20.0), c)


def test_streams_and_graphs():
    """Two streams with workspaces of their own, and a captured call replayed
    with other inputs and lengths."""
    c = case(21, [2500, 700], [3, 4], 8, 2, 128, 16, BF)
    want = reference(c, softcap=20.0)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got, err = run(c, softcap=20.0, stream=s)
    assert err == 0
    close(got, want, c)
    for qlens, maxq in (([3, 4], 8), ([100, 90], 128)):
        c = case(22, [2500, 700], qlens, 8, 2, 128, 16, BF)
        d = {k: c[k].to(DEV) for k in ("q", "k", "v", "tables", "cu", "lens")}
        out = torch.zeros_like(d["q"])
        ws = pkv.ChunkWorkspace(2, out.shape[0], 8, 2, 128, 16, d["tables"].shape[1], maxq)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            pkv.pkv_chunk_attention(out, d["q"], d["k"], d["v"], d["tables"], d["cu"], d["lens"], c["scale"], softcap=20.0,
                                    max_q_len=maxq, workspace=ws, err_flags=err, stream=s)
        for lens in ([2500, 700], [900, 120]):
            c["lens"] = torch.tensor(lens, dtype=torch.int32)
            d["lens"].copy_(c["lens"])
            out.fill_(7.0)
            g.replay()
            torch.cuda.synchronize()
            assert int(err) == 0
            close(out.cpu(), reference(c, softcap=20.0), c, f"{lens}")


@pytest.mark.parametrize("dtype,D", [(BF, 128), (F32, 64), (HF, 256), (BF, 80)])
def test_blocks_past_32_bit_offsets(dtype, D):
    """Blocks behind 2^32 elements of the cache (10 to 17 GB)."""
    base = -(-(1 << 32) // (16 * 8 * D)) + 5
    for qlens in ([1, 2], [150, 40]):
        c = case(24, [300, 77], qlens, 16, 8, D, 16, dtype)
        want = reference(c, softcap=20.0)
        big = []
        for name in ("k", "v"):
            t = torch.empty(base + len(c[name]), 16, 8, D, dtype=dtype, device=DEV)
            t[base:] = c[name].to(DEV)
            big.append(t)
        tables = torch.where(c["tables"] < 99999, c["tables"] + base, 2 ** 31 - 1).to(torch.int32)
        got, err = run({**c, "k": big[0], "v": big[1], "tables": tables}, softcap=20.0)
        assert err == 0
        close(got, want, c, f"{qlens}")
        del big, t
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("odd", ["q", "k", "v", "out", "qkv", "all"])
def test_tensors_that_start_anywhere(dtype, odd):
    """Pointers aligned to an element only: the same values on the CUDA cores."""
    for D, qlens in ((128, [1, 2]), (128, [60, 90]), (64, [3, 7]), (80, [40, 1])):
        c = case(25 + D, [200, 333], qlens, 4, 2, D, 16, dtype)
        want = reference(c, softcap=20.0, window=90)

        def place(t, at):
            flat = torch.zeros(t.numel() + 1, dtype=dtype, device=DEV)
            v = flat[at:at + t.numel()].view(t.shape)
            v.copy_(t)
            return v

        put = {n: place(c[n], int(n in odd or odd == "all")) for n in ("q", "k", "v")}
        out = place(torch.full_like(c["q"], 7.0), int(odd in ("out", "all")))
        for part in (0, 128):
            got, err = run({**c, **put}, out=out, partition_size=part, softcap=20.0, window=90)
            assert err == 0
            close(got, want, c, f"{D} {qlens} {part}")


def test_no_queries_at_all():
    """A padded step in which no sequence has a new token: nothing is written."""
    for dtype, D in ((BF, 128), (F32, 64), (HF, 256)):
        for B, total in ((1, 3), (5, 200)):
            c = case(26, [90] * B, [0] * B, 4, 2, D, 16, dtype)
            c["q"] = torch.full((total, 4, D), float("nan"), dtype=dtype)
            for part in (0, 128):
                got, err = run(c, partition_size=part, softcap=9.0)
                assert err == 0 and (got == 7).all()


def test_calls_that_run_at_once():
    """Calls on four streams, each with a workspace of its own, give the bits of
    the calls one by one."""
    shapes = [(BF, 128, [900, 700], [300, 200]), (BF, 128, [4000, 900], [2, 3]), (F32, 64, [300, 400], [40, 2]),
              (HF, 256, [600, 333], [90, 100])]
    state, want = [], []
    for i, (dtype, D, lens, qlens) in enumerate(shapes):
        c = case(60 + i, lens, qlens, 8, 2, D, 16, dtype)
        d = {k: c[k].to(DEV) for k in ("q", "k", "v", "tables", "cu", "lens")}
        ws = pkv.ChunkWorkspace(2, len(d["q"]), 8, 2, D, 16, d["tables"].shape[1], max(qlens), max(lens), 128)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        call = lambda out, stream, c=c, d=d, ws=ws, err=err, lens=lens, qlens=qlens: pkv.pkv_chunk_attention(
            out, d["q"], d["k"], d["v"], d["tables"], d["cu"], d["lens"], c["scale"], softcap=20.0, max_q_len=max(qlens),
            max_context_len=max(lens), partition_size=128, workspace=ws, err_flags=err, stream=stream)
        out = torch.zeros_like(d["q"])
        call(out, None)
        torch.cuda.synchronize()
        state.append((call, d, err, torch.cuda.Stream()))
        want.append(out)
    for _ in range(20):
        outs = [torch.zeros_like(d["q"]) for _, d, _, _ in state]
        torch.cuda.synchronize()
        for (call, _, _, stream), out in zip(state, outs):
            for _ in range(3):
                call(out, stream)
        torch.cuda.synchronize()
        for (_, _, err, _), out, w in zip(state, outs, want):
            assert int(err) == 0 and torch.equal(out, w)


def test_results_repeat_bit_by_bit():
    for dtype, D, q in ((BF, 128, [3, 5]), (BF, 128, [200, 100]), (HF, 256, [2, 2]), (F32, 64, [20, 3])):
        c = case(23, [1500, 400], q, 8, 2, D, 16, dtype)
        a, b = (run(c, softcap=10.0, partition_size=128)[0] for _ in range(2))
        assert torch.equal(a, b)
