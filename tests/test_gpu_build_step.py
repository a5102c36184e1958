"""pkv_build_step on the GPU against its plain restatement: growth over block
edges, blocks given back and taken again in the same step, prompts, padding,
refused steps, in-place loops, streams, graphs and the host block manager."""
import random

import pytest
import torch

import paged_kv_cache_67_gb300 as pkv
from step_reference import build_step

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
I32, I64 = torch.int32, torch.int64


def case(seed, B, bs, len_hi, new_hi, spare=0, zero=0.3, prompts=0.1):
    r = random.Random(seed)
    cached = [0 if r.random() < zero else r.randint(1, len_hi) for _ in range(B)]
    held_tok = [c + r.randint(0, spare) for c in cached]
    new = [0 if r.random() < zero else r.randint(1, new_hi) for _ in range(B)]
    for b in range(B):
        if r.random() < prompts:
            cached[b], new[b] = 0, r.randint(1, len_hi)
        if r.random() < 0.1:
            cached[b] = new[b] = 0
    held = [max(-(-h // bs), -(-c // bs)) for h, c in zip(held_tok, cached)]
    mb = max([-(-(c + n) // bs) for c, n in zip(cached, new)] + held) + r.randint(0, 2)
    used = sum(held)
    nb = used + sum(max(0, -(-(c + n) // bs) - h) for c, n, h in zip(cached, new, held)) + r.randint(0, 5)
    perm = list(range(nb))
    r.shuffle(perm)
    tables, at = [], 0
    for h in held:
        tables.append(perm[at:at + h] + [99999] * (mb - h))
        at += h
    free = perm[at:] + [-7] * used
    return dict(tables=tables, held=held, free=free, count=nb - used, cached=cached, new=new, bs=bs, nb=nb)


def run(c, max_tokens, in_place=False, err=None, stream=None):
    t = lambda x: torch.tensor(x, dtype=I32, device=DEV)
    B = len(c["held"])
    mb = len(c["tables"][0]) if B else 0
    d = dict(tables=t(c["tables"]).view(B, mb), held=t(c["held"]), free=t(c["free"]), count=t([c["count"]]),
             cached=t(c["cached"]), new=t(c["new"]))
    d["held_out"] = d["held"] if in_place else torch.full((B,), -5, dtype=I32, device=DEV)
    d["count_out"] = d["count"] if in_place else torch.full((1,), -5, dtype=I32, device=DEV)
    d["lens"] = d["cached"] if in_place else torch.full((B,), -5, dtype=I32, device=DEV)
    d["cu"] = torch.full((B + 1,), -5, dtype=I32, device=DEV)
    d["slots"] = torch.full((max_tokens,), -5, dtype=I64, device=DEV)
    d["positions"] = torch.full((max_tokens,), -5, dtype=I32, device=DEV)
    flags = torch.zeros(1, dtype=I32, device=DEV) if err is None else err
    pkv.pkv_build_step(d["tables"], d["held"], d["held_out"], d["free"], d["count"], d["count_out"], d["cached"],
                       d["new"], d["lens"], d["cu"], d["slots"], d["positions"], c["nb"], c["bs"], err_flags=flags,
                       stream=stream)
    torch.cuda.synchronize()
    got = {k: d[n].tolist() for k, n in (("tables", "tables"), ("held", "held_out"), ("free", "free"), ("lens", "lens"),
                                         ("cu", "cu"), ("slots", "slots"), ("positions", "positions"))}
    got["count"] = int(d["count_out"])
    return got, int(flags)


def want_of(c, max_tokens):
    return build_step(c["tables"], c["held"], c["free"], c["count"], c["cached"], c["new"], c["bs"], max_tokens, c["nb"])


def check(c, extra=0, in_place=False):
    T = sum(c["new"]) + extra
    want = want_of(c, T)
    assert "why" not in want
    got, flags = run(c, T, in_place)
    assert flags == 0
    for k in want:
        assert got[k] == want[k], k


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("seed,B,bs,len_hi,new_hi,spare", [
    (1, 1, 16, 40, 1, 0), (2, 3, 1, 9, 4, 3), (3, 31, 16, 100, 1, 0), (4, 33, 8, 300, 20, 30), (5, 256, 16, 2047, 1, 5),
    (6, 1023, 32, 64, 3, 40), (7, 1024, 16, 64, 3, 0), (8, 1025, 16, 64, 7, 17), (9, 5000, 4, 12, 2, 3), (10, 7, 7, 3000, 900, 9)])
def test_against_plain(seed, B, bs, len_hi, new_hi, spare, in_place):
    c = case(seed, B, bs, len_hi, new_hi, spare)
    check(c, extra=0, in_place=in_place)
    check(c, extra=seed * 3 + 1, in_place=in_place)


def test_many_tokens_use_the_cluster():
    """More tokens than one CTA takes: the cluster's CTAs share one step."""
    c = case(21, 700, 16, 400, 60, 20, prompts=0.4)
    assert sum(c["new"]) > 3 * 4096
    check(c, extra=5000)
    check(c, extra=5000, in_place=True)


def test_largest_batch():
    check(case(22, 16384, 16, 30, 2, 3), extra=7)


@pytest.mark.parametrize("B", [8192, 8193, 16384])
def test_largest_batches_in_place(B):
    """Two steps that carry their state in place, on either side of the batch up
    to which the lengths stay in shared memory.  Blocks of 4 and up to 9 new
    tokens: most requests would want other blocks for c + 2n than for c + n."""
    c = case(B, B, 4, 30, 9, 3)
    check(c, extra=7, in_place=True)
    c["tables"] = [row + [99999] * 3 for row in c["tables"]]     # room and blocks for a second step
    spare = list(range(c["nb"], c["nb"] + 4 * B))
    c.update(free=spare + c["free"], count=c["count"] + len(spare), nb=c["nb"] + len(spare))
    t = lambda x: torch.tensor(x, dtype=I32, device=DEV)
    d = {k: t(c[k]) for k in ("tables", "held", "free", "cached", "new")}
    count, cu, err = t([c["count"]]), t([0] * (B + 1)), t([0])
    T = 9 * B + 40 * B // 4
    slots, pos = torch.zeros(T, dtype=I64, device=DEV), torch.zeros(T, dtype=I32, device=DEV)
    r = random.Random(B)
    for step in range(2):
        want = want_of(c, T)
        assert "why" not in want
        pkv.pkv_build_step(d["tables"], d["held"], d["held"], d["free"], count, count, d["cached"], d["new"], d["cached"],
                           cu, slots, pos, c["nb"], 4, err_flags=err)
        torch.cuda.synchronize()
        assert int(err) == 0
        for k, v in (("tables", d["tables"]), ("held", d["held"]), ("free", d["free"]), ("lens", d["cached"]), ("cu", cu),
                     ("slots", slots), ("positions", pos)):
            assert v.tolist() == want[k], (step, k)
        assert int(count) == want["count"]
        c.update(tables=want["tables"], held=want["held"], free=want["free"], count=want["count"], cached=want["lens"],
                 new=[r.randint(0, 9) for _ in range(B)])
        d["new"].copy_(t(c["new"]))


def test_all_idle_and_empty():
    c = dict(tables=[[3, 9], [9, 9]], held=[1, 0], free=[0, 1, 2, -1], count=3, cached=[5, 0], new=[0, 0], bs=16, nb=4)
    check(c, extra=3)
    got, flags = run(dict(tables=[], held=[], free=[4], count=1, cached=[], new=[], bs=16, nb=8), 3)
    assert flags == 0 and got["slots"] == [-1] * 3 and got["cu"] == [0] and got["count"] == 1


def test_blocks_released_and_taken_in_one_step():
    """A request ends with its blocks the only free ones: another grows into
    them in the same step, last released first."""
    c = dict(tables=[[4, 2, 7], [1, 99, 99]], held=[3, 1], free=[-1] * 8, count=0, cached=[0, 10], new=[0, 25], bs=16, nb=8)
    check(c)
    got, _ = run(c, 25)
    assert got["tables"][1] == [1, 7, 2] and got["count"] == 1 and got["free"][:3] == [4, 2, 7]


REFUSED = [("negative cached", dict(cached=[-1, 10]), "invalid"), ("negative new", dict(new=[1, -1]), "invalid"),
           ("held over the row", dict(held=[4, 1]), "invalid"), ("held negative", dict(held=[-1, 1]), "invalid"),
           ("fewer blocks than cached", dict(held=[0, 0]), "invalid"), ("row too short", dict(new=[200, 1]), "invalid"),
           ("huge", dict(new=[2**31 - 1, 1]), "invalid"), ("count negative", dict(count=-1), "invalid"),
           ("count over", dict(count=9), "invalid"), ("stack overflows", dict(count=8, cached=[0, 10], new=[0, 1]), "invalid"),
           ("no blocks", dict(count=0, new=[8, 0], cached=[16, 10]), "blocks")]


@pytest.mark.parametrize("what,change,why", REFUSED)
@pytest.mark.parametrize("in_place", [False, True])
def test_refused_steps_change_nothing(what, change, why, in_place):
    c = dict(tables=[[4, 99, 99], [1, 99, 99]], held=[1, 1], free=[5, 6, 0, -1, -1, -1, -1, -1], count=3, cached=[3, 10],
             new=[1, 1], bs=16, nb=8)
    c.update(change)
    T = 8
    assert want_of(c, T) == {"why": why}
    got, flags = run(c, T, in_place)
    assert flags == (pkv.FLAG_STEP_INVALID if why == "invalid" else pkv.FLAG_OUT_OF_BLOCKS)
    assert got["tables"] == c["tables"] and got["free"] == c["free"] and got["held"] == c["held"]
    assert got["count"] == c["count"]
    assert got["slots"] == [-1] * T and got["positions"] == [0] * T and got["cu"] == [0, 0, 0] and got["lens"] == [0, 0]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,new", [(2, 2 ** 30), (4, 2 ** 29), (4096, 2 ** 20), (16384, 131072), (8192, 131072), (1024, 2 ** 20)])
def test_totals_past_the_bound_are_refused(B, new, in_place):
    """2^30, 2^31 and 2^32 new tokens in all, a block each: no sum may wrap."""
    c = dict(tables=[[b] for b in range(B)], held=[1] * B, free=[-1] * 4, count=0, cached=[0] * B, new=[new] * B, bs=new, nb=B)
    assert want_of(c, 8) == {"why": "invalid"}
    got, flags = run(c, 8, in_place)
    assert flags == pkv.FLAG_STEP_INVALID
    assert got["tables"] == c["tables"] and got["free"] == c["free"] and got["held"] == c["held"] and got["count"] == 0
    assert got["slots"] == [-1] * 8 and got["positions"] == [0] * 8 and got["cu"] == [0] * (B + 1) and got["lens"] == [0] * B


def test_the_largest_total():
    """One token less than the bound is a step; the lists hold its first tokens."""
    c = dict(tables=[[0], [1]], held=[1, 0], free=[1, -1], count=1, cached=[0, 0], new=[2 ** 30 - 2, 1], bs=2 ** 30, nb=2)
    got, flags = run(c, 3)
    assert flags == pkv.FLAG_TOKENS_OVER
    assert got["cu"] == [0, 2 ** 30 - 2, 2 ** 30 - 1] and got["lens"] == c["new"] and got["held"] == [1, 1]
    assert got["slots"] == [0, 1, 2] and got["positions"] == [0, 1, 2] and got["count"] == 0


@pytest.mark.parametrize("room", [0, 1, 9, 24])
def test_more_tokens_than_the_lists_hold(room):
    """The lists hold the first max_tokens; the rest of the step is done."""
    c = dict(tables=[[4, 99, 99], [1, 99, 99]], held=[1, 1], free=[5, 6, 0, -1], count=3, cached=[3, 10], new=[15, 10], bs=16, nb=8)
    got, flags = run(c, room)
    assert flags == pkv.FLAG_TOKENS_OVER
    assert got == want_of(c, room) and got["cu"] == [0, 15, 25]


def test_bad_entries_are_flagged():
    """A table or free entry outside the pool: that token's slot is -1."""
    c = dict(tables=[[8, 99], [1, 99]], held=[1, 1], free=[-3, 6], count=1, cached=[3, 15], new=[2, 3], bs=16, nb=8)
    got, flags = run(c, 6)
    assert flags == pkv.FLAG_BLOCK_OUT_OF_RANGE
    assert got["slots"] == [-1, -1, 31, -1, -1, -1] and got["positions"] == [3, 4, 15, 16, 17, 0]


def test_loop_in_place_matches_block_by_block_growth():
    """Forty in-place decode steps in a captured graph: every step equals the
    restatement applied to the state before it."""
    r = random.Random(5)
    c = case(31, 12, 4, 30, 1, 0, zero=0.0, prompts=0.0)
    mb, nb = 40, 600
    c["tables"] = [row[:h] + [99999] * (mb - h) for row, h in zip(c["tables"], c["held"])]
    used = [x for row, h in zip(c["tables"], c["held"]) for x in row[:h]]
    rest = [x for x in range(nb) if x not in set(used)]
    r.shuffle(rest)
    c.update(free=rest + [-1] * len(used), count=len(rest), nb=nb, new=[1] * 12)
    t = lambda x: torch.tensor(x, dtype=I32, device=DEV)
    d = {k: t(c[k]) for k in ("tables", "held", "free", "cached", "new")}
    count, cu = t([c["count"]]), torch.zeros(13, dtype=I32, device=DEV)
    slots, pos = torch.zeros(64, dtype=I64, device=DEV), torch.zeros(64, dtype=I32, device=DEV)
    err = torch.zeros(1, dtype=I32, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        pkv.pkv_build_step(d["tables"], d["held"], d["held"], d["free"], count, count, d["cached"], d["new"], d["cached"],
                           cu, slots, pos, nb, 4, err_flags=err, stream=side)
    state = dict(c)
    for step in range(40):
        new = [r.randint(0, 4) for _ in range(12)]
        turned = [r.randint(0, 2) for _ in range(12)]          # drafts turned down since the last step
        state["cached"] = [max(0, x - y) for x, y in zip(state["cached"], turned)]
        state["new"] = new
        if step % 9 == 8:
            state["cached"][step % 12], state["new"][step % 12] = 0, 0
        d["cached"].copy_(t(state["cached"]))
        d["new"].copy_(t(state["new"]))
        want = want_of(state, 64)
        assert "why" not in want
        g.replay()
        torch.cuda.synchronize()
        assert int(err) == 0
        for k, v in (("tables", d["tables"]), ("held", d["held"]), ("free", d["free"]), ("lens", d["cached"]), ("cu", cu),
                     ("slots", slots), ("positions", pos)):
            assert v.tolist() == want[k], (step, k)
        assert int(count) == want["count"]
        state.update(tables=want["tables"], held=want["held"], free=want["free"], count=want["count"], cached=want["lens"])


def test_other_stream():
    c = case(41, 50, 16, 100, 5, 3)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        check(c, 3)


def test_agrees_with_the_host_block_manager():
    """Decode appends: slots and lengths equal the host manager's once both
    hold the same tables."""
    bm = pkv.BlockManager(64, 16, prefix_caching=False)
    lens = [5, 16, 31, 33]
    for i, n in enumerate(lens):
        bm.add_sequence(i, list(range(n)))
    tables, _ = bm.build_batch(range(4), 8)
    held = [-(-n // 16) for n in lens]
    slots = bm.append_tokens(range(4), [1, 2, 3, 4])
    after, lens_after = bm.build_batch(range(4), 8)
    grown = [b for b in range(4) if lens[b] % 16 == 0]
    free = [int(after[b, held[b]]) for b in grown][::-1]        # the stack's top is the first block taken
    got, flags = run(dict(tables=tables.tolist(), held=held, free=free, count=len(free), cached=lens, new=[1] * 4, bs=16, nb=64), 4)
    assert flags == 0 and got["slots"] == slots.tolist() and got["lens"] == lens_after.tolist()
    assert got["tables"] == after.tolist()
