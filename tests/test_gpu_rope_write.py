"""pkv_rope_write on the GPU against its 64-bit restatement.

Tolerance.  y = x c - z s in fp32 with one fused multiply-add: the product z s
is rounded (2^-24 |z s|) and the result (2^-24 |y|), then y is rounded to the
output type (half a step, relative eps / 2).  With |c|, |s| <= 1 every element
is within eps(dtype) / 2 * |y| + 2^-23 (|x| + |z|) of the exact value; the
16-bit types' subnormal spacing adds half a step of it (fp16: 2^-25)."""
import pytest
import torch

import paged_kv_cache_67_gb300 as pkv
from step_reference import rope

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def table(max_pos, rot):
    pairs = rot // 2
    ang = torch.arange(max_pos, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / max(pairs, 1))
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def case(seed, T, H, KVH, D, rot, axes, dtype, bs=16, max_pos=97, pads=0, extra=0, shift=0):
    """q, k, v as slices of one projection's output (`extra` more columns, the
    storage shifted by `shift` elements)."""
    g = torch.Generator().manual_seed(seed)
    width = (H + 2 * KVH) * D + extra
    flat = torch.randn(T * width + shift, generator=g).to(dtype)
    qkv = flat[shift:].view(T, width)
    nb = -(-(T + 5) // bs) + 2
    slots = torch.randperm(nb * bs, generator=g)[:T]
    slots[torch.randperm(T, generator=g)[:pads]] = -1
    pos = torch.randint(0, max_pos, (axes, T), generator=g, dtype=torch.int32)
    pair_axis = torch.randint(0, axes, (rot // 2,), generator=g).tolist()
    return dict(flat=flat, shift=shift, width=width, T=T, H=H, KVH=KVH, D=D, slots=slots, pos=pos, pair_axis=pair_axis,
                cos_sin=table(max_pos, rot), k_cache=torch.randn(nb, bs, KVH, D, generator=g).to(dtype),
                v_cache=torch.randn(nb, bs, KVH, D, generator=g).to(dtype), q=qkv[:, :H * D].unflatten(1, (H, D)),
                k=qkv[:, H * D:(H + KVH) * D].unflatten(1, (KVH, D)),
                v=qkv[:, (H + KVH) * D:(H + 2 * KVH) * D].unflatten(1, (KVH, D)), dtype=dtype)


def run(c, interleaved=False, in_place=False, stream=None, pair_axis="own"):
    d = lambda t: t.to(DEV)
    H, KVH, D, T = c["H"], c["KVH"], c["D"], c["T"]
    qkv = d(c["flat"])[c["shift"]:].view(T, c["width"])
    q, k, v = (qkv[:, a * D:b * D].unflatten(1, (b - a, D)) for a, b in ((0, H), (H, H + KVH), (H + KVH, H + 2 * KVH)))
    if in_place:
        q = q.contiguous()
    q_out = q if in_place else torch.full((T, H, D), 7.0, dtype=c["dtype"], device=DEV)
    kc, vc = d(c["k_cache"]).clone(), d(c["v_cache"]).clone()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.pkv_rope_write(q_out, kc, vc, q, k, v, d(c["cos_sin"]), d(c["pos"]), d(c["slots"]),
                       pair_axis=c["pair_axis"] if pair_axis == "own" else pair_axis, interleaved=interleaved,
                       err_flags=err, stream=stream)
    torch.cuda.synchronize()
    return q_out.cpu(), kc.cpu(), vc.cpu(), int(err)


def close(got, want, x, dtype, pairs, interleaved, what):
    """Element by element with the tolerance of the module's text."""
    x = x.double().abs()
    z = x.clone()
    if interleaved:
        z[..., 0:2 * pairs:2], z[..., 1:2 * pairs:2] = x[..., 1:2 * pairs:2], x[..., 0:2 * pairs:2]
    else:
        z[..., :pairs], z[..., pairs:2 * pairs] = x[..., pairs:2 * pairs], x[..., :pairs]
    tol = torch.finfo(dtype).eps / 2 * want.abs() + 2.0 ** -23 * (x + z) + (2.0 ** -25 if dtype == torch.float16 else 0)
    off = (got.double() - want).abs()
    assert (off <= tol).all(), f"{what}: {(off - tol).max().item():.3e} over"


def check(c, interleaved=False, in_place=False, stream=None):
    q_out, kc, vc, err = run(c, interleaved, in_place, stream)
    assert err == 0
    dt, KVH, D = c["dtype"], c["KVH"], c["D"]
    pairs = c["cos_sin"].shape[1] // 2
    keep = (c["slots"] >= 0).nonzero()[:, 0]
    slots = c["slots"][keep]
    for name, x, got in (("q", c["q"], q_out), ("k", c["k"], None)):
        want = rope(x, c["cos_sin"], c["pos"], c["pair_axis"], interleaved)[keep]
        got = q_out[keep] if got is not None else kc.view(-1, KVH, D)[slots]
        close(got, want, x[keep], dt, pairs, interleaved, name)
        assert torch.equal(got[..., 2 * pairs:], x[keep][..., 2 * pairs:]), name   # the rest is copied bit by bit
    assert torch.equal(vc.view(-1, KVH, D)[slots], c["v"][keep])
    # nothing else changed: padding rows of q_out, other cache rows
    pad = (c["slots"] < 0).nonzero()[:, 0]
    assert torch.equal(q_out[pad], c["q"][pad] if in_place else torch.full_like(q_out[pad], 7.0))
    rest = torch.ones(kc.shape[0] * kc.shape[1], dtype=torch.bool)
    rest[slots] = False
    assert torch.equal(kc.view(-1, KVH, D)[rest], c["k_cache"].view(-1, KVH, D)[rest])
    assert torch.equal(vc.view(-1, KVH, D)[rest], c["v_cache"].view(-1, KVH, D)[rest])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (128, 64), (80, 80), (96, 32), (256, 64), (512, 512), (512, 256), (20, 10), (9, 4), (64, 0)])
def test_shapes(D, rot, dtype, interleaved):
    check(case(D + rot, 23, 6, 2, D, rot, 3, dtype, pads=4), interleaved)


@pytest.mark.parametrize("T", [1, 2, 63, 300, 5000])
@pytest.mark.parametrize("H,KVH", [(4, 4), (32, 8), (7, 1), (64, 8)])
def test_token_counts_and_heads(T, H, KVH):
    check(case(T + H, T, H, KVH, 64, 64, 4, torch.bfloat16, pads=T // 5))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("extra,shift", [(0, 1), (3, 0), (8, 4), (2, 2), (4, 8)])
def test_alignments(extra, shift, dtype):
    """Rows that start anywhere: narrower vectors, the same values."""
    check(case(extra * 9 + shift, 31, 4, 2, 64, 64, 3, dtype, extra=extra, shift=shift, pads=2))
    check(case(extra * 9 + shift, 31, 4, 2, 64, 32, 3, dtype, extra=extra, shift=shift), interleaved=True)


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place(interleaved):
    check(case(5, 40, 8, 2, 128, 96, 3, torch.bfloat16, pads=3), interleaved, in_place=True)


def test_one_axis_default():
    c = case(6, 17, 4, 2, 64, 64, 1, torch.bfloat16)
    a, b = run(c, pair_axis=None), run(c)
    assert all(torch.equal(x, y) for x, y in zip(a[:3], b[:3]))
    c["pos"] = c["pos"][0]
    a = run(c, pair_axis=None)
    assert all(torch.equal(x, y) for x, y in zip(a[:3], b[:3]))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,T,rot", [(torch.bfloat16, 2101, 128), (torch.float16, 2101, 64), (torch.float32, 1051, 128)])
def test_more_than_the_cache_level_holds(dtype, T, rot, interleaved):
    """Past 64 MB of rows the stores are marked as streaming: the same values."""
    H, KVH, D = 128, 16, 128
    assert T * (H + 2 * KVH) * D * torch.finfo(dtype).bits // 8 > 64 << 20
    check(case(12, T, H, KVH, D, rot, 3, dtype, max_pos=3000, pads=100), interleaved)


def test_slots_past_32_bit_offsets():
    """Blocks behind 2^32 elements of the cache."""
    c = case(13, 40, 8, 8, 128, 128, 3, torch.bfloat16, pads=3)
    want, base = run(c), (1 << 32) // (16 * 8 * 128) + 7
    d = lambda t: t.to(DEV)
    q, k, v = (d(c[n]).contiguous() for n in "qkv")
    caches = [torch.empty(base + len(c["k_cache"]), 16, 8, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for big, name in zip(caches, ("k_cache", "v_cache")):
        big[base:] = d(c[name])
    q_out = torch.full_like(q, 7.0)
    pkv.pkv_rope_write(q_out, *caches, q, k, v, d(c["cos_sin"]), d(c["pos"]),
                       d(torch.where(c["slots"] < 0, c["slots"], c["slots"] + base * 16)), pair_axis=c["pair_axis"])
    torch.cuda.synchronize()
    for got, w in zip((q_out, caches[0][base:], caches[1][base:]), want):
        assert torch.equal(got.cpu(), w)
    del caches, big
    torch.cuda.empty_cache()


def test_positions_broadcast_over_the_axes():
    """Text: one position for every axis, as an expanded tensor (stride 0)."""
    for T in (1, 21):
        c = case(11, T, 4, 2, 64, 64, 3, torch.bfloat16)
        c["pos"] = c["pos"][:1].repeat(3, 1)
        want = run(c)
        d = lambda t: t.to(DEV)
        q, k, v = (d(c[n]).contiguous() for n in "qkv")
        q_out, kc, vc = torch.full_like(q, 7.0), d(c["k_cache"]), d(c["v_cache"])
        pkv.pkv_rope_write(q_out, kc, vc, q, k, v, d(c["cos_sin"]), d(c["pos"][0]).expand(3, T), d(c["slots"]),
                           pair_axis=c["pair_axis"])
        for got, w in zip((q_out, kc, vc), want):
            assert torch.equal(got.cpu(), w)


def test_values_that_are_not_finite_stay_in_their_pair():
    c = case(7, 9, 4, 2, 64, 64, 2, torch.bfloat16)
    c["q"][3, 1, 5] = float("nan")
    c["k"][4, 0, 40] = float("inf")
    q_out, kc, _, err = run(c)
    assert err == 0
    assert q_out.isnan().nonzero().tolist() == [[3, 1, 5], [3, 1, 37]]
    k = kc.view(-1, 2, 64)[c["slots"]]
    assert set(map(tuple, (~k.isfinite()).nonzero().tolist())) <= {(4, 0, 8), (4, 0, 40)}


def test_bad_positions_and_slots_are_flagged_and_skipped():
    c = case(8, 12, 4, 2, 64, 64, 3, torch.bfloat16)
    c["pair_axis"] = [0] * 16 + [2] * 16            # axis 1 turns nothing: its positions do not matter
    c["pos"][1] = -1000
    check(c)
    c["pos"][0, 2], c["pos"][2, 5], c["slots"][7] = -1, 97, 10 ** 12
    c["pos"][0, 9], c["slots"][9] = 97, -1          # a padding token's position does not matter
    q_out, kc, vc, err = run(c)
    assert err == pkv.FLAG_POSITION | pkv.FLAG_SLOT_OUT_OF_RANGE
    for t in (2, 5, 9):
        assert (q_out[t] == 7).all()
    assert not (q_out[7] == 7).any()
    written = [i for i in range(12) if i not in (2, 5, 7, 9)]
    rest = torch.ones(kc.shape[0] * 16, dtype=torch.bool)
    rest[c["slots"][written]] = False
    for got, was in ((kc, c["k_cache"]), (vc, c["v_cache"])):
        assert torch.equal(got.view(-1, 2, 64)[rest], was.view(-1, 2, 64)[rest])


def test_plain_write_is_the_unrotated_form():
    """rot_dim 0 writes what pkv_write writes."""
    c = case(9, 33, 4, 2, 64, 0, 1, torch.float16, pads=5)
    _, kc, vc, err = run(c)
    k2, v2 = c["k_cache"].to(DEV), c["v_cache"].to(DEV)
    pkv.pkv_write(k2, v2, c["k"].to(DEV).contiguous(), c["v"].to(DEV).contiguous(), c["slots"].to(DEV))
    assert err == 0 and torch.equal(kc, k2.cpu()) and torch.equal(vc, v2.cpu())


def test_stream_and_graph_replay():
    c = case(10, 64, 8, 2, 128, 128, 3, torch.bfloat16)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        check(c, stream=s)
    d = {k: c[k].to(DEV) for k in ("k_cache", "v_cache", "cos_sin", "pos", "slots")}
    q, k, v = (c[n].to(DEV).contiguous() for n in "qkv")
    q_out = torch.zeros_like(q)
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        pkv.pkv_rope_write(q_out, d["k_cache"], d["v_cache"], q, k, v, d["cos_sin"], d["pos"], d["slots"],
                           pair_axis=c["pair_axis"], stream=s)
    for shift in (0, 1):
        q.copy_(c["q"].roll(shift, 0))
        g.replay()
        torch.cuda.synchronize()
        want = rope(c["q"].roll(shift, 0), c["cos_sin"], c["pos"], c["pair_axis"], False)
        close(q_out.cpu(), want, c["q"].roll(shift, 0), torch.bfloat16, 64, False, "replay")
