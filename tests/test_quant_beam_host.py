"""The quantised cache's and beam search's operators on the CPU: what their C
entry points refuse before any CUDA call, workspace sizes, the binding's checks,
and pins of the restatements that the GPU tests compare with."""
import ctypes
import math

import pytest
import torch

import quant_beam_reference as ref
from paged_kv_cache_67_gb300 import build as libbuild

OK, INVALID, CUDA, UNSUPPORTED, WORKSPACE = 0, 1, 3, 2, 4
FAKE = 1 << 20  # an aligned address that is never dereferenced


def at(i):
    return FAKE + (i << 40)


@pytest.fixture(scope="module")
def pkv():
    libbuild.build()
    import paged_kv_cache_67_gb300 as m
    m.load_library()
    return m


def _rows(lib, read=False, **kw):
    names = ("k_codes", "v_codes", "k_params", "v_params", "k", "v", "slots")
    p = {n: at(i) for i, n in enumerate(names)}
    p.update({k: v for k, v in kw.items() if k in names})
    D, KVH = kw.get("D", 64), kw.get("KVH", 2)
    codes = (p["k_codes"], p["v_codes"], p["k_params"], p["v_params"])
    first = (p["k"], p["v"], *codes) if read else (*codes, p["k"], p["v"])
    fn = lib.pkv_quant_read if read else lib.pkv_quant_write
    return fn(*first, p["slots"], kw.get("T", 3), kw.get("ks", KVH * D), kw.get("vs", KVH * D), kw.get("nb", 8),
              kw.get("bs", 16), KVH, D, kw.get("fmt", 0), kw.get("dt", 1), kw.get("err"), None)


@pytest.mark.parametrize("read", [False, True])
def test_quant_rows_refusals(pkv, read):
    lib = pkv.load_library()
    assert _rows(lib, read, T=0) == OK
    for bad in ({"T": -1}, {"T": 1 << 31}, {"D": 0}, {"D": -4}, {"nb": -1}, {"nb": 1 << 31}, {"bs": 0}, {"KVH": 0},
                {"fmt": 3}, {"fmt": -1}, {"dt": 3}, {"ks": 127}, {"vs": 127}, {"fmt": 2, "D": 63}, {"k_codes": None},
                {"v_codes": None}, {"k_params": None}, {"v_params": None}, {"k": None}, {"v": None}, {"slots": None},
                {"k": at(4) + 1}, {"k_params": at(2) + 2}, {"slots": at(6) + 4}, {"err": FAKE + 2}):
        assert _rows(lib, read, **bad) == INVALID, bad
    assert _rows(lib, read, D=513) == UNSUPPORTED
    # what is written overlaps nothing else
    for bad in ([{"k": at(0)}, {"v_codes": at(0) + 64}, {"v_params": at(2) + 4}, {"k_params": at(6)}] if not read else
                [{"k": at(5)}, {"k": at(0) + 64}, {"v": at(3)}, {"k": at(6)}]):
        assert _rows(lib, read, **bad) == INVALID, bad


def _decode(lib, **kw):
    names = ("out", "q", "k_codes", "v_codes", "k_params", "v_params", "tables", "lens", "ws")
    p = {n: at(i) for i, n in enumerate(names)}
    p.update({k: v for k, v in kw.items() if k in names})
    f = ctypes.c_float
    return lib.pkv_quant_decode_attention(
        *[p[n] for n in names[:8]], kw.get("B", 2), kw.get("H", 8), kw.get("KVH", 2), kw.get("D", 64), kw.get("bs", 16),
        kw.get("mb", 8), kw.get("nb", 32), f(kw.get("scale", 0.125)), f(kw.get("cap", 0.0)), kw.get("window", 0),
        kw.get("fmt", 0), kw.get("dt", 1), kw.get("maxn", 0), kw.get("P", 0), p["ws"], kw.get("wsb", 1 << 40),
        kw.get("err"), None)


def test_quant_decode_refusals(pkv):
    lib = pkv.load_library()
    assert _decode(lib, B=0) == OK
    for bad in ({"B": -1}, {"B": 65536}, {"H": 0}, {"H": 7}, {"KVH": 0}, {"D": 0}, {"bs": 0}, {"mb": -1}, {"nb": -1},
                {"nb": 1 << 31}, {"scale": math.inf}, {"scale": math.nan}, {"cap": -1.0}, {"cap": math.inf},
                {"cap": math.nan}, {"cap": 1e-45}, {"window": -1}, {"fmt": 3}, {"dt": 3}, {"fmt": 2, "D": 65},
                {"maxn": -1}, {"P": -128}, {"P": 64}, {"out": None}, {"q": None}, {"k_codes": None}, {"v_codes": None},
                {"k_params": None}, {"v_params": None}, {"tables": None}, {"lens": None}, {"out": at(0) + 1},
                {"q": at(1) + 1}, {"k_params": at(4) + 2}, {"tables": at(6) + 2}, {"lens": at(7) + 1},
                {"err": FAKE + 1}, {"out": at(1)}, {"out": at(2) + 128}, {"ws": at(7)}, {"ws": at(0)}):
        assert _decode(lib, **bad) == INVALID, bad
    assert _decode(lib, D=513) == UNSUPPORTED
    for bad in ({"ws": None}, {"ws": at(8) + 128}, {"wsb": 1000}):
        assert _decode(lib, **bad) == WORKSPACE, bad


def test_quant_decode_workspace(pkv):
    size = pkv.pkv_quant_decode_workspace_size
    assert size(4, 6, 4, 64, 16, 8) == 0 and size(4, 8, 2, 600, 16, 8) == 0 and size(4, 8, 2, 64, 16, 8, 0, 100) == 0
    assert size(4, 8, 2, 64, 16, 8, 0, 128) > 0
    # the size for no window serves every window, format and dtype
    lib = pkv.load_library()
    if torch.cuda.is_available():
        return
    for B, H, KVH, D, bs, mb, P in ((1, 32, 8, 128, 16, 2048, 0), (64, 32, 8, 128, 16, 256, 0), (3, 12, 2, 80, 24, 999, 0),
                                    (128, 16, 1, 256, 32, 256, 0), (2, 8, 2, 64, 16, 500, 256), (1, 5, 1, 72, 1, 9000, 128)):
        need = size(B, H, KVH, D, bs, mb, 0, P)
        for window in (0, 1, 100, 129, 1000, 1025, 5000, 1 << 20):
            for dt in (0, 1, 2):
                for fmt in (0, 1, 2):
                    assert _decode(lib, B=B, H=H, KVH=KVH, D=D, bs=bs, mb=mb, P=P, window=window, dt=dt, fmt=fmt,
                                   nb=8, wsb=need) not in (WORKSPACE, INVALID)


def _select(lib, **kw):
    names = ("scores_out", "parents", "tokens", "finished_out", "logits", "scores", "finished", "ws")
    p = {n: at(i) for i, n in enumerate(names)}
    p.update({k: v for k, v in kw.items() if k in names})
    V = kw.get("V", 1000)
    return lib.pkv_beam_select(*[p[n] for n in names[:7]], kw.get("B", 2), kw.get("W", 4), kw.get("K", 4), V,
                               kw.get("stride", V), kw.get("end", 2), kw.get("dt", 1), p["ws"], kw.get("wsb", 1 << 40),
                               kw.get("err"), None)


def test_beam_select_refusals(pkv):
    lib = pkv.load_library()
    assert _select(lib, B=0) == OK
    for bad in ({"B": -1}, {"W": 0}, {"K": 0}, {"V": 0}, {"stride": 999}, {"end": -2}, {"end": 1000}, {"dt": 3},
                {"scores_out": None}, {"parents": None}, {"tokens": None}, {"finished_out": None}, {"logits": None},
                {"scores": None}, {"scores": at(5) + 2}, {"logits": at(4) + 1}, {"parents": at(1) + 2},
                {"err": FAKE + 2}, {"parents": at(2)}, {"scores_out": at(4) + 64}, {"scores_out": at(5) + 4},
                {"finished_out": at(6) + 1}, {"ws": at(5)}, {"K": 3, "scores_out": at(5)}):
        assert _select(lib, **bad) == INVALID, bad
    for bad in ({"W": 33}, {"K": 33}, {"V": (1 << 21) + 1}, {"B": 16385}):
        assert _select(lib, **bad) == UNSUPPORTED, bad
    for bad in ({"ws": None}, {"ws": at(7) + 64}, {"wsb": 100}):
        assert _select(lib, **bad) == WORKSPACE, bad
    if not torch.cuda.is_available():      # in place, and without `finished`
        assert _select(lib, scores_out=at(5), finished_out=at(6)) == CUDA
        assert _select(lib, finished=None) == CUDA
    size = pkv.pkv_beam_select_workspace_size
    assert size(2, 4, 4, 0) == 0 and size(2, 33, 4, 10) == 0 and size(2, 4, 33, 10) == 0 and size(1, 1, 1, 1) > 0


def _reorder(lib, **kw):
    names = ("tables_out", "lens_out", "slots", "tables", "lens", "parents", "owned", "finished")
    p = {n: at(i) for i, n in enumerate(names)}
    p.update({k: v for k, v in kw.items() if k in names})
    pools = kw.get("pools", [at(10), at(11)])
    n = len(pools)
    block, rows = kw.get("block", [4096] * n), kw.get("rows", [256] * n)
    arr = lambda t, x: (t * max(1, n))(*x)
    return lib.pkv_beam_reorder(*[p[k] for k in names], kw.get("B", 2), kw.get("W", 4), kw.get("K", 4),
                                kw.get("mb", 8), kw.get("nb", 64), kw.get("bs", 16), kw.get("n", n),
                                kw.get("arr", arr(ctypes.c_void_p, pools)), arr(ctypes.c_int64, block),
                                arr(ctypes.c_int64, rows), kw.get("err"), None)


def test_beam_reorder_refusals(pkv):
    lib = pkv.load_library()
    assert _reorder(lib, B=0) == OK
    for bad in ({"B": -1}, {"W": 0}, {"K": 0}, {"mb": 0}, {"nb": -1}, {"nb": 1 << 31}, {"bs": 0}, {"n": -1},
                {"arr": None}, {"tables_out": None}, {"lens_out": None}, {"slots": None}, {"tables": None},
                {"lens": None}, {"parents": None}, {"owned": None}, {"tables": at(3) + 2}, {"slots": at(2) + 4},
                {"err": FAKE + 2}, {"tables_out": at(3)}, {"lens_out": at(4)}, {"slots": at(5)}, {"tables_out": at(6) + 64},
                {"pools": [at(10), at(10) + 4096]}, {"pools": [at(3)]}, {"pools": [at(0)]}, {"block": [-1, 4096]},
                {"rows": [257, 256]}, {"rows": [-1, 0]}, {"pools": [None, at(10)]}):
        assert _reorder(lib, **bad) == INVALID, bad
    for bad in ({"W": 33}, {"K": 33}, {"B": 16385}, {"pools": [at(10 + i) for i in range(257)]}):
        assert _reorder(lib, **bad) == UNSUPPORTED, bad


def test_binding_checks(pkv):
    t = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype)
    i8, i32, i64 = torch.int8, torch.int32, torch.int64
    c, p, k, slots = t(4, 16, 2, 64, dtype=i8), t(4, 2, 16), t(3, 2, 64), t(3, dtype=i64)
    for bad in ((c.float(), c.float(), p, p, k, k, slots), (c, c, t(4, 16, 2), p, k, k, slots),
                (c, c, p, p, t(3, 2, 32), t(3, 2, 32), slots), (c, c, p, p, k, k, slots.int()),
                (c, c, p, p, k, k.half(), slots), (c, c, p, p, k.transpose(0, 1).contiguous().transpose(0, 1), k, slots),
                (t(4, 16, 2, 32, dtype=torch.uint8), t(4, 16, 2, 32, dtype=torch.uint8), p, p, k, k, slots),
                (c, c, p, p, k, k, slots)):                                # the last: not on a GPU
        with pytest.raises(ValueError):
            pkv.pkv_quant_write(*bad)
    q = t(2, 8, 64)
    with pytest.raises(ValueError):
        pkv.pkv_quant_decode_attention(q, q, c, c, p, p, t(2, 4, dtype=i32), t(2, dtype=i64), 0.1)
    with pytest.raises(ValueError):
        pkv.pkv_beam_select(t(2, 4), t(2, 4, dtype=i32), t(2, 4, dtype=i32), t(2, 4, dtype=torch.uint8),
                            t(2, 4, 10).transpose(1, 2).contiguous().transpose(1, 2), t(2, 4))
    with pytest.raises(ValueError):
        pkv.pkv_beam_reorder(t(1, 2, 3, dtype=i32), t(1, 2, dtype=i32), t(1, 2, dtype=i64), t(1, 2, 3, dtype=i32),
                             t(1, 2, dtype=i32), t(1, 2, dtype=i32), t(1, 2, 3, dtype=i32), 16)


def test_reference_quantise_pins():
    x = torch.tensor([[1.0, -2.0, 0.5, 0.0], [0.0, 0.0, 0.0, 0.0], [math.inf, 1.0, 2.0, 3.0], [1e-40, 0, 0, 0]])
    c, s, _ = ref.quantise(x, "int8")
    assert c[0].tolist() == [64, -127, 32, 0]                              # 63.5 -> 64, 31.75 -> 32
    assert s[0] == (torch.tensor(2.0) * torch.tensor(1 / 127.0)).double() and s[1] == 0 and s[3] == 0 and s[2].isnan()
    c, s, z = ref.quantise(torch.tensor([[-1.0, 2.0, 0.0, 0.5], [3.0, 1.0, 1.5, 0.2]]), "int4")
    assert z.tolist() == [5, 0] and c[0].tolist() == [0, 15, 5, 7] and c[1].tolist() == [15, 5, 8, 1]   # 2.5 -> 2, 7.5 -> 8
    g = torch.Generator().manual_seed(0)
    x = torch.randn(50, 64, generator=g)
    c, s, _ = ref.quantise(x, "e4m3")
    want = (x * (448.0 / x.abs().amax(1, keepdim=True))).to(torch.float8_e4m3fn)
    assert torch.equal(c.float(), want.float())
    assert torch.equal(ref.stored(c, "e4m3").view(torch.uint8), want.view(torch.uint8))


def test_reference_beam_pins():
    # two beams, three tokens: equal rows tie, the lower beam goes first
    x = torch.zeros(1, 2, 3)
    s, p, t, f = ref.beam_select(x, torch.zeros(1, 2), None, 4, 1)
    assert p.tolist() == [[0, 0, 0, 1]] and t.tolist() == [[0, 1, 2, 0]] and f.tolist() == [[0, 1, 0, 0]]
    assert torch.allclose(s, torch.full((1, 4), -math.log(3.0), dtype=torch.float64))
    # one prompt of 3 tokens in blocks of 2 (block 9, then 4 half full), two children of it
    t, n, s, c = ref.beam_reorder([[9, 4, 0]], [3], [0, 0, -1], [[9, 4, 6], [9, 5, 7], [9, 8, 3]], None, 2)
    assert t == [[9, 4, 6], [9, 5, 7], [9, 8, 3]] and n == [4, 4, 0] and s == [9, 11, -1] and c == [(4, 5, 1)]


def test_beam_select_workspace_of_the_largest_serves_all(pkv):
    """A workspace for B, W, K, V serves every smaller one: a loop's requests finish."""
    lib, size = pkv.load_library(), pkv.pkv_beam_select_workspace_size
    if torch.cuda.is_available():
        return                                                             # (the calls below have no memory behind them)
    for B, W, K, V in ((10, 4, 4, 128256), (64, 8, 8, 128256), (16, 4, 4, 32000), (300, 2, 32, 50257), (16384, 1, 1, 50),
                       (3, 32, 32, 1 << 21), (40, 16, 8, 300001)):
        need = size(B, W, K, V)
        for b in sorted({1, 2, 3, B // 2 or 1, B - 1 or 1, B, *range(1, min(B, 40))}):
            for w in sorted({1, W // 2 or 1, W}):
                for k in sorted({1, K}):
                    for v in sorted({1, 2048, 2049, V // 3 + 1, V - 1 or 1, V}):
                        if v > V or b > B:
                            continue
                        assert size(b, w, k, v) <= need, (B, W, K, V, b, w, k, v)
                        for dt in (0, 1, 2):
                            assert _select(lib, B=b, W=w, K=k, V=v, dt=dt, end=-1, wsb=need) == CUDA, (B, W, K, V, b, w, k, v, dt)


def test_quant_decode_workspace_of_the_largest_serves_all(pkv):
    """A workspace for a batch and a context length serves smaller ones, on the
    tensor cores and on the CUDA cores (head_dim 40; unaligned codes)."""
    lib, size = pkv.load_library(), pkv.pkv_quant_decode_workspace_size
    if torch.cuda.is_available():
        return
    for B, H, KVH, D, bs, mb, P in ((400, 4, 1, 40, 16, 20, 0), (200, 8, 2, 40, 16, 128, 0), (64, 32, 8, 64, 16, 256, 0),
                                    (2000, 6, 1, 72, 16, 300, 0), (300, 16, 1, 256, 32, 256, 0), (40, 5, 1, 40, 1, 5000, 256),
                                    (20000, 4, 4, 40, 16, 30, 128)):
        need = size(B, H, KVH, D, bs, mb, 0, P)
        for b in sorted({1, 2, B // 7 or 1, B // 2 or 1, B - 1, B, *range(1, min(B, 80)), *(x for x in range(290, 320) if x <= B)}):
            for n in (0, 1, 130, mb * bs // 3 + 1, mb * bs):
                assert size(b, H, KVH, D, bs, mb, n, P) <= need, (B, b, n)
                for odd in (0, 1):
                    for dt in (0, 1):
                        assert _decode(lib, B=b, H=H, KVH=KVH, D=D, bs=bs, mb=mb, maxn=n, P=P, dt=dt, nb=8, k_codes=at(2) + odd,
                                       wsb=need) == CUDA, (B, b, n, odd, dt)


def test_quant_read_side_by_side(pkv):
    """Rows of K and V in one buffer are not an overlap, rows that meet are."""
    lib = pkv.load_library()
    row, far = 2 * 64 * 2, 1 << 30                                         # bytes of a token's row (bf16)
    call = lambda shift, stride=256, other=None, T=5: _rows(lib, True, k=at(4) + far, v=at(4) + far + shift, T=T, ks=stride,
                                                            vs=other or stride)
    for bad in (call(0), call(row - 2), call(-row + 2), call(2 * row - 2), call(2 * row + 2), call(8 * row + 2), call(4, 300), call(row, 256, 300),
                call(row, 129), call(-8 * row - row + 2), call(0, T=1), call(row - 2, T=1)):
        assert bad == INVALID
    if not torch.cuda.is_available():
        for fine in (call(row), call(-row), call(row, 257), call(-row, 300), call(3 * row), call(row + 40, 300), call(9 * row + row),
                     call(row, 256, 300, T=1), call(100 * row, 256, 300)):
            assert fine == CUDA


@pytest.mark.parametrize("read", [False, True])
def test_quant_rows_flags_apart(pkv, read):
    """The flags are an argument that what is written overlaps as little as the others."""
    lib = pkv.load_library()
    for i in (4, 5) if read else (0, 1, 2, 3):
        assert _rows(lib, read, err=at(i) + 8) == INVALID, i
    if not torch.cuda.is_available():
        for i in (0, 1, 2, 3) if read else (4, 5):
            assert _rows(lib, read, err=at(i) + (1 << 30)) == CUDA, i
