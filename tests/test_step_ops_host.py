"""The step operators on the CPU: what their C entry points refuse before any
CUDA call, the chunk plan and workspace sizes, and the binding's checks."""
import ctypes

import pytest
import torch

from paged_kv_cache_67_gb300 import build as libbuild

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4
FAKE = 1 << 20  # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def pkv():
    libbuild.build()
    import paged_kv_cache_67_gb300 as m
    m.load_library()
    return m


def _step(lib, **kw):
    names = ("tables", "held", "held_out", "free", "count", "count_out", "cached", "new", "lens", "cu", "slots", "pos")
    ptr = {n: FAKE + (i << 24) for i, n in enumerate(names)}
    ptr.update({k: v for k, v in kw.items() if k in names})
    return lib.pkv_build_step(*[ptr[n] for n in names], kw.get("B", 4), kw.get("mb", 8), kw.get("nb", 64),
                              kw.get("bs", 16), kw.get("cap", 64), kw.get("T", 32), kw.get("err"), None)


def test_build_step_refusals(pkv):
    lib = pkv.load_library()
    assert _step(lib, B=0, T=0) == OK
    for bad in ({"B": -1}, {"mb": -1}, {"nb": -1}, {"bs": 0}, {"cap": -1}, {"T": -1}, {"nb": 1 << 31}):
        assert _step(lib, **bad) == INVALID, bad
    assert _step(lib, B=16385) == UNSUPPORTED
    assert _step(lib, T=1 << 30) == UNSUPPORTED
    for name in ("tables", "held", "held_out", "free", "count", "count_out", "cached", "new", "lens", "cu", "slots",
                 "pos"):
        assert _step(lib, **{name: None}) == INVALID, name
        assert _step(lib, **{name: FAKE + 2}) == INVALID, name
    assert _step(lib, slots=FAKE + (20 << 24) + 4) == INVALID       # int64, 4-byte aligned only
    # overlaps: an output inside another argument, or an in-place pair that is shifted
    assert _step(lib, lens=FAKE + (7 << 24)) == INVALID             # context_lens on new_lens
    assert _step(lib, held_out=FAKE + (1 << 24) + 4) == INVALID     # held_out one entry into held
    assert _step(lib, cu=FAKE + (6 << 24)) == INVALID
    assert _step(lib, pos=FAKE + (10 << 24) + 64) == INVALID


def test_build_step_bounds(pkv):
    """The largest sizes and the first ones past them: what is refused says so,
    what is not fails for want of a device alone."""
    lib = pkv.load_library()
    assert _step(lib, cap=1 << 30) == UNSUPPORTED
    assert _step(lib, cap=1 << 31) == INVALID
    far = {n: FAKE + (i << 36) for i, n in enumerate(("tables", "held", "held_out", "free", "count", "count_out", "cached",
                                                      "new", "lens", "cu", "slots", "pos"))}
    if not torch.cuda.is_available():
        assert _step(lib, **far, cap=(1 << 30) - 1, T=(1 << 30) - 1, B=16384) not in (OK, INVALID, UNSUPPORTED)


def _rope(lib, **kw):
    D, H, KVH = kw.get("D", 64), kw.get("H", 4), kw.get("KVH", 2)
    axis = kw.get("axis")
    arr = None if axis is None else (ctypes.c_uint8 * len(axis))(*axis)
    return lib.pkv_rope_write(
        kw.get("q_out", 4 * FAKE), kw.get("kc", FAKE), kw.get("vc", FAKE), kw.get("q", FAKE + 4096), kw.get("k", FAKE),
        kw.get("v", FAKE), kw.get("cs", FAKE), kw.get("pos", FAKE), arr, kw.get("slots", FAKE), kw.get("T", 3),
        kw.get("qs", H * D), kw.get("ks", KVH * D), kw.get("vs", KVH * D), kw.get("ps", 3), kw.get("axes", 1), H, KVH,
        D, kw.get("rot", 64), 0, kw.get("maxp", 128), kw.get("nb", 8), kw.get("bs", 16), kw.get("dt", 1), None, None)


def test_rope_write_refusals(pkv):
    lib = pkv.load_library()
    assert _rope(lib, T=0) == OK
    for bad in ({"T": -1}, {"T": 1 << 31}, {"D": 0, "rot": 0}, {"rot": 63}, {"rot": 66}, {"rot": -2}, {"axes": 0},
                {"axes": 5}, {"maxp": -1}, {"nb": -1}, {"bs": 0}, {"H": 0}, {"KVH": 0}, {"dt": 7}, {"qs": 255},
                {"ks": 127}, {"vs": 127}, {"axes": 3, "ps": 2}, {"axis": [0] * 31 + [1]}, {"q_out": None},
                {"kc": None}, {"vc": None}, {"q": None}, {"k": None}, {"v": None}, {"cs": None}, {"pos": None},
                {"slots": None}, {"q": FAKE + 1}, {"cs": FAKE + 2}, {"pos": FAKE + 2}, {"slots": FAKE + 4},
                {"q_out": FAKE + 4096, "qs": 512}, {"q_out": FAKE + 4100}, {"q_out": FAKE - 8}):
        assert _rope(lib, **bad) == INVALID, bad
    assert _rope(lib, D=513, rot=64) == UNSUPPORTED


def test_rope_write_refuses_outputs_on_other_arguments(pkv):
    """q_out on a cache or a table, first and last byte, and a cache on the other."""
    lib = pkv.load_library()
    cache, row = 8 * 16 * 2 * 64 * 2, 4 * 64 * 2          # bytes of a cache, of a token's q
    far = {"q_out": 16 * FAKE, "q": 32 * FAKE, "k": 48 * FAKE, "v": 64 * FAKE, "kc": 80 * FAKE, "vc": 96 * FAKE,
           "cs": 112 * FAKE, "pos": 128 * FAKE, "slots": 144 * FAKE}
    for name, size in (("q", 3 * row), ("k", row // 2 * 3), ("v", row // 2 * 3), ("kc", cache), ("vc", cache),
                       ("cs", 128 * 64 * 4), ("pos", 12), ("slots", 24)):
        for at in (far[name], far[name] - 3 * row + 8, (far[name] + size - 1) // 8 * 8):
            if name != "q" or at != far["q"]:
                assert _rope(lib, **{**far, "q_out": at}) == INVALID, (name, at - far[name])
    assert _rope(lib, **{**far, "vc": far["kc"] + cache - 16}) == INVALID
    assert _rope(lib, **{**far, "vc": far["kc"]}) == INVALID


def _chunk(lib, **kw):
    g = kw.get
    return lib.pkv_chunk_attention(
        g("out", FAKE), g("q", FAKE), g("kc", FAKE), g("vc", FAKE), g("tables", FAKE), g("cu", FAKE), g("lens", FAKE),
        g("slopes"), g("prefix"), g("starts"), g("B", 2), g("total", 6), g("H", 4), g("KVH", 2), g("D", 64),
        g("bs", 16), g("mb", 4), g("nb", 8), ctypes.c_float(g("scale", 0.1)), ctypes.c_float(g("cap", 0.0)), g("window", 0),
        g("dt", 1), g("max_q", 0), g("max_n", 0), g("P", 0), g("ws"), g("wsb", 0), None, None)


def test_chunk_refusals(pkv):
    lib = pkv.load_library()
    assert _chunk(lib, B=0) == OK and _chunk(lib, total=0) == OK
    for bad in ({"B": -1}, {"B": 65536}, {"total": -1}, {"H": 3}, {"KVH": 0}, {"D": 0}, {"bs": 0}, {"mb": -1},
                {"nb": -1}, {"cap": -1.0}, {"cap": float("nan")}, {"cap": float("inf")}, {"cap": 1e-40}, {"scale": float("nan")}, {"scale": float("inf")}, {"window": -1}, {"dt": 5},
                {"max_q": -1}, {"max_n": -1}, {"P": 64}, {"P": -128}, {"out": None}, {"q": None}, {"kc": None},
                {"vc": None}, {"tables": None}, {"cu": None}, {"lens": None}, {"q": FAKE + 1}, {"slopes": FAKE + 2},
                {"prefix": FAKE + 2}, {"starts": FAKE + 1}, {"tables": FAKE + 2}):
        assert _chunk(lib, **bad) == INVALID, bad
    assert _chunk(lib, D=513) == UNSUPPORTED
    assert _chunk(lib) == WORKSPACE                               # none given
    need = pkv.pkv_chunk_workspace_size(2, 6, 4, 2, 64, 16, 4)
    assert _chunk(lib, ws=FAKE, wsb=1024) == WORKSPACE            # too small
    assert _chunk(lib, ws=FAKE + 128, wsb=need) == WORKSPACE      # misaligned


def test_chunk_refuses_more_rows_than_32_bits_count(pkv):
    """2^31 packed (query, head) rows of a KV head and more."""
    lib = pkv.load_library()
    for kw in ({"D": 1, "H": 65535, "KVH": 1, "total": 40000}, {"D": 2, "H": 16384, "KVH": 1, "total": 131072, "dt": 0},
               {"D": 64, "H": 2, "KVH": 1, "total": 1 << 30}):
        assert _chunk(lib, **kw) == UNSUPPORTED, kw
        assert _chunk(lib, **kw, max_q=1000) == WORKSPACE, kw     # with a bound on the queries it is a call
    assert _chunk(lib, D=1, H=65535, KVH=1, total=32767) == WORKSPACE


def test_chunk_refuses_outputs_on_other_arguments(pkv):
    """out and the workspace on any other argument, first and last byte."""
    lib = pkv.load_library()
    names = ("out", "q", "kc", "vc", "tables", "cu", "lens", "slopes", "prefix", "starts", "ws")
    far = {n: (i + 1) * 16 * FAKE for i, n in enumerate(names)}
    need = pkv.pkv_chunk_workspace_size(2, 6, 4, 2, 64, 16, 4)
    rows, cache = 6 * 4 * 64 * 2, 8 * 16 * 2 * 64 * 2
    sizes = {"out": rows, "q": rows, "kc": cache, "vc": cache, "tables": 32, "cu": 12, "lens": 8, "slopes": 16,
             "prefix": 8, "starts": 24, "ws": 65536 * 4}
    for written in ("out", "ws"):
        for name in names:
            if name == written:
                continue
            step = 16 if written == "out" else 256
            for at in (far[name], far[name] - (sizes[written] - 1) // step * step, far[name] + (sizes[name] - 1) // step * step):
                assert _chunk(lib, **{**far, written: at}, wsb=need) == INVALID, (written, name, at - far[name])


def test_chunk_plan_and_workspace(pkv):
    size, plan = pkv.pkv_chunk_workspace_size, pkv.pkv_chunk_plan
    assert size(2, 6, 3, 2, 64, 16, 4) == 0                       # H % KVH
    assert size(2, 6, 4, 2, 64, 16, 4, 0, 0, 100) == 0            # partition not a multiple of 128
    assert plan(2, 6, 3, 2, 64, 16, 4)[0] == 0
    front = 65536 * 4
    for dt in (torch.bfloat16, torch.float32):
        for B, q, H, KVH, D, bs, mb in ((1, 1, 8, 1, 64, 16, 2048), (64, 64, 32, 8, 128, 16, 256), (3, 700, 6, 2, 80, 24, 99),
                                        (8, 8 * 4, 32, 8, 128, 16, 2048), (1, 8192, 32, 8, 128, 16, 512), (2, 40, 8, 2, 64, 16, 12000)):
            for window in (0, 1, 100, 1000, 5000, 32000, 150000):
                for part in (0, 128, 1024):
                    for max_q in (0, -(-q // B)):
                        P, parts, kernel = plan(B, q, H, KVH, D, bs, mb, max_q, 0, window, False, part, dt)
                        assert P % 128 == 0 and 1 <= parts <= 256
                        # every part a unit can touch has a place
                        mq = max_q or q
                        span = min(bs * mb, window + mq + 63) if window else bs * mb
                        assert parts == -(-span // P)
                        least = -(-(-(-span // 256)) // 128) * 128
                        assert part == 0 or P == min(max(part, least), -(-span // 128) * 128)
                        rows = q * H
                        al = lambda x: (x + 255) // 256 * 256
                        need = front + (0 if parts == 1 else 2 * al(rows * parts * 4) + rows * parts * D * 4)
                        assert size(B, q, H, KVH, D, bs, mb, max_q, 0, part) >= need


@pytest.mark.parametrize("keys", [1 << 20, (1 << 20) + 16, 1 << 24, (1 << 28) + 16, 1 << 30])
@pytest.mark.parametrize("part", [0, 1 << 20, 1 << 21, 1 << 29, (1 << 31) - 128])
def test_parts_stay_inside_the_kernels_time_limits(pkv, keys, part):
    """tcgen05: no part longer than 2^20 keys, or than a 256th of the context."""
    P, parts, kernel = pkv.pkv_chunk_plan(2, 512, 8, 2, 128, 16, keys // 16, 256, 0, 0, False, part)
    assert kernel == 2 and P <= max(1 << 20, -(-keys // 256 // 128) * 128 + 128) and parts == -(-keys // P) <= 256
    rows = 512 * 8
    need = 65536 * 4 + (0 if parts == 1 else 2 * rows * parts * 4 + rows * parts * 128 * 4)
    assert pkv.pkv_chunk_workspace_size(2, 512, 8, 2, 128, 16, keys // 16, 256, 0, part) >= need


def test_binding_refuses_before_any_call(pkv):
    """Wrong shapes, types and devices raise ValueError on the host."""
    z = lambda *s, dt=torch.int32: torch.zeros(*s, dtype=dt)
    args = [z(2, 4), z(2), z(2), z(8), z(1), z(1), z(2), z(2), z(2), z(3), z(6, dt=torch.int64), z(6)]
    with pytest.raises(ValueError):
        pkv.pkv_build_step(*args, 8, 16)                          # host tensors
    for i, wrong in ((0, z(2, 4, dt=torch.int64)), (1, z(3)), (3, z(2, 4)), (4, z(2)), (9, z(2)), (10, z(6)), (11, z(5))):
        bad = list(args)
        bad[i] = wrong
        with pytest.raises(ValueError):
            pkv.pkv_build_step(*bad, 8, 16)
    f = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    rope = dict(q_out=f(3, 4, 64), k_cache=f(2, 16, 2, 64), v_cache=f(2, 16, 2, 64), q=f(3, 4, 64), k=f(3, 2, 64),
                v=f(3, 2, 64), cos_sin=torch.zeros(8, 64), positions=z(3), slot_mapping=z(3, dt=torch.int64))
    for change in ({}, {"q": f(3, 4, 32)}, {"k": f(2, 2, 64)}, {"q_out": f(3, 4, 64).float()}, {"cos_sin": torch.zeros(8, 66)},
                   {"cos_sin": torch.zeros(8, 64).double()}, {"positions": z(4)}, {"slot_mapping": z(3)},
                   {"pair_axis": [0] * 31}, {"pair_axis": [1] * 32}, {"q": f(3, 64, 4).transpose(1, 2)}):
        with pytest.raises(ValueError):
            pkv.pkv_rope_write(**{**rope, **change})
    chunk = dict(out=f(3, 4, 64), q=f(3, 4, 64), k_cache=f(2, 16, 2, 64), v_cache=f(2, 16, 2, 64), block_tables=z(2, 2),
                 cu_seqlens_q=z(3), context_lens=z(2), scale=0.1)
    for change in ({}, {"out": f(2, 4, 64)}, {"cu_seqlens_q": z(2)}, {"slopes": torch.zeros(3)}, {"prefix_lens": z(3)},
                   {"kv_starts": z(2)}, {"block_tables": z(3, 2)}, {"q": f(3, 4, 64).float()}):
        with pytest.raises(ValueError):
            pkv.pkv_chunk_attention(**{**chunk, **change})
