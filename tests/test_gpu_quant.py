"""pkv_quant_write, pkv_quant_read and pkv_quant_decode_attention against their
restatement in 64 bits.

Tolerances, from the arithmetic.  Write: every code, scale and zero point is
fixed to the bit by the definition, so the comparison is exact.  Read: one
fp32 product (half a step of 2^-24), then the output type's rounding: for fp32
the product itself is the output, exactly rounded, and equality is asked of all
three.  Decode: with A the largest scale * sum |q_d k_d| log2 e of a visible
key, a score is off by A (2^-22 for the two halves of a query + 2^-23 a sum of
16 products, D / 16 of them, + 2^-21 for its scale and cap); a weight by that
times ln 2 and 2^-21 for ex2, on either side of the division; sums over n keys
by 2^-23 a step of 32 keys; bf16's weights, held in fp16, by its half step, 2^-11; the output by its own
half step.  All times the largest visible |v|, or |out| at most that."""
import math

import pytest
import torch

import paged_kv_cache_67_gb300 as pkv
import quant_beam_reference as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def empty_cache(nb, bs, kvh, d, fmt, fill=0x7f, params=math.nan):
    """A cache whose unwritten rows are poison: e4m3 NaN codes, NaN scales."""
    dd = d // 2 if fmt == "int4" else d
    codes = [torch.full((nb, bs, kvh, dd), fill, dtype=torch.uint8).view(ref.FORMATS[fmt]) for _ in range(2)]
    shape = (nb, kvh, bs) + ((2,) if fmt == "int4" else ())
    return codes + [torch.full(shape, params) for _ in range(2)]


def rows_like(T, kvh, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, 2, kvh, d, generator=g) * torch.exp(torch.randn(2, kvh, d, generator=g) * 0.5)
    return x.to(dtype)


def write_reference(cache, k, v, slots, fmt):
    """`cache` (CPU) after the write."""
    out = [t.clone() for t in cache]
    bs = out[0].shape[1]
    for s, x in enumerate((k, v)):
        c, scale, zero = ref.quantise(x, fmt)
        for i, slot in enumerate(slots.tolist()):
            if not 0 <= slot < out[0].shape[0] * bs:
                continue
            b, o = divmod(slot, bs)
            out[s].view(torch.uint8)[b, o] = ref.stored(c[i], fmt).view(torch.uint8)
            out[2 + s][b, :, o] = torch.stack([scale[i], zero[i]], -1).float() if fmt == "int4" else scale[i].float()
    return out


def same(got, want, what=""):
    for g, w in zip(got, want):
        g, w = g.cpu(), w.cpu()
        if g.dtype == torch.float32:
            assert torch.equal(torch.isnan(g), torch.isnan(w)), what
            g, w = g.nan_to_num(0.0), w.nan_to_num(0.0)
        else:
            g, w = g.view(torch.uint8), w.view(torch.uint8)
        assert torch.equal(g, w), (what, int((g != w).sum()))


SHAPES = [(1, 64), (2, 80), (8, 128), (3, 96), (1, 256), (2, 192), (1, 512), (5, 2), (2, 36), (1, 130)]


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "int4"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kvh,d", SHAPES)
def test_write_and_read(fmt, dtype, kvh, d):
    bs = 16 if d > 64 else 3
    T = 37
    nb = -(-T * 2 // bs)
    x = rows_like(T, kvh, d, dtype, 1)
    x[3] = 0                                                    # zeros
    x[4, 0, 0, 0], x[5, 1, 0, -1] = math.inf, math.nan          # not finite
    x[6] = x[6].abs() + 1                                       # one sign
    x[7] = -x[7].abs() - 1
    x[8, :, :, 0] = 300.0                                       # an outlier
    if dtype != torch.float16:
        x[9] *= 1e-32
        x[10] *= 1e-30
        x[11] = x[11].sign() * 3e38                             # a range over fp32's
    slots = torch.randperm(nb * bs, generator=torch.Generator().manual_seed(2))[:T].to(torch.int64)
    slots[20], slots[21], slots[22] = -1, nb * bs, 1 << 40      # padding, past the pool
    cache = empty_cache(nb, bs, kvh, d, fmt)
    want = write_reference(cache, x[:, 0], x[:, 1], slots, fmt)
    dev = [t.to(DEV) for t in cache]
    xd = x.to(DEV)                                              # k and v side by side: strided rows
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.pkv_quant_write(*dev, xd[:, 0], xd[:, 1], slots.to(DEV), err_flags=err)
    torch.cuda.synchronize()
    assert int(err) == pkv.FLAG_SLOT_OUT_OF_RANGE
    same(dev, want, "write")
    # read back, some slots twice
    back = torch.cat([slots, slots[:5]])
    out = [torch.full((T + 5, kvh, d), 7.0, dtype=dtype, device=DEV) for _ in range(2)]
    err.zero_()
    pkv.pkv_quant_read(*out, *dev, back.to(DEV), err_flags=err)
    torch.cuda.synchronize()
    assert int(err) == pkv.FLAG_SLOT_OUT_OF_RANGE
    for s in range(2):
        for i, slot in enumerate(back.tolist()):
            if 0 <= slot < nb * bs:
                b, o = divmod(slot, bs)
                # (a product of a code and a float32: fp32 rounds it once, then the type)
                w = ref.values(want[s][b, o], want[2 + s][b, :, o], fmt).float().to(dtype)
            else:
                w = torch.full((kvh, d), 7.0, dtype=dtype)
            g = out[s][i].cpu()
            assert torch.equal(torch.isnan(g), torch.isnan(w)), (i, s)
            assert torch.equal(g.nan_to_num(0.0), w.nan_to_num(0.0)), (i, s)


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "int4"])
@pytest.mark.parametrize("dtype", TYPES)
def test_rows_anywhere(fmt, dtype):
    """Tensors that start at any element, strides of any size, one token."""
    kvh, d, bs, nb = 2, 64, 4, 6
    for T, shift, pad in ((1, 0, 0), (5, 1, 0), (5, 2, 3), (9, 3, 8), (9, 0, 6)):
        x = rows_like(T, kvh, d, dtype, T + shift)
        row = kvh * d + pad
        flat = torch.zeros(2, shift + T * row, dtype=dtype, device=DEV)
        views = [flat[s][shift:].view(T, row)[:, :kvh * d].view(T, kvh, d) for s in range(2)]
        for s in range(2):
            views[s].copy_(x[:, s])
        slots = torch.randperm(nb * bs, generator=torch.Generator().manual_seed(T))[:T].to(torch.int64)
        cache = empty_cache(nb, bs, kvh, d, fmt)
        want = write_reference(cache, x[:, 0], x[:, 1], slots, fmt)
        # codes that start at an odd byte
        dev = []
        for i, t in enumerate(cache):
            buf = torch.zeros(t.numel() + 3, dtype=torch.uint8 if i < 2 else torch.float32, device=DEV)
            buf = buf[shift % 4:][:t.numel()]
            dev.append((buf.view(t.dtype) if i < 2 else buf).view(t.shape).copy_(t.to(DEV)))
        pkv.pkv_quant_write(*dev, *views, slots.to(DEV))
        same(dev, want, (T, shift, pad))
        before = flat.clone()
        for v in views:
            v.zero_()
        pkv.pkv_quant_read(*views, *dev, slots.to(DEV))
        gap = flat[:, shift:].view(2, T, row)[:, :, kvh * d:]
        assert torch.equal(gap, before[:, shift:].view(2, T, row)[:, :, kvh * d:])
        for s in range(2):
            for i, slot in enumerate(slots.tolist()):
                b, o = divmod(slot, bs)
                w = ref.values(want[s][b, o], want[2 + s][b, :, o], fmt).float().to(dtype)
                assert torch.equal(views[s][i].cpu(), w)


def test_rows_past_32_bits():
    """A cache of more than 2^32 bytes: rows at its far end."""
    nb, bs, kvh, d = 40000, 16, 64, 128                          # 5.2 GB of codes each
    codes = [torch.zeros(nb, bs, kvh, d, dtype=torch.int8, device=DEV) for _ in range(2)]
    params = [torch.zeros(nb, kvh, bs, device=DEV) for _ in range(2)]
    x = rows_like(3, kvh, d, torch.bfloat16, 5)
    slots = torch.tensor([nb * bs - 1, 0, nb * bs - 17])
    pkv.pkv_quant_write(*codes, *params, x[:, 0].to(DEV), x[:, 1].to(DEV), slots.to(DEV))
    out = [torch.zeros(3, kvh, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    pkv.pkv_quant_read(*out, *codes, *params, slots.to(DEV))
    for s in range(2):
        c, scale, zero = ref.quantise(x[:, s], "int8")
        assert torch.equal(out[s].cpu(), (c * scale[..., None]).float().to(torch.bfloat16))
        assert int((params[s] != 0).sum()) == 3 * kvh
    # and the decode over them: one sequence in the last blocks
    q = torch.randn(1, kvh, d, device=DEV).to(torch.bfloat16)
    tables = torch.tensor([[nb - 1, nb - 2]], dtype=torch.int32, device=DEV)
    o = torch.empty_like(q)
    lens = torch.tensor([16], dtype=torch.int32, device=DEV)
    ws = pkv.QuantDecodeWorkspace(1, kvh, kvh, d, bs, 2)
    pkv.pkv_quant_decode_attention(o, q, *codes, *params, tables, lens, 0.05, workspace=ws)
    k, v = (ref.values(c[nb - 1].cpu(), p[nb - 1].transpose(0, 1).cpu(), "int8") for c, p in zip(codes, params))
    want = ref.decode(q[0].cpu(), k, v, 0.05)
    assert (o[0].cpu().double() - want).abs().max() <= 2 * HALF[torch.bfloat16] * v.abs().max()


# ------------------------------------------------------------------- decode

class Case:
    def __init__(self, lens, H, KVH, D, bs, fmt, dtype, seed=0, qscale=1.0, spread=0.0, spare=3):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.fmt, self.dtype = lens, fmt, dtype
        self.H, self.KVH, self.D, self.bs = H, KVH, D, bs
        need = [-(-n // bs) for n in lens]
        self.nb = sum(need) + spare
        perm = torch.randperm(self.nb, generator=g).to(torch.int32)
        self.tables = torch.full((len(lens), max(need + [1]) + 1), 99999, dtype=torch.int32)
        self.cache = empty_cache(self.nb, bs, KVH, D, fmt)
        self.k, self.v, at = [], [], 0
        for b, n in enumerate(lens):
            self.tables[b, :need[b]] = perm[at:at + need[b]]
            x = torch.randn(2, n, KVH, D, generator=g)
            x *= torch.exp2(spread * torch.randn(2, n, 1, 1, generator=g))
            for s, keep in ((0, self.k), (1, self.v)):
                codes, params = self._codes(x[s], g, fmt, spread, s)
                for t in range(n):
                    blk, o = int(perm[at + t // bs]), t % bs
                    self.cache[s].view(torch.uint8)[blk, o] = codes[t].view(torch.uint8)
                    self.cache[2 + s][blk, :, o] = params[t]
                keep.append(ref.values(codes, params, fmt) if n else torch.zeros(0, KVH, D, dtype=torch.float64))
            at += need[b]
        self.q = (torch.randn(len(lens), H, D, generator=g) * qscale).to(dtype)

    @staticmethod
    def _codes(x, g, fmt, spread, s):
        """Codes and params straight from tensor arithmetic (any valid cache will do)."""
        n, kvh, d = x.shape
        if fmt == "int4":
            c = torch.randint(0, 16, (n, kvh, d), generator=g)
            p = torch.stack([0.2 * torch.exp2(spread * torch.randn(n, kvh, generator=g)),
                             torch.randint(0, 16, (n, kvh), generator=g).float()], -1)
            return ref.stored(c, fmt), p
        top = 127.0 if fmt == "int8" else 448.0
        scale = x.abs().amax(-1) / top if n else torch.zeros(0, kvh)
        c = x / scale[..., None]
        return (c.round().to(torch.int8) if fmt == "int8" else c.clamp(-448, 448).to(torch.float8_e4m3fn)), scale

    def on(self, dev):
        return [t.to(dev) for t in (self.q, *self.cache, self.tables, torch.tensor(self.lens, dtype=torch.int32))]

    def run(self, scale, softcap=0.0, window=0, P=0, max_n=0, flags=0, ws=None):
        q, kc, vc, kp, vp, tables, lens = self.on(DEV)
        out = torch.full_like(q, math.nan)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        ws = ws or pkv.QuantDecodeWorkspace(len(self.lens), self.H, self.KVH, self.D, self.bs, tables.shape[1], max_n, P)
        for _ in range(2):                                     # the second finds the workspace as the first left it
            pkv.pkv_quant_decode_attention(out, q, kc, vc, kp, vp, tables, lens, scale, softcap=softcap, window=window,
                                           max_context_len=max_n, partition_size=P, workspace=ws, err_flags=err)
        torch.cuda.synchronize()
        assert int(err) == flags
        return out.cpu()

    def check(self, out, scale, softcap=0.0, window=0):
        G = self.H // self.KVH
        for b, n in enumerate(self.lens):
            lo = max(0, n - window) if window else 0
            want = ref.decode(self.q[b], self.k[b], self.v[b], scale, softcap, window)
            if n == 0:
                assert torch.equal(out[b].double(), want)
                continue
            for h in range(self.H):
                k, v = self.k[b][lo:n, h // G], self.v[b][lo:n, h // G]
                A = abs(scale) * float((k.abs() @ self.q[b, h].double().abs()).max()) * 1.4427
                x = A * (2.0 ** -22 + self.D / 16 * 2.0 ** -23 + 2.0 ** -21)
                tol = 2 * (x * 0.6932 + 2.0 ** -21) + 2.0 ** -23 * (n / 32 + 8) + HALF[self.dtype]
                if self.dtype == torch.bfloat16:
                    tol += 2.0 ** -11
                off = float((out[b, h].double() - want[h]).abs().max())
                assert off <= tol * float(v.abs().max()), (b, n, h, off / float(v.abs().max()), tol)


FMTS = ["int8", "e4m3", "int4"]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H,KVH,D,bs", [(4, 4, 64, 16), (8, 2, 128, 16), (8, 1, 128, 32), (16, 1, 256, 32), (12, 2, 96, 16),
                                        (7, 1, 80, 16), (10, 2, 192, 24), (33, 3, 128, 1), (4, 2, 72, 16), (3, 1, 512, 7),
                                        (24, 1, 64, 5), (2, 2, 10, 16)])
def test_decode_shapes(fmt, dtype, H, KVH, D, bs):
    case = Case([1, 0, 31, 32, 33, 257, 700], H, KVH, D, bs, fmt, dtype, seed=D + H)
    scale = 1 / math.sqrt(D)
    case.check(case.run(scale), scale)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("softcap,window,P", [(0.0, 0, 128), (30.0, 0, 0), (30.0, 100, 128), (0.0, 1, 0), (0.0, 33, 128),
                                              (1e6, 0, 0), (0.0, 128, 0), (2.0, 1000, 256)])
def test_decode_forms(fmt, dtype, softcap, window, P):
    case = Case([900, 1, 128, 129, 500], 8, 2, 128, 16, fmt, dtype, seed=3, qscale=2.0)
    scale = 1 / math.sqrt(128)
    case.check(case.run(scale, softcap, window, P), scale, softcap, window)
    case = Case([300, 7], 6, 1, 40, 9, fmt, dtype, seed=4, qscale=2.0)          # the CUDA cores
    case.check(case.run(0.2, softcap, window, P), 0.2, softcap, window)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", TYPES)
def test_decode_spread_scales(fmt, dtype):
    """Rows whose scales lie far apart, negative softmax scale, queries at the
    ends of their type's range, zero queries."""
    case = Case([400, 64], 4, 2, 128, 16, fmt, dtype, seed=9, qscale=0.2, spread=3.0)
    case.check(case.run(0.02), 0.02)
    case.check(case.run(-0.02), -0.02)
    tiny = 2.0 ** -13 if dtype == torch.float16 else 2.0 ** -90
    case.q = (case.q.double() * tiny).to(dtype)
    case.check(case.run(0.02 / tiny), 0.02 / tiny)
    case.q.zero_()
    case.check(case.run(0.5), 0.5)


@pytest.mark.parametrize("fmt", FMTS)
def test_decode_zero_and_nan_rows(fmt):
    case = Case([200, 200, 200], 8, 2, 128, 16, fmt, torch.bfloat16, seed=11)
    bs = 16
    # sequence 0: every value row of head 0 is zero; sequence 1: one NaN scale in head 1
    for t in range(200):
        blk = int(case.tables[0, t // bs])
        case.cache[3][blk, 0, t % bs] = 0.0
    case.v[0][:, 0] = 0.0
    case.cache[2][int(case.tables[1, 77 // bs]), 1, 77 % bs] = math.nan
    out = case.run(0.09)
    assert torch.isnan(out[1, 4:]).all() and not torch.isnan(out[1, :4]).any()
    assert torch.equal(out[0, :4], torch.zeros(4, 128, dtype=torch.bfloat16))
    keep = case.lens
    case.lens = [200]                                               # (sequence 0's second head)
    want = ref.decode(case.q[0], case.k[0], case.v[0], 0.09)
    assert (out[0, 4:].double() - want[4:]).abs().max() <= 2 * HALF[torch.bfloat16] * case.v[0].abs().max()
    case.lens = keep


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [128, 40])
def test_decode_flags(fmt, D):
    case = Case([100, 50, 60], 4, 2, D, 16, fmt, torch.bfloat16, seed=1)
    good = case.run(0.1)
    bad = case.tables.clone()
    case.tables[1, 2] = case.nb + 5                                 # a bad entry: its sequence alone
    out = case.run(0.1, flags=pkv.FLAG_BLOCK_OUT_OF_RANGE)
    assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    case.tables = bad
    case.lens = [-3, 1 << 20, 60]
    out = case.run(0.1, flags=pkv.FLAG_CONTEXT_NEGATIVE | pkv.FLAG_CONTEXT_TOO_LONG | pkv.FLAG_BLOCK_OUT_OF_RANGE)
    assert torch.equal(out[0], torch.zeros_like(out[0])) and torch.equal(out[2], good[2])
    case.lens = [100, 50, 60]
    out = case.run(0.1, max_n=60, flags=pkv.FLAG_CONTEXT_OVER_HINT)
    assert torch.equal(out[1:], good[1:])


@pytest.mark.parametrize("D", [128, 40])
def test_decode_table_without_columns(D):
    """A table of no columns holds no context: lengths are flagged, rows are
    zeros, and the entry that is not there is not read."""
    import ctypes
    lib = pkv.load_library()
    case = Case([40, 0], 4, 2, D, 16, "int8", torch.bfloat16)
    q, kc, vc, kp, vp, tables, lens = case.on(DEV)
    tables.fill_(0x7fffffff)
    out = torch.full_like(q, math.nan)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device=DEV)
    f, p = ctypes.c_float, lambda t: ctypes.c_void_p(t.data_ptr())
    for max_n in (0, 5):
        out.fill_(math.nan)
        assert lib.pkv_quant_decode_attention(p(out), p(q), p(kc), p(vc), p(kp), p(vp), p(tables), p(lens), 2, 4, 2, D, 16, 0,
                                              case.nb, f(0.1), f(0.0), 0, 0, 1, max_n, 0, p(ws), ws.numel(), p(err), None) == 0
        torch.cuda.synchronize()
        assert int(err) == pkv.FLAG_CONTEXT_TOO_LONG
        assert torch.equal(out, torch.zeros_like(out))


@pytest.mark.parametrize("fmt", FMTS)
def test_decode_long_split(fmt):
    """One long context over many parts, and repeated bit for bit."""
    case = Case([20000], 4, 1, 128, 16, fmt, torch.float32, seed=2)
    scale = 1 / math.sqrt(128)
    out = case.run(scale)
    case.check(out, scale)
    assert torch.equal(out, case.run(scale))
    case.check(case.run(scale, P=128), scale)


def test_decode_many_units():
    """More (sequence, head) units than the workspace counts: whole."""
    B, KVH, D, bs = 16400, 4, 64, 16
    g = torch.Generator().manual_seed(0)
    codes = [torch.randint(-127, 128, (8, bs, KVH, D), generator=g, dtype=torch.int8) for _ in range(2)]
    params = [torch.rand(8, KVH, bs, generator=g) * 0.02 for _ in range(2)]
    tables = torch.randint(0, 8, (B, 20), generator=g, dtype=torch.int32)
    lens = torch.randint(0, 300, (B,), generator=g, dtype=torch.int32)
    q = torch.randn(B, KVH, D, generator=g).to(torch.bfloat16)
    out = torch.full_like(q, math.nan, device=DEV)
    ws = pkv.QuantDecodeWorkspace(B, KVH, KVH, D, bs, 20, 0, 128)
    pkv.pkv_quant_decode_attention(out, q.to(DEV), *[t.to(DEV) for t in codes + params], tables.to(DEV), lens.to(DEV),
                                   0.125, partition_size=128, workspace=ws)
    out = out.cpu()
    for b in range(0, B, 1171):
        n = int(lens[b])
        k, v = (ref.values(c[tables[b].long()].flatten(0, 1)[:n], p[tables[b].long()].transpose(1, 2).flatten(0, 1)[:n], "int8")
                for c, p in zip(codes, params))
        want = ref.decode(q[b], k, v, 0.125)
        assert (out[b].double() - want).abs().max() <= 1.1 * HALF[torch.bfloat16] * 127 * 0.02


@pytest.mark.parametrize("fmt", FMTS)
def test_decode_streams_and_graph(fmt):
    """Two calls on two streams with workspaces of their own, and a captured
    step (write, then decode) replayed on new inputs."""
    cases = [Case([300, 90], 8, 2, 128, 16, fmt, torch.bfloat16, seed=s) for s in (21, 22)]
    alone = [c.run(0.1) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    dev = [c.on(DEV) for c in cases]
    outs = [torch.full_like(d[0], math.nan) for d in dev]
    wss = [pkv.QuantDecodeWorkspace(2, 8, 2, 128, 16, c.tables.shape[1]) for c in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for d, o, ws, st in zip(dev, outs, wss, streams):
            pkv.pkv_quant_decode_attention(o, *d[:5], d[5], d[6], 0.1, workspace=ws, stream=st)
    torch.cuda.synchronize()
    for o, a in zip(outs, alone):
        assert torch.equal(o.cpu(), a)
    # captured: sequence b's next token goes to position lens[b]
    c, d = cases[0], dev[0]
    k, v = torch.zeros(2, 2, 128, dtype=torch.bfloat16, device=DEV), torch.zeros(2, 2, 128, dtype=torch.bfloat16, device=DEV)
    slots, lens = torch.full((2,), -1, dtype=torch.int64, device=DEV), d[6].clone()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        pkv.pkv_quant_write(*d[1:5], k, v, slots, stream=side)
        pkv.pkv_quant_decode_attention(outs[0], d[0], *d[1:5], d[5], lens, 0.1, workspace=wss[0], stream=side)
    history = [[x.clone() for x in c.k], [x.clone() for x in c.v]]
    for step in range(3):
        x = rows_like(2, 2, 128, torch.bfloat16, 40 + step)
        k.copy_(x[:, 0]), v.copy_(x[:, 1])
        n = [int(t) for t in lens]
        slots.copy_(torch.tensor([int(c.tables[b, n[b] // 16]) * 16 + n[b] % 16 for b in range(2)]))
        lens += 1
        graph.replay()
        torch.cuda.synchronize()
        for s in range(2):
            codes, scale, zero = ref.quantise(x[:, s], fmt)
            for b in range(2):
                row = scale[b][:, None] * (codes[b] - (zero[b][:, None] if fmt == "int4" else 0))
                history[s][b] = torch.cat([history[s][b], row[None]])
        for b in range(2):
            want = ref.decode(d[0][b].cpu(), history[0][b], history[1][b], 0.1)
            top = float(history[1][b].abs().max())
            assert (outs[0][b].cpu().double() - want).abs().max() <= 1.1 * HALF[torch.bfloat16] * top


@pytest.mark.parametrize("fmt", FMTS)
def test_prefill_over_read_back(fmt):
    """A chunk of new queries over a quantised context: its rows read back into
    a 16-bit paged cache, then pkv_chunk_attention."""
    D, KVH, H, bs, n, ql = 128, 2, 8, 16, 200, 40
    case = Case([n], H, KVH, D, bs, fmt, torch.bfloat16, seed=30)
    d = case.on(DEV)
    nb = -(-n // bs)
    pos = torch.arange(n, device=DEV)
    slots = d[5][0].long()[pos // bs] * bs + pos % bs
    scratch = [torch.zeros(nb, bs, KVH, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    pkv.pkv_quant_read(*[t.view(-1, KVH, D)[:n] for t in scratch], *d[1:5], slots)
    q = torch.randn(ql, H, D, device=DEV).to(torch.bfloat16)
    out = torch.empty_like(q)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    tables = torch.arange(nb, dtype=torch.int32, device=DEV)[None]
    ws = pkv.ChunkWorkspace(1, ql, H, KVH, D, bs, nb, ql, n)
    pkv.pkv_chunk_attention(out, q, *scratch, tables, i32([0, ql]), i32([n]), 0.088, max_q_len=ql, max_context_len=n,
                            workspace=ws)
    k, v = (x[0].to(torch.bfloat16).double() for x in (case.k, case.v))
    for i in range(ql):
        m = n - ql + i + 1
        want = ref.decode(q[i].cpu(), k[:m], v[:m], 0.088)
        assert (out[i].cpu().double() - want).abs().max() <= (2.0 ** -7 + 2.0 ** -18) * float(v[:m].abs().max())


def off_by(case, b, h, scale):
    """What the 32-bit arithmetic of a score, its weight and the sums may be off
    by, of the largest |v| (see the head; the weights' two parts: 2^-22)."""
    G, n = case.H // case.KVH, case.lens[b]
    k = case.k[b][:, h // G].abs()
    A = abs(scale) * float((k @ case.q[b, h].double().abs()).max()) * 1.4427
    x = A * (2.0 ** -22 + case.D / 16 * 2.0 ** -23 + 2.0 ** -21)
    return 2 * (x * 0.6932 + 2.0 ** -21) + 2.0 ** -22 + 2.0 ** -23 * (n / 32 + 8)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H,KVH,D", [(4, 4, 64), (8, 2, 128), (4, 1, 256), (8, 1, 128), (16, 2, 96)])
def test_decode_weights_keep_their_bits(fmt, dtype, H, KVH, D):
    """Weights are not rounded to 16 bits.  Few keys of nearly equal weight and
    values of both signs: outputs near 0, whose own rounding is small, show what
    a weight lost.  Each is off by its own half step and the 32-bit form's."""
    case = Case([2, 3, 5, 37, 64], H, KVH, D, 16, fmt, dtype, seed=50 + D, qscale=0.1)
    scale = 1 / math.sqrt(D)
    out = case.run(scale)
    for b in range(len(case.lens)):
        want = ref.decode(case.q[b], case.k[b], case.v[b], scale)
        for h in range(H):
            top = float(case.v[b][:, h // (H // KVH)].abs().max())
            # (an output below fp16's normal numbers: half of 2^-24)
            room = HALF[dtype] * want[h].abs() + 1.01 * off_by(case, b, h, scale) * top + 2.0 ** -25
            off = (out[b, h].double() - want[h]).abs()
            assert (off <= room).all(), (b, h, float((off - room).max()))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H,KVH", [(8, 2), (8, 1)])
def test_decode_large_queries(fmt, dtype, H, KVH):
    """Queries up to the end of their type's range, with a scale to match: a
    score is what it is for ordinary ones."""
    case = Case([400, 33], H, KVH, 128, 16, fmt, dtype, seed=60, qscale=0.05)
    q = case.q.clone()
    for power in (99, 101, 110, 124):
        case.q = (q.double() * 2.0 ** power).to(dtype)
        case.check(case.run(0.5 * 2.0 ** -power), 0.5 * 2.0 ** -power)
    case.q = torch.zeros_like(q)
    case.q[..., 5] = torch.finfo(dtype).max
    case.check(case.run(2.0 ** -126), 2.0 ** -126)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("H,KVH", [(8, 2), (8, 1)])
def test_decode_large_queries_of_small_keys(fmt, H, KVH):
    """A query of 2^120 and keys of 2^-100: the score is in range (one key: its
    value comes out), though the query times the codes is not."""
    case = Case([1], H, KVH, 128, 16, fmt, torch.float32, seed=61)
    case.q = case.q * 2.0 ** 120
    p = case.cache[2][..., 0] if fmt == "int4" else case.cache[2]
    p *= 2.0 ** -100
    out = case.run(1.0)
    want = case.v[0][0].repeat_interleave(H // KVH, 0)
    assert (out[0].double() - want).abs().max() <= 2.0 ** -20 * want.abs().max()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad", [0, 5])
def test_read_into_one_buffer(fmt, dtype, pad):
    """K and V read back side by side, as one projection's output has them (the
    layout that the write takes)."""
    kvh, d, bs, nb, T = 2, 64, 16, 4, 40
    x = rows_like(T, kvh, d, dtype, 3).to(DEV)
    slots = torch.randperm(nb * bs, generator=torch.Generator().manual_seed(4))[:T].to(DEV)
    cache = [t.to(DEV) for t in empty_cache(nb, bs, kvh, d, fmt)]
    pkv.pkv_quant_write(*cache, x[:, 0], x[:, 1], slots)
    apart = [torch.zeros(T, kvh, d, dtype=dtype, device=DEV) for _ in range(2)]
    pkv.pkv_quant_read(*apart, *cache, slots)
    for first in (0, 1):
        buf = torch.full((T, 2 * kvh * d + pad), 7.0, dtype=dtype, device=DEV)
        halves = [buf[:, i * kvh * d:(i + 1) * kvh * d].view(T, kvh, d) for i in (first, 1 - first)]
        pkv.pkv_quant_read(*halves, *cache, slots)
        for got, want in zip(halves, apart):
            assert torch.equal(got, want)
        assert (buf[:, 2 * kvh * d:] == 7).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H,KVH,D,bs", [(32, 8, 64, 16), (16, 16, 64, 32), (64, 8, 64, 16), (8, 8, 128, 24), (24, 8, 96, 16)])
def test_decode_eight_heads_at_once(fmt, dtype, H, KVH, D, bs):
    """Eight KV heads (or head groups) a token: warps of two CTAs walk the same
    tokens.  Ragged lengths, empty sequences, splits and joins, windows."""
    case = Case([0, 1, 700, 31, 32, 0, 33, 257, 2100, 0], H, KVH, D, bs, fmt, dtype, seed=70 + H + D)
    scale = 1 / math.sqrt(D)
    out = case.run(scale)
    case.check(out, scale)
    assert torch.equal(out, case.run(scale))
    case.check(case.run(scale, P=128), scale)
    case.check(case.run(scale, 20.0, 100), scale, 20.0, 100)
    case.check(case.run(scale, window=33, P=1 << 20), scale, window=33)


@pytest.mark.parametrize("shift", [0, 1])
def test_decode_more_units_than_counters(shift):
    """The CUDA cores: (sequence, KV head) units past the workspace's counters
    are not split, whatever partition is asked for.  A head size of 40, and one
    of 64 whose codes begin at an odd byte."""
    B, KVH, D, bs = 16400, 4, 64 if shift else 40, 16
    g = torch.Generator().manual_seed(1)
    codes = [torch.randint(-127, 128, (8, bs, KVH, D), generator=g, dtype=torch.int8) for _ in range(2)]
    params = [torch.rand(8, KVH, bs, generator=g) * 0.02 for _ in range(2)]
    tables = torch.randint(0, 8, (B, 19), generator=g, dtype=torch.int32)
    lens = torch.randint(0, 301, (B,), generator=g, dtype=torch.int32)
    q = torch.randn(B, KVH, D, generator=g).to(torch.bfloat16)
    dev = []
    for t in codes:
        buf = torch.zeros(t.numel() + shift, dtype=torch.int8, device=DEV)[shift:]
        dev.append(buf.view(t.shape).copy_(t.to(DEV)))
    dev += [t.to(DEV) for t in params]
    out = torch.full_like(q, math.nan, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = pkv.QuantDecodeWorkspace(B, KVH, KVH, D, bs, 19, 0, 128)
    for _ in range(2):
        pkv.pkv_quant_decode_attention(out, q.to(DEV), *dev, tables.to(DEV), lens.to(DEV), 0.05, partition_size=128,
                                       workspace=ws, err_flags=err)
    out = out.cpu()
    assert int(err) == 0 and torch.isfinite(out).all()
    for b in [*range(0, B, 211), *range(B - 30, B)]:           # (the last are past the counters)
        n = int(lens[b])
        k, v = (ref.values(c[tables[b].long()].flatten(0, 1)[:n], p[tables[b].long()].transpose(1, 2).flatten(0, 1)[:n], "int8")
                for c, p in zip(codes, params))
        want = ref.decode(q[b], k, v, 0.05)
        if n == 0:
            assert torch.equal(out[b].double(), want)
            continue
        # a score's sum of D products and 5 steps of a warp's, its weight's, the sums' over n keys
        A = 0.05 * float((k.abs() * q[b].double().abs()).sum(-1).max()) * 1.4427
        tol = 2 * (A * (D / 32 + 8) * 2.0 ** -23 * 0.6932 + 2.0 ** -21) + 2.0 ** -23 * (n / 8 + 16)
        room = HALF[torch.bfloat16] * want.abs() + 1.01 * tol * v.abs().amax((0, 2))[:, None]
        assert ((out[b].double() - want).abs() <= room).all()
