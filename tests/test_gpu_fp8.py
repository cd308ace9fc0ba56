"""The 8-bit floating-point operators on the GPU against the format's
definition and fp64 sums.

Quantising and reading back are exact steps, so codes, scales and values are
compared bit for bit.  Products: an output y of value ref may be off by
  L * gamma_n * S   the fp32 sum of n terms (S = sum |a b| + |bias| + |R|,
                    gamma_n with u = 2^-23: the matrix cores' additions need
                    not round to nearest), through the activation's slope L,
  2^-15 |ref|       one fp32 evaluation of the activation,
  half a step       of the output type at |ref| plus the above,
and for 16-bit outputs, within the sum,
  7 * 2^-13 * T     the 8-bit matrix instructions add the products of eight
                    neighbouring k in fixed point: each is cut off, towards zero, at
                    2^(e - 13), e the largest sum of two codes' exponents among the eight
                    (a subnormal code has the smallest normal one).  The product
                    that e comes from loses nothing, so seven lose less than that
                    each, and 2^e is at most the sum of the eight 2^(sum of exponents):
                    T = P_A . P_B^T, P the powers of two with the codes' exponents
                    (0 for a code of zero) times their scales.
test_sums_of_eight checks that rule itself, product by product."""
import numpy as np
import pytest

import fp8_ref as f8
import test_gpu_mxfp4 as mx4
from gpu_helpers import O
from oracle.compare import ETA_ACT, gamma, slope_bound, ulp
from test_gpu_mxfp4 import TD, dev, edges_intact, f64, guarded

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

FD = {"f8e4m3": torch.float8_e4m3fn, "f8e5m2": torch.float8_e5m2}


@pytest.fixture(scope="module")
def ba():
    import conv_bias_activation_amd as m
    return m


def codes_dev(c, fmt):
    return torch.from_numpy(np.ascontiguousarray(c)).cuda().view(FD[fmt])


def packed(ba, rows, K, fmt, block_rows=1):
    """Guarded room for codes and scales."""
    cs, ss = ba.fp8_shapes(rows, K, block_rows)
    codes, cbuf = guarded(cs, torch.uint8, 0xA5)
    scales, sbuf = guarded(ss, torch.uint8, 0xA5)
    return codes.view(FD[fmt]), scales, cbuf, sbuf


def check_quantized(codes, scales, cbuf, sbuf, x, fmt, block_rows):
    want_c, want_s = f8.quantize(x, fmt, block_rows)
    got_c = codes.view(torch.uint8).cpu().numpy()
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(got_c, want_c), np.argwhere(got_c != want_c)[:4]
    assert edges_intact(cbuf, codes.numel(), 0xA5) and edges_intact(sbuf, scales.numel(), 0xA5)


# ---- quantisation -------------------------------------------------------------------

def special_rows(rows, K, dt, seed):
    """Normal values of many sizes with zeros, ties, the formats' and the
    type's borders, subnormals, infinities and NaN among the blocks."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, K)) * np.exp2(rng.integers(-12, 6, (rows, 1)))
    kind = np.repeat(rng.integers(0, 12, (rows, -(-K // 128))), 128, axis=1)[:, :K]
    info = torch.finfo(TD[dt])
    x = np.where(kind == 0, 0.0, x)
    x = np.where(kind == 1, -0.0, x)
    x = np.where(kind == 2, rng.choice([1.0625, 1.1875, -1.3125, 28.0, 1.75, -30.0, 448.0, 0.001953125], (rows, K)), x)
    x = np.where(kind == 3, info.smallest_normal * rng.uniform(-1, 1, (rows, K)), x)
    x = np.where(kind == 4, info.max * rng.uniform(0, 1, (rows, K)), x)
    pick = rng.integers(0, 32, (rows, K)) == 0
    x = np.where((kind == 5) & pick, rng.choice([np.inf, -np.inf], (rows, K)), x)
    x = np.where((kind == 6) & pick, np.nan, x)
    x = np.where(kind == 7, np.where(pick, np.inf, np.where(x > 0, np.nan, -0.0)), x)
    with np.errstate(over="ignore"):
        t = torch.from_numpy(x).to(TD[dt])
    return t, t.double().numpy()


SHAPES = [(1, 1), (1, 128), (3, 127), (5, 129), (2, 511), (7, 513), (64, 256), (127, 512), (129, 640), (130, 1003), (257, 384),
          (1021, 1000)]


@pytest.mark.parametrize("fmt", list(FD))
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("axis", [1, 0])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,K", SHAPES)
def test_quantize_is_exact(ba, rows, K, dt, axis, block_rows, fmt):
    t, x = special_rows(rows, K, dt, 11 * rows + K)
    X = (t.t().contiguous() if axis == 0 else t).cuda()
    q = packed(ba, rows, K, fmt, block_rows)
    out = ba.fp8_quantize(X, q[0], q[1], axis=axis)
    torch.cuda.synchronize()
    assert out[0] is q[0] and out[1] is q[1]
    check_quantized(*q, x, fmt, block_rows)


@pytest.mark.parametrize("fmt", list(FD))
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("axis", [1, 0])
@pytest.mark.parametrize("neighbours", [True, False])
def test_quantize_every_16_bit_pattern(ba, dt, fmt, axis, neighbours):
    # neighbours: values of like size in a block, so that each is near its top; else of every size
    words = np.arange(65536, dtype=np.uint16)
    words = words.reshape(512, 128) if neighbours else words.reshape(128, 512).T
    t = torch.from_numpy(np.ascontiguousarray(words).view(np.int16)).view(TD[dt])
    q = packed(ba, 512, 128, fmt)
    ba.fp8_quantize((t.t().contiguous() if axis == 0 else t).cuda(), q[0], q[1], axis=axis)
    check_quantized(*q, t.double().numpy(), fmt, 1)


@pytest.mark.parametrize("fmt", list(FD))
@pytest.mark.parametrize("axis", [1, 0])
def test_quantize_fp32_borders(ba, fmt, axis):
    # a block's top on either side of the largest value times a power of two, over
    # fp32's whole range, and values on either side of the ties below it
    big = f8.FMT[fmt][2]
    rng = np.random.default_rng(3)
    tops = np.float32(big) * np.exp2(np.arange(-140, 112, dtype=np.float64)).astype(np.float32)
    tops = np.concatenate([np.nextafter(tops, np.float32(0)), tops, np.nextafter(tops, np.float32(np.inf))]).astype(np.float32)
    tops = tops[np.isfinite(tops)]
    mid = rng.integers(2, 32, (len(tops), 127)) / 32.0 * np.exp2(rng.integers(-8, 0, (len(tops), 127)))
    x = (tops[:, None].astype(np.float64) * mid / 1.75).astype(np.float32)
    x = np.where(rng.integers(0, 2, x.shape) == 1, np.nextafter(x, np.float32(0)), x)
    x = np.concatenate([tops[:, None], x], 1).astype(np.float32)
    t = torch.from_numpy(x)
    q = packed(ba, len(tops), 128, fmt)
    ba.fp8_quantize((t.t().contiguous() if axis == 0 else t).cuda(), q[0], q[1], axis=axis)
    check_quantized(*q, x.astype(np.float64), fmt, 1)


@pytest.mark.parametrize("fmt", list(FD))
@pytest.mark.parametrize("axis", [1, 0])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,K", [(66, 130), (67, 512), (129, 96)])
def test_views_aligned_for_one_value(ba, rows, K, dt, axis, fmt):
    t, x = special_rows(rows, K, dt, 5)
    src = t.t().contiguous() if axis == 0 else t
    X, _ = guarded(tuple(src.shape), TD[dt], 0, shift=1)
    X.copy_(src)
    q = packed(ba, rows, K, fmt)
    ba.fp8_quantize(X, q[0], q[1], axis=axis)
    check_quantized(*q, x, fmt, 1)
    Y, buf = guarded(tuple(src.shape), TD[dt], 3, shift=1)
    ba.fp8_dequantize(q[0], q[1], Y, axis=axis)
    v = torch.from_numpy(f8.values(*f8.quantize(x, fmt), K, fmt)).to(TD[dt])
    got = (Y.t() if axis == 0 else Y).cpu()
    assert torch.equal(got.isnan(), v.isnan())
    assert torch.equal(got.nan_to_num(7.0), v.nan_to_num(7.0))
    assert edges_intact(buf, Y.numel(), 3, shift=1)


@pytest.mark.parametrize("fmt", list(FD))
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("axis", [1, 0])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,K", SHAPES[:-1])
def test_dequantize_is_exact(ba, rows, K, dt, axis, block_rows, fmt):
    # every code and every scale byte
    rng = np.random.default_rng(rows + K)
    codes, scales = f8.random_packed(rng, rows, K, fmt, block_rows, 0, 255)
    codes[:, :K] = rng.integers(0, 256, (rows, K), dtype=np.uint8)
    Y, buf = guarded((K, rows) if axis == 0 else (rows, K), TD[dt], 3)
    assert ba.fp8_dequantize(codes_dev(codes, fmt), dev(scales), Y, axis=axis) is Y
    v = f8.values(codes, scales, K, fmt, block_rows)
    with np.errstate(over="ignore"):
        want = torch.from_numpy(v.astype(np.float16) if dt == "f16" else v.astype(np.float32)).to(TD[dt])
    got = (Y.t() if axis == 0 else Y).cpu()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))
    assert edges_intact(buf, Y.numel(), 3)


# ---- products ------------------------------------------------------------------------

def powers(codes, scales, K, fmt, block_rows):
    """2^exponent of each code (0 for zero) times its scale, fp64 [rows, K]."""
    bits, bias, _ = f8.FMT[fmt]
    c = codes.astype(np.int64) & 127
    p = np.where(c == 0, 0.0, np.ldexp(1.0, np.maximum(c >> bits, 1) - bias))
    s = np.ldexp(1.0, scales[:, :codes.shape[1] // 128].astype(np.int64) - 127)
    return (p * np.repeat(np.repeat(s, 128, 1), block_rows, 0)[:len(c)])[:, :K]


class Operand:
    def __init__(self, rng, rows, K, fmt, block_rows=1, lo=None, hi=None, codes=None):
        lo, hi = (lo, hi) if lo is not None else (118, 124) if fmt == "f8e4m3" else (111, 116)
        self.c, self.s = f8.random_packed(rng, rows, K, fmt, block_rows, lo, hi)
        if codes is not None:
            self.c[:, :K] = codes
        self.K, self.fmt, self.block_rows = K, fmt, block_rows

    @property
    def dev(self):
        return codes_dev(self.c, self.fmt), dev(self.s)

    @property
    def values(self):
        return f8.values(self.c, self.s, self.K, self.fmt, self.block_rows)

    @property
    def powers(self):
        return powers(self.c, self.s, self.K, self.fmt, self.block_rows)


def reference(a, b, bias, R, act, alpha, out):
    """fp64 result and each output's allowance (module docstring)."""
    if out == "f32":
        return mx4.reference(a.values, b.values, bias, R, act, alpha, out)
    av, bv = a.values, b.values
    z, s = av @ bv.T, np.abs(av) @ np.abs(bv).T
    for t in (bias, R):
        if t is not None:
            z, s = z + t, s + np.abs(t)
    ref = O().act(np.ascontiguousarray(z), act, alpha).reshape(z.shape)
    E = gamma(a.K + 2, 2.0 ** -23) * s + 7 * 2.0 ** -13 * (a.powers @ b.powers.T)
    if act == "sigmoid":
        u = np.exp(-np.maximum(np.abs(z) - E, 0.0))      # s(1 - s) at the point of [z - E, z + E] nearest 0
        L = u / (1.0 + u) ** 2
    else:
        L = slope_bound(z, E, act, alpha)
    d = L * E + ETA_ACT * np.abs(ref)
    return ref, d + 0.5 * ulp(np.abs(ref) + d, out)


def run_case(ba, M, N, K, fa="f8e4m3", fb="f8e4m3", out="f32", act="none", bias_dt="f32", residual=False, pre=False,
             blocks=(1, 128), seed=0, shift=0):
    rng = np.random.default_rng(seed + 7 * M + 13 * N + K)
    alpha = float(np.float32(0.05))
    a, b = Operand(rng, M, K, fa, blocks[0]), Operand(rng, N, K, fb, blocks[1])
    bias = dev(rng.standard_normal(N), bias_dt) if bias_dt else None
    R = dev(rng.standard_normal((M, N)), out) if residual else None
    C, buf = guarded((M, N), TD[out], 3, shift)
    Z, zbuf = guarded((M, N), TD[out], 5, shift) if pre else (None, None)
    args = (*a.dev, *b.dev, bias)
    if residual:
        R2, _ = guarded((M, N), TD[out], 0, shift)
        R2.copy_(R)
        got = ba.gemm_fp8_bias_add_act(*args, R2, C, act, alpha, Z=Z)
    else:
        got = ba.gemm_fp8_bias_act(*args, C, act, alpha, Z=Z)
    torch.cuda.synchronize()
    assert got is C
    for what, o, f in ((C, buf, act),) + (((Z, zbuf, "none"),) if pre else ()):
        ref, tol = reference(a, b, None if bias is None else f64(bias), None if R is None else f64(R), f, alpha, out)
        err = np.abs(f64(what) - ref)
        worst = np.unravel_index(np.argmax(err / tol), err.shape)
        assert (err <= tol).all(), (ba.last_tile_config(), f, worst, f64(what)[worst], ref[worst], tol[worst])
        assert edges_intact(o, M * N, 5 if what is Z else 3, shift)


SIZES = [(1, 1, 1), (1, 16, 32), (1, 4096, 512), (2, 17, 33), (7, 250, 4100), (16, 64, 128), (17, 65, 129), (33, 130, 500),
         (48, 96, 1024), (64, 64, 512), (65, 1001, 1503), (128, 256, 1024), (256, 128, 640), (300, 520, 2050),
         (512, 512, 256), (1000, 72, 96), (1, 300, 9000), (3, 5, 7), (40, 64, 8), (2800, 2900, 130), (2049, 4100, 520),
         (3000, 2816, 1800)]


@pytest.mark.parametrize("out", ["f32", "f16"])
@pytest.mark.parametrize("blocks", [(1, 128), (1, 1), (128, 1), (128, 128)])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(ba, M, N, K, blocks, out):
    if blocks != (1, 128) and M * N > 2 ** 20:
        M, N = min(M, 1200), min(N, 1300)
    run_case(ba, M, N, K, out=out, blocks=blocks)


@pytest.mark.parametrize("fa,fb", [("f8e4m3", "f8e4m3"), ("f8e4m3", "f8e5m2"), ("f8e5m2", "f8e4m3"), ("f8e5m2", "f8e5m2")])
@pytest.mark.parametrize("M,N,K", [(16, 40, 128), (37, 50, 300), (70, 33, 1100), (300, 700, 40), (1030, 1100, 24)])
def test_sums_of_eight(ba, M, N, K, fa, fb):
    # 16-bit outputs against the sum of the products as the instructions cut them
    # off: what is left is the fp32 sum and the output's rounding
    rng = np.random.default_rng(K)
    a, b = Operand(rng, M, K, fa), Operand(rng, N, K, fb)
    C = torch.empty((M, N), dtype=torch.float16, device="cuda")
    ba.gemm_fp8_bias_act(*a.dev, *b.dev, None, C)
    av, bv, ap, bp = (np.pad(t, ((0, 0), (0, -K % 8))) for t in (a.values, b.values, a.powers, b.powers))
    z, s = np.zeros((M, N)), np.abs(av) @ np.abs(bv).T
    for k in range(0, K, 8):
        p = av[:, None, k:k + 8] * bv[None, :, k:k + 8]
        unit = (ap[:, None, k:k + 8] * bp[None, :, k:k + 8]).max(-1, keepdims=True) * 2.0 ** -13
        z += (np.trunc(p / np.where(unit == 0, 1.0, unit)) * unit).sum(-1)
    E = gamma(K + 2, 2.0 ** -23) * s
    assert (np.abs(f64(C) - z) <= E + 0.5 * ulp(np.abs(z) + E, "f16")).all()


@pytest.mark.parametrize("out", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(3, 70, 900), (20, 40, 700), (65, 301, 1030), (1100, 1160, 900), (2305, 2310, 390)])
def test_sums_without_rounding(ba, M, N, K, out):
    # codes of -2 .. 2 and equal scales: every sum is exact, so are the bits (bf16: up to the output's rounding)
    rng = np.random.default_rng(K)
    small = [np.flatnonzero(np.isin(f8.table(f), [-2.0, -1.0, 0.0, 1.0, 2.0])).astype(np.uint8) for f in FD]
    a = Operand(rng, M, K, "f8e4m3", 1, 127, 127, rng.choice(small[0], (M, K)))
    b = Operand(rng, N, K, "f8e5m2", 128, 126, 126, rng.choice(small[1], (N, K)))
    C = torch.empty((M, N), dtype=TD[out], device="cuda")
    ba.gemm_fp8_bias_act(*a.dev, *b.dev, None, C)
    assert np.array_equal(f64(C), torch.from_numpy(a.values @ b.values.T).to(TD[out]).double().numpy())


@pytest.mark.parametrize("fa,fb", [("f8e4m3", "f8e5m2"), ("f8e5m2", "f8e4m3"), ("f8e5m2", "f8e5m2")])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(3, 70, 300), (20, 40, 700), (65, 301, 1030), (1100, 1160, 900), (2305, 2310, 390)])
def test_formats(ba, M, N, K, fa, fb, out):
    run_case(ba, M, N, K, fa, fb, out, blocks=(1, 1))


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("act", ["none", "relu", "leaky_relu", "tanh", "gelu", "sigmoid"])
def test_epilogue(ba, out, act):
    i = ["none", "relu", "leaky_relu", "tanh", "gelu", "sigmoid"].index(act)
    for M, N in ((5, 200), (20, 264), (130, 261)):
        run_case(ba, M, N, 384, "f8e4m3", "f8e4m3", out, act, ["f32", "f16", "bf16", None][(i + M) % 4], residual=(i + M) % 2 == 0,
                 pre=(i + N) % 2 == 0)


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("act,bias_dt,residual,pre", [("none", None, True, True), ("leaky_relu", "bf16", False, True),
                                                      ("gelu", "f32", False, False), ("gelu", "f16", True, True),
                                                      ("tanh", "f32", True, False), ("sigmoid", None, False, True)])
@pytest.mark.parametrize("M,N,K,kernel", [
    (5, 200, 1100, "stream, 16 n x 16 m"), (16, 301, 1100, "stream, 16 n x 16 m"), (32, 4096, 1100, "stream, 32 n x 16 m"), (31, 4091, 1100, "stream, 32 n x 16 m"),
    (64, 4096, 1100, "64 m x 32 n"), (49, 4081, 1100, "64 m x 32 n"), (256, 4096, 7000, "64 m x 64 n, k over 4"), (200, 4035, 7000, "64 m x 64 n, k over 4"),
    (256, 4096, 1100, "64 m x 64 n, k over 1"), (200, 4035, 1100, "64 m x 64 n, k over 1"), (1100, 1160, 200, "64 m x 64 n, k over 1"),
    (900, 4096, 2200, "128 m x 128 n, k over 1 groups of waves, 4 stages"), (911, 4081, 2200, "128 m x 128 n, k over 1 groups of waves, 4 stages"),
    (1500, 1600, 200, "128 m x 128 n, k over 1 groups of waves, 2 stages"), (1541, 1603, 200, "128 m x 128 n, k over 1 groups of waves, 2 stages"),
    (3328, 4104, 1100, "256 m x 256 n"), (3329, 4099, 1100, "256 m x 256 n")])
def test_epilogue_of_every_kernel(ba, M, N, K, kernel, act, bias_dt, residual, pre, out):
    # rows of whole 16-byte stores and ragged ones, last tiles of few rows and columns
    run_case(ba, M, N, K, "f8e4m3", "f8e5m2", out, act, bias_dt, residual, pre)
    if out == "f32":
        kernel = kernel.replace("256", "128")
    assert kernel in ba.last_tile_config()


@pytest.mark.parametrize("out", ["f32", "f16"])
@pytest.mark.parametrize("K", [1, 64, 128, 129, 256, 300, 384, 512, 513, 640, 768, 1024, 1025, 1100, 1280, 1700, 2177, 4200])
@pytest.mark.parametrize("M,N", [(4, 500), (32, 4096), (60, 4096), (250, 4000), (480, 4000), (900, 4096), (1100, 1160), (1500, 1600), (3329, 4104)])
def test_reduction_lengths(ba, M, N, K, out):
    if M > 3000 and (K < 1000 or out == "f32"):          # (the 256x256 tile: 16-bit outputs, longer reductions)
        M, N = 1400, 1500
    run_case(ba, M, N, K, out=out, seed=3, blocks=(1, 1))


@pytest.mark.parametrize("M,N,K", [(1, 33, 8064), (2, 17, 8065), (16, 40, 8192), (20, 33, 8449), (17, 64, 10240),
                                   (5, 5000, 8200), (32, 20, 16384), (520, 2100, 8200)])
def test_long_reductions(ba, M, N, K):
    run_case(ba, M, N, K, act="relu", seed=17)
    run_case(ba, M, N, K, out="bf16", seed=18)


@pytest.mark.parametrize("out,blocks", [("f32", (1, 1)), ("f16", (1, 128)), ("bf16", (128, 1))])
@pytest.mark.parametrize("M,N,K", [(1024, 4096, 13200), (1000, 3969, 13569), (513, 6001, 10500), (4096, 1024, 13200), (130, 16000, 4200)])
def test_large_operands_of_one_round(ba, M, N, K, out, blocks):
    run_case(ba, M, N, K, "f8e5m2", "f8e4m3", out, "gelu", "f32", residual=True, pre=True, blocks=blocks, seed=23)
    assert "128 m x 128 n, k over 1 groups of waves, 4 stages, a wave ahead" in ba.last_tile_config()


@pytest.mark.parametrize("M,N,K", [(3, 70, 300), (130, 301, 260), (256, 512, 512), (1100, 1160, 300)])
def test_outputs_aligned_for_one_value(ba, M, N, K):
    run_case(ba, M, N, K, "f8e4m3", "f8e4m3", "bf16", "gelu", "bf16", residual=True, pre=True, shift=1)


def test_no_reduction(ba):
    # K = 0: act(bias)
    for M in (5, 700):
        A, B = (torch.empty((r, 0), dtype=FD["f8e4m3"], device="cuda") for r in (M, 1400))
        As, Bs = (torch.empty((r, 0), dtype=torch.uint8, device="cuda") for r in (M, 1400))
        bias = torch.linspace(-1, 1, 1400, device="cuda")
        C, Z = torch.full((M, 1400), 9.0, device="cuda"), torch.full((M, 1400), 9.0, device="cuda")
        ba.gemm_fp8_bias_act(A, As, B, Bs, bias, C, "relu", Z=Z)
        assert torch.equal(C, bias.relu().expand(M, 1400)) and torch.equal(Z, bias.expand(M, 1400))


def test_nothing_to_do(ba):
    A, As = torch.empty((0, 128), dtype=FD["f8e4m3"], device="cuda"), torch.empty((0, 4), dtype=torch.uint8, device="cuda")
    B, Bs = torch.zeros((8, 128), device="cuda").to(FD["f8e4m3"]), torch.zeros((8, 4), dtype=torch.uint8, device="cuda")
    C = torch.empty((0, 8), device="cuda")
    assert ba.gemm_fp8_bias_act(A, As, B, Bs, None, C) is C
    assert ba.gemm_fp8_bias_act(B, Bs, A, As, None, C.t().contiguous()).shape == (8, 0)
    X = torch.empty((0, 100), device="cuda")
    ba.fp8_quantize(X, A, As)
    ba.fp8_dequantize(A, As, X)
    ba.fp8_quantize(X.t().contiguous(), A, As, axis=0)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M", [4, 40, 300, 1500])
@pytest.mark.parametrize("fmt", list(FD))
def test_nonfinite_values_stay_in_their_rows(ba, M, fmt, out):
    rng = np.random.default_rng(5)
    N, K = 1300, 700
    a, b = Operand(rng, M, K, fmt), Operand(rng, N, K, fmt)
    b.s[17, 3] = 255                                     # column 17 of C is NaN
    a.s[2, 5] = 255
    a.c[1, 40] = 0x7F                                    # NaN
    if fmt == "f8e5m2":
        a.c[3, 40] = 0x7C                                # infinity
    C = torch.empty((M, N), dtype=TD[out], device="cuda")
    ba.gemm_fp8_bias_act(*a.dev, *b.dev, None, C)
    got = f64(C)
    assert np.isnan(got[[1, 2]]).all() and np.isnan(got[:, 17]).all()
    keep_m, keep_n = ~np.isin(np.arange(M), [1, 2]), np.arange(N) != 17
    if fmt == "f8e5m2":
        w = b.values[:, 40]                              # inf * w: signed infinity, NaN where w is 0
        assert np.array_equal(got[3, keep_n], np.where(w == 0, np.nan, np.sign(w) * np.inf)[keep_n], equal_nan=True)
        keep_m[3] = False
        a.c[3, 40] = 0
    a.s[2, 5], b.s[17, 3], a.c[1, 40] = 120, 120, 0
    ref, tol = reference(a, b, None, None, "none", 0.0, out)
    at = np.ix_(keep_m, keep_n)
    assert (np.abs(got[at] - ref[at]) <= tol[at]).all()


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(9, 33, 77), (33, 1200, 200), (1030, 1100, 400)])
def test_rest_of_a_row_does_not_reach_the_next(ba, M, N, K, out):
    # NaN right behind every ragged end: rows of codes and scales past the last row
    rng = np.random.default_rng(8)
    a, b = Operand(rng, M, K, "f8e4m3"), Operand(rng, N, K, "f8e4m3", 128)
    pad = lambda t, fill: torch.cat([dev(t).reshape(-1), torch.full((65536,), fill, dtype=torch.uint8, device="cuda")])[:t.size].view(t.shape)  # noqa: E731
    C = torch.empty((M, N), dtype=TD[out], device="cuda")
    ba.gemm_fp8_bias_act(pad(a.c, 0x7F).view(FD["f8e4m3"]), pad(a.s, 255), pad(b.c, 0x7F).view(FD["f8e4m3"]), pad(b.s, 255), None, C)
    ref, tol = reference(a, b, None, None, "none", 0.0, out)
    assert (np.abs(f64(C) - ref) <= tol).all()


@pytest.mark.parametrize("M,N", [(20, 48), (1100, 1160)])
@pytest.mark.parametrize("out,lo,hi", [("bf16", 0, 6), ("bf16", 20, 24), ("bf16", 200, 204), ("bf16", 236, 242), ("f32", 3, 8),
                                       ("f32", 20, 24), ("f32", 200, 204), ("f32", 232, 237)])
def test_scales_far_from_one(ba, M, N, out, lo, hi):
    # (an fp32 output's operands: values within bf16's range)
    rng = np.random.default_rng(lo)
    a, b = Operand(rng, M, 300, "f8e4m3", 1, 243 - hi, 243 - lo), Operand(rng, N, 300, "f8e4m3", 1, lo, hi)
    C = torch.empty((M, N), dtype=TD[out], device="cuda")
    ba.gemm_fp8_bias_act(*a.dev, *b.dev, None, C)
    ref, tol = reference(a, b, None, None, "none", 0.0, out)
    assert (np.abs(f64(C) - ref) <= tol).all()


@pytest.mark.parametrize("M,N", [(70, 136), (1030, 1160)])
def test_residual_in_place_and_equal_bits(ba, M, N):
    rng = np.random.default_rng(9)
    K = 640
    a = (*Operand(rng, M, K, "f8e4m3").dev, *Operand(rng, N, K, "f8e4m3", 128).dev, None)
    R = dev(rng.standard_normal((M, N)), "bf16")
    C1, C2, Z1, Z2 = torch.empty_like(R), R.clone(), torch.empty_like(R), torch.empty_like(R)
    ba.gemm_fp8_bias_add_act(*a, R, C1, "tanh", Z=Z1)
    ba.gemm_fp8_bias_add_act(*a, C2, C2, "tanh", Z=Z2)
    assert torch.equal(C1, C2) and torch.equal(Z1, Z2)
    for _ in range(3):
        C2.zero_()
        ba.gemm_fp8_bias_add_act(*a, R, C2, "tanh")
        assert torch.equal(C1, C2)


def test_both_ways_of_the_binding_agree(ba):
    # the C++ way takes these calls itself; with a stream given they go through ctypes
    n = ba._binding._native
    assert n is not None
    g = torch.Generator(device="cuda").manual_seed(2)
    x, w = torch.randn(33, 300, generator=g, device="cuda").half(), torch.randn(300, 72, generator=g, device="cuda")
    u8 = lambda shape: torch.empty(shape, dtype=torch.uint8, device="cuda")  # noqa: E731
    st = torch.cuda.current_stream()
    got = []
    for stream in (None, st, st.cuda_stream):
        wc, ws = map(u8, ba.fp8_shapes(72, 300, 128))
        xc, xs = map(u8, ba.fp8_shapes(33, 300))
        wc, xc = wc.view(FD["f8e4m3"]), xc.view(FD["f8e5m2"])
        ba.fp8_quantize(w, wc, ws, axis=0, stream=stream)
        ba.fp8_quantize(x, xc, xs, stream=stream)
        back = ba.fp8_dequantize(xc, xs, torch.empty_like(x), stream=stream)
        R = torch.ones(33, 72, device="cuda")
        C = [torch.empty(33, 72, device="cuda") for _ in range(4)]
        ba.gemm_fp8_bias_act(xc, xs, wc, ws, None, C[0], "leaky_relu", 0.25, stream=stream)
        ba.gemm_fp8_bias_act(xc, xs, wc, ws, x[0, :72].contiguous(), C[1], "tanh", Z=C[3], stream=stream)
        ba.gemm_fp8_bias_add_act(xc, xs, wc, ws, None, R, C[2], stream=stream)
        got.append([wc.view(torch.uint8), ws, xc.view(torch.uint8), xs, back, *C])
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))
    assert n.f8_quantize(x, xc, xs, 1) is True
    assert n.f8_gemm(xc, xs, wc, ws, None, R, None, C[2], "none", 0.0) is True
    assert n.f8_gemm(xc, xs, wc, ws, None, R.half(), None, C[2], "none", 0.0) is False


# ---- streams and graphs -----------------------------------------------------------------

@pytest.mark.parametrize("M,N,K", [(4, 512, 512), (256, 512, 512), (1100, 1160, 640), (2304, 2304, 256)])
def test_side_stream_and_graph_replays(ba, M, N, K):
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    w = torch.randn(K, N, generator=g, device="cuda").bfloat16()
    room = lambda rows, k, b: tuple(torch.empty(s, dtype=d, device="cuda")  # noqa: E731
                                    for s, d in zip(ba.fp8_shapes(rows, k, b), (FD["f8e4m3"], torch.uint8)))
    wq, xq = room(N, K, 128), room(M, K, 1)
    bias = torch.randn(N, generator=g, device="cuda")
    C, Z = torch.empty((M, N), dtype=torch.bfloat16, device="cuda"), torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    back = torch.empty_like(x)

    def layer(stream=None):
        ba.fp8_quantize(w, *wq, axis=0, stream=stream)
        ba.fp8_quantize(x, *xq, stream=stream)
        ba.fp8_dequantize(*xq, back, stream=stream)
        ba.gemm_fp8_bias_act(*xq, *wq, bias, C, "gelu", Z=Z, stream=stream)

    outs = (C, Z, back)
    layer()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    [t.zero_() for t in outs]
    side.wait_stream(torch.cuda.current_stream())
    layer(side)                                          # an explicit stream, not the current one
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    base = x.clone()
    for r in range(3):
        x.copy_(base * (1.0 - 0.25 * r))
        [t.zero_() for t in outs]
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        layer()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, outs)), r
