"""The MXFP4 operators on the GPU against the format's definition and fp64
sums.

Quantising and reading back are exact steps, so codes, scales and values are
compared bit for bit.  Products: an output y of value ref may be off by
  L * gamma_n * S   the fp32 sum of n terms (S = sum |a b| + |bias| + |R|,
                    gamma_n with u = 2^-23: the matrix cores' additions need
                    not round to nearest), through the activation's slope L,
  2^-15 |ref|       one fp32 evaluation of the activation,
  half a step       of the output type at |ref| plus the above."""
import numpy as np
import pytest

import mxfp4_ref as mx
from gpu_helpers import O
from oracle.compare import ETA_ACT, gamma, slope_bound, ulp

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TD = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def ba():
    import conv_bias_activation_amd as m
    return m


def dev(a, dt=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t.to(TD[dt]) if dt else t).cuda()


def f64(t):
    return t.detach().cpu().double().numpy()


def guarded(shape, dtype, fill, shift=0):
    """A view of `shape` with 64 elements of `fill` around it (shift: more in
    front), and the whole buffer."""
    n = int(np.prod(shape))
    buf = torch.full((n + 128 + shift,), fill, dtype=dtype, device="cuda")
    return buf[64 + shift:64 + shift + n].view(shape), buf


def edges_intact(buf, n, fill, shift=0):
    return bool((buf[:64 + shift] == fill).all()) and bool((buf[64 + shift + n:] == fill).all())


# ---- quantisation -------------------------------------------------------------------

def special_rows(rows, K, dt, seed):
    """Normal values of many sizes with zeros, ties, subnormals, the type's
    largest values, infinities and NaN among the blocks."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, K)) * np.exp2(rng.integers(-12, 6, (rows, 1)))
    kind = rng.integers(0, 12, (rows, -(-K // 32)))
    kind = np.repeat(kind, 32, axis=1)[:, :K]
    info = torch.finfo(TD[dt])
    x = np.where(kind == 0, 0.0, x)
    x = np.where(kind == 1, -0.0, x)
    x = np.where(kind == 2, rng.choice([0.25, 0.75, -1.25, 1.75, -2.5, 3.5, 5.0, 4.0], (rows, K)), x)
    x = np.where(kind == 3, info.smallest_normal * rng.uniform(-1, 1, (rows, K)), x)
    x = np.where(kind == 4, info.max * rng.uniform(0, 1, (rows, K)), x)
    pick = rng.integers(0, 32, (rows, K)) == 0
    x = np.where((kind == 5) & pick, np.inf, x)
    x = np.where((kind == 6) & pick, np.nan, x)
    t = torch.from_numpy(x).to(TD[dt])
    return t, t.double().numpy()


@pytest.mark.parametrize("axis", [1, 0])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 32), (3, 31), (5, 33), (2, 127), (7, 129), (64, 256), (65, 512),
                                    (130, 1003), (257, 384), (1021, 1000)])
def test_quantize_is_exact(ba, rows, K, dt, axis):
    t, x = special_rows(rows, K, dt, 11 * rows + K)
    X = (t.t().contiguous() if axis == 0 else t).cuda()
    cs, ss = ba.mxfp4_shapes(rows, K)
    codes, cbuf = guarded(cs, torch.uint8, 0xA5)
    scales, sbuf = guarded(ss, torch.uint8, 0xA5)
    out = ba.mxfp4_quantize(X, codes, scales, axis=axis)
    torch.cuda.synchronize()
    assert out[0] is codes and out[1] is scales
    want_c, want_s = mx.quantize(x)
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)
    assert edges_intact(cbuf, codes.numel(), 0xA5) and edges_intact(sbuf, scales.numel(), 0xA5)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("neighbours", [True, False])
def test_quantize_every_16_bit_pattern(ba, dt, neighbours):
    words = np.arange(65536, dtype=np.uint16)
    words = words.reshape(2048, 32) if neighbours else words.reshape(32, 2048).T
    X = torch.from_numpy(np.ascontiguousarray(words).view(np.int16)).view(TD[dt]).cuda()
    codes = torch.empty((2048, 64), dtype=torch.uint8, device="cuda")
    scales = torch.empty((2048, 4), dtype=torch.uint8, device="cuda")
    ba.mxfp4_quantize(X, codes, scales)
    want_c, want_s = mx.quantize(f64(X))
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)


@pytest.mark.parametrize("axis", [1, 0])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("K", [96, 130, 512])
def test_quantize_of_a_shifted_view(ba, dt, axis, K):
    # X and Y aligned for one value only
    t, x = special_rows(67, K, dt, 5)
    src = t.t().contiguous() if axis == 0 else t
    X, _ = guarded(tuple(src.shape), TD[dt], 0, shift=1)
    X.copy_(src)
    codes = torch.empty(ba.mxfp4_shapes(67, K)[0], dtype=torch.uint8, device="cuda")
    scales = torch.empty(ba.mxfp4_shapes(67, K)[1], dtype=torch.uint8, device="cuda")
    ba.mxfp4_quantize(X, codes, scales, axis=axis)
    want_c, want_s = mx.quantize(x)
    assert np.array_equal(scales.cpu().numpy(), want_s) and np.array_equal(codes.cpu().numpy(), want_c)
    Y, buf = guarded(tuple(src.shape), TD[dt], 3, shift=1)
    ba.mxfp4_dequantize(codes, scales, Y, axis=axis)
    v = torch.from_numpy(mx.values(want_c, want_s, K)).to(TD[dt])
    assert torch.equal((Y.t() if axis == 0 else Y).cpu().nan_to_num(7.0), v.nan_to_num(7.0))
    assert edges_intact(buf, Y.numel(), 3, shift=1)


@pytest.mark.parametrize("axis", [1, 0])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 31), (5, 33), (2, 127), (7, 129), (64, 256), (130, 1003), (257, 384)])
def test_dequantize_is_exact(ba, rows, K, dt, axis):
    rng = np.random.default_rng(rows + K)
    codes, scales = mx.random_packed(rng, rows, K, 0, 255)          # every scale byte
    Y, buf = guarded((K, rows) if axis == 0 else (rows, K), TD[dt], 3)
    assert ba.mxfp4_dequantize(dev(codes), dev(scales), Y, axis=axis) is Y
    v = mx.values(codes, scales, K)
    with np.errstate(over="ignore"):
        want = torch.from_numpy(v.astype(np.float16) if dt == "f16" else v.astype(np.float32)).to(TD[dt])
    got = (Y.t() if axis == 0 else Y).cpu()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))
    assert edges_intact(buf, Y.numel(), 3)


# ---- products ------------------------------------------------------------------------

def reference(av, bv, bias, R, act, alpha, out):
    """fp64 result and each output's allowance (module docstring)."""
    z = av @ bv.T
    s = np.abs(av) @ np.abs(bv).T
    for t in (bias, R):
        if t is not None:
            z = z + t
            s = s + np.abs(t)
    ref = O().act(np.ascontiguousarray(z), act, alpha).reshape(z.shape)
    E = gamma(av.shape[1] + 2, 2.0 ** -23) * s
    if act == "sigmoid":
        # s(1 - s) at the point of [z - E, z + E] nearest 0, without forming
        # 1 - s (which cancels to 0 from |z| = 37 on)
        u = np.exp(-np.maximum(np.abs(z) - E, 0.0))
        L = u / (1.0 + u) ** 2
    else:
        L = slope_bound(z, E, act, alpha)
    d = L * E + ETA_ACT * np.abs(ref)
    return ref, d + 0.5 * ulp(np.abs(ref) + d, out)


def operand(ba, rng, rows, K, kind):
    """(A, a_scales, float64 values) of a left operand: MXFP4 or 16-bit."""
    if kind == "mxfp4":
        c, s = mx.random_packed(rng, rows, K)
        return dev(c), dev(s), mx.values(c, s, K)
    A = dev(rng.standard_normal((rows, K)), kind)
    return A, None, f64(A)


def run_case(ba, M, N, K, kind, out, act="none", bias_dt="f32", residual=False, seed=0, shift=0):
    rng = np.random.default_rng(seed + 7 * M + 13 * N + K)
    alpha = float(np.float32(0.05))
    A, As, av = operand(ba, rng, M, K, kind)
    if shift and As is None:
        A2, _ = guarded((M, K), A.dtype, 0, shift)
        A2.copy_(A)
        A = A2
    c, s = mx.random_packed(rng, N, K)
    bias = dev(rng.standard_normal(N), bias_dt) if bias_dt else None
    R = dev(rng.standard_normal((M, N)), out) if residual else None
    C, buf = guarded((M, N), TD[out], 3, shift)
    if residual:
        R2, _ = guarded((M, N), TD[out], 0, shift)
        R2.copy_(R)
        got = ba.gemm_mxfp4_bias_add_act(A, As, dev(c), dev(s), bias, R2, C, act, alpha)
    else:
        got = ba.gemm_mxfp4_bias_act(A, As, dev(c), dev(s), bias, C, act, alpha)
    torch.cuda.synchronize()
    assert got is C
    ref, tol = reference(av, mx.values(c, s, K), None if bias is None else f64(bias),
                         None if R is None else f64(R), act, alpha, out)
    err = np.abs(f64(C) - ref)
    worst = np.unravel_index(np.argmax(err / tol), err.shape)
    assert (err <= tol).all(), (ba.last_tile_config(), worst, f64(C)[worst], ref[worst], tol[worst])
    assert edges_intact(buf, M * N, 3, shift)


SIZES = [(1, 1, 1), (1, 16, 32), (1, 4096, 512), (2, 17, 33), (7, 250, 4100), (16, 64, 128), (17, 65, 129), (33, 130, 500),
         (48, 96, 1024), (64, 64, 512), (65, 1001, 1503), (128, 256, 1024), (256, 128, 640), (300, 520, 2050),
         (512, 512, 256), (1000, 72, 96), (1, 300, 9000), (3, 5, 7), (40, 64, 8), (2800, 2900, 130), (2049, 4100, 520),
         (3000, 2816, 1800)]


@pytest.mark.parametrize("kind", ["mxfp4", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(ba, M, N, K, kind):
    run_case(ba, M, N, K, kind, "f32")


@pytest.mark.parametrize("kind", ["mxfp4", "bf16", "f16"])
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("act", ["none", "relu", "leaky_relu", "tanh", "gelu", "sigmoid"])
def test_epilogue(ba, kind, out, act):
    i = ["none", "relu", "leaky_relu", "tanh", "gelu", "sigmoid"].index(act)
    for M, N in ((5, 200), (130, 264)):
        run_case(ba, M, N, 384, kind, out, act, ["f32", "f16", "bf16", None][(i + M) % 4], residual=(i + M) % 2 == 0)


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("act,bias_dt,residual", [("none", None, True), ("leaky_relu", "bf16", False), ("gelu", "f32", False),
                                                  ("gelu", "f16", True), ("tanh", "f32", True), ("sigmoid", None, False)])
@pytest.mark.parametrize("M,N,tile", [(1100, 1160, "128 m x 128 n"), (1030, 1217, "128 m x 128 n"),
                                      (2304, 4104, "256 m x 256 n"), (2305, 4099, "256 m x 256 n")])
def test_epilogue_of_the_tiles(ba, M, N, tile, act, bias_dt, residual, out):
    # rows of whole 16-byte stores and ragged ones, a last tile of one row
    run_case(ba, M, N, 200, "mxfp4", out, act, bias_dt, residual)
    assert tile in ba.last_tile_config()


@pytest.mark.parametrize("K", [1, 128, 129, 256, 300, 512, 513, 640, 768, 1100, 1280, 1281, 1700])
@pytest.mark.parametrize("M,N", [(1100, 1160), (2305, 4104)])
def test_reduction_lengths_of_the_tiles(ba, M, N, K):
    run_case(ba, M, N, K, "mxfp4", "f32", seed=3)
    assert "tile" in ba.last_tile_config()


@pytest.mark.parametrize("kind", ["mxfp4", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(1, 33, 8064), (2, 17, 8065), (16, 40, 8192), (20, 33, 8449), (17, 64, 10240),
                                   (5, 5000, 8200), (32, 20, 16384), (520, 2100, 8200)])
def test_long_reductions(ba, M, N, K, kind):
    run_case(ba, M, N, K, kind, "f32", act="relu", seed=17)


@pytest.mark.parametrize("kind", ["mxfp4", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(3, 70, 300), (130, 301, 260), (256, 512, 512), (1100, 1160, 300)])
def test_operands_aligned_for_one_value(ba, kind, M, N, K):
    run_case(ba, M, N, K, kind, "bf16", "gelu", "bf16", residual=True, shift=1)


@pytest.mark.parametrize("kind", ["mxfp4", "bf16"])
def test_no_reduction(ba, kind):
    # K = 0: act(bias)
    A = torch.empty((5, 0), dtype=torch.uint8 if kind == "mxfp4" else torch.bfloat16, device="cuda")
    As = torch.empty((5, 0), dtype=torch.uint8, device="cuda") if kind == "mxfp4" else None
    B = torch.empty((40, 0), dtype=torch.uint8, device="cuda")
    bias = torch.linspace(-1, 1, 40, device="cuda")
    C = torch.full((5, 40), 9.0, device="cuda")
    ba.gemm_mxfp4_bias_act(A, As, B, B, bias, C, "relu")
    assert torch.equal(C, bias.relu().expand(5, 40))


@pytest.mark.parametrize("kind", ["mxfp4", "bf16", "f16"])
@pytest.mark.parametrize("M", [4, 40, 300])
def test_nonfinite_values_stay_in_their_rows(ba, kind, M):
    rng = np.random.default_rng(5)
    N, K = 96, 700
    A, As, av = operand(ba, rng, M, K, kind)
    c, s = mx.random_packed(rng, N, K)
    s[17, 3] = 255                                       # column 17 of C is NaN
    if kind == "mxfp4":
        As[2, 5] = 255
    else:
        A[2, 655] = float("nan")
        A[3, 40] = float("inf")
    C = torch.empty((M, N), device="cuda")
    ba.gemm_mxfp4_bias_act(A, As, dev(c), dev(s), None, C)
    got = f64(C)
    assert np.isnan(got[2]).all() and np.isnan(got[:, 17]).all()
    keep_m, keep_n = np.arange(M) != 2, np.arange(N) != 17
    if kind != "mxfp4":
        w = mx.values(c, s, K)[:, 40]                    # inf * w: signed infinity, NaN where w is 0
        want = np.where(w == 0, np.nan, np.sign(w) * np.inf)[keep_n]
        assert np.array_equal(got[3, keep_n], want, equal_nan=True)
        keep_m &= np.arange(M) != 3
    ref, tol = reference(av[keep_m], mx.values(c, s, K)[keep_n], None, None, "none", 0.0, "f32")
    assert (np.abs(got[np.ix_(keep_m, keep_n)] - ref) <= tol).all()


@pytest.mark.parametrize("kind", ["mxfp4", "bf16", "f16"])
def test_rest_of_a_row_does_not_reach_the_next(ba, kind):
    # NaN right behind every ragged end: rows of A, codes and scales past the last row
    rng = np.random.default_rng(8)
    M, N, K = 9, 33, 77
    A, As, av = operand(ba, rng, M, K, kind)
    c, s = mx.random_packed(rng, N, K)
    pad = lambda t, fill: torch.cat([t.reshape(-1), torch.full((4096,), fill, dtype=t.dtype, device="cuda")])
    a = pad(A, float("nan") if As is None else 0x77)[:A.numel()].view(A.shape)
    a_s = None if As is None else pad(As, 255)[:As.numel()].view(As.shape)
    b = pad(dev(c), 0x77)[:c.size].view(c.shape)
    b_s = pad(dev(s), 255)[:s.size].view(s.shape)
    C = torch.empty((M, N), device="cuda")
    ba.gemm_mxfp4_bias_act(a, a_s, b, b_s, None, C)
    ref, tol = reference(av, mx.values(c, s, K), None, None, "none", 0.0, "f32")
    assert (np.abs(f64(C) - ref) <= tol).all()


@pytest.mark.parametrize("kind,lo,hi,x", [("mxfp4", 20, 24, 1.0), ("mxfp4", 230, 234, 1.0), ("bf16", 2, 6, 1e30),
                                          ("bf16", 236, 240, 1e-30), ("f16", 60, 64, 6e4), ("f16", 150, 154, 6e-8),
                                          ("f16", 100, 145, 1.0), ("f16", 118, 128, 6e-8), ("f16", 115, 139, 1.0)])
def test_scales_far_from_one(ba, kind, lo, hi, x):
    rng = np.random.default_rng(lo)
    M, N, K = 20, 48, 300
    if kind == "mxfp4":
        ca, sa = mx.random_packed(rng, M, K, 254 - hi, 254 - lo)
        A, As, av = dev(ca), dev(sa), mx.values(ca, sa, K)
    else:
        A, As = dev(rng.uniform(-x, x, (M, K)), kind), None
        av = f64(A)
    c, s = mx.random_packed(rng, N, K, lo, hi)
    C = torch.empty((M, N), device="cuda")
    ba.gemm_mxfp4_bias_act(A, As, dev(c), dev(s), None, C)
    ref, tol = reference(av, mx.values(c, s, K), None, None, "none", 0.0, "f32")
    assert (np.abs(f64(C) - ref) <= tol).all()


@pytest.mark.parametrize("kind", ["mxfp4", "bf16", "f16"])
def test_residual_in_place_and_equal_bits(ba, kind):
    rng = np.random.default_rng(9)
    M, N, K = 70, 136, 640
    A, As, av = operand(ba, rng, M, K, kind)
    c, s = mx.random_packed(rng, N, K)
    b, bs = dev(c), dev(s)
    R = dev(rng.standard_normal((M, N)), "bf16")
    C1, C2 = torch.empty_like(R), R.clone()
    ba.gemm_mxfp4_bias_add_act(A, As, b, bs, None, R, C1, "tanh")
    ba.gemm_mxfp4_bias_add_act(A, As, b, bs, None, C2, C2, "tanh")
    assert torch.equal(C1, C2)
    for _ in range(3):
        C2.zero_()
        ba.gemm_mxfp4_bias_add_act(A, As, b, bs, None, R, C2, "tanh")
        assert torch.equal(C1, C2)


def test_both_ways_of_the_binding_agree(ba):
    # the C++ way takes these calls itself; with a stream given they go through ctypes
    n = ba._binding._native
    assert n is not None
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(33, 300, generator=g, device="cuda").half()
    w = torch.randn(300, 72, generator=g, device="cuda")
    u8 = lambda shape: torch.empty(shape, dtype=torch.uint8, device="cuda")
    st = torch.cuda.current_stream()
    got = []
    for stream in (None, st, st.cuda_stream):
        wc, ws = map(u8, ba.mxfp4_shapes(72, 300))
        xc, xs = map(u8, ba.mxfp4_shapes(33, 300))
        ba.mxfp4_quantize(w, wc, ws, axis=0, stream=stream)
        ba.mxfp4_quantize(x, xc, xs, stream=stream)
        back = ba.mxfp4_dequantize(xc, xs, torch.empty_like(x), stream=stream)
        R = torch.ones(33, 72, device="cuda")
        C = [torch.empty(33, 72, device="cuda") for _ in range(3)]
        ba.gemm_mxfp4_bias_act(xc, xs, wc, ws, None, C[0], "leaky_relu", 0.25, stream=stream)
        ba.gemm_mxfp4_bias_act(x, None, wc, ws, x[0, :72].contiguous(), C[1], "tanh", stream=stream)
        ba.gemm_mxfp4_bias_add_act(x, None, wc, ws, None, R, C[2], stream=stream)
        got.append([wc, ws, xc, xs, back, *C])
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))
    assert n.quantize(x, got[0][2], got[0][3], 1) is True
    assert n.gemm(x, None, wc, ws, None, R, C[2], "none", 0.0) is True
    assert n.gemm(x, None, wc, ws, None, R.half(), C[2], "none", 0.0) is False


# ---- streams and graphs -----------------------------------------------------------------

@pytest.mark.parametrize("M,N,K", [(4, 512, 512), (256, 512, 512), (1024, 1024, 512)])
def test_side_stream_and_graph_replays(ba, M, N, K):
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    w = torch.randn(K, N, generator=g, device="cuda").bfloat16()
    u8 = lambda shape: torch.empty(shape, dtype=torch.uint8, device="cuda")
    wc, ws = map(u8, ba.mxfp4_shapes(N, K))
    xc, xs = map(u8, ba.mxfp4_shapes(M, K))
    bias = torch.randn(N, generator=g, device="cuda")
    C, D = torch.empty((M, N), dtype=torch.bfloat16, device="cuda"), torch.empty((M, N), device="cuda")

    def layer(stream=None):
        ba.mxfp4_quantize(w, wc, ws, axis=0, stream=stream)
        ba.mxfp4_quantize(x, xc, xs, stream=stream)
        ba.gemm_mxfp4_bias_act(xc, xs, wc, ws, bias, C, "gelu", stream=stream)
        ba.gemm_mxfp4_bias_act(x, None, wc, ws, bias, D, "none", stream=stream)

    layer()
    torch.cuda.synchronize()
    want = C.clone(), D.clone()
    side = torch.cuda.Stream()
    C.zero_(), D.zero_()
    side.wait_stream(torch.cuda.current_stream())
    layer(side)                                          # an explicit stream, not the current one
    side.synchronize()
    assert torch.equal(C, want[0]) and torch.equal(D, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    base = x.clone()
    for r in range(3):
        x.copy_(base * (1.0 - 0.25 * r))
        C.zero_(), D.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = C.clone(), D.clone()
        layer()
        torch.cuda.synchronize()
        assert torch.equal(got[0], C) and torch.equal(got[1], D), r
