"""The MXFP4 operators with one tensor just under 2^31 bytes (the library's
limit for its 32-bit offsets), where the offsets of rows past the last one
pass 2^31 or wrap round 2^32.  Codes, scales and values read back are compared
bit for bit on sampled rows, the last ones among them, products with fp64 sums
and the allowance of test_gpu_mxfp4; products over very long rows are of a few
values, so that their sums are exact."""
import numpy as np
import pytest

import mxfp4_ref as mx
from test_gpu_mxfp4 import TD, dev, f64, reference

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

LIMIT = 1 << 31


@pytest.fixture(scope="module")
def ba():
    import conv_bias_activation_amd as m
    return m


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def u8(shape):
    return torch.empty(shape, dtype=torch.uint8, device="cuda")


def just_under(nbytes):
    assert LIMIT - (1 << 20) < nbytes < LIMIT, nbytes


def sample(n, seed, edge=64):
    """Sorted indices below n: the first and last `edge` and some between."""
    rng = np.random.default_rng(seed)
    return np.unique(np.concatenate([np.arange(min(edge, n)), np.arange(max(n - edge, 0), n), rng.integers(0, n, 64)]))


def take(t, idx, dim=0):
    return t.index_select(dim, torch.from_numpy(idx).to(t.device))


# ---- quantise and read back ------------------------------------------------------------

# X of almost 2 GiB, and a small X whose padded codes are (one value a row, one group)
@pytest.mark.parametrize("dt,rows,K", [("bf16", 32767, 32768), ("f32", 16383, 32767), ("f16", (1 << 25) - 1, 1)])
@pytest.mark.parametrize("axis", [1, 0])
def test_round_trip(ba, axis, dt, rows, K):
    es = 4 if dt == "f32" else 2
    just_under(max(rows * K * es, ba.mxfp4_shapes(rows, K)[0][1] * rows))
    g = torch.Generator(device="cuda").manual_seed(rows)
    X = torch.randn((K, rows) if axis == 0 else (rows, K), generator=g, device="cuda", dtype=TD[dt])
    codes, scales = map(u8, ba.mxfp4_shapes(rows, K))
    ba.mxfp4_quantize(X, codes, scales, axis=axis)
    Y = torch.empty_like(X)
    ba.mxfp4_dequantize(codes, scales, Y, axis=axis)
    torch.cuda.synchronize()
    idx = sample(rows, 5)
    x, y = (take(t, idx, 1 - axis) for t in (X, Y))
    x, y = (t.t() if axis == 0 else t for t in (x, y))
    want_c, want_s = mx.quantize(f64(x))
    assert np.array_equal(take(codes, idx).cpu().numpy(), want_c)
    assert np.array_equal(take(scales, idx).cpu().numpy(), want_s)
    assert np.array_equal(f64(y), mx.values(want_c, want_s, K))     # (normal values: exact in every type)


# ---- products ------------------------------------------------------------------------------

def packed_rows(g, rows, K):
    """Random codes (K a multiple of 128) and scales on the device."""
    G = K // 128
    c = torch.randint(0, 256, (rows, 64 * G), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.randint(120, 128, (rows, 4 * G), generator=g, device="cuda", dtype=torch.uint8)
    return c, s


def values_of(c, s, idx, K):
    return mx.values(take(c, idx).cpu().numpy(), take(s, idx).cpu().numpy(), K)


def check(C, mi, ni, av, bv, bias, R, out):
    pick = lambda t: f64(take(take(t, mi), ni, 1))  # noqa: E731
    ref, tol = reference(av, bv, None if bias is None else f64(bias)[ni], None if R is None else pick(R), "none", 0.0, out)
    assert (np.abs(pick(C) - ref) <= tol).all()


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_16_bit_activations(ba, kind):
    M, N, K = 32767, 70, 32768
    just_under(M * K * 2)
    g = torch.Generator(device="cuda").manual_seed(1)
    A = torch.randn(M, K, generator=g, device="cuda", dtype=TD[kind])
    b, bs = packed_rows(g, N, K)
    C = torch.empty((M, N), device="cuda")
    ba.gemm_mxfp4_bias_act(A, None, b, bs, None, C)
    mi, ni = sample(M, 2), np.arange(N)
    check(C, mi, ni, f64(take(A, mi)), values_of(b, bs, ni, K), None, None, "f32")


def test_short_rows_of_activations(ba):
    M, N, K = LIMIT // 14, 2, 7
    just_under(M * K * 2)
    g = torch.Generator(device="cuda").manual_seed(2)
    A = torch.randn(M, K, generator=g, device="cuda", dtype=torch.bfloat16)
    c, s = mx.random_packed(np.random.default_rng(2), N, K)
    C = torch.empty((M, N), dtype=torch.float16, device="cuda")
    ba.gemm_mxfp4_bias_act(A, None, dev(c), dev(s), None, C)
    mi, ni = sample(M, 3), np.arange(N)
    check(C, mi, ni, f64(take(A, mi)), mx.values(c, s, K), None, None, "f16")


@pytest.mark.parametrize("kind", ["mxfp4", "bf16", "f16"])
@pytest.mark.parametrize("M", [1, 9])
def test_codes_of_many_rows(ba, kind, M):
    # MXFP4 A: the tiled kernel, 16-bit A: the streaming one
    N, K = (1 << 25) - 1, 128
    just_under(N * 64)
    g = torch.Generator(device="cuda").manual_seed(3)
    b, bs = packed_rows(g, N, K)
    if kind == "mxfp4":
        A, As = packed_rows(g, M, K)
        av = values_of(A, As, np.arange(M), K)
    else:
        A, As = torch.randn(M, K, generator=g, device="cuda", dtype=TD[kind]), None
        av = f64(A)
    bias = torch.randn(N, generator=g, device="cuda")
    C = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    ba.gemm_mxfp4_bias_act(A, As, b, bs, bias, C)
    mi, ni = np.arange(M), sample(N, 4)
    check(C, mi, ni, av, values_of(b, bs, ni, K), bias, None, "bf16")


@pytest.mark.parametrize("out,M,N", [("f32", 32769, 16383), ("bf16", 32767, 32767), ("f16", 32760, 32768)])
@pytest.mark.parametrize("kind", ["mxfp4", "bf16"])
def test_output_and_residual(ba, kind, out, M, N):
    K = 128
    just_under(M * N * (4 if out == "f32" else 2))
    g = torch.Generator(device="cuda").manual_seed(4)
    b, bs = packed_rows(g, N, K)
    if kind == "mxfp4":
        A, As = packed_rows(g, M, K)
    else:
        A, As = torch.randn(M, K, generator=g, device="cuda", dtype=TD[kind]), None
    bias = torch.randn(N, generator=g, device="cuda")
    R = torch.randn(M, N, generator=g, device="cuda", dtype=TD[out])
    C = torch.empty_like(R)
    ba.gemm_mxfp4_bias_add_act(A, As, b, bs, bias, R, C)
    mi, ni = sample(M, 5), sample(N, 6)
    av = values_of(A, As, mi, K) if kind == "mxfp4" else f64(take(A, mi))
    check(C, mi, ni, av, values_of(b, bs, ni, K), bias, R, out)


@pytest.mark.parametrize("kind", ["mxfp4", "bf16", "f16"])
@pytest.mark.parametrize("M,N", [(1, 1), (1, 2)])
def test_one_very_long_row(ba, kind, M, N):
    # rows 2 .. 15 of the blocks, which do not exist, have offsets past 2^31 and round 2^32
    K = (1 << 30) - 64
    G = (K + 127) // 128
    at = np.array([0, 1, 31, 32, 127, 128, 255, 256, 65535, 1 << 20, K // 2, K - 257, K - 130, K - 65, K - 64, K - 2, K - 1])
    rng = np.random.default_rng(7)
    wv = rng.choice([-3.0, -1.5, -1.0, 0.5, 2.0, 6.0], (N, at.size))
    xv = rng.choice([-4.0, -1.5, 0.5, 1.0, 3.0], (M, at.size))

    def pack(v):
        codes, scales = (torch.zeros(s, dtype=torch.uint8, device="cuda") for s in ba.mxfp4_shapes(len(v), K))
        scales.fill_(127)
        nib = np.zeros(v.shape, np.int64)
        for i, m in enumerate(mx.MAGS):
            nib[np.abs(v) == m] = i
        nib |= (v < 0) << 3
        for r in range(len(v)):
            for k, n in zip(at, nib[r]):
                codes[r, int(k) >> 1] |= int(n) << (4 * (int(k) & 1))
        return codes, scales

    b, bs = pack(wv)
    assert b.shape == (N, 64 * G)
    if kind == "mxfp4":
        A, As = pack(xv)
    else:
        just_under(M * K * 2)
        A, As = torch.zeros(M, K, dtype=TD[kind], device="cuda"), None
        for k, v in zip(at, xv[0]):
            A[0, int(k)] = v
    C = torch.empty((M, N), device="cuda")
    ba.gemm_mxfp4_bias_act(A, As, b, bs, None, C)
    assert np.array_equal(f64(C), xv @ wv.T)             # a few small multiples of 1/4: exact
