"""What the sums of the 8-bit products are good to, with a few channels far
larger than the others: with a 16-bit C the documented bound of the 8-bit matrix
instructions' cut-off, with f32_sums that of an fp32 sum.

Allowance of the sum, besides fp32's gamma_n S (S the sum of the terms' sizes, u = 2^-23
as in test_gpu_fp8): 7 * 2^-13 times the sum, over eights of neighbouring k, of the
largest product of the two values' powers of two; none with f32_sums.  Then half a
step of C at the value plus that."""
import numpy as np
import pytest

import fp8_ref as f8
import test_gpu_mxfp4 as mx4
from oracle.compare import gamma, ulp
from test_gpu_fp8 import Operand, codes_dev, powers
from test_gpu_mxfp4 import TD, dev, edges_intact, f64, guarded

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

E4 = "f8e4m3"


@pytest.fixture(scope="module")
def ba():
    import conv_bias_activation_amd as m
    return m


def channels(rng, M, N, K, kind):
    """Rows of A and of B whose every eighth channel is `size` times the others."""
    x, w, eighth = rng.standard_normal((M, K)), rng.standard_normal((N, K)), np.arange(K) % 8 == 0
    if kind == "one sign":
        return np.where(eighth, 400, 1) * np.abs(x), np.abs(w)
    size = {"cancelling 100": 100.0, "cancelling 400": 400.0}[kind]
    sign = np.where(np.arange(K) // 8 % 2 == 0, 1.0, -1.0)
    return np.where(eighth, size, np.abs(x)), np.where(eighth, sign, np.abs(w))


def sums(a, b, rows, cols, K):
    """Of some rows and columns, fp64: the results, the sums of the terms' sizes
    and those of the eights' largest powers."""
    (ac, asc), (bc, bsc) = (a[0][rows], a[1][rows]), (b[0][cols], b[1][cols])
    av, bv = f8.values(ac, asc, K, E4), f8.values(bc, bsc, K, E4)
    ap, bp = powers(ac, asc, K, E4, 1), powers(bc, bsc, K, E4, 1)
    top = np.zeros((len(av), len(bv)))
    for k in range(0, K, 8):
        top += (ap[:, None, k:k + 8] * bp[None, :, k:k + 8]).max(-1)
    return av @ bv.T, np.abs(av) @ np.abs(bv).T, top


# a shape for each of the kernels: streaming (16, 32 rows of B), tiles of 64x32, 64x64, 128x128 and 256x256
SHAPES = [(8, 40, 4096), (32, 4096, 1024), (64, 4096, 1024), (256, 4096, 1024), (900, 4096, 2200), (1500, 1600, 200), (3328, 4104, 1032)]


@pytest.mark.parametrize("out", ["f16", "bf16"])
@pytest.mark.parametrize("kind", ["one sign", "cancelling 100", "cancelling 400"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_large_channels(ba, M, N, K, kind, out):
    rng = np.random.default_rng(M + K)
    a, b = (f8.quantize(t, E4) for t in channels(rng, M, N, K, kind))
    A, B = ((codes_dev(c, E4), dev(s)) for c, s in (a, b))
    rows, cols = rng.permutation(M)[:12], rng.permutation(N)[:24]
    ref, size, top = sums(a, b, rows, cols, K)
    for f32_sums in (False, True):
        C = torch.full((M, N), 7.0, dtype=TD[out], device="cuda")
        assert ba.gemm_fp8_bias_act(*A, *B, None, C, f32_sums=f32_sums) is C
        assert (", fp32 sums" in ba.last_tile_config()) == f32_sums
        E = gamma(K + 2, 2.0 ** -23) * size + (0 if f32_sums else 7 * 2.0 ** -13 * top)
        got = f64(C)[np.ix_(rows, cols)]
        # 4096 / 8 terms of one sign, 400 * 0.8 * 0.8 each, add up to 1.3e5: from 65520, half a step
        # past fp16's largest value, a result rounds to infinity
        most = 65520.0 if out == "f16" else np.inf
        assert (got[ref - E >= most] == np.inf).all()
        at = ref + E < most
        assert at.any() or kind == "one sign"
        err, tol = np.abs(got - ref)[at], (E + 0.5 * ulp(np.abs(ref) + E, out))[at]
        assert (err <= tol).all(), (f32_sums, ba.last_tile_config(), (err / tol).max())


# ---- f32_sums in every kernel and form ------------------------------------------------------

def run(ba, M, N, K, fa, fb, out, act, bias_dt, residual, pre, blocks=(1, 128), shift=0, stream=None):
    rng = np.random.default_rng(M + N + K)
    alpha = float(np.float32(0.05))
    a, b = Operand(rng, M, K, fa, blocks[0]), Operand(rng, N, K, fb, blocks[1])
    bias = dev(rng.standard_normal(N), bias_dt) if bias_dt else None
    C, buf = guarded((M, N), TD[out], 3, shift)
    Z, zbuf = guarded((M, N), TD[out], 5, shift) if pre else (None, None)
    R = None
    if residual:
        R, _ = guarded((M, N), TD[out], 0, shift)
        R.copy_(dev(rng.standard_normal((M, N)), out))
        ba.gemm_fp8_bias_add_act(*a.dev, *b.dev, bias, R, C, act, alpha, Z=Z, stream=stream, f32_sums=True)
    else:
        ba.gemm_fp8_bias_act(*a.dev, *b.dev, bias, C, act, alpha, Z=Z, stream=stream, f32_sums=True)
    torch.cuda.synchronize()
    for what, o, f in ((C, buf, act),) + (((Z, zbuf, "none"),) if pre else ()):
        ref, tol = mx4.reference(a.values, b.values, None if bias is None else f64(bias), None if R is None else f64(R), f, alpha, out)
        err = np.abs(f64(what) - ref)
        assert (err <= tol).all(), (ba.last_tile_config(), f, (err / tol).max())
        assert edges_intact(o, M * N, 5 if what is Z else 3, shift)
    return ba.last_tile_config()


@pytest.mark.parametrize("out", ["f16", "bf16"])
@pytest.mark.parametrize("act,bias_dt,residual,pre", [("none", None, True, True), ("leaky_relu", "bf16", False, True), ("gelu", "f32", False, False),
                                                      ("tanh", "f16", True, False)])
@pytest.mark.parametrize("M,N,K,kernel", [
    (5, 200, 1100, "stream, 16 n x 16 m"), (31, 4091, 1100, "stream, 32 n x 16 m"), (49, 4081, 1100, "64 m x 32 n"),
    (200, 4035, 7000, "64 m x 64 n, k over 4"), (200, 4035, 1100, "64 m x 64 n, k over 1"), (911, 4081, 2200, "128 m x 128 n, k over 1 groups of waves, 4 stages"),
    (1541, 1603, 200, "128 m x 128 n, k over 1 groups of waves, 2 stages"), (3329, 4099, 260, "128 m x 128 n")])
def test_every_kernel(ba, M, N, K, kernel, act, bias_dt, residual, pre, out):
    got = run(ba, M, N, K, "f8e4m3", "f8e5m2", out, act, bias_dt, residual, pre)
    assert kernel in got and got.endswith(", fp32 sums"), got


@pytest.mark.parametrize("out", ["f16", "bf16"])
def test_a_wave_ahead(ba, out):
    assert run(ba, 1000, 3969, 13569, "f8e4m3", "f8e5m2", out, "none", None, True, True).endswith("4 stages, a wave ahead, fp32 sums")


@pytest.mark.parametrize("fa,fb", [("f8e4m3", "f8e4m3"), ("f8e5m2", "f8e4m3"), ("f8e5m2", "f8e5m2")])
@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (3, 70, 300), (65, 301, 1030), (1100, 1160, 129)])
def test_formats_and_ragged_sizes(ba, M, N, K, fa, fb, out):
    run(ba, M, N, K, fa, fb, out, "sigmoid", "f32", True, True, blocks=(128, 1), shift=1)


@pytest.mark.parametrize("M,N,K", [(9, 130, 700), (300, 520, 1100)])
def test_equal_bits_with_an_fp32_output_and_by_both_ways(ba, M, N, K):
    # the same sums as with an fp32 C, rounded once; and through ctypes
    rng = np.random.default_rng(4)
    a = (*Operand(rng, M, K, "f8e4m3").dev, *Operand(rng, N, K, "f8e5m2", 128).dev, None)
    C32 = ba.gemm_fp8_bias_act(*a, torch.empty((M, N), device="cuda"))
    for t in (torch.float16, torch.bfloat16):
        for stream in (None, torch.cuda.current_stream()):
            Z = torch.empty((M, N), dtype=t, device="cuda")
            C = ba.gemm_fp8_bias_act(*a, torch.empty((M, N), dtype=t, device="cuda"), Z=Z, stream=stream, f32_sums=True)
            assert torch.equal(C, C32.to(t)) and torch.equal(Z, C)
    n = ba._binding._native
    assert n.f8_gemm_f32_sums(*a, None, None, C, "none", 0.0) is True
    assert n.f8_gemm_f32_sums(*a, Z.float(), None, C, "none", 0.0) is False


def test_side_stream_and_graph_replays(ba):
    rng = np.random.default_rng(6)
    M, N, K = 300, 1160, 640
    A, B = Operand(rng, M, K, "f8e4m3").dev, Operand(rng, N, K, "f8e4m3", 128).dev
    C = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    want = ba.gemm_fp8_bias_act(*A, *B, None, C, "gelu", f32_sums=True).clone()
    side = torch.cuda.Stream()
    C.zero_()
    side.wait_stream(torch.cuda.current_stream())
    ba.gemm_fp8_bias_act(*A, *B, None, C, "gelu", stream=side, f32_sums=True)
    side.synchronize()
    assert torch.equal(C, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ba.gemm_fp8_bias_act(*A, *B, None, C, "gelu", f32_sums=True)
    for _ in range(3):
        C.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(C, want)
