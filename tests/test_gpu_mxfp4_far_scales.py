"""Products whose MXFP4 scales lie at the ends of the byte's range, where a
code times its scale leaves what 16-bit operands hold (byte 253 with magnitudes
of 4 and 6, byte 254 from 2 on) or becomes a subnormal (bytes 0 and 1).  The
products themselves are ordinary numbers; the allowance is that of
test_gpu_mxfp4 (an fp32 sum, each product exact)."""
import numpy as np
import pytest

import mxfp4_ref as mx
from test_gpu_mxfp4 import dev, f64, reference

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ba():
    import conv_bias_activation_amd as m
    return m


def activations(rng, M, K, kind, x):
    A = dev(rng.uniform(-x, x, (M, K)), kind)
    A[0] = 0                                             # a row of zeros stays exactly zero
    return A, f64(A)


def check(C, av, bv):
    ref, tol = reference(av, bv, None, None, "none", 0.0, "f32")
    got = f64(C)
    assert (np.abs(got - ref) <= tol).all(), (np.isnan(got).sum(), np.isinf(got).sum())


# blocks of 16 n x 16 m of the streaming kernel: 1x1, 1x2, 1x4, 2x4, 4x4, 4x1 and 4x2, one unit under way and two, rows of
# fewer than eight values
SIZES = [(3, 48, 300), (20, 48, 300), (40, 70, 300), (40, 8192, 260), (64, 16384, 260), (3, 16384, 260), (20, 16384, 260),
         (2, 40, 8200), (20, 40, 8200), (3, 33, 7), (2, 5, 1)]


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_largest_scales(ba, kind, M, N, K):
    rng = np.random.default_rng(M + N + K)
    A, av = activations(rng, M, K, kind, 2.0 ** -14)
    c, s = mx.random_packed(rng, N, K, 250, 254)
    C = torch.empty((M, N), device="cuda")
    ba.gemm_mxfp4_bias_act(A, None, dev(c), dev(s), None, C)
    check(C, av, mx.values(c, s, K))


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("byte", [253, 254])
def test_one_large_block_among_ordinary_ones(ba, kind, byte):
    # the other columns keep their accuracy, an infinity and a NaN stay where they belong
    rng = np.random.default_rng(byte)
    M, N, K = 9, 40, 1100
    A, av = activations(rng, M, K, kind, 2.0 ** -14)
    c, s = mx.random_packed(rng, N, K)
    s[5, 13] = byte
    s[21, 13] = 255
    A[2, 13 * 32 + 3] = float("inf")
    C = torch.empty((M, N), device="cuda")
    ba.gemm_mxfp4_bias_act(A, None, dev(c), dev(s), None, C)
    bv, got = mx.values(c, s, K), f64(C)
    assert np.isnan(got[:, 21]).all()
    w = bv[:, 13 * 32 + 3]
    want = np.where(np.isnan(w) | (w == 0), np.nan, np.sign(w) * np.inf)
    assert np.array_equal(got[2], want, equal_nan=True)
    m, n = np.arange(M) != 2, np.arange(N) != 21
    check(C[torch.from_numpy(m).cuda()][:, torch.from_numpy(n).cuda()], av[m], bv[n])


@pytest.mark.parametrize("kind,x", [("bf16", 1e30), ("f16", 6e4)])
@pytest.mark.parametrize("M,N,K", [(3, 48, 300), (40, 70, 300), (3, 33, 7)])
def test_smallest_scales(ba, kind, x, M, N, K):
    rng = np.random.default_rng(M + N)
    A, av = activations(rng, M, K, kind, x)
    c, s = mx.random_packed(rng, N, K, 0, 1)
    C = torch.empty((M, N), device="cuda")
    ba.gemm_mxfp4_bias_act(A, None, dev(c), dev(s), None, C)
    check(C, av, mx.values(c, s, K))


@pytest.mark.parametrize("M,N,K", [(3, 48, 300), (40, 70, 300), (3, 33, 7)])
def test_subnormal_bf16_activations(ba, M, N, K):
    rng = np.random.default_rng(M + N)
    A, av = activations(rng, M, K, "bf16", 2.0 ** -126)
    c, s = mx.random_packed(rng, N, K, 196, 202)
    C = torch.empty((M, N), device="cuda")
    ba.gemm_mxfp4_bias_act(A, None, dev(c), dev(s), None, C)
    check(C, av, mx.values(c, s, K))


@pytest.mark.parametrize("large", ["A", "B"])
@pytest.mark.parametrize("M,N,K", [(3, 48, 300), (40, 70, 300), (1100, 1160, 300)])
def test_two_mxfp4_operands_of_opposite_scales(ba, large, M, N, K):
    rng = np.random.default_rng(M)
    lo, hi = mx.random_packed(rng, M, K, 0, 1), mx.random_packed(rng, N, K, 253, 254)
    if large == "A":
        lo, hi = mx.random_packed(rng, M, K, 253, 254), mx.random_packed(rng, N, K, 0, 1)
    C = torch.empty((M, N), device="cuda")
    ba.gemm_mxfp4_bias_act(dev(lo[0]), dev(lo[1]), dev(hi[0]), dev(hi[1]), None, C)
    check(C, mx.values(*lo, K), mx.values(*hi, K))


@pytest.mark.parametrize("kind", ["mxfp4", "bf16"])
@pytest.mark.parametrize("M,N,K", [(9, 40, 1100), (40, 8192, 260), (1100, 1160, 300)])
def test_a_nan_block_leaves_the_other_columns_bits(ba, kind, M, N, K):
    # byte 255 is what the quantiser writes for a block with an infinity or a NaN
    rng = np.random.default_rng(M)
    if kind == "mxfp4":
        A, As = map(dev, mx.random_packed(rng, M, K))
    else:
        A, As = dev(rng.standard_normal((M, K)), kind), None
    c, s = mx.random_packed(rng, N, K)
    want, got = torch.empty((M, N), device="cuda"), torch.empty((M, N), device="cuda")
    ba.gemm_mxfp4_bias_act(A, As, dev(c), dev(s), None, want)
    rows = [5, 21]
    s[5, 0], s[21, K // 64] = 255, 255
    ba.gemm_mxfp4_bias_act(A, As, dev(c), dev(s), None, got)
    keep = torch.ones(N, dtype=torch.bool, device="cuda")
    keep[rows] = False
    assert bool(got[:, rows].isnan().all())
    assert torch.equal(got[:, keep], want[:, keep])


@pytest.mark.parametrize("kind", ["mxfp4", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(3, 48, 300), (40, 70, 130), (1100, 1160, 300), (3, 33, 7)])
def test_scales_of_the_padding_do_not_matter(ba, kind, M, N, K):
    # zero codes past K with any scale but NaN
    rng = np.random.default_rng(M + K)
    packed = [mx.random_packed(rng, rows, K) for rows in (N, M)]
    A = None if kind == "mxfp4" else dev(rng.standard_normal((M, K)), kind)
    got = []
    for fill in (None, 1, 253, 254):
        for _, s in packed:
            s[:, -(-K // 32):] = 0 if fill is None else fill
        (b, bs), (a, a_s) = packed
        C = torch.empty((M, N), device="cuda")
        ba.gemm_mxfp4_bias_act(dev(a) if A is None else A, dev(a_s) if A is None else None, dev(b), dev(bs), None, C)
        got.append(C)
    assert all(torch.equal(got[0], c) for c in got[1:])
