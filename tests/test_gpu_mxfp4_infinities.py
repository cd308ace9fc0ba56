"""Activations of the MXFP4 products at infinite sums: for every output type
the same as the other products of the library, and as the formulas evaluated
in 64 bits (GELU of -infinity is -inf * Phi(-inf) = NaN)."""
import numpy as np
import pytest

from gpu_helpers import O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TD = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def ba():
    import conv_bias_activation_amd as m
    return m


# M, N of the streaming kernel, of 128x128 and of 256x256 tiles; K = 4: a lane per output
@pytest.mark.parametrize("kind,M,N,K", [("bf16", 5, 40, 64), ("f16", 40, 40, 64), ("bf16", 5, 40, 4), ("mxfp4", 5, 40, 64),
                                        ("mxfp4", 1100, 1160, 128), ("mxfp4", 2304, 4104, 128)])
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("act", ["none", "relu", "leaky_relu", "tanh", "gelu", "sigmoid"])
def test_infinite_sums(ba, act, out, kind, M, N, K):
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.randn(N, K, generator=g, device="cuda")
    u8 = lambda shape: torch.empty(shape, dtype=torch.uint8, device="cuda")  # noqa: E731
    b, bs = ba.mxfp4_quantize(w, *map(u8, ba.mxfp4_shapes(N, K)))
    x = torch.zeros(M, K, device="cuda")
    if kind == "mxfp4":
        A, As = ba.mxfp4_quantize(x, *map(u8, ba.mxfp4_shapes(M, K)))
    else:
        A, As = x.to(TD[kind]), None
    z = torch.full((N,), 0.5, device="cuda")
    z[1::4], z[2::4], z[3::4] = float("inf"), float("-inf"), float("nan")
    C = torch.empty((M, N), dtype=TD[out], device="cuda")
    ba.gemm_mxfp4_bias_act(A, As, b, bs, z, C, act, 0.25)
    want = O().act(np.ascontiguousarray(z.cpu().double().numpy()), act, 0.25)
    got = C.cpu().double().numpy()
    for i in (1, 2, 3):
        same = np.array_equal(got[:, i::4], np.broadcast_to(want[i::4], (M, len(want[i::4]))), equal_nan=True)
        assert same, (got[0, i], want[i])
    # the library's own product of the same zeros and bias
    D = torch.empty((M, N), dtype=TD[out], device="cuda")
    ba.gemm_bias_act(torch.zeros(M, 8, device="cuda"), torch.zeros(8, N, device="cuda"), z, D, act, 0.25)
    for i in (1, 2, 3):
        same = torch.equal(C[:, i::4].nan_to_num(7.0, 8.0, 9.0), D[:, i::4].nan_to_num(7.0, 8.0, 9.0))
        assert same, (C[0, i], D[0, i])
