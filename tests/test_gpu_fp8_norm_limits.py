"""The 8-bit, layer norm and gradient calls on tensors just under 2 GiB: the
last rows, columns and values against the same call on a copy of them, or
against fp64 sums (with the allowances of test_gpu_fp8)."""
import numpy as np
import pytest

import fp8_ref as f8
from oracle.compare import gamma, ulp
from test_gpu_fp8 import FD, powers
from test_gpu_mxfp4 import f64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def ba():
    import conv_bias_activation_amd as m
    return m


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def normal(*shape, dtype=torch.float32, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = torch.empty(shape, dtype=dtype, device="cuda")
    for part in out.split(max(1, 2 ** 27 // shape[1])):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
    return out


def room(ba, rows, K, block_rows=1, fmt="f8e4m3"):
    c, s = ba.fp8_shapes(rows, K, block_rows)
    return torch.empty(c, dtype=FD[fmt], device="cuda"), torch.empty(s, dtype=torch.uint8, device="cuda")


def same(a, b):
    v = lambda t: t.contiguous().view(torch.uint8)  # noqa: E731
    return torch.equal(v(a), v(b))


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,K,dt", [(16383, 65536, BF16), (65535, 16384, BF16), (8191, 65536, torch.float32)])
def test_quantise(ba, rows, K, dt, block_rows):
    x = normal(rows, K, dtype=dt)
    q = ba.fp8_quantize(x, *room(ba, rows, K, block_rows))
    cut = (rows - 200) // 128 * 128                      # whole blocks of rows
    want = ba.fp8_quantize(x[cut:].contiguous(), *room(ba, rows - cut, K, block_rows))
    assert same(q[0][cut:], want[0]) and same(q[1][cut // block_rows:], want[1])
    y = ba.fp8_dequantize(*q, torch.empty_like(x))
    assert same(y[cut:], ba.fp8_dequantize(*want, torch.empty_like(x[cut:])))
    assert float((y[:100].float() - x[:100].float()).norm() / x[:100].float().norm()) < 0.05


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,K,dt", [(65536, 16383, BF16), (16383, 65535, BF16), (65536, 8191, torch.float32)])
def test_quantise_down_columns(ba, rows, K, dt, block_rows):
    x = normal(K, rows, dtype=dt)
    q = ba.fp8_quantize(x, *room(ba, rows, K, block_rows), axis=0)
    cut = (rows - 200) // 128 * 128
    part = x[:, cut:].contiguous()
    want = ba.fp8_quantize(part, *room(ba, rows - cut, K, block_rows), axis=0)
    assert same(q[0][cut:], want[0]) and same(q[1][cut // block_rows:], want[1])
    y = ba.fp8_dequantize(*q, torch.empty_like(x), axis=0)
    assert same(y[:, cut:], ba.fp8_dequantize(*want, torch.empty_like(part), axis=0))


def test_codes_of_two_gib(ba):
    # one value a row: 128 bytes of codes each
    rows = 2 ** 24 - 1
    x = normal(rows, 1, seed=3)
    q = ba.fp8_quantize(x, *room(ba, rows, 1))
    y = ba.fp8_dequantize(*q, torch.empty_like(x))
    assert ((y - x).abs() <= 2.0 ** -4 * x.abs()).all()  # (a draw can be zero)
    w = ba.fp8_quantize(torch.full((3, 1), 1.0, device="cuda"), *room(ba, 3, 1))
    C = ba.gemm_fp8_bias_act(*q, *w, None, torch.empty((rows, 3), device="cuda"))
    assert torch.equal(C, y.expand(rows, 3))


def test_one_column(ba):
    # X [K, 1]: the longest grid of the column kernels
    K = 2 ** 30 - 1
    x = normal(1, K, dtype=BF16).view(K, 1)
    q = ba.fp8_quantize(x, *room(ba, 1, K), axis=0)
    y = ba.fp8_dequantize(*q, torch.empty_like(x), axis=0)
    cut = (K - 1000) // 512 * 512
    want = ba.fp8_quantize(x[cut:].contiguous(), *room(ba, 1, K - cut), axis=0)
    assert same(q[0][:, cut:], want[0]) and same(q[1][:, cut // 128:], want[1])
    assert same(y[cut:], ba.fp8_dequantize(*want, torch.empty_like(x[cut:]), axis=0))
    r = ba.fp8_quantize(x.view(1, K), *room(ba, 1, K))
    assert same(r[0], q[0]) and same(r[1], q[1]) and same(ba.fp8_dequantize(*r, torch.empty_like(x).view(1, K)).view(K, 1), y)


@pytest.mark.parametrize("M,N", [(1, 2 ** 30 - 1), (2 ** 30 - 1, 1)])
def test_no_reduction(ba, M, N):
    # K = 0 and as many outputs as there can be: act(bias)
    e = lambda n: (torch.empty((n, 0), dtype=FD["f8e4m3"], device="cuda"), torch.empty((n, 0), dtype=torch.uint8, device="cuda"))  # noqa: E731
    bias = normal(1, N, dtype=BF16).view(N)
    C = torch.full((M, N), 7.0, dtype=BF16, device="cuda")
    ba.gemm_fp8_bias_act(*e(M), *e(N), bias, C, "relu")
    assert torch.equal(C, bias.relu().expand(M, N))


def check(C, q, w, K, out, rows, cols):
    """C[rows][:, cols] against fp64 (both slices)."""
    ac, asc, bc, bsc = (t[s].view(torch.uint8).cpu().numpy() for t, s in ((q[0], rows), (q[1], rows), (w[0], cols), (w[1], cols)))
    av, bv = f8.values(ac, asc, K, "f8e4m3"), f8.values(bc, bsc, K, "f8e4m3")
    ref = av @ bv.T
    E = gamma(K + 2, 2.0 ** -23) * (np.abs(av) @ np.abs(bv).T)
    if out != "f32":
        E = E + 7 * 2.0 ** -13 * (powers(ac, asc, K, "f8e4m3", 1) @ powers(bc, bsc, K, "f8e4m3", 1).T)
    got = f64(C[rows][:, cols])
    assert (np.abs(got - ref) <= E + 0.5 * ulp(np.abs(ref) + E, out)).all()


@pytest.mark.parametrize("M,N,out", [(32768, 16383, "f32"), (32767, 32768, "bf16"), (16, 2 ** 26 - 1, "bf16")])
def test_output_of_two_gib(ba, M, N, out):
    K = 16 if N > 2 ** 20 else 130
    if N > 2 ** 20:                                      # (rows of B: 128 bytes each)
        N = 2 ** 24 - 1
        M = 63
    q = ba.fp8_quantize(normal(M, K), *room(ba, M, K))
    w = ba.fp8_quantize(normal(N, K, seed=1), *room(ba, N, K))
    C = torch.empty((M, N), dtype={"f32": torch.float32, "bf16": BF16}[out], device="cuda")
    ba.gemm_fp8_bias_act(*q, *w, None, C)
    for rows in (slice(0, 40), slice(M - 40, M)):
        for cols in (slice(0, 300), slice(N - 300, N)):
            check(C, q, w, K, out, rows, cols)


@pytest.mark.parametrize("rows,K,other", [(32767, 65536, 40), (16383, 131072, 300), (1023, 2097152, 5)])
@pytest.mark.parametrize("left", [True, False])
def test_operand_of_two_gib(ba, rows, K, other, left):
    big, small = room(ba, rows, K), room(ba, other, K)
    for (c, s), seed in ((big, 0), (small, 1)):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for part in c.view(torch.uint8).split(max(1, 2 ** 28 // K)):
            part.copy_(torch.randint(0, 120, part.shape, generator=g, dtype=torch.uint8, device="cuda"))
        s.fill_(115)
    M, N = (rows, other) if left else (other, rows)
    C = torch.empty((M, N), dtype=BF16, device="cuda")
    ba.gemm_fp8_bias_act(*(big if left else small), *(small if left else big), None, C)
    for part in (slice(0, 20), slice(rows - 20, rows)):
        if left:
            check(C, big, small, K, "bf16", part, slice(0, other))
        else:
            check(C, small, big, K, "bf16", slice(0, other), part)


@pytest.mark.parametrize("rows,N,dt", [(32767, 16384, torch.float32), (16383, 65536, BF16), (2 ** 23 - 1, 128, BF16), (2 ** 22 - 1, 250, BF16), (3, 357913939, BF16)])
def test_layer_norm(ba, rows, N, dt):
    x = normal(rows, N, dtype=dt)
    ga, be = torch.randn(N, device="cuda"), torch.randn(N, device="cuda")
    stats = lambda n: [torch.empty(n, device="cuda") for _ in range(2)]  # noqa: E731
    m, r = stats(rows)
    y = ba.layer_norm(x, ga, be, torch.empty_like(x), m, r)
    last = min(rows, 3000)
    m2, r2 = stats(last)
    part = x[-last:].contiguous()
    assert torch.equal(y[-last:], ba.layer_norm(part, ga, be, torch.empty_like(part), m2, r2))
    assert torch.equal(m[-last:], m2) and torch.equal(r[-last:], r2)
    # the gradient: rows alone decide dX; the sums against torch's in fp64
    ws = torch.empty(ba.layer_norm_grad_workspace_size(rows, N), dtype=torch.uint8, device="cuda")
    dx, dg, db = ba.layer_norm_grad(y, x, ga, m, r, torch.empty_like(x), torch.empty(N, device="cuda"), torch.empty(N, device="cuda"), workspace=ws)
    want = ba.layer_norm_grad(y[-last:].contiguous(), part, ga, m2, r2, torch.empty_like(part))[0]
    assert torch.equal(dx[-last:], want)
    g = torch.zeros(2, N, dtype=torch.float64, device="cuda")
    size = torch.zeros(2, N, dtype=torch.float64, device="cuda")
    for i in range(0, rows, max(1, 2 ** 26 // N)):
        s = slice(i, i + max(1, 2 ** 26 // N))
        d = y[s].double()
        t = d * (x[s].double() - m[s, None].double()) * r[s, None].double()
        for k, v in enumerate((t, d)):
            g[k] += v.sum(0)
            size[k] += v.abs().sum(0)
    # a sum runs through a few thousand additions at most, not through all rows
    for got, ref, s in zip((dg, db), g, size):
        assert ((got.double() - ref).abs() <= 2.0 ** -24 * 20000 * s).all()


@pytest.mark.parametrize("M,N,dt", [(32767, 16384, torch.float32), (2 ** 23 - 1, 128, BF16), (3, 357913939, BF16)])
def test_act_grad(ba, M, N, dt):
    z = normal(M, N, dtype=dt)
    ws = torch.empty(ba.bias_act_grad_workspace_size(M, N), dtype=torch.uint8, device="cuda")
    dz, db = ba.bias_act_grad(z, z, torch.empty_like(z), torch.empty(N, device="cuda"), "tanh", workspace=ws)
    rows = min(M, 1000)
    part = z[-rows:].contiguous()
    assert torch.equal(dz[-rows:], ba.bias_act_grad(part, part, torch.empty_like(part), None, "tanh")[0])
    if N < 2 ** 20:
        ref = torch.zeros(N, dtype=torch.float64, device="cuda")
        for p in z.split(2 ** 26 // N):
            d = p.double()
            ref += (d * (1 - torch.tanh(d) ** 2)).sum(0)
        assert ((db.double() - ref).abs() <= 2.0 ** -24 * 70000 * z[:1000].float().abs().mean() * M).all()
    else:
        assert torch.allclose(db, (z.float() * (1 - torch.tanh(z.float()) ** 2)).sum(0), rtol=1e-4, atol=1e-5)
