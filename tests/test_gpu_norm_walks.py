"""Layer norm of so many rows that a workgroup walks several of them, with the
next row's values under way: every forward kernel that does, against the fp64 formula
(allowances of test_gpu_norm), aligned for one value, and in place.

A workgroup walks from 8192 workgroups of 256 threads on (2048 of 1024), with 32 values a
thread from 2560 on; rows = that many workgroups' rows, and some of their second."""
import pytest

from test_gpu_mxfp4 import TD, edges_intact, guarded
from test_gpu_norm import D, U

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

EPS = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -24, "f32": 2.0 ** -149}


@pytest.fixture(scope="module")
def ba():
    import conv_bias_activation_amd as m
    return m


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def ok(got, ref, tol, what):
    over = (got.double() - ref).abs() / tol
    assert bool(got.isfinite().all()) and float(over.max()) <= 1, (what, float(over.max()), int(over.argmax()))


def stream(rows, N, dt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, N, generator=g, device="cuda") * torch.exp(0.6 * torch.randn(N, generator=g, device="cuda"))
    return (x + 2 * torch.randn(rows, 1, generator=g, device="cuda")).to(TD[dt])


def run(ba, rows, N, dt, kernel, shift=0):
    x = stream(rows, N, dt, N)
    g = torch.Generator(device="cuda").manual_seed(1)
    ga, be = (a + 0.3 * torch.randn(N, generator=g, device="cuda") for a in (1.0, 0.0))
    X, xbuf = guarded((rows, N), TD[dt], 2, shift)
    X.copy_(x)
    Y, buf = guarded((rows, N), TD[dt], 3, shift)
    mean, mbuf = guarded((rows,), torch.float32, 5)
    rstd, rbuf = guarded((rows,), torch.float32, 5)
    ba.layer_norm(X, ga, be, Y, mean, rstd)
    assert kernel in ba.last_tile_config(), ba.last_tile_config()
    assert torch.equal(X, x) and edges_intact(xbuf, rows * N, 2, shift)
    assert edges_intact(buf, rows * N, 3, shift) and edges_intact(mbuf, rows, 5) and edges_intact(rbuf, rows, 5)
    for i in range(0, rows, 4096):
        s = slice(i, i + 4096)
        d = x[s].double()
        m = d.mean(1)
        d = d - m[:, None]
        r = 1 / (d.square().mean(1) + 1e-5).sqrt()
        ok(mean[s], m, U * m.abs() + D * U * d.abs().mean(1) + 2.0 ** -149, "mean")
        ok(rstd[s], r, (D + 16) * U * r, "rstd")
        xh = d * r[:, None] * ga.double()
        y = xh + be.double()
        tol = (D + 16) * U * (xh.abs() + ga.double().abs()) + 4 * U * be.double().abs()
        # half a step of the output's type at |y| + tol: no more than eps / 2 of it
        ok(Y[s], y, tol + EPS[dt] * (y.abs() + tol) + TINY[dt], "y")
    # in place, with the next row already read: the same bits
    m2, r2 = torch.empty_like(mean), torch.empty_like(rstd)
    assert ba.layer_norm(X, ga, be, X, m2, r2) is X
    assert torch.equal(X, Y) and torch.equal(m2, mean) and torch.equal(r2, rstd) and edges_intact(xbuf, rows * N, 2, shift)


KERNELS = [(2048, 1025, 64, 32), (10240 + 777, 2048, 64, 32), (2 * 10240 + 5, 1200, 64, 32), (10240 + 3, 2047, 64, 32),
           (2048, 2049, 256, 16), (8192 + 1000, 4096, 256, 16), (2 * 8192 + 1, 2056, 256, 16), (8192 + 77, 4095, 256, 16),
           (2049, 4100, 256, 32), (2560 + 600, 8192, 256, 32), (2 * 2560 + 1, 5120, 256, 32), (2560 + 77, 8191, 256, 32),
           (2048 + 300, 16384, 1024, 16), (2 * 2048 + 1, 8193, 1024, 16), (32768 + 100, 1000, 64, 16), (32768 + 100, 777, 64, 16),
           (2 * 32768 + 1, 300, 64, 8), (131072 + 50, 100, 16, 8), (131072 + 50, 128, 16, 8)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,N,threads,values", KERNELS)
def test_walks(ba, rows, N, threads, values, dt):
    run(ba, rows, N, dt, f"layer norm, {threads} threads a row, {values} values a thread")


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,N,threads,values", [(10240 + 9, 1536, 64, 32), (8192 + 9, 2500, 256, 16), (2560 + 9, 4104, 256, 32)])
def test_walks_aligned_for_one_value(ba, rows, N, threads, values, dt):
    run(ba, rows, N, dt, f"layer norm, {threads} threads a row, {values} values a thread", shift=1)
