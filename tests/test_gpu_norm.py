"""Layer norm, its gradient and the gradient of the bias-and-activation epilogue
on the GPU against fp64 formulas and against differences.

Allowances, with u = 2^-24 and D = 160, more than the additions that any value
of a row's sum passes through (a thread's 64 values and 16 steps between threads; in
rows past 16384 values, 8 of each 8192 and those steps):
  mean    u |mean| + D u s, s the mean of |x - mean|: the second sum corrects the first's rounding
  rstd    (D + 16) u of it: a sum of N squares, its mean, square root and quotient
  y       (D + 16) u (|xhat gamma| + |gamma|) + 4 u |beta|, + half a step of its type
  dx      (D + 16) u rstd (|g| + mean|g| + |xhat| mean|g xhat|), + half a step
  dgamma, dbeta, dbias: gamma_(rows + 8) times the sum of the terms' magnitudes and
          each term's own error (4 u of |dy xhat|), + half a step of their type
  dz      |dy| times the slope's error, + half a step: u of the product for none,
          ReLU and LeakyReLU; 2^-20 of the slope for tanh and sigmoid (exponential,
          reciprocal and three products, an ulp or two each); 2^-16 (Phi + |z phi|)
          for GELU, whose exponents' arguments round (8e-6 of Phi, as much of phi)."""
import math

import numpy as np
import pytest

from oracle.compare import gamma as gamma_n, ulp
from test_gpu_mxfp4 import TD, edges_intact, f64, guarded

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U, D = 2.0 ** -24, 160


@pytest.fixture(scope="module")
def ba():
    import conv_bias_activation_amd as m
    return m


def put(t, shift=0):
    """t on the device; shift: aligned for one value only."""
    v, _ = guarded(tuple(t.shape), t.dtype, 0, shift)
    v.copy_(t)
    return v


def ok(got, ref, tol, what):
    err = np.abs(got - ref)
    assert np.isfinite(got).all(), what
    worst = np.unravel_index(np.argmax(err / tol), err.shape)
    assert (err <= tol).all(), (what, worst, got[worst], ref[worst], tol[worst])


def rows_of(rows, N, dt, seed, kind="stream"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, N, generator=g, dtype=torch.float64)
    if kind == "stream":
        x = x * torch.exp(0.6 * torch.randn(N, generator=g, dtype=torch.float64)) + 2 * torch.randn(rows, 1, generator=g, dtype=torch.float64)
    elif kind == "offset":                               # the offset far above the deviation
        x = x + 3000.0
    elif kind == "small":
        x = x * 1e-6
    return x.to(TD[dt])


def weights(N, dt, seed):
    g = torch.Generator().manual_seed(seed)
    return [(a + 0.3 * torch.randn(N, generator=g)).to(TD[dt]) for a in (1.0, 0.0)]


# ---- layer norm -------------------------------------------------------------------------

def norm_reference(x, ga, be, eps):
    mean = x.mean(1, keepdims=True)
    d = x - mean
    rstd = 1 / np.sqrt((d * d).mean(1, keepdims=True) + eps)
    xh = d * rstd
    y = xh * ga + be
    tol = (D + 16) * U * (np.abs(xh * ga) + np.abs(ga)) + 4 * U * np.abs(be) + np.zeros_like(x)
    return mean[:, 0], rstd[:, 0], y, tol, U * np.abs(mean[:, 0]) + D * U * np.abs(d).mean(1) + 2.0 ** -149


def run_norm(ba, rows, N, dtx, dty, dtw="f32", which="both", kind="stream", eps=1e-5, stats=True, shift=0):
    x = rows_of(rows, N, dtx, 7 * rows + N, kind)
    ga, be = weights(N, dtw, N)
    X = put(x, shift)
    Y, buf = guarded((rows, N), TD[dty], 3, shift)
    mean, mbuf = guarded((rows,), torch.float32, 5)
    rstd, rbuf = guarded((rows,), torch.float32, 5)
    g, b = (put(ga, shift) if which in ("both", "gamma") else None), (put(be, shift) if which in ("both", "beta") else None)
    out = ba.layer_norm(X, g, b, Y, mean if stats else None, rstd if stats else None, eps)
    torch.cuda.synchronize()
    assert out is Y
    rm, rr, ry, tol, mtol = norm_reference(f64(x), 1.0 if g is None else f64(ga), 0.0 if b is None else f64(be), eps)
    ok(f64(Y), ry, tol + 0.5 * ulp(np.abs(ry) + tol, dty), ba.last_tile_config())
    assert edges_intact(buf, rows * N, 3, shift)
    if stats:
        ok(f64(mean), rm, mtol, "mean")
        ok(f64(rstd), rr, (D + 16) * U * rr, "rstd")
        assert edges_intact(mbuf, rows, 5) and edges_intact(rbuf, rows, 5)


NS = [1, 2, 7, 8, 9, 64, 127, 128, 129, 500, 512, 513, 1000, 1024, 2047, 2048, 2049, 4096, 4100, 8192, 8193, 16384, 16385]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N", NS)
def test_norm_lengths(ba, N, dt):
    for rows in (1, 3, 37):
        run_norm(ba, rows, N, dt, dt)


@pytest.mark.parametrize("N", [16384, 16385, 40000, 65537, 70001, 200000])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_norm_long_rows(ba, N, dt):
    run_norm(ba, 3, N, dt, dt, dt)


@pytest.mark.parametrize("dtx", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dty", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dtw", ["bf16", "f16", "f32"])
def test_norm_types(ba, dtx, dty, dtw):
    run_norm(ba, 33, 1000, dtx, dty, dtw)
    run_norm(ba, 5, 100, dtx, dty, dtw, stats=False)


@pytest.mark.parametrize("which", ["gamma", "beta", "neither"])
@pytest.mark.parametrize("N", [100, 5000])
def test_norm_without_weights(ba, N, which):
    run_norm(ba, 9, N, "bf16", "f32", which=which)


@pytest.mark.parametrize("kind,eps", [("offset", 1e-5), ("offset", 0.0), ("small", 1e-12), ("small", 0.0), ("stream", 3.0)])
@pytest.mark.parametrize("N", [96, 1000, 4096, 70000])
def test_norm_distributions(ba, N, kind, eps):
    run_norm(ba, 5, N, "f32", "f32", kind=kind, eps=eps)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N", [77, 512, 1003, 4096, 9000, 65540])
def test_norm_aligned_for_one_value(ba, N, dt):
    run_norm(ba, 7, N, dt, dt, dt, shift=1)


@pytest.mark.parametrize("rows", [16, 17, 4097, 70000])
def test_norm_many_rows(ba, rows):
    run_norm(ba, rows, 48, "bf16", "bf16")


@pytest.mark.parametrize("N", [64, 700, 4096, 70000])
def test_norm_of_rows_that_do_not_vary(ba, N):
    # zeros, and a value that fp32 sums exactly: y = beta; with eps = 0 NaN
    x = torch.zeros(4, N, device="cuda")
    x[1] = 2.0
    x[3] = torch.randn(N, device="cuda")
    be = torch.randn(N, device="cuda")
    y, mean, rstd = torch.empty_like(x), torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
    ba.layer_norm(x, None, be, y, mean, rstd)
    assert torch.equal(y[:3], be.expand(3, N)) and mean[:3].tolist() == [0.0, 2.0, 0.0]
    assert torch.allclose(rstd[:3], torch.full((3,), 1e5 ** 0.5, device="cuda"), rtol=1e-6)
    ba.layer_norm(x, None, be, y, mean, rstd, 0.0)
    assert y[:3].isnan().all() and y[3].isfinite().all()


@pytest.mark.parametrize("N", [64, 700, 4096, 9000, 70000])
def test_norm_nonfinite_values_stay_in_their_rows(ba, N):
    x = torch.randn(40, N, generator=torch.Generator().manual_seed(1)).cuda()
    y0, y = torch.empty_like(x), torch.empty_like(x)
    ba.layer_norm(x, None, None, y0)
    x[3, N // 2], x[18, 0], x[39, N - 1] = float("nan"), float("inf"), float("-inf")
    ba.layer_norm(x, None, None, y)
    bad = torch.zeros(40, dtype=torch.bool)
    bad[[3, 18, 39]] = True
    assert y[bad.cuda()].isnan().all() and torch.equal(y[~bad.cuda()], y0[~bad.cuda()])


@pytest.mark.parametrize("N", [64, 700, 4096, 9000, 70000])
def test_statistics_of_rows_with_nonfinite_values(ba, N):
    x = torch.randn(5, N, generator=torch.Generator().manual_seed(2)).cuda()
    x[1, N // 2], x[2, 0], x[3, N - 1] = float("nan"), float("inf"), float("-inf")
    y, mean, rstd = torch.empty_like(x), torch.empty(5, device="cuda"), torch.empty(5, device="cuda")
    ba.layer_norm(x, None, None, y, mean, rstd)
    assert not mean[1:4].isfinite().any() and rstd[1:4].isnan().all()
    assert mean[[0, 4]].isfinite().all() and rstd[[0, 4]].isfinite().all()


@pytest.mark.parametrize("N", [100, 4096, 70000])
def test_norm_in_place_and_equal_bits(ba, N):
    x = rows_of(50, N, "bf16", 3).cuda()
    y = ba.layer_norm(x, None, None, torch.empty_like(x))
    for _ in range(3):
        assert torch.equal(ba.layer_norm(x, None, None, torch.empty_like(x)), y)
    assert ba.layer_norm(x, None, None, x) is x and torch.equal(x, y)


# ---- its gradient -------------------------------------------------------------------------

def grad_reference(dy, x, ga, mean, rstd):
    mean, rstd = mean[:, None], rstd[:, None]
    xh = (x - mean) * rstd
    g = dy * ga
    s1, s2 = g.mean(1, keepdims=True), (g * xh).mean(1, keepdims=True)
    dx = rstd * (g - s1 - xh * s2)
    tol = (D + 16) * U * rstd * (np.abs(g) + np.abs(g).mean(1, keepdims=True) + np.abs(xh) * np.abs(g * xh).mean(1, keepdims=True))
    k = gamma_n(x.shape[0] + 8, U) + 4 * U
    return dx, tol, [((dy * xh).sum(0), k * np.abs(dy * xh).sum(0)), (dy.sum(0), k * np.abs(dy).sum(0))]


def run_grad(ba, rows, N, dtx, dty, dtw="f32", have_gamma=True, want=(True, True), kind="stream", shift=0):
    x = rows_of(rows, N, dtx, 3 * rows + N, kind)
    dy = (rows_of(rows, N, "f32", rows + N, "plain") * torch.exp(torch.randn(rows, 1, generator=torch.Generator().manual_seed(N)))).to(TD[dty])
    ga = weights(N, dtw, N)[0]
    xf = f64(x)
    mean = xf.mean(1)
    rstd = 1 / np.sqrt(((xf - mean[:, None]) ** 2).mean(1) + 1e-5)
    mean, rstd = (torch.from_numpy(a.astype(np.float32)) for a in (mean, rstd))
    dX, buf = guarded((rows, N), TD[dtx], 3, shift)
    outs = [guarded((N,), TD[dtw], 5, shift) if w else (None, None) for w in want]
    size = ba.layer_norm_grad_workspace_size(rows, N)
    ws, wbuf = guarded((size,), torch.uint8, 0xA5)
    got = ba.layer_norm_grad(put(dy, shift), put(x, shift), put(ga, shift) if have_gamma else None, put(mean), put(rstd), dX, outs[0][0], outs[1][0],
                             workspace=ws if any(want) else None)
    torch.cuda.synchronize()
    assert got[0] is dX and got[1] is outs[0][0] and got[2] is outs[1][0]
    rdx, tol, rw = grad_reference(f64(dy), xf, f64(ga) if have_gamma else 1.0, f64(mean), f64(rstd))
    name = ba.last_tile_config()
    ok(f64(dX), rdx, tol + 0.5 * ulp(np.abs(rdx) + tol, dtx), name)
    assert edges_intact(buf, rows * N, 3, shift) and edges_intact(wbuf, size, 0xA5)
    for (o, b), (ref, t) in zip(outs, rw):
        if o is not None:
            ok(f64(o), ref, t + 0.5 * ulp(np.abs(ref) + t, dtw), name)
            assert edges_intact(b, N, 5, shift)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N", NS + [32768, 32769, 40001])
def test_grad_lengths(ba, N, dt):
    for rows in (1, 3, 37):
        run_grad(ba, rows, N, dt, dt)


@pytest.mark.parametrize("rows,N", [(70000, 8), (5000, 130), (4097, 1000), (2500, 2048), (1200, 5000), (700, 16000), (300, 33000)])
def test_grad_many_rows(ba, rows, N):
    run_grad(ba, rows, N, "f32", "f32")


@pytest.mark.parametrize("dtx", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dty", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dtw", ["bf16", "f16", "f32"])
def test_grad_types(ba, dtx, dty, dtw):
    run_grad(ba, 33, 1000, dtx, dty, dtw)


@pytest.mark.parametrize("want", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("N", [100, 3000, 40000])
def test_grad_of_some(ba, N, want):
    run_grad(ba, 19, N, "bf16", "f32", have_gamma=False, want=want)
    run_grad(ba, 19, N, "bf16", "f32", want=want)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N", [77, 512, 1003, 4096, 9000, 33333])
def test_grad_aligned_for_one_value(ba, N, dt):
    run_grad(ba, 7, N, dt, dt, dt, shift=1)


@pytest.mark.parametrize("N", [96, 4096])
def test_grad_of_an_offset(ba, N):
    run_grad(ba, 9, N, "f32", "f32", kind="offset")


@pytest.mark.parametrize("N", [100, 4096])
def test_grad_in_place_and_equal_bits(ba, N):
    x, dy = rows_of(300, N, "bf16", 3).cuda(), rows_of(300, N, "bf16", 4).cuda()
    mean, rstd = x.float().mean(1), 1 / x.float().std(1)
    ws = torch.empty(ba.layer_norm_grad_workspace_size(300, N), dtype=torch.uint8, device="cuda")
    new = lambda: [torch.empty(N, device="cuda") for _ in range(2)]  # noqa: E731
    want = ba.layer_norm_grad(dy, x, None, mean, rstd, torch.empty_like(x), *new(), workspace=ws)
    for place in ("apart", "apart", "x", "dy"):
        a, b = x.clone(), dy.clone()
        out = {"apart": torch.empty_like(x), "x": a, "dy": b}[place]
        got = ba.layer_norm_grad(b, a, None, mean, rstd, out, *new(), workspace=ws)
        assert all(torch.equal(p, q) for p, q in zip(got, want)), place


def test_grad_without_rows(ba):
    X = torch.empty((0, 70), device="cuda")
    v = torch.empty(0, device="cuda")
    dg, db = torch.full((70,), 3.0, device="cuda"), torch.full((70,), 3.0, device="cuda")
    ba.layer_norm_grad(X, X, None, v, v, X, dg, db, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert not dg.any() and not db.any()
    ba.layer_norm(X, None, None, X)
    E = torch.empty((5, 0), device="cuda")
    v = torch.empty(5, device="cuda")
    ba.layer_norm(E, None, None, E)
    ba.layer_norm_grad(E, E, None, v, v, E)


@pytest.mark.parametrize("N", [60, 600, 5000])
def test_grad_against_differences(ba, N):
    # <dx, v> against the change of sum(dy y) along v, y the fp64 formula:
    # the central difference's own error is h^2 / 6 times a third derivative, below
    # 1e-6 of the sums of magnitudes at h = 1e-3 and unit deviation
    rows = 6
    rng = np.random.default_rng(N)
    x, dy, v = (rng.standard_normal((rows, N)).astype(np.float32).astype(np.float64) for _ in range(3))
    ga, be = (f64(t) for t in weights(N, "f32", 1))
    f = lambda x, ga, be: (dy * norm_reference(x, ga, be, 1e-5)[2]).sum(1)  # noqa: E731
    X, dY, G = (torch.from_numpy(a.astype(np.float32)).cuda() for a in (x, dy, ga))
    mean, rstd, Y = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.empty_like(X)
    ba.layer_norm(X, G, torch.from_numpy(be.astype(np.float32)).cuda(), Y, mean, rstd)
    ws = torch.empty(ba.layer_norm_grad_workspace_size(rows, N), dtype=torch.uint8, device="cuda")
    dx, dg, db = ba.layer_norm_grad(dY, X, G, mean, rstd, torch.empty_like(X), torch.empty_like(G), torch.empty_like(G), workspace=ws)
    h = 1e-3
    want = (f(x + h * v, ga, be) - f(x - h * v, ga, be)) / (2 * h)
    scale = np.abs(dy).sum(1)
    assert (np.abs((f64(dx) * v).sum(1) - want) <= 2e-5 * scale).all()
    for got, lo, hi in ((dg, (ga - v[0], be), (ga + v[0], be)), (db, (ga, be - v[0]), (ga, be + v[0]))):
        want = (f(x, *hi) - f(x, *lo)).sum() / 2         # linear in the weights
        assert abs((f64(got) * v[0]).sum() - want) <= 2e-5 * scale.sum()


# ---- the epilogue's gradient ----------------------------------------------------------------

ACTS = ["none", "relu", "leaky_relu", "tanh", "gelu", "sigmoid"]


def slope(z, act, alpha):
    """act'(z) and the allowance for it, fp64."""
    if act == "none":
        return np.ones_like(z), 0 * z
    if act == "relu":
        return (z > 0).astype(np.float64), 0 * z
    if act == "leaky_relu":
        s = np.where(z >= 0, 1.0, alpha)
        return s, U * np.abs(s)
    if act in ("tanh", "sigmoid"):
        k = 2.0 if act == "tanh" else 1.0
        u = np.exp(-k * np.abs(z))
        s = k * k * u / (1 + u) ** 2
        return s, 2.0 ** -20 * s + 2.0 ** -146           # (subnormal exponentials)
    t = torch.from_numpy(np.clip(z, -60.0, 60.0))
    phi = 0.5 * torch.special.erfc(-t / math.sqrt(2)).numpy()
    zphi = np.clip(z, -60, 60) * np.exp(-np.clip(z, -60, 60) ** 2 / 2) / math.sqrt(2 * math.pi)
    return phi + zphi, 2.0 ** -16 * (phi + np.abs(zphi)) + 2.0 ** -146


def run_act(ba, M, N, dt, act, dtb="f32", want=(True, True), shift=0, alpha=0.05, wide=False):
    alpha = float(np.float32(alpha))
    g = torch.Generator().manual_seed(M + 3 * N)
    z = (torch.randn(M, N, generator=g, dtype=torch.float64) * (20 if wide else 1.5)).to(TD[dt])
    dy = torch.randn(M, N, generator=g, dtype=torch.float64).to(TD[dt])
    dZ, buf = guarded((M, N), TD[dt], 3, shift) if want[0] else (None, None)
    db, bbuf = guarded((N,), TD[dtb], 5, shift) if want[1] else (None, None)
    size = ba.bias_act_grad_workspace_size(M, N)
    ws, wbuf = guarded((size,), torch.uint8, 0xA5)
    got = ba.bias_act_grad(put(dy, shift), None if act == "none" and M % 2 else put(z, shift), dZ, db, act, alpha, workspace=ws if want[1] else None)
    torch.cuda.synchronize()
    assert got[0] is dZ and got[1] is db
    s, se = slope(f64(z), act, alpha)
    ref = f64(dy) * s
    tol = np.abs(f64(dy)) * se + U * np.abs(ref)
    if want[0]:
        ok(f64(dZ), ref, tol + 0.5 * ulp(np.abs(ref) + tol, dt), (act, ba.last_tile_config()))
        assert edges_intact(buf, M * N, 3, shift)
    if want[1]:
        rb, t = ref.sum(0), gamma_n(M + 8, U) * np.abs(ref).sum(0) + tol.sum(0) * 1.01
        ok(f64(db), rb, t + 0.5 * ulp(np.abs(rb) + t, dtb), (act, ba.last_tile_config()))
        assert edges_intact(bbuf, N, 5, shift) and edges_intact(wbuf, size, 0xA5)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("act", ACTS)
def test_act_grad(ba, act, dt):
    for M, N in ((1, 1), (1, 4096), (3, 7), (37, 100), (300, 1003), (5000, 24)):
        run_act(ba, M, N, dt, act, ["f32", "f16", "bf16"][N % 3])
    run_act(ba, 64, 600, dt, act, wide=True)


@pytest.mark.parametrize("M,N", [(70000, 3), (9000, 64), (4097, 520), (1, 100000), (2, 16385), (513, 512), (2049, 1000)])
def test_act_grad_sizes(ba, M, N):
    run_act(ba, M, N, "bf16", "gelu")


@pytest.mark.parametrize("want", [(True, False), (False, True)])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_act_grad_of_some(ba, act, want):
    run_act(ba, 333, 1001, "bf16", act, want=want)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N", [5, 77, 512, 1003])
def test_act_grad_aligned_for_one_value(ba, N, dt):
    run_act(ba, 41, N, dt, "sigmoid", dt, shift=1)


@pytest.mark.parametrize("act", ACTS)
def test_act_grad_at_the_ends(ba, act):
    # where the slope has a limit: infinities, zeros of both signs, the largest values
    z = torch.tensor([[float("inf"), float("-inf"), 0.0, -0.0, 3e38, -3e38, 1e-40, -1e-40]], device="cuda")
    dz = torch.empty_like(z)
    ba.bias_act_grad(torch.full_like(z, 2.0), z, dz, None, act, 0.25)
    want = {"none": [2] * 8, "relu": [2, 0, 0, 0, 2, 0, 2, 0], "leaky_relu": [2, .5, 2, 2, 2, .5, 2, .5],
            "tanh": [0, 0, 2, 2, 0, 0, 2, 2], "gelu": [2, 0, 1, 1, 2, 0, 1, 1], "sigmoid": [0, 0, .5, .5, 0, 0, .5, .5]}[act]
    assert torch.allclose(dz.cpu(), torch.tensor([want], dtype=torch.float32), rtol=2e-5, atol=0)
    z.fill_(float("nan"))                                # not above zero, and "elsewhere" for LeakyReLU
    ba.bias_act_grad(torch.full_like(z, 2.0), z, dz, None, act, 0.25)
    want = {"none": 2.0, "relu": 0.0, "leaky_relu": 0.5}.get(act)
    assert dz.isnan().all() if want is None else bool((dz == want).all())


@pytest.mark.parametrize("act", ["gelu", "tanh", "sigmoid"])
def test_act_grad_against_differences(ba, act):
    z = np.linspace(-6, 6, 1001)[None].astype(np.float32).astype(np.float64)
    h = 1e-4
    t = lambda a: torch.from_numpy(a)  # noqa: E731
    f = {"gelu": lambda a: a * 0.5 * torch.special.erfc(t(-a / math.sqrt(2))).numpy(), "tanh": np.tanh, "sigmoid": lambda a: 1 / (1 + np.exp(-a))}[act]
    want = (f(z + h) - f(z - h)) / (2 * h)               # its error: h^2 / 6 of a third derivative below 2, and 1e-16 / h
    Z = torch.from_numpy(z.astype(np.float32)).cuda()
    dZ, _ = ba.bias_act_grad(torch.ones_like(Z), Z, torch.empty_like(Z), None, act)
    assert (np.abs(f64(dZ) - want) <= 2e-8 + 2.0 ** -16 * 1.2).all()


@pytest.mark.parametrize("act", ["relu", "gelu"])
def test_act_grad_in_place_and_equal_bits(ba, act):
    g = torch.Generator(device="cuda").manual_seed(3)
    dy, z = (torch.randn(777, 1030, generator=g, device="cuda").bfloat16() for _ in range(2))
    ws = torch.empty(ba.bias_act_grad_workspace_size(777, 1030), dtype=torch.uint8, device="cuda")
    want = ba.bias_act_grad(dy, z, torch.empty_like(z), torch.empty(1030, device="cuda"), act, workspace=ws)
    for place in ("apart", "apart", "dy", "z"):
        a, b = dy.clone(), z.clone()
        out = {"apart": torch.empty_like(z), "dy": a, "z": b}[place]
        got = ba.bias_act_grad(a, b, out, torch.empty(1030, device="cuda"), act, workspace=ws)
        assert all(torch.equal(p, q) for p, q in zip(got, want)), place


def test_act_grad_without_rows(ba):
    e = torch.empty((0, 70), device="cuda")
    db = torch.full((70,), 3.0, device="cuda")
    ba.bias_act_grad(e, e, e, db, "gelu", workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert not db.any()
    e = torch.empty((7, 0), device="cuda")
    ba.bias_act_grad(e, e, e, torch.empty(0, device="cuda"), "gelu", workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))


# ---- binding, streams and graphs ----------------------------------------------------------------

def test_both_ways_of_the_binding_agree(ba):
    n = ba._binding._native
    assert n is not None
    x, dy = rows_of(65, 300, "bf16", 1).cuda(), rows_of(65, 300, "f32", 2).cuda()
    ga, be = (t.cuda() for t in weights(300, "f16", 3))
    st = torch.cuda.current_stream()
    ws = torch.empty(ba.layer_norm_grad_workspace_size(65, 300) + ba.bias_act_grad_workspace_size(65, 300), dtype=torch.uint8, device="cuda")
    got = []
    for stream in (None, st, st.cuda_stream):
        y, mean, rstd = torch.empty(65, 300, device="cuda"), torch.empty(65, device="cuda"), torch.empty(65, device="cuda")
        ba.layer_norm(x, ga, be, y, mean, rstd, 1e-3, stream=stream)
        g = ba.layer_norm_grad(dy, x, ga, mean, rstd, torch.empty_like(x), torch.empty_like(ga), torch.empty_like(ga), workspace=ws, stream=stream)
        a = ba.bias_act_grad(dy, y, torch.empty_like(dy), torch.empty(300, device="cuda").half(), "leaky_relu", 0.3, workspace=ws, stream=stream)
        got.append([y, mean, rstd, *g, *a])
    for other in got[1:]:
        assert all(torch.equal(p, q) for p, q in zip(got[0], other))
    assert n.norm(x, ga, be, y, mean, rstd, 1e-3) is True
    assert n.norm(x, ga, be.float(), y, mean, rstd, 1e-3) is False
    assert n.norm_grad(dy, x, ga, mean, rstd, torch.empty_like(x), torch.empty_like(ga), None, ws) is True
    assert n.norm_grad(dy, x, ga, mean, rstd, y, None, None, None) is False
    assert n.act_grad(dy, y, torch.empty_like(dy), None, "tanh", 0.0, None) is True
    assert n.act_grad(dy, y, x, None, "tanh", 0.0, None) is False


@pytest.mark.parametrize("rows,N", [(5, 64), (300, 1000), (1024, 4096), (20, 40000)])
def test_side_stream_and_graph_replays(ba, rows, N):
    x, dy = rows_of(rows, N, "bf16", 1).cuda(), rows_of(rows, N, "bf16", 2, "plain").cuda()
    ga, be = (t.cuda() for t in weights(N, "f32", 3))
    ws = torch.empty(max(ba.layer_norm_grad_workspace_size(rows, N), ba.bias_act_grad_workspace_size(rows, N)), dtype=torch.uint8, device="cuda")
    y, dx, dz = (torch.empty_like(x) for _ in range(3))
    mean, rstd, dg, db, dbias = (torch.empty(k, device="cuda") for k in (rows, rows, N, N, N))
    outs = (y, dx, dz, mean, rstd, dg, db, dbias)

    def step(stream=None):
        ba.layer_norm(x, ga, be, y, mean, rstd, stream=stream)
        ba.bias_act_grad(dy, y, dz, dbias, "gelu", workspace=ws, stream=stream)
        ba.layer_norm_grad(dz, x, ga, mean, rstd, dx, dg, db, workspace=ws, stream=stream)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    [t.zero_() for t in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    base = x.clone()
    for r in range(3):
        x.copy_(base * (1.0 - 0.25 * r))
        [t.zero_() for t in outs]
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, outs)), r
