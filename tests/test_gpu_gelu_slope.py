"""GELU's slope in bias_act_grad, value by value, at the accuracy of fp32 for
tensors of every type: dbias is fp32 and adds the slopes before dZ's rounding.

GELU'(z) is h = phi(x) (M(x) - x) for z < 0 and 1 - h for z > 0, x = |z|, M = Phi(-x) / phi(x)
as t Q(t), t = 1 / (1 + 0.32 x), Q of degree 9.  Allowance, u = 2^-24, as a share of
S = Phi(z) + |z phi(z)|, which is phi (M + x) for z < 0 and no less than 1/2 for z > 0:
  M   t is off by 3 u (its sum half a step, the reciprocal an ulp), and |dM / dt| t is at most
      (1 / 0.32) (1 + 0.32 x) (1 - x M), 3.1 at x = 0: 9.4 u of phi; the steps of Q round to u
      of their values, whose sizes add up to 3.4, the coefficients add 2.2 and the fit
      0.7: 15.7 u of phi in all where M + x is least, M = 1.25, i.e. 12.6 u of S;
  phi the exponential an ulp (2 u), its argument's rest, the constant and three products u each: 6 u;
  1 - h   u;
together 19.6 u, and half a step of 2^-149 below the normal values.
A 16-bit z has no second part of its exponent e = z^2 log2(e) / 2: the product rounds to u of
it and its constant is 1.33e-8 off, 0.22 u, and 2^e is off by ln 2 times that: 1.22 * 0.7213 * 0.6931
z^2 u = 0.61 z^2 u of phi."""
import math

import numpy as np
import pytest

from test_gpu_mxfp4 import TD, f64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24


@pytest.fixture(scope="module")
def ba():
    import conv_bias_activation_amd as m
    return m


def values(dt):
    """Every finite 16-bit value, or fp32 values of every size."""
    if dt == "f32":
        z = np.concatenate([np.linspace(-14, 14, 60001), [s * 2.0 ** e * f for s in (1, -1) for e in range(-140, 127, 3) for f in (1, 1.3)]])
        return torch.from_numpy(z.astype(np.float32))
    t = torch.from_numpy(np.arange(65536, dtype=np.uint16).view(np.int16)).view(TD[dt])
    return t[t.isfinite()].contiguous()


def near(got, z, dt):
    t = torch.from_numpy(np.clip(z, -60.0, 60.0))
    phi = 0.5 * torch.special.erfc(-t / math.sqrt(2)).numpy()
    zphi = t.numpy() * np.exp(-t.numpy() ** 2 / 2) / math.sqrt(2 * math.pi)
    err, tol = np.abs(got - (phi + zphi)), (20 + (0 if dt == "f32" else 0.61 * t.numpy() ** 2)) * U * (phi + np.abs(zphi)) + 2.0 ** -149
    worst = np.argmax(err / tol)
    assert (err <= tol).all(), (z[worst], got[worst], (phi + zphi)[worst], (err / tol)[worst])


@pytest.mark.parametrize("rows", [1, 40, 3000])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_slope_in_the_sums(ba, dt, rows):
    # one row has a gradient (of one), the others none: the sums are the slopes
    z = values(dt)
    n = z.numel() if rows < 3000 else 2000
    z = z[:: -(-z.numel() // n)].contiguous()
    n = z.numel()
    Z = z.cuda().expand(rows, n).contiguous()
    dY = torch.zeros_like(Z)
    dY[rows // 2] = 1
    db = torch.empty(n, device="cuda")
    ws = torch.empty(ba.bias_act_grad_workspace_size(rows, n), dtype=torch.uint8, device="cuda")
    ba.bias_act_grad(dY, Z, None, db, "gelu", workspace=ws)
    near(f64(db), f64(z), dt)


def test_slope_of_fp32_tensors(ba):
    z = values("f32").cuda()[None]
    dZ, _ = ba.bias_act_grad(torch.ones_like(z), z, torch.empty_like(z), None, "gelu")
    near(f64(dZ)[0], f64(z)[0], "f32")
