"""Coefficients of the device GELU gradient.

For x >= 0, GELU'(-x) = Phi(-x) - x phi(x) = phi(x) (M(x) - x) with M = Phi(-x) / phi(x),
the ratio of the normal distribution's tail to its density, and GELU'(x) = 1 - GELU'(-x).
M is smooth and falls from sqrt(pi / 2) like 1 / x, so the kernels evaluate
it as t * Q(t), t = 1 / (1 + a x), Q a polynomial fitted here by least squares
on Chebyshev nodes of t in (0, 1], reweighted towards the largest relative
error: degree 9, the smallest that leaves less than the float32 steps do (degree 8
4.6e-7, 9 4.3e-8).  Run it to reprint the constants of act_grad.hip and the error of
the gradient's float32 evaluation against scipy in float64, relative to
Phi + |z phi|.
"""
import numpy as np
from scipy.special import erfcx, ndtr


def mills(x):
    return np.sqrt(np.pi / 2) * erfcx(x / np.sqrt(2))


def fit(a, deg, nodes=4000, rounds=40):
    t = np.clip((1 - np.cos(np.pi * (np.arange(nodes) + 0.5) / nodes)) / 2, 1e-9, 1.0)
    y = mills((1 / t - 1) / a) / t
    V, w = np.vander(t, deg + 1, increasing=True) / y[:, None], np.ones(nodes)
    for _ in range(rounds):
        c, *_ = np.linalg.lstsq(V * w[:, None], w, rcond=None)
        r = np.abs(V @ c - 1)
        w *= np.sqrt(0.3 + r / r.max())
        w /= w.max()
    return c.astype(np.float32)


def eval_f32(c, a, z):
    """GELU'(z), one float32 rounding per operation, the exponential exact."""
    f32, f64 = np.float32, np.float64
    fma = lambda p, q, r: (p.astype(f64) * q + r).astype(f32)  # noqa: E731
    x = np.abs(z).astype(f32)
    t = (f32(1) / fma(x, f32(a), f32(1))).astype(f32)
    q = np.full_like(x, c[-1])
    for ci in c[-2::-1]:
        q = fma(q, t, ci)
    phi = (f32(0.398942280) * np.exp(-0.5 * x.astype(f64) ** 2).astype(f32)).astype(f32)
    h = (phi * fma(t, q, -x)).astype(f32)
    return np.where(z < 0, h, (f32(1) - h).astype(f32))


if __name__ == "__main__":
    z = np.linspace(-13, 13, 1300001).astype(np.float32)
    zd = z.astype(np.float64)
    zphi = zd * np.exp(-0.5 * zd ** 2) / np.sqrt(2 * np.pi)
    a, deg = 0.32, 9
    c = fit(a, deg)
    err = np.abs(eval_f32(c, a, z) - (ndtr(zd) + zphi)) / (ndtr(zd) + np.abs(zphi))
    print(f"a = {a}, degree {deg}: error {err.max():.2e}")
    print(", ".join(f"{v:.9e}f" for v in c))
