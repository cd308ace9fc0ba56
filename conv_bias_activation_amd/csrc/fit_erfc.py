"""Coefficients of the device erfc used by the GELU epilogue.

For x >= 0 the kernels evaluate erfc(x) = t * exp(-x^2 + P(t)) with
t = 1 / (1 + x/2) and P a polynomial of degree 9: the functional form of the
Chebyshev-fitted erfc of Press, Teukolsky, Vetterling and Flannery
(Numerical Recipes, section 6.2), whose exponent is smooth in t on the whole
half-line.  The coefficients here are this script's own least-squares fit of
P(t) = ln(erfc(x) / t) + x^2 on Chebyshev nodes of t in [1/6, 1]
(x in [0, 10]; past x = 10 erfc is below the float32 range); negative
arguments use erfc(-x) = 2 - erfc(x).  Run it to reprint the constants used
in device_common.hpp (and mx_act.hpp) and the maximum relative error of the float32
evaluation (Horner with fused multiply-adds, exp through exp2) against
scipy.special.erfc in float64.

fit_short() is the same form for outputs that are next rounded to 16 bits, in
GELU's own variable: 2 Phi(-z) = t * 2^(-z^2 log2(e) / 2 + Q(t)) for z in
[0, 14] with t = 1 / (1 + 0.35 z) and Q of degree 5, the smallest that keeps
the relative error below 2^-17 (0.35 is the best multiple of 0.05 for it),
fitted by least squares reweighted towards the largest error.
"""
import numpy as np
from scipy.special import erfc

DEG, NODES, XMAX = 9, 800, 10.0
LOG2E = 1.4426950408889634


def fit():
    tmin = 1.0 / (1.0 + XMAX / 2.0)
    k = np.arange(NODES)
    t = tmin + (np.cos((2 * k + 1) * np.pi / (2 * NODES)) + 1) / 2 * (1.0 - tmin)
    x = 2.0 * (1.0 / t - 1.0)
    f = np.log(erfc(x) / t) + x * x
    c, *_ = np.linalg.lstsq(np.vander(t, DEG + 1, increasing=True), f, rcond=None)
    return c.astype(np.float32)


def eval_f32(c, xs):
    """The device's evaluation order, one float32 rounding per operation."""
    f32 = np.float32
    xs = xs.astype(f32)
    t = (f32(1.0) / (f32(1.0) + f32(0.5) * xs)).astype(f32)
    p = np.full_like(xs, c[-1])
    for ci in c[-2::-1]:
        p = (p.astype(np.float64) * t + ci).astype(f32)              # fma
    e = (p.astype(np.float64) - xs.astype(np.float64) * xs).astype(f32)   # fma(-x, x, p)
    y = (t * np.exp2((e * f32(LOG2E)).astype(f32).astype(np.float64)).astype(f32)).astype(f32)
    return y


def max_rel_error(c, lo=0.0, hi=9.0):
    xs = np.linspace(lo, hi, 900001).astype(np.float32)
    ref = erfc(xs.astype(np.float64))
    y = eval_f32(c, xs).astype(np.float64)
    return float(np.max(np.abs(y - ref) / ref))


def fit_short(a=0.35, deg=5, zmax=14.0, nodes=4000, rounds=40):
    from scipy.special import log_ndtr
    tmin = 1.0 / (1.0 + a * zmax)
    k = np.arange(nodes)
    u = np.cos((2 * k + 1) * np.pi / (2 * nodes))
    t = tmin + (u + 1) / 2 * (1.0 - tmin)
    z = (1.0 / t - 1.0) / a
    f = (log_ndtr(-z) + np.log(2.0)) * LOG2E + z * z * (LOG2E / 2) - np.log2(t)
    cheb = np.polynomial.chebyshev
    V, w, best = cheb.chebvander(u, deg), np.ones(nodes), None
    for _ in range(rounds):
        c, *_ = np.linalg.lstsq(V * w[:, None], f * w, rcond=None)
        e = np.abs(V @ c - f)
        if best is None or e.max() < best[0]:
            best = e.max(), c
        w *= (e / e.max() + 0.05) ** 0.5
        w /= w.mean()
    # Chebyshev in u -> powers of t, u = (2 t - 1 - tmin) / (1 - tmin)
    poly = np.polynomial.Polynomial(cheb.cheb2poly(best[1]))
    in_t = poly(np.polynomial.Polynomial([-(1 + tmin) / (1 - tmin), 2 / (1 - tmin)]))
    return in_t.coef.astype(np.float32), best[0] / LOG2E


if __name__ == "__main__":
    c = fit()
    for i, v in enumerate(c):
        print(f"c{i} = {float(v):.9e}f")
    for lo, hi in ((0.0, 1.0), (1.0, 4.0), (4.0, 9.0)):
        print(f"max relative error of the float32 evaluation on [{lo}, {hi}]: {max_rel_error(c, lo, hi):.3e}")
    c, err = fit_short()
    for i, v in enumerate(c):
        print(f"q{i} = {float(v):.9e}f")
    print(f"largest relative error of fit_short: {err:.3e}")
