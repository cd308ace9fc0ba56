"""The trained layer of examples/fp8_training_layer.py: every step against the
fp64 formula over what went into it (the intermediates as stored and
quantised), with the allowances that test_gpu_fp8 and test_gpu_norm derive; and
the whole against fp64 differences."""
import importlib.util
import os
import sys

import numpy as np
import pytest

import fp8_ref as f8
from oracle.compare import gamma as gamma_n, ulp
from test_gpu_fp8 import reference
from test_gpu_mxfp4 import f64
from test_gpu_norm import D, U, grad_reference, norm_reference, ok, slope

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "fp8_training_layer.py")
    spec = importlib.util.spec_from_file_location("fp8_training_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


class Packed:
    """What quantising x gives, as test_gpu_fp8's reference wants it."""
    def __init__(self, x, fmt, block_rows=1):
        x = np.ascontiguousarray(x)
        self.c, self.s = f8.quantize(x, fmt, block_rows)
        self.K, self.fmt, self.block_rows = x.shape[1], fmt, block_rows

    @property
    def values(self):
        return f8.values(self.c, self.s, self.K, self.fmt, self.block_rows)

    @property
    def powers(self):
        from test_gpu_fp8 import powers
        return powers(self.c, self.s, self.K, self.fmt, self.block_rows)


def near(got, ref_tol, what):
    ok(f64(got), *ref_tol, what)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("tokens", [1, 70, 600])
def test_layer(example, tokens, dt):
    width, hidden, E4, E5 = 200, 1160, "f8e4m3", "f8e5m2"
    t = {"bf16": torch.bfloat16, "f16": torch.float16}[dt]
    layer = example.Layer(width, hidden, t, seed=tokens)
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x = torch.randn(tokens, width, generator=g, device="cuda").to(t)
    dy = torch.randn(tokens, width, generator=g, device="cuda").to(t)
    y = torch.empty_like(x)
    assert layer.forward(x, y) is y
    _, n, mean, rstd, z, h = layer.kept
    dx, dw1, db1, dw2, db2, dga, dbe = layer.backward(dy)
    torch.cuda.synchronize()

    # forward
    rm, rr, rn, tol, mtol = norm_reference(f64(x), f64(layer.gamma), f64(layer.beta), 1e-5)
    ok(f64(n), rn, tol + 0.5 * ulp(np.abs(rn) + tol, dt), "norm")
    ok(f64(mean), rm, mtol, "mean")
    ok(f64(rstd), rr, (D + 16) * U * rr, "rstd")
    a, w = Packed(f64(n), E4), Packed(f64(layer.w1), E4, 128)
    near(z, reference(a, w, f64(layer.b1), None, "none", 0.0, dt), "z")
    near(h, reference(a, w, f64(layer.b1), None, "gelu", 0.0, dt), "h")
    near(y, reference(Packed(f64(h), E4), Packed(f64(layer.w2), E4, 128), f64(layer.b2), f64(x), "none", 0.0, dt), "y")

    # backward of the second product
    d = f64(dy)
    s = gamma_n(tokens + 8, U) * np.abs(d).sum(0)
    ok(f64(db2), d.sum(0), s + 2.0 ** -149 + U * np.abs(d.sum(0)), "db2")
    near(dw2, reference(Packed(d.T, E5), Packed(f64(h).T, E4), None, None, "none", 0.0, dt), "dw2")
    # dh is overwritten by dz: form it as stored, from the same call
    dh = torch.empty_like(h)
    example.ba.gemm_fp8_bias_act(*example.quantized(dy, example.E5M2), *example.quantized(layer.w2, example.E4M3, 0, 128), None, dh)
    near(dh, reference(Packed(d, E5), Packed(f64(layer.w2).T, E4, 128), None, None, "none", 0.0, dt), "dh")
    # and of the first
    dz, _ = example.ba.bias_act_grad(dh, z, torch.empty_like(dh), None, "gelu")
    sl, sle = slope(f64(z), "gelu", 0.0)
    ref = f64(dh) * sl
    tol = np.abs(f64(dh)) * sle + U * np.abs(ref)
    ok(f64(dz), ref, tol + 0.5 * ulp(np.abs(ref) + tol, dt), "dz")
    ok(f64(db1), ref.sum(0), gamma_n(tokens + 8, U) * np.abs(ref).sum(0) + 1.01 * tol.sum(0) + U * np.abs(ref.sum(0)), "db1")
    near(dw1, reference(Packed(f64(dz).T, E5), Packed(f64(n).T, E4), None, None, "none", 0.0, dt), "dw1")
    dn = torch.empty_like(x)
    example.ba.gemm_fp8_bias_act(*example.quantized(dz, example.E5M2), *example.quantized(layer.w1, example.E4M3, 0, 128), None, dn)
    near(dn, reference(Packed(f64(dz), E5), Packed(f64(layer.w1).T, E4, 128), None, None, "none", 0.0, dt), "dn")
    rdx, tol, rw = grad_reference(f64(dn), f64(x), f64(layer.gamma), f64(mean), f64(rstd))
    tol = tol + 0.5 * ulp(np.abs(rdx) + tol, dt)         # as layer_norm_grad rounds it, then the sum with dy
    ok(f64(dx), rdx + d, tol + 0.5 * ulp(np.abs(rdx + d) + tol, dt), "dx")
    for got, (r, tw) in zip((dga, dbe), rw):
        ok(f64(got), r, tw + U * np.abs(r), "dgamma, dbeta")


def test_gradients_against_differences(example):
    # Along directions v: the gradient's product with v against the change of
    # sum(dy y) of the fp64 layer.  What the 8-bit steps leave: each value of e4m3 is off by
    # 2^-4 of itself at most and of e5m2 by 2^-3, in no one direction, so a sum of n products
    # loses some 2^-3 / sqrt(n) of the sum of their sizes; 0.1 of the 2-norms is three times what
    # that gives for these sizes (n = 256 at least).
    width, hidden, tokens = 256, 512, 384
    layer = example.Layer(width, hidden, torch.bfloat16, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    x, dy = (torch.randn(tokens, width, generator=g, device="cuda").bfloat16() for _ in range(2))
    layer.forward(x, torch.empty_like(x))
    got = layer.backward(dy)
    names = ("x", "w1", "b1", "w2", "b2", "gamma", "beta")
    at = dict(zip(names, (t.double().cpu() for t in (x, layer.w1, layer.b1, layer.w2, layer.b2, layer.gamma, layer.beta))))

    def total(p):
        d = p["x"] - p["x"].mean(1, keepdim=True)
        n = d / (d.square().mean(1, keepdim=True) + 1e-5).sqrt() * p["gamma"] + p["beta"]
        z = n @ p["w1"].t() + p["b1"]
        h = 0.5 * z * torch.special.erfc(-z / 2 ** 0.5)
        return float((dy.double().cpu() * (p["x"] + h @ p["w2"].t() + p["b2"])).sum())

    for name, grad in zip(names, got):
        gd = grad.double().cpu()
        v = gd / gd.norm()                               # the direction in which the gradient says most
        step = 1e-4 * float(at[name].norm())
        slope_v = (total({**at, name: at[name] + step * v}) - total({**at, name: at[name] - step * v})) / (2 * step)
        assert abs(float((gd * v).sum()) - slope_v) <= 0.1 * abs(slope_v), (name, float((gd * v).sum()), slope_v)


def test_example_runs(example, monkeypatch, capsys):
    monkeypatch.setattr(sys, "argv", ["fp8_training_layer.py", "--tokens", "300", "--width", "256", "--hidden", "640"])
    example.main()
    assert "forward and backward" in capsys.readouterr().out


def test_two_layers_on_two_streams(example):
    # each with tensors and workspaces of its own, at once
    x = torch.randn(500, 256, device="cuda").bfloat16()
    layers = [example.Layer(256, 768, seed=s) for s in (1, 2)]
    want = []
    for layer in layers:
        y = layer.forward(x, torch.empty_like(x)).clone()
        want.append([y, *(t.clone() for t in layer.backward(x))])
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in layers], [None, None]
    for _ in range(3):
        for i, (layer, s) in enumerate(zip(layers, streams)):
            with torch.cuda.stream(s):
                y = layer.forward(x, torch.empty_like(x))
                got[i] = [y, *layer.backward(x)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_a_captured_training_step(example):
    x = torch.randn(300, 256, device="cuda").bfloat16()
    dy = torch.randn(300, 256, device="cuda").bfloat16()
    layer, y = example.Layer(256, 768, seed=3), torch.empty(300, 256, device="cuda").bfloat16()
    layer.forward(x, y), layer.backward(dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(x, y)
        grads = layer.backward(dy)
    base = x.clone()
    for r in range(3):
        x.copy_(base * (1 + r))
        graph.replay()
        torch.cuda.synchronize()
        got = [y.clone(), *(t.clone() for t in grads)]
        other = layer.forward(x, torch.empty_like(y))
        want = [other, *layer.backward(dy)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), r
