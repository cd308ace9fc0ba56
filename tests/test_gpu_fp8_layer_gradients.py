"""The gradients of examples/fp8_training_layer.py against those of the same layer
in fp64, whole: a term, a row or a column that is missing shows, which a
comparison along the gradient itself does not.

Allowance, a share of the fp64 gradient's 2-norm.  A value of e4m3 is off by 2^-4 of
itself at most and one of e5m2 by 2^-3, each in its own direction; a sum of products of
such values is then off by sqrt(a^2 + b^2) of its 2-norm at most, a and b the shares of its
operands (16-bit roundings are nothing beside them):
  z, h, y      sqrt(2) 2^-4 = 0.09 of z; h less than that share of z's part, say 0.09
  dh, dw2      e5m2 by e4m3: sqrt(2^-6 + 2^-8) = 0.14; dw2 with h's own 0.09: 0.17
  dz, db1      dh's 0.14 and the slope at a z that is 0.09 off: 0.17
  dn, dw1      0.17 and 0.14: 0.22, and so dx, dgamma and dbeta."""
import pytest

from test_gpu_fp8_layer import example  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

NAMES = ("x", "w1", "b1", "w2", "b2", "gamma", "beta")
ALLOWED = dict(x=0.22, w1=0.22, b1=0.17, w2=0.17, b2=1e-3, gamma=0.22, beta=0.22)


def fp64_gradients(layer, x, dy):
    leaves = [t.double().cpu().requires_grad_() for t in (x, layer.w1, layer.b1, layer.w2, layer.b2, layer.gamma, layer.beta)]
    xf, w1, b1, w2, b2, ga, be = leaves
    d = xf - xf.mean(1, keepdim=True)
    n = d / (d.square().mean(1, keepdim=True) + 1e-5).sqrt() * ga + be
    z = n @ w1.t() + b1
    h = 0.5 * z * torch.special.erfc(-z / 2 ** 0.5)
    (xf + h @ w2.t() + b2).backward(dy.double().cpu())
    return [t.grad for t in leaves]


def off(got, ref):
    return float((got - ref).norm() / ref.norm())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("width,hidden,tokens", [(256, 512, 384), (200, 1160, 70), (512, 1536, 1100)])
def test_whole_gradients(example, width, hidden, tokens, dt):  # noqa: F811
    layer = example.Layer(width, hidden, dt, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    x, dy = (torch.randn(tokens, width, generator=g, device="cuda").to(dt) for _ in range(2))
    layer.forward(x, torch.empty_like(x))
    got = [t.double().cpu() for t in layer.backward(dy)]
    for name, a, b in zip(NAMES, got, fp64_gradients(layer, x, dy)):
        assert off(a, b) <= ALLOWED[name], (name, off(a, b))
        if b.dim() == 2:                                 # each quarter by itself
            for i in range(2):
                for j in range(2):
                    q = tuple(slice(k * n // 2, (k + 1) * n // 2) for k, n in zip((i, j), b.shape))
                    assert off(a[q], b[q]) <= 1.2 * ALLOWED[name], (name, i, j)
    # x's gradient without dy, which the layer's sum passes on as it is: the way through the products
    way = dy.double().cpu()
    ref = fp64_gradients(layer, x, dy)[0] - way
    assert off(got[0] - way, ref) <= ALLOWED["x"]


def test_the_allowance_sees_what_is_missing(example):  # noqa: F811
    # on the fp64 gradients: without half of the rows, of the columns, or without a term
    layer = example.Layer(256, 512, torch.bfloat16, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    x, dy = (torch.randn(384, 256, generator=g, device="cuda").bfloat16() for _ in range(2))
    grads = dict(zip(NAMES, fp64_gradients(layer, x, dy)))
    way = dy.double().cpu()
    for lost in (way, grads["x"] - way):
        assert off(grads["x"] - lost, grads["x"]) > 2 * ALLOWED["x"]
    for name, t in grads.items():
        half = t.clone()
        half[: len(half) // 2] = 0
        assert off(half, t) > 2 * ALLOWED[name]
