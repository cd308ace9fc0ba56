"""The feed-forward layer of examples/mxfp4_feed_forward.py, its two products
each against fp64 sums over what went into it (the intermediate as stored and
quantised), with the allowance that test_gpu_mxfp4 derives."""
import importlib.util
import os

import numpy as np
import pytest

import mxfp4_ref as mx
from test_gpu_mxfp4 import f64, reference

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def layer():
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "mxfp4_feed_forward.py")
    spec = importlib.util.spec_from_file_location("mxfp4_feed_forward", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def stored(codes, scales, n, k):
    return mx.values(codes[:n].cpu().numpy(), scales[:n].cpu().numpy(), k)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,in_place", [(1, False), (64, True), (65, False), (1100, True)])
def test_layer(layer, tokens, in_place, dt):
    width, hidden = 200, 1160
    t = {"bf16": torch.bfloat16, "f16": torch.float16}[dt]
    g = torch.Generator(device="cuda").manual_seed(tokens)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    w1, w2 = (rand(width, hidden) / 14).to(t), (rand(hidden, width) / 34).to(t)
    b1, b2 = rand(hidden), rand(width).to(t)
    ff = layer.FeedForward(w1, b1, w2, b2, 1200)
    v1, v2 = stored(*ff.w1, hidden, width), stored(*ff.w2, width, hidden)
    want_c, want_s = mx.quantize(np.ascontiguousarray(f64(w1).T))
    assert np.array_equal(ff.w1[0].cpu().numpy(), want_c) and np.array_equal(ff.w1[1].cpu().numpy(), want_s)

    x = rand(tokens, width).to(t)
    x0 = f64(x)
    y = x if in_place else torch.empty_like(x)
    assert ff(x, y) is y
    torch.cuda.synchronize()
    h = f64(ff.h[:tokens])
    few = tokens <= ff.FEW
    a1 = x0 if few else stored(*ff.xq, tokens, width)
    a2 = h if few else stored(*ff.hq, tokens, hidden)
    if not few:
        want_c, want_s = mx.quantize(h)
        assert np.array_equal(ff.hq[0][:tokens].cpu().numpy(), want_c)
        assert np.array_equal(ff.hq[1][:tokens].cpu().numpy(), want_s)
    for got, (ref, tol) in ((h, reference(a1, v1, f64(b1), None, "gelu", 0.0, dt)),
                            (f64(y), reference(a2, v2, f64(b2), x0, "none", 0.0, dt))):
        assert (np.abs(got - ref) <= tol).all()
