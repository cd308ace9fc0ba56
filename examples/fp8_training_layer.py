"""A feed-forward layer behind a layer norm, run and trained with 8-bit products:

    y = x + W2 . gelu(W1 . norm(x) + b1) + b2        (one row of x per token)

Weights are kept in 16 bits and quantised in blocks of 128 x 128, activations
and gradients (e5m2) with a scale for each 128 values along whatever index a
product sums over: a row for the layer's own products and dX = dZ . W, a column for
dW = dZ^T . X.  The backward pass takes the gradient of y and leaves those of x, the
weights, the biases and the norm.

    python examples/fp8_training_layer.py [--tokens 4096] [--width 1024] [--hidden 4096]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import conv_bias_activation_amd as ba  # noqa: E402

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


def quantized(x, f8, axis=1, block_rows=1):
    """x's rows (axis 1) or columns (axis 0) in 8 bits."""
    rows, k = x.shape if axis == 1 else x.shape[::-1]
    codes, scales = ba.fp8_shapes(rows, k, block_rows)
    return ba.fp8_quantize(x, torch.empty(codes, dtype=f8, device=x.device),
                           torch.empty(scales, dtype=torch.uint8, device=x.device), axis=axis)


class Layer:
    def __init__(self, width, hidden, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.w1, self.w2 = (rand(hidden, width) / width ** 0.5).to(dtype), (rand(width, hidden) / hidden ** 0.5).to(dtype)
        self.b1, self.b2 = 0.1 * rand(hidden), 0.1 * rand(width)
        self.gamma, self.beta = 1 + 0.1 * rand(width), 0.1 * rand(width)

    def forward(self, x, y):
        """y from x [tokens, width]; keeps what backward wants."""
        tokens, hidden = x.shape[0], self.w1.shape[0]
        n, mean, rstd = torch.empty_like(x), x.new_empty(tokens, dtype=torch.float32), x.new_empty(tokens, dtype=torch.float32)
        ba.layer_norm(x, self.gamma, self.beta, n, mean, rstd)
        z, h = x.new_empty(tokens, hidden), x.new_empty(tokens, hidden)
        ba.gemm_fp8_bias_act(*quantized(n, E4M3), *quantized(self.w1, E4M3, block_rows=128), self.b1, h, "gelu", Z=z)
        ba.gemm_fp8_bias_add_act(*quantized(h, E4M3), *quantized(self.w2, E4M3, block_rows=128), self.b2, x, y)
        self.kept = x, n, mean, rstd, z, h
        return y

    def backward(self, dy):
        """The gradients of x, w1, b1, w2, b2, gamma and beta."""
        x, n, mean, rstd, z, h = self.kept
        dx, dn, dh = torch.empty_like(x), torch.empty_like(x), torch.empty_like(h)
        dw1, dw2 = torch.empty_like(self.w1), torch.empty_like(self.w2)
        db1, db2, dgamma, dbeta = (torch.empty_like(t) for t in (self.b1, self.b2, self.gamma, self.beta))
        need = max(ba.bias_act_grad_workspace_size(*h.shape), ba.bias_act_grad_workspace_size(*x.shape),
                   ba.layer_norm_grad_workspace_size(*x.shape))
        ws = torch.empty(need, dtype=torch.uint8, device=x.device)
        # the second product: y = x + h . w2^T + b2
        ba.bias_act_grad(dy, None, None, db2, workspace=ws)
        ba.gemm_fp8_bias_act(*quantized(dy, E5M2), *quantized(self.w2, E4M3, 0, 128), None, dh)
        ba.gemm_fp8_bias_act(*quantized(dy, E5M2, 0), *quantized(h, E4M3, 0), None, dw2)
        # the first: h = gelu(z), z = n . w1^T + b1
        dz, _ = ba.bias_act_grad(dh, z, dh, db1, "gelu", workspace=ws)
        ba.gemm_fp8_bias_act(*quantized(dz, E5M2), *quantized(self.w1, E4M3, 0, 128), None, dn)
        ba.gemm_fp8_bias_act(*quantized(dz, E5M2, 0), *quantized(n, E4M3, 0), None, dw1)
        ba.layer_norm_grad(dn, x, self.gamma, mean, rstd, dx, dgamma, dbeta, workspace=ws)
        dx += dy
        return dx, dw1, db1, dw2, db2, dgamma, dbeta


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--tokens", type=int, default=4096)
    p.add_argument("--width", type=int, default=1024)
    p.add_argument("--hidden", type=int, default=4096)
    a = p.parse_args()
    layer = Layer(a.width, a.hidden)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.tokens, a.width, generator=g, device="cuda").bfloat16()
    dy = torch.randn(a.tokens, a.width, generator=g, device="cuda").bfloat16()
    y = torch.empty_like(x)
    layer.forward(x, y)
    grads = layer.backward(dy)
    # the same layer in fp32
    leaves = [t.float().requires_grad_() for t in (x, layer.w1, layer.b1, layer.w2, layer.b2, layer.gamma, layer.beta)]
    xf, w1, b1, w2, b2, ga, be = leaves
    n = torch.nn.functional.layer_norm(xf, (a.width,), ga, be)
    want = xf + torch.nn.functional.gelu(n @ w1.t() + b1) @ w2.t() + b2
    want.backward(dy.float())
    off = lambda got, ref: float((got.float() - ref).norm() / ref.norm())  # noqa: E731
    print(f"y differs from the fp32 layer by {off(y, want.detach()):.4f}")
    for name, got, leaf in zip(("x", "w1", "b1", "w2", "b2", "gamma", "beta"), grads, leaves):
        print(f"gradient of {name:5s} by {off(got, leaf.grad):.4f}")
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(20):
        layer.forward(x, y)
        layer.backward(dy)
    end.record()
    torch.cuda.synchronize()
    us = start.elapsed_time(end) / 20 * 1e3
    print(f"{a.tokens} tokens, forward and backward: {us:.0f} us, {12e-6 * a.tokens * a.width * a.hidden / us:.0f} TFLOP/s")


if __name__ == "__main__":
    main()
