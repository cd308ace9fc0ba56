"""A feed-forward layer whose weights are kept in MXFP4:

    y = x + W2 . gelu(W1 . x + b1) + b2        (one row of x per token)

The weights are quantised once, from the [inputs, outputs] matrices a model
stores.  A prompt quantises its activations too and multiplies MXFP4 by MXFP4;
a few tokens at a time keep their 16-bit activations, since then the weights'
bytes set the time.  The residual is added in the second product's epilogue.

    python examples/mxfp4_feed_forward.py [--width 4096] [--hidden 16384]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import conv_bias_activation_amd as ba  # noqa: E402


def packed(rows, k):
    """Codes and scales of `rows` rows of k values."""
    return tuple(torch.empty(s, dtype=torch.uint8, device="cuda") for s in ba.mxfp4_shapes(rows, k))


class FeedForward:
    FEW = 64          # tokens up to which the activations stay in 16 bits

    def __init__(self, w1, b1, w2, b2, max_tokens):
        """w1 [width, hidden], w2 [hidden, width], 16-bit; b1, b2 fp32 or 16-bit."""
        self.width, self.hidden = w1.shape
        self.b1, self.b2 = b1, b2
        # each output's weights are a column: blocks of 32 along the inputs, axis 0
        self.w1 = ba.mxfp4_quantize(w1, *packed(self.hidden, self.width), axis=0)
        self.w2 = ba.mxfp4_quantize(w2, *packed(self.width, self.hidden), axis=0)
        self.h = torch.empty(max_tokens, self.hidden, dtype=w1.dtype, device="cuda")
        self.xq, self.hq = packed(max_tokens, self.width), packed(max_tokens, self.hidden)

    def __call__(self, x, y):
        """x, y [tokens, width]; y may be x."""
        n = x.shape[0]
        h = self.h[:n]
        if n <= self.FEW:
            ba.gemm_mxfp4_bias_act(x, None, *self.w1, self.b1, h, "gelu")
            return ba.gemm_mxfp4_bias_add_act(h, None, *self.w2, self.b2, x, y)
        xq = ba.mxfp4_quantize(x, self.xq[0][:n], self.xq[1][:n])
        ba.gemm_mxfp4_bias_act(*xq, *self.w1, self.b1, h, "gelu")
        hq = ba.mxfp4_quantize(h, self.hq[0][:n], self.hq[1][:n])
        return ba.gemm_mxfp4_bias_add_act(*hq, *self.w2, self.b2, x, y)


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--width", type=int, default=4096)
    p.add_argument("--hidden", type=int, default=16384)
    a = p.parse_args()
    torch.manual_seed(0)
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    w1 = (torch.randn(a.width, a.hidden, device="cuda") / a.width ** 0.5).bfloat16()
    w2 = (torch.randn(a.hidden, a.width, device="cuda") / a.hidden ** 0.5).bfloat16()
    b1, b2 = torch.randn(a.hidden, device="cuda"), torch.randn(a.width, device="cuda")
    ff = FeedForward(w1, b1, w2, b2, 4096)
    # the weights that the codes stand for, as the 16-bit layer would hold them
    v1 = ba.mxfp4_dequantize(*ff.w1, torch.empty_like(w1), axis=0)
    v2 = ba.mxfp4_dequantize(*ff.w2, torch.empty_like(w2), axis=0)
    held = sum(t.numel() for t in (*ff.w1, *ff.w2))
    print(f"weights: {2 * (w1.numel() + w2.numel()) / 2**20:.0f} MiB in bf16, {held / 2**20:.0f} MiB in MXFP4")
    for n in (1, 16, 64, 512, 4096):
        x, y = torch.randn(n, a.width, **bf16), torch.empty(n, a.width, **bf16)
        ff(x, y)
        xf = x.float()
        want = xf + torch.nn.functional.gelu(xf @ v1.float() + b1) @ v2.float() + b2
        err = float((y.float() - want).norm() / want.norm())
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(20):
            ff(x, y)
        end.record()
        torch.cuda.synchronize()
        print(f"{n:5d} tokens: {start.elapsed_time(end) / 20 * 1e3:8.1f} us, "
              f"difference from 16-bit activations {err:.4f}", flush=True)


if __name__ == "__main__":
    main()
