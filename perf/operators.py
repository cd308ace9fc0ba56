"""The MXFP4 operators (4-bit floating point in blocks of 32 values that share a power-of-two scale), case by case.

Three kinds of pass:
  round_trip  X is quantised to MXFP4 and read back in its own type
  linear      act(X . W^T + bias (+ R)): the activations are quantised within the call, W is held in MXFP4
  tokens      act(X . W^T + bias (+ R)): 16-bit activations as they are, W is held in MXFP4 (few tokens at a time)

Storage: a row of K values is padded with zeros to whole groups of 128; codes are uint8 [rows, 64 * groups], the even value in
the low four bits; scales are uint8 [rows, 4 * groups], the value 2^(byte - 127) each.
"""
import math

import torch

own = False

BF16, F16, F32 = "bfloat16", "float16", "float32"


def listed():
    return [
        # one token's activations, quantised before a layer and checked by reading them back: latency alone
        dict(name="round_trip_one_token", op="round_trip", rows=1, K=4096, x=BF16, axis=1),
        # ragged activations in fp32, the last block of a row incomplete
        dict(name="round_trip_ragged", op="round_trip", rows=1021, K=1003, x=F32, axis=1),
        # the activations of a long prompt
        dict(name="round_trip_prompt", op="round_trip", rows=32768, K=4096, x=BF16, axis=1),
        # a [K, N] weight, whose blocks run down its columns
        dict(name="round_trip_weight", op="round_trip", rows=4096, K=4096, x=F16, axis=0),
        # a few sequences decoding together
        dict(name="linear_decode", op="linear", M=8, N=4096, K=4096, x=BF16, y=BF16, bias=F32, act="gelu", alpha=0.0, residual=False),
        # the small LeakyReLU product of this repository's workloads
        dict(name="linear_leaky_1024x640x256", op="linear", M=1024, N=640, K=256, x=F16, y=F32, bias=F32, act="leaky_relu", alpha=0.001, residual=False),
        # nothing a multiple of anything, with a residual
        dict(name="linear_ragged", op="linear", M=333, N=1001, K=1503, x=F16, y=F16, bias=F16, act="none", alpha=0.0, residual=True),
        # the square product of this repository's workloads
        dict(name="linear_gelu_4096", op="linear", M=4096, N=4096, K=4096, x=BF16, y=BF16, bias=F32, act="gelu", alpha=0.0, residual=False),
        # its largest one: a long prompt through a narrow layer
        dict(name="linear_leaky_32768x4096x1024", op="linear", M=32768, N=4096, K=1024, x=BF16, y=BF16, bias=F32, act="leaky_relu", alpha=0.01, residual=False),
        # one token through one layer
        dict(name="tokens_1", op="tokens", M=1, N=4096, K=4096, x=BF16, y=BF16, bias=BF16, act="relu", alpha=0.0, residual=False),
        # a ragged batch of tokens with a residual and an fp32 result
        dict(name="tokens_ragged", op="tokens", M=37, N=1001, K=1503, x=F16, y=F32, bias=F32, act="sigmoid", alpha=0.0, residual=True),
        # many sequences decoding together
        dict(name="tokens_256", op="tokens", M=256, N=4096, K=4096, x=BF16, y=BF16, bias=F32, act="none", alpha=0.0, residual=True),
    ]


def _log_int(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm; one in three is a multiple of 64 where it is that large."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v >= 64 and rng.random() < 1 / 3:
        v -= v % 64
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["round_trip", "linear", "linear", "tokens", "tokens"])
    if op == "round_trip":
        while True:
            rows, K = _log_int(rng, 1, 32768), _log_int(rng, 1, 16384)
            if rows * K <= 32768 * 4096:
                return dict(op=op, rows=rows, K=K, x=rng.choice([BF16, F16, F32]), axis=rng.choice([1, 1, 0]))
    x = rng.choice([BF16, BF16, F16])
    act = rng.choice(["none", "relu", "leaky_relu", "tanh", "gelu", "sigmoid"])
    while True:
        M, N, K = _log_int(rng, 1, 32768 if op == "linear" else 512), _log_int(rng, 64, 16384), _log_int(rng, 64, 16384)
        if M * N * K <= (4096 ** 3 if op == "linear" else 512 * 4096 * 4096) and M * N <= 2 ** 27 and M * K <= 2 ** 27:
            return dict(op=op, M=M, N=N, K=K, x=x, y=rng.choice([x, x, F32]), bias=rng.choice([F32, x]), act=act,
                        alpha=0.01 if act == "leaky_relu" else 0.0, residual=rng.random() < 0.4)


# ---- inputs ----------------------------------------------------------------------------------------------------------------

def _activations(g, rows, K, dtype):
    """Normal values whose channels differ in size, a few of them by much; one row in sixteen of many is all zero (padding)."""
    size = torch.exp(0.6 * torch.randn(K, generator=g, device="cuda"))
    size = torch.where(torch.rand(K, generator=g, device="cuda") < 0.01, size * 20, size)
    x = torch.randn(rows, K, generator=g, device="cuda") * size
    if rows >= 64:
        x[torch.rand(rows, generator=g, device="cuda") < 1 / 16] = 0
    return x.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = getattr(torch, case["x"])
    if case["op"] == "round_trip":
        rows, K = case["rows"], case["K"]
        x = _activations(g, rows, K, dtype)
        x = x.t().contiguous() if case["axis"] == 0 else x
        groups = -(-K // 128)
        return dict(case=case, x=x, y=torch.empty_like(x), codes=torch.empty(rows, 64 * groups, dtype=torch.uint8, device="cuda"),
                    scales=torch.empty(rows, 4 * groups, dtype=torch.uint8, device="cuda"))
    M, N, K = case["M"], case["N"], case["K"]
    x = _activations(g, M, K, dtype)
    w_codes, w_scales = _quantize(torch.randn(N, K, generator=g, device="cuda") / math.sqrt(K))
    bias = (0.5 * torch.randn(N, generator=g, device="cuda")).to(getattr(torch, case["bias"]))
    out = getattr(torch, case["y"])
    r = torch.randn(M, N, generator=g, device="cuda").to(out) if case["residual"] else None
    state = dict(case=case, x=x, w_codes=w_codes, w_scales=w_scales, bias=bias, r=r, y=torch.empty(M, N, dtype=out, device="cuda"))
    if case["op"] == "linear":
        groups = w_codes.shape[1] // 64
        state["codes"] = torch.empty(M, 64 * groups, dtype=torch.uint8, device="cuda")
        state["scales"] = torch.empty(M, 4 * groups, dtype=torch.uint8, device="cuda")
    return state


# ---- the plain form --------------------------------------------------------------------------------------------------------

def _quantize(x):
    """Rows of X (blocks along them) -> codes, scales."""
    rows, K = x.shape
    x = torch.nn.functional.pad(x.float(), (0, -K % 128)).view(rows, -1, 32)
    top = x.abs().amax(-1, keepdim=True)
    e = (torch.frexp(top)[1] - 3).clamp(-127, 127)  # floor(log2 top) - 2
    e = torch.where(top == 0, -127, e)
    a = torch.ldexp(x.abs(), -e)
    code = (a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)  # ties to the even code
    code = code | (torch.signbit(x).byte() << 3)
    code = code.view(rows, -1)
    return code[:, ::2] | (code[:, 1::2] << 4), (e + 127).byte().view(rows, -1)


def _dequantize(codes, scales, K):
    """Codes, scales -> fp32 values [rows, K]."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    v = table[torch.stack([codes & 15, codes >> 4], -1).int()].view(codes.shape[0], -1, 32)
    return torch.ldexp(v, scales.int().unsqueeze(-1) - 127).view(codes.shape[0], -1)[:, :K]


def _act(z, case):
    a = case["act"]
    if a == "relu":
        return z.clamp_min(0)
    if a == "leaky_relu":
        return torch.where(z >= 0, z, case["alpha"] * z)
    if a == "tanh":
        return torch.tanh(z)
    if a == "gelu":
        return 0.5 * z * torch.special.erfc(z * -math.sqrt(0.5))
    if a == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    return z


def run(state):
    case, x, y = state["case"], state["x"], state["y"]
    if own:
        import conv_bias_activation_amd as ba

        if case["op"] == "round_trip":
            ba.mxfp4_quantize(x, state["codes"], state["scales"], axis=case["axis"])
            return ba.mxfp4_dequantize(state["codes"], state["scales"], y, axis=case["axis"])
        a, a_scales = x, None
        if case["op"] == "linear":
            a, a_scales = ba.mxfp4_quantize(x, state["codes"], state["scales"])
        if state["r"] is None:
            return ba.gemm_mxfp4_bias_act(a, a_scales, state["w_codes"], state["w_scales"], state["bias"], y, case["act"], case["alpha"])
        return ba.gemm_mxfp4_bias_add_act(a, a_scales, state["w_codes"], state["w_scales"], state["bias"], state["r"], y, case["act"], case["alpha"])
    if case["op"] == "round_trip":
        rows = x.t() if case["axis"] == 0 else x
        v = _dequantize(*_quantize(rows), case["K"]).to(x.dtype)
        return v.t().contiguous() if case["axis"] == 0 else v
    a = _dequantize(*_quantize(x), case["K"]) if case["op"] == "linear" else x.float()
    z = torch.matmul(a, _dequantize(state["w_codes"], state["w_scales"], case["K"]).t()) + state["bias"].float()
    if state["r"] is not None:
        z = z + state["r"].float()
    return _act(z, case).to(y.dtype)


# ---- what a pass cannot do without -----------------------------------------------------------------------------------------

_SIZE = {BF16: 2, F16: 2, F32: 4}


def work(case):
    if case["op"] == "round_trip":
        n = case["rows"] * case["K"]
        # X read, codes and scales written, read again, Y written
        return {"bytes": 2 * n * _SIZE[case["x"]] + 2 * (n / 2 + n / 32), "flops": 2 * n}
    M, N, K = case["M"], case["N"], case["K"]
    w = M * K * _SIZE[case["x"]] + N * K * (1 / 2 + 1 / 32) + N * _SIZE[case["bias"]] + M * N * _SIZE[case["y"]] * (2 if case["residual"] else 1)
    return {"bytes": w, "flops": 2 * M * N * K}


# ---- from the definition, in 64 bits ---------------------------------------------------------------------------------------

def _nearest(x):
    """X (rows, blocks along them) with each block rounded to its 4-bit values, in 64 bits."""
    rows, K = x.shape
    n = -(-K // 32)
    v = torch.zeros(rows, 32 * n, dtype=torch.float64, device=x.device)
    v[:, :K] = x.double()
    v = v.view(rows, n, 32)
    top = v.abs().max(-1, keepdim=True).values
    scale = torch.exp2((torch.floor(torch.log2(top.clamp_min(1e-300))) - 2).clamp(-127, 127))
    t = v / scale
    # the spacing of the values is 1/2 below 2, 1 from 2 to 4 and 2 from there: round to it, halves to even
    step = torch.where(t.abs() < 2, 0.5, torch.where(t.abs() < 4, 1.0, 2.0)).double()
    q = torch.round(t / step) * step
    return (q.clamp(-6, 6) * scale).view(rows, -1)[:, :K]


def _value(codes, scales, K):
    nib = torch.stack([codes & 15, codes >> 4], 2).reshape(codes.shape[0], -1).long()
    sign, ex, man = 1 - 2 * (nib >> 3), (nib >> 1) & 3, nib & 1
    mag = torch.where(ex == 0, 0.5 * man.double(), (1 + 0.5 * man.double()) * torch.exp2((ex - 1).double()))
    s = torch.exp2(scales.double() - 127).repeat_interleave(32, 1)
    return (sign * mag * s)[:, :K]


def exact(case, seed):
    state = prepare(case, seed)
    x = state["x"]
    if case["op"] == "round_trip":
        return _nearest(x.t()).t().contiguous() if case["axis"] == 0 else _nearest(x)
    a = _nearest(x) if case["op"] == "linear" else x.double()
    z = a @ _value(state["w_codes"], state["w_scales"], case["K"]).t().contiguous()
    z = z + state["bias"].double()
    if state["r"] is not None:
        z = z + state["r"].double()
    act = case["act"]
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "leaky_relu":
        return torch.maximum(z, z * case["alpha"])
    if act == "tanh":
        return 1 - 2 / (torch.exp(2 * z) + 1)
    if act == "gelu":
        return z * torch.special.erfc(-z / math.sqrt(2)) / 2
    if act == "sigmoid":
        return torch.sigmoid(z)
    return z
