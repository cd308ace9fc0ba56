"""Operators of a layer in 8-bit floating point and of its training, case by case.

Six kinds of pass:
  round_trip   X is quantised to 8-bit floating point (a power-of-two scale for each 128 values of a row, or each 128 x 128 of a
               matrix) and read back in its own type
  linear       act(X . W^T + bias (+ R)): the activations are quantised within the call, W is held in 8 bits (128 x 128); with
               `pre` the sums before the activation come too, as a backward pass wants them
  act_grad     dZ = dY * act'(Z) and the bias's gradient, the column sums of dZ
  linear_grad  the backward pass of a linear layer: dZ and the bias's gradient, then dX = dZ . W and dW = dZ^T . X in 8 bits (the
               gradient in e5m2), every operand quantised within the call along its own reduction; dX and dW in X's and W's type
  norm         layer norm, with the row's mean and 1 / deviation where a backward pass follows
  norm_grad    its backward pass: dX and the gradients of its weight and bias

Storage: a row of K values is padded with zeros to whole blocks of 128; codes are float8_e4m3fn or float8_e5m2
[rows, 128 * ceil(K / 128)]; scales are uint8 [rows, 4 * ceil(K / 512)], or [ceil(rows / 128), 4 * ceil(K / 512)] for blocks of
128 rows, the value 2^(byte - 127) each.
"""
import math

import torch

own = False

BF16, F16, F32 = "bfloat16", "float16", "float32"
E4M3, E5M2 = "float8_e4m3fn", "float8_e5m2"


def listed():
    return [
        # the activations of a long prompt
        dict(name="round_trip_prompt", op="round_trip", rows=32768, K=4096, x=BF16, f8=E4M3, axis=1, block_rows=1),
        # a [K, N] weight in blocks of 128 x 128, turned so that its columns become rows
        dict(name="round_trip_weight", op="round_trip", rows=4096, K=4096, x=F16, f8=E4M3, axis=0, block_rows=128),
        # a few sequences decoding together
        dict(name="linear_decode", op="linear", M=8, N=4096, K=4096, x=BF16, y=BF16, bias=F32, act="gelu", alpha=0.0, residual=False, pre=False),
        # the square product of this repository's workloads
        dict(name="linear_gelu_4096", op="linear", M=4096, N=4096, K=4096, x=BF16, y=BF16, bias=F32, act="gelu", alpha=0.0, residual=False, pre=False),
        # nothing a multiple of anything
        dict(name="act_grad_ragged", op="act_grad", M=1021, N=1003, x=F32, act="tanh", alpha=0.0),
        # the hidden layer of a feed-forward block, a batch of training
        dict(name="act_grad_gelu", op="act_grad", M=8192, N=16384, x=BF16, act="gelu", alpha=0.0),
        # a small ragged layer
        dict(name="linear_grad_ragged", op="linear_grad", M=333, N=1001, K=1503, x=F16, act="leaky_relu", alpha=0.25),
        # the largest product of this repository's workloads, trained
        dict(name="linear_grad_32768x4096x1024", op="linear_grad", M=32768, N=4096, K=1024, x=BF16, act="relu", alpha=0.0),
        # one token before a layer: latency alone
        dict(name="norm_one_token", op="norm", rows=1, N=4096, x=BF16, w=F32, stats=False),
        # a long prompt, or a batch of training
        dict(name="norm_prompt", op="norm", rows=32768, N=4096, x=BF16, w=F32, stats=True),
        # nothing a multiple of anything
        dict(name="norm_grad_ragged", op="norm_grad", rows=1021, N=1003, x=F32, w=F32),
        # a batch of training
        dict(name="norm_grad_batch", op="norm_grad", rows=32768, N=4096, x=BF16, w=F32),
    ]


def _log_int(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm; one in three is a multiple of 64 where it is that large."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v >= 64 and rng.random() < 1 / 3:
        v -= v % 64
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["round_trip", "linear", "linear", "act_grad", "linear_grad", "norm", "norm_grad"])
    x = rng.choice([BF16, BF16, F16, F32])
    if op in ("round_trip", "norm", "norm_grad", "act_grad"):
        while True:
            rows, n = _log_int(rng, 1, 32768), _log_int(rng, 1 if op == "round_trip" else 8, 16384)
            if rows * n <= 2 ** 27:
                break
        if op == "round_trip":
            return dict(op=op, rows=rows, K=n, x=x, f8=rng.choice([E4M3, E4M3, E5M2]), axis=rng.choice([1, 1, 0]), block_rows=rng.choice([1, 1, 128]))
        if op == "act_grad":
            act = rng.choice(["none", "relu", "leaky_relu", "tanh", "gelu", "sigmoid"])
            return dict(op=op, M=rows, N=n, x=x, act=act, alpha=0.01 if act == "leaky_relu" else 0.0)
        case = dict(op=op, rows=rows, N=n, x=x, w=rng.choice([F32, x]))
        if op == "norm":
            case["stats"] = rng.random() < 0.5
        return case
    x = rng.choice([BF16, BF16, F16])
    while True:
        M, N, K = _log_int(rng, 1, 32768), _log_int(rng, 64, 16384), _log_int(rng, 64, 16384)
        if M * N * K <= 4096 ** 3 // (1 if op == "linear" else 2) and M * N <= 2 ** 27 and M * K <= 2 ** 27:
            break
    if op == "linear_grad":
        act = rng.choice(["none", "relu", "leaky_relu"])
        return dict(op=op, M=M, N=N, K=K, x=x, act=act, alpha=0.25 if act == "leaky_relu" else 0.0)
    act = rng.choice(["none", "relu", "leaky_relu", "tanh", "gelu", "sigmoid"])
    return dict(op=op, M=M, N=N, K=K, x=x, y=rng.choice([x, x, F32]), bias=rng.choice([F32, x]), act=act,
                alpha=0.01 if act == "leaky_relu" else 0.0, residual=rng.random() < 0.3, pre=rng.random() < 0.3)


# ---- inputs ----------------------------------------------------------------------------------------------------------------

def _shapes(rows, K, block_rows=1):
    return (rows, 128 * (-(-K // 128))), (-(-rows // block_rows), 4 * (-(-K // 512)))


def _packed(rows, K, f8, block_rows=1):
    """Room for the codes and scales of `rows` rows of K values."""
    codes, scales = _shapes(rows, K, block_rows)
    return torch.empty(codes, dtype=getattr(torch, f8), device="cuda"), torch.empty(scales, dtype=torch.uint8, device="cuda")


def _activations(g, rows, K, dtype):
    """Normal values whose channels differ in size, a few of them by much; one row in sixteen of many is all zero (padding)."""
    size = torch.exp(0.6 * torch.randn(K, generator=g, device="cuda"))
    size = torch.where(torch.rand(K, generator=g, device="cuda") < 0.01, size * 20, size)
    x = torch.randn(rows, K, generator=g, device="cuda") * size
    if rows >= 64:
        x[torch.rand(rows, generator=g, device="cuda") < 1 / 16] = 0
    return x.to(dtype)


def _gradients(g, rows, n, dtype):
    """Gradients: rows of very different sizes, one in sixteen of many without any (a masked token)."""
    x = torch.randn(rows, n, generator=g, device="cuda") * torch.exp(torch.randn(rows, 1, generator=g, device="cuda") - 4)
    if rows >= 64:
        x[torch.rand(rows, generator=g, device="cuda") < 1 / 16] = 0
    return x.to(dtype)


def _stream(g, rows, n, dtype):
    """A residual stream: rows with an offset of their own, channels of different sizes."""
    size = torch.exp(0.6 * torch.randn(n, generator=g, device="cuda"))
    return (torch.randn(rows, n, generator=g, device="cuda") * size + 2 * torch.randn(rows, 1, generator=g, device="cuda")).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, dtype = case["op"], getattr(torch, case["x"])
    if op == "round_trip":
        rows, K = case["rows"], case["K"]
        x = _activations(g, rows, K, dtype)
        x = x.t().contiguous() if case["axis"] == 0 else x
        return dict(case=case, x=x, y=torch.empty_like(x), q=_packed(rows, K, case["f8"], case["block_rows"]))
    if op in ("norm", "norm_grad"):
        rows, n = case["rows"], case["N"]
        w = getattr(torch, case["w"])
        x = _stream(g, rows, n, dtype)
        gamma = (1 + 0.3 * torch.randn(n, generator=g, device="cuda")).to(w)
        state = dict(case=case, x=x, gamma=gamma)
        if op == "norm":
            state["beta"] = (0.3 * torch.randn(n, generator=g, device="cuda")).to(w)
            state["y"] = torch.empty_like(x)
            state["stats"] = [torch.empty(rows, device="cuda") for _ in range(2)] if case["stats"] else [None, None]
            return state
        mean = x.double().mean(1)
        state["mean"] = mean.float()
        state["rstd"] = (1 / torch.sqrt((x.double() - mean[:, None]).square().mean(1) + 1e-5)).float()
        state["dy"] = _gradients(g, rows, n, dtype)
        state["dx"] = torch.empty_like(x)
        state["dw"] = [torch.empty_like(gamma) for _ in range(2)]
        state["workspace"] = None
        if own:
            import conv_bias_activation_amd as ba

            state["workspace"] = torch.empty(ba.layer_norm_grad_workspace_size(rows, n), dtype=torch.uint8, device="cuda")
        return state
    if op == "act_grad":
        M, N = case["M"], case["N"]
        z = (1.5 * torch.randn(M, N, generator=g, device="cuda")).to(dtype)
        state = dict(case=case, dy=_gradients(g, M, N, dtype), z=z, dz=torch.empty_like(z))
        state["dbias"] = torch.empty(N, device="cuda")
        state["workspace"] = _act_grad_workspace(M, N)
        return state
    M, N, K = case["M"], case["N"], case["K"]
    x = _activations(g, M, K, dtype)
    w = torch.randn(N, K, generator=g, device="cuda") / math.sqrt(K)
    if op == "linear":
        bias = (0.5 * torch.randn(N, generator=g, device="cuda")).to(getattr(torch, case["bias"]))
        out = getattr(torch, case["y"])
        r = torch.randn(M, N, generator=g, device="cuda").to(out) if case["residual"] else None
        y = torch.empty(M, N, dtype=out, device="cuda")
        return dict(case=case, x=x, w=_quantize(w, E4M3, 128), bias=bias, r=r, y=y, z=torch.empty_like(y) if case["pre"] else None,
                    q=_packed(M, K, E4M3))
    z = torch.randn(M, N, generator=g, device="cuda").to(dtype)
    state = dict(case=case, x=x, w=w.to(dtype), z=z, dy=_gradients(g, M, N, dtype), dz=torch.empty_like(z))
    state["dbias"] = torch.empty(N, device="cuda")
    state["dx"], state["dw"] = torch.empty_like(x), torch.empty_like(state["w"])
    state["workspace"] = _act_grad_workspace(M, N)
    state["dz_rows"], state["w_cols"] = _packed(M, N, E5M2), _packed(K, N, E4M3, 128)
    state["dz_cols"], state["x_cols"] = _packed(N, M, E5M2), _packed(K, M, E4M3)
    return state


def _act_grad_workspace(M, N):
    if not own:
        return None
    import conv_bias_activation_amd as ba

    return torch.empty(ba.bias_act_grad_workspace_size(M, N), dtype=torch.uint8, device="cuda")


# ---- the plain form --------------------------------------------------------------------------------------------------------

_TOP = {E4M3: 8, E5M2: 15}  # the largest value is 1.75 times 2 to this


def _pow2(e):
    """2 to the whole number e in fp32, from its bits (exp2 and ldexp need not be exact on a GPU)."""
    return ((e.long() + 1023) << 52).view(torch.float64).float()


def _blocks(x, block_rows):
    """Rows of x padded to [row blocks, rows of a block, k blocks, 128]."""
    rows, K = x.shape
    x = torch.nn.functional.pad(x, (0, -K % 128, 0, -rows % block_rows))
    return x.view(x.shape[0] // block_rows, block_rows, -1, 128)


def _quantize(x, f8, block_rows=1):
    """Rows of x -> codes, scales."""
    rows = x.shape[0]
    v = _blocks(x.float(), block_rows)
    top = v.abs().amax((1, 3))
    m, e = torch.frexp(top)  # top = m * 2^e, m from 1/2 to 1
    e = (e - 1 - _TOP[f8] + (m > 0.875).int()).clamp(-127, 127)
    e = torch.where(top == 0, -127, e)
    codes = (v * _pow2(-e[:, None, :, None])).to(getattr(torch, f8)).view(v.shape[0] * block_rows, -1)[:rows]
    scales = (e + 127).to(torch.uint8)
    return codes.contiguous(), torch.nn.functional.pad(scales, (0, -scales.shape[1] % 4)).contiguous()


def _dequantize(codes, scales, K):
    """Codes, scales -> fp32 values [rows, K]."""
    rows, blocks = codes.shape[0], codes.shape[1] // 128
    e = scales[:, :blocks].int() - 127
    if scales.shape[0] != rows:
        e = e.repeat_interleave(128, 0)[:rows]
    return (codes.float().view(rows, blocks, 128) * _pow2(e.unsqueeze(-1))).view(rows, -1)[:, :K]


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


def _act_slope(z, case):
    a = case["act"]
    if a == "relu":
        return (z > 0).float()
    if a == "leaky_relu":
        return torch.where(z >= 0, 1.0, case["alpha"])
    if a == "tanh":
        u = torch.exp(-2 * z.abs())
        return 4 * u / (1 + u).square()
    if a == "gelu":
        return 0.5 * torch.special.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if a == "sigmoid":
        u = torch.exp(-z.abs())
        return u / (1 + u).square()
    return torch.ones_like(z)


def _own(state):
    import conv_bias_activation_amd as ba

    case, op = state["case"], state["case"]["op"]
    if op == "round_trip":
        ba.fp8_quantize(state["x"], *state["q"], axis=case["axis"])
        return ba.fp8_dequantize(*state["q"], state["y"], axis=case["axis"])
    if op == "linear":
        q = ba.fp8_quantize(state["x"], *state["q"])
        if state["r"] is None:
            y = ba.gemm_fp8_bias_act(*q, *state["w"], state["bias"], state["y"], case["act"], case["alpha"], Z=state["z"])
        else:
            y = ba.gemm_fp8_bias_add_act(*q, *state["w"], state["bias"], state["r"], state["y"], case["act"], case["alpha"], Z=state["z"])
        return (y, state["z"]) if case["pre"] else y
    if op == "norm":
        mean, rstd = state["stats"]
        y = ba.layer_norm(state["x"], state["gamma"], state["beta"], state["y"], mean, rstd)
        return (y, mean, rstd) if case["stats"] else y
    if op == "norm_grad":
        return ba.layer_norm_grad(state["dy"], state["x"], state["gamma"], state["mean"], state["rstd"], state["dx"], *state["dw"],
                                  workspace=state["workspace"])
    dz, dbias = ba.bias_act_grad(state["dy"], state["z"], state["dz"], state["dbias"], case["act"], case["alpha"], workspace=state["workspace"])
    if op == "act_grad":
        return dz, dbias
    d = ba.fp8_quantize(dz, *state["dz_rows"])
    wt = ba.fp8_quantize(state["w"], *state["w_cols"], axis=0)
    dx = ba.gemm_fp8_bias_act(*d, *wt, None, state["dx"])
    dt = ba.fp8_quantize(dz, *state["dz_cols"], axis=0)
    xt = ba.fp8_quantize(state["x"], *state["x_cols"], axis=0)
    dw = ba.gemm_fp8_bias_act(*dt, *xt, None, state["dw"])
    return dx, dw, dbias


def run(state):
    if own:
        return _own(state)
    case, op = state["case"], state["case"]["op"]
    if op == "round_trip":
        x = state["x"].t() if case["axis"] == 0 else state["x"]
        v = _dequantize(*_quantize(x, case["f8"], case["block_rows"]), case["K"]).to(x.dtype)
        return v.t().contiguous() if case["axis"] == 0 else v
    if op == "linear":
        a = _dequantize(*_quantize(state["x"], E4M3), case["K"])
        z = torch.matmul(a, _dequantize(*state["w"], case["K"]).t()) + state["bias"].float()
        if state["r"] is not None:
            z = z + state["r"].float()
        y = _act(z, case).to(state["y"].dtype)
        return (y, z.to(y.dtype)) if case["pre"] else y
    if op == "norm":
        x = state["x"].float()
        mean = x.mean(1, keepdim=True)
        d = x - mean
        rstd = 1 / torch.sqrt(d.square().mean(1, keepdim=True) + 1e-5)
        y = (d * rstd * state["gamma"].float() + state["beta"].float()).to(state["x"].dtype)
        return (y, mean.view(-1), rstd.view(-1)) if case["stats"] else y
    if op == "norm_grad":
        dy, rstd = state["dy"].float(), state["rstd"][:, None]
        xh = (state["x"].float() - state["mean"][:, None]) * rstd
        gr = dy * state["gamma"].float()
        dx = rstd * (gr - gr.mean(1, keepdim=True) - xh * (gr * xh).mean(1, keepdim=True))
        return dx.to(state["x"].dtype), (dy * xh).sum(0).to(state["gamma"].dtype), dy.sum(0).to(state["gamma"].dtype)
    d = state["dy"].float() * _act_slope(state["z"].float(), case)
    dz, dbias = d.to(state["dy"].dtype), d.sum(0)
    if op == "act_grad":
        return dz, dbias
    M, N = case["M"], case["N"]
    d = _dequantize(*_quantize(dz, E5M2), N)
    w = _dequantize(*_quantize(state["w"].t(), E4M3, 128), N)
    dx = torch.matmul(d, w.t()).to(state["x"].dtype)
    d = _dequantize(*_quantize(dz.t(), E5M2), M)
    x = _dequantize(*_quantize(state["x"].t(), E4M3), M)
    return dx, torch.matmul(d, x.t()).to(state["w"].dtype), dbias


# ---- what a pass cannot do without -----------------------------------------------------------------------------------------

_SIZE = {BF16: 2, F16: 2, F32: 4}


def work(case):
    op, s = case["op"], _SIZE[case["x"]]
    if op == "round_trip":
        n, blocks = case["rows"] * case["K"], case["rows"] * case["K"] / (128 * case["block_rows"])
        # X read, codes and scales written, read again, Y written
        return {"bytes": 2 * n * s + 2 * (n + blocks), "flops": 2 * n}
    if op == "norm":
        n = case["rows"] * case["N"]
        return {"bytes": 2 * n * s + 2 * case["N"] * _SIZE[case["w"]] + (8 * case["rows"] if case["stats"] else 0), "flops": 8 * n}
    if op == "norm_grad":
        n = case["rows"] * case["N"]
        return {"bytes": 3 * n * s + 3 * case["N"] * _SIZE[case["w"]] + 8 * case["rows"], "flops": 14 * n}
    if op == "act_grad":
        n = case["M"] * case["N"]
        return {"bytes": 3 * n * s + 4 * case["N"], "flops": 4 * n}
    M, N, K = case["M"], case["N"], case["K"]
    if op == "linear":
        outs = 1 + case["residual"] + case["pre"]
        w = M * K * s + N * K * (1 + 1 / 128 ** 2) + N * _SIZE[case["bias"]] + M * N * _SIZE[case["y"]] * outs
        return {"bytes": w, "flops": 2 * M * N * K}
    # dY, Z, X and W read, dX, dW and the bias's gradient written
    return {"bytes": s * (2 * M * N + 2 * M * K + 2 * N * K) + 4 * N, "flops": 4 * M * N * K}


# ---- from the definition, in 64 bits ---------------------------------------------------------------------------------------

_FORMAT = {E4M3: (3, -6, 448.0), E5M2: (2, -14, 57344.0)}  # mantissa bits, exponent of the smallest normal value, largest value


def _two_to(e):
    return torch.tensor([2.0 ** i for i in range(-400, 400)], dtype=torch.float64, device=e.device)[e.long() + 400]


def _nearest(x, f8, block_rows=1):
    """x (rows, blocks along them) with each value rounded to the nearest one of its block, in 64 bits."""
    bits, low, top = _FORMAT[f8]
    rows, K = x.shape
    v = torch.zeros(-(-rows // block_rows) * block_rows, -(-K // 128) * 128, dtype=torch.float64, device=x.device)
    v[:rows, :K] = x.double()
    v = v.view(-1, block_rows, v.shape[1] // 128, 128)
    most = v.abs().amax((1, 3), keepdim=True)
    # the smallest power of two that brings the largest value within the format's range; the logarithm is only a first guess
    e = torch.ceil(torch.log2(most.clamp_min(1e-60) / top)) + 1
    for _ in range(2):
        e = torch.where(most <= top * _two_to(e - 1), e - 1, e)
    scale = _two_to(e.clamp(-127, 127))
    t = v / scale
    _, ex = torch.frexp(t.abs())
    step = _two_to((ex - 1).clamp_min(low) - bits)
    return (torch.round(t / step) * step * scale).view(v.shape[0] * block_rows, -1)[:rows, :K]


def _value(codes, scales, K, block_rows):
    """What codes and scales stand for, from their bits."""
    b = codes.view(torch.uint8).long()
    bits, low, _ = _FORMAT[E4M3 if codes.dtype == torch.float8_e4m3fn else E5M2]
    ex, man = (b & 127) >> bits, (b & ((1 << bits) - 1)).double() / (1 << bits)
    mag = torch.where(ex == 0, man * 2.0 ** low, (1 + man) * _two_to(ex - 1 + low))
    s = _two_to(scales.long() - 127).repeat_interleave(128, 1).repeat_interleave(block_rows, 0)
    return ((1 - 2 * (b >> 7)) * mag * s[:b.shape[0], :b.shape[1]])[:, :K]


def _exact_act(z, case):
    act = case["act"]
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "leaky_relu":
        return torch.maximum(z, z * case["alpha"])
    if act == "tanh":
        return torch.tanh(z)
    if act == "gelu":
        return z * torch.special.erfc(-z / math.sqrt(2)) / 2
    if act == "sigmoid":
        return torch.sigmoid(z)
    return z


def _exact_slope(z, case):
    act = case["act"]
    if act == "relu":
        return torch.where(z > 0, 1.0, 0.0).double()
    if act == "leaky_relu":
        return torch.where(z < 0, case["alpha"], 1.0).double()
    if act == "tanh":
        return 1 / torch.cosh(z).square()
    if act == "gelu":
        return torch.special.erfc(-z / math.sqrt(2)) / 2 + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "sigmoid":
        return torch.sigmoid(z) * torch.sigmoid(-z)
    return torch.ones_like(z)


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "round_trip":
        x = state["x"]
        if case["axis"] == 0:
            return _nearest(x.t(), case["f8"], case["block_rows"]).t().contiguous()
        return _nearest(x, case["f8"], case["block_rows"])
    if op == "linear":
        z = _nearest(state["x"], E4M3) @ _value(*state["w"], case["K"], 128).t().contiguous() + state["bias"].double()
        if state["r"] is not None:
            z = z + state["r"].double()
        y = _exact_act(z, case)
        return (y, z) if case["pre"] else y
    if op == "norm":
        x = state["x"].double()
        n = x.shape[1]
        mean = x.sum(1) / n
        var = (x - mean[:, None]).pow(2).sum(1) / n
        rstd = (var + 1e-5).pow(-0.5)
        y = (x - mean[:, None]) * rstd[:, None] * state["gamma"].double() + state["beta"].double()
        return (y, mean, rstd) if case["stats"] else y
    if op == "norm_grad":
        dy, rstd, n = state["dy"].double(), state["rstd"].double()[:, None], case["N"]
        xh = (state["x"].double() - state["mean"].double()[:, None]) * rstd
        gr = dy * state["gamma"].double()
        a, b = gr.sum(1, keepdim=True) / n, (gr * xh).sum(1, keepdim=True) / n
        return (gr - a - xh * b) * rstd, (dy * xh).sum(0), dy.sum(0)
    dz = state["dy"].double() * _exact_slope(state["z"].double(), case)
    dbias = dz.sum(0)
    if op == "act_grad":
        return dz, dbias
    dz = dz.to(state["dz"].dtype)  # as it is stored
    dx = _nearest(dz, E5M2) @ _nearest(state["w"].t(), E4M3, 128).t().contiguous()
    dw = _nearest(dz.t(), E5M2) @ _nearest(state["x"].t(), E4M3).t().contiguous()
    return dx, dw, dbias
