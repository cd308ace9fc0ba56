"""Refusals of the 8-bit floating-point, layer norm and gradient calls: of the
C ABI by status (no call reaches the GPU: every check comes before), and of the
binding by message."""
import ctypes

import numpy as np
import pytest

import fp8_ref as f8

ba = pytest.importorskip("conv_bias_activation_amd")
torch = pytest.importorskip("torch")
L = ba.lib
P = 0x10000000          # an aligned address that nothing reads
OK, INVALID, UNSUPPORTED = 0, 1, 2
F32, F16, BF16, I8, I32, MX, E4, E5 = range(8)


def dts(a, b=0, c=0, d=0):
    return a | b << 8 | c << 16 | d << 24


# ---- sizes ----------------------------------------------------------------------------

@pytest.mark.parametrize("rows,K,block", [(0, 0, 1), (0, 9, 1), (9, 0, 128), (1, 1, 1), (1, 1, 128), (128, 512, 128), (129, 513, 128),
                                          (1000, 1003, 1), (4096, 4096, 128)])
def test_packed_size(rows, K, block):
    c, s = ctypes.c_size_t(7), ctypes.c_size_t(7)
    assert L.fp8_packed_size(rows, K, block, c, s) == OK
    want = f8.shapes(rows, K, block)
    assert (c.value, s.value) == (want[0][0] * want[0][1], want[1][0] * want[1][1])
    assert ba.fp8_shapes(rows, K, block) == want


@pytest.mark.parametrize("args,status", [((-1, 1, 1), INVALID), ((1, -1, 1), INVALID), ((1, 1, 2), INVALID), ((1, 1, 0), INVALID),
                                         ((2 ** 31, 1, 1), UNSUPPORTED), ((1, 2 ** 31, 1), UNSUPPORTED), ((2 ** 24, 1, 1), UNSUPPORTED),
                                         ((2 ** 24 - 1, 128, 1), OK)])
def test_packed_size_refusals(args, status):
    c, s = ctypes.c_size_t(7), ctypes.c_size_t(7)
    assert L.fp8_packed_size(*args, c, s) == status
    assert status == OK or (c.value, s.value) == (7, 7)
    assert L.fp8_packed_size(1, 1, 1, None, s) == INVALID and L.fp8_packed_size(1, 1, 1, c, None) == INVALID


def test_shapes_refuse_other_blocks():
    with pytest.raises(ValueError, match="block_rows must be 1 or 128"):
        ba.fp8_shapes(4, 4, 64)


# ---- quantisation --------------------------------------------------------------------------

QUANT = dict(X=P, codes=P, scales=P, rows=4, K=200, axis=1, block=1, dt=dts(BF16, E4))
QUANT_BAD = [(dict(rows=-1), INVALID), (dict(K=-1), INVALID), (dict(axis=2), INVALID), (dict(axis=-1), INVALID), (dict(block=64), INVALID),
             (dict(X=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(X=P + 1), INVALID),
             (dict(X=P + 2, dt=dts(F32, E4)), INVALID), (dict(codes=P + 8), INVALID), (dict(scales=P + 2), INVALID),
             (dict(dt=dts(I8, E4)), UNSUPPORTED), (dict(dt=dts(BF16, MX)), UNSUPPORTED), (dict(dt=dts(BF16, BF16)), UNSUPPORTED),
             (dict(dt=dts(BF16, E4, 1)), UNSUPPORTED), (dict(dt=dts(BF16, E4, 0, 1)), UNSUPPORTED), (dict(dt=dts(E4, E4)), UNSUPPORTED),
             (dict(rows=2 ** 31), UNSUPPORTED), (dict(K=2 ** 31), UNSUPPORTED), (dict(rows=2 ** 24, K=1), UNSUPPORTED),
             (dict(rows=2 ** 15, K=2 ** 15), UNSUPPORTED), (dict(rows=2 ** 15, K=2 ** 14, dt=dts(F32, E4)), UNSUPPORTED)]


@pytest.mark.parametrize("f", ["fp8_quantize", "fp8_dequantize"])
@pytest.mark.parametrize("bad,status", QUANT_BAD)
def test_quantise_status(f, bad, status):
    a = {**QUANT, **bad}
    p = (a["X"], a["codes"], a["scales"]) if f == "fp8_quantize" else (a["codes"], a["scales"], a["X"])
    assert getattr(L, f)(*p, a["rows"], a["K"], a["axis"], a["block"], a["dt"], None) == status


def test_quantise_nothing():
    for rows, K in ((0, 5), (5, 0), (0, 0)):
        assert L.fp8_quantize(None, None, None, rows, K, 1, 1, dts(F32, E5), None) == OK
        assert L.fp8_dequantize(None, None, None, rows, K, 0, 128, dts(F32, E5), None) == OK


# ---- products ----------------------------------------------------------------------------------

GEMM = dict(A=P, As=P, ab=1, B=P, Bs=P, bb=128, bias=P, R=P, Z=P + 4096, C=P + 8192, M=4, N=6, K=200, dt=dts(E4, E5, F32, BF16), act=4)
GEMM_BAD = [(dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-1), INVALID), (dict(act=6), INVALID), (dict(act=-1), INVALID),
            (dict(ab=2), INVALID), (dict(bb=0), INVALID), (dict(A=None), INVALID), (dict(As=None), INVALID), (dict(B=None), INVALID),
            (dict(Bs=None), INVALID), (dict(C=None), INVALID), (dict(A=P + 8), INVALID), (dict(Bs=P + 1), INVALID), (dict(C=P + 1), INVALID),
            (dict(R=P + 1), INVALID), (dict(Z=P + 1), INVALID), (dict(bias=P + 2), INVALID), (dict(Z=P + 8192), INVALID), (dict(Z=P), INVALID),
            (dict(dt=dts(MX, E4, F32, BF16)), UNSUPPORTED), (dict(dt=dts(E4, BF16, F32, BF16)), UNSUPPORTED),
            (dict(dt=dts(E4, E4, I32, BF16)), UNSUPPORTED), (dict(dt=dts(E4, E4, F32, I32)), UNSUPPORTED), (dict(dt=dts(E4, E4, F32, E4)), UNSUPPORTED),
            (dict(M=2 ** 31), UNSUPPORTED), (dict(N=2 ** 31), UNSUPPORTED), (dict(K=2 ** 31), UNSUPPORTED),
            (dict(M=2 ** 15, N=2 ** 15), UNSUPPORTED), (dict(M=2 ** 16, K=2 ** 15), UNSUPPORTED), (dict(N=2 ** 16, K=2 ** 15), UNSUPPORTED),
            (dict(M=1, N=2 ** 29, K=0), UNSUPPORTED)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("bad,status", GEMM_BAD)
def test_product_status(bad, status, residual):
    a = {**GEMM, **bad}
    if not residual and "R" in bad or not residual and bad == dict(Z=P):
        return
    common = (a["A"], a["As"], a["ab"], a["B"], a["Bs"], a["bb"], a["bias"])
    tail = (a["Z"], a["C"], a["M"], a["N"], a["K"], a["dt"], a["act"], 0.0, None)
    if residual:
        assert L.gemm_fp8_bias_add_act(*common, a["R"], *tail) == status
    else:
        assert L.gemm_fp8_bias_act(*common, *tail) == status


def test_product_nothing_and_missing_residual():
    d = dts(E4, E4, F32, F32)
    for M, N in ((0, 5), (5, 0)):
        assert L.gemm_fp8_bias_act(None, None, 1, None, None, 1, None, None, None, M, N, 7, d, 0, 0.0, None) == OK
        assert L.gemm_fp8_bias_add_act(None, None, 1, None, None, 1, None, None, None, None, M, N, 7, d, 0, 0.0, None) == OK
    assert L.gemm_fp8_bias_add_act(P, P, 1, P, P, 1, None, None, None, P, 2, 2, 7, d, 0, 0.0, None) == INVALID


# ---- layer norm and gradients -----------------------------------------------------------------------

NORM = dict(X=P, ga=P, be=P, Y=P + 4096, mean=P, rstd=P, rows=4, N=200, eps=1e-5, dt=dts(BF16, F32, 0, F16))
NORM_BAD = [(dict(rows=-1), INVALID), (dict(N=-1), INVALID), (dict(eps=-1e-9), INVALID), (dict(eps=float("nan")), INVALID),
            (dict(eps=float("inf")), INVALID), (dict(X=None), INVALID), (dict(Y=None), INVALID), (dict(mean=None), INVALID),
            (dict(rstd=None), INVALID), (dict(X=P + 1), INVALID), (dict(Y=P + 1), INVALID), (dict(ga=P + 2), INVALID), (dict(be=P + 1), INVALID),
            (dict(mean=P + 2), INVALID), (dict(rstd=P + 2), INVALID), (dict(Y=P), INVALID), (dict(dt=dts(I8, F32, 0, F16)), UNSUPPORTED),
            (dict(dt=dts(F16, I32, 0, F16)), UNSUPPORTED), (dict(dt=dts(F16, F32, 0, E4)), UNSUPPORTED), (dict(dt=dts(F16, F32, 1, F16)), UNSUPPORTED),
            (dict(rows=2 ** 31), UNSUPPORTED), (dict(N=2 ** 31), UNSUPPORTED), (dict(rows=2 ** 15, N=2 ** 15), UNSUPPORTED),
            (dict(rows=1, N=2 ** 29), UNSUPPORTED), (dict(rows=2 ** 29, N=1), UNSUPPORTED), (dict(rows=2 ** 15, N=2 ** 14, dt=dts(F16, F32, 0, F32)), UNSUPPORTED)]


@pytest.mark.parametrize("bad,status", NORM_BAD)
def test_norm_status(bad, status):
    a = {**NORM, **bad}
    assert L.layer_norm(a["X"], a["ga"], a["be"], a["Y"], a["mean"], a["rstd"], a["rows"], a["N"], a["eps"], a["dt"], None) == status


NG = dict(dY=P + 4096, X=P + 8192, ga=P, mean=P, rstd=P, dX=P + 16384, dg=P, db=P, rows=4, N=200, dt=dts(BF16, F32, 0, F16), ws=P, n=1 << 20)
NG_BAD = [(dict(rows=-1), INVALID), (dict(N=-1), INVALID), (dict(dY=None), INVALID), (dict(X=None), INVALID), (dict(dX=None), INVALID),
          (dict(mean=None), INVALID), (dict(rstd=None), INVALID), (dict(ws=None), INVALID), (dict(ws=P + 8), INVALID), (dict(n=4 * 2 * 200 - 1), INVALID),
          (dict(n=0, dg=None), INVALID), (dict(dY=P + 1), INVALID), (dict(X=P + 1), INVALID), (dict(dX=P + 1), INVALID), (dict(ga=P + 1), INVALID),
          (dict(dg=P + 1), INVALID), (dict(db=P + 2), INVALID), (dict(mean=P + 1), INVALID), (dict(dX=P + 4096), INVALID),
          (dict(dX=P + 8192, N=40000), INVALID), (dict(dX=P + 4096, N=40000, dt=dts(F16, F32, 0, F16)), INVALID),
          (dict(dt=dts(E4, F32, 0, F16)), UNSUPPORTED), (dict(rows=2 ** 16, N=2 ** 15), UNSUPPORTED)]


@pytest.mark.parametrize("bad,status", NG_BAD)
def test_norm_grad_status(bad, status):
    a = {**NG, **bad}
    assert L.layer_norm_grad(a["dY"], a["X"], a["ga"], a["mean"], a["rstd"], a["dX"], a["dg"], a["db"], a["rows"], a["N"], a["dt"], a["ws"],
                             a["n"], None) == status


AG = dict(dY=P, Z=P + 4096, dZ=P + 8192, db=P, M=4, N=200, dt=dts(BF16, 0, F32), act=4, ws=P, n=1 << 20)
AG_BAD = [(dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(act=6), INVALID), (dict(act=-1), INVALID), (dict(dY=None), INVALID),
          (dict(Z=None), INVALID), (dict(dZ=None, db=None), INVALID), (dict(ws=None), INVALID), (dict(ws=P + 4), INVALID), (dict(n=4 * 200 - 1), INVALID),
          (dict(dY=P + 1), INVALID), (dict(Z=P + 1), INVALID), (dict(dZ=P + 1), INVALID), (dict(db=P + 2), INVALID),
          (dict(dt=dts(I8, 0, F32)), UNSUPPORTED), (dict(dt=dts(BF16, 0, I32)), UNSUPPORTED), (dict(dt=dts(BF16, 1, F32)), UNSUPPORTED),
          (dict(dt=dts(BF16, 0, F32, 1)), UNSUPPORTED), (dict(M=2 ** 15, N=2 ** 15), UNSUPPORTED),
          (dict(M=1, N=2 ** 29), UNSUPPORTED)]


@pytest.mark.parametrize("bad,status", AG_BAD)
def test_act_grad_status(bad, status):
    a = {**AG, **bad}
    assert L.bias_act_grad(a["dY"], a["Z"], a["dZ"], a["db"], a["M"], a["N"], a["dt"], a["act"], 0.0, a["ws"], a["n"], None) == status


def test_nothing_to_do():
    assert L.layer_norm(None, None, None, None, None, None, 0, 5, 0.0, dts(F32), None) == OK
    assert L.layer_norm(None, None, None, None, None, None, 5, 0, 0.0, dts(F32), None) == OK
    assert L.layer_norm_grad(None, None, None, None, None, None, None, None, 5, 0, dts(F32), None, 0, None) == OK
    assert L.bias_act_grad(None, None, None, None, 5, 0, dts(F32), 0, 0.0, None, 0, None) == OK
    for f in (ba.layer_norm_grad_workspace_size, ba.bias_act_grad_workspace_size):
        assert f(0, 5) == f(5, 0) == f(-1, 5) == 0 and f(1, 1) > 0 and f(2 ** 20, 512) <= 2 ** 26


# ---- the binding's own messages -----------------------------------------------------------------------

def e4(*shape):
    return torch.zeros(shape, dtype=torch.uint8).view(torch.float8_e4m3fn)


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def z(*shape, dt=torch.float32):
    return torch.zeros(shape, dtype=dt)


PACK, TYPES, DEVICE = r"codes must be \[rows, 128 b\]", "codes must be float8", "must be a device tensor"
# X [300, 200]: codes [300, 256], scales [300, 4] or [3, 4]
QUANT_MSG = {
    "X of one dimension": (dict(X=z(60000)), "must be 2-D"), "no such axis": (dict(axis=2), "axis must be 0 or 1"),
    "the other axis": (dict(axis=0), "codes and scales must be"), "X of more rows": (dict(X=z(301, 200)), "codes and scales must be"),
    "X longer": (dict(X=z(300, 257)), "codes and scales must be"), "codes uint8": (dict(codes=u8(300, 256)), TYPES),
    "codes fp16": (dict(codes=z(300, 256, dt=torch.float16)), TYPES), "scales int8": (dict(scales=z(300, 4, dt=torch.int8)), TYPES),
    "codes no whole blocks": (dict(codes=e4(300, 200)), PACK), "scales too narrow": (dict(scales=u8(300, 2)), PACK),
    "scales too wide": (dict(scales=u8(300, 8)), PACK), "scales of other rows": (dict(scales=u8(299, 4)), PACK),
    "scales of two row blocks": (dict(scales=u8(2, 4)), PACK), "codes of one dimension": (dict(codes=e4(76800)), PACK),
    "X fp64": (dict(X=z(300, 200, dt=torch.float64)), "unsupported tensor dtype"), "on the host": ({}, DEVICE),
    "on the host, blocks of 128 rows": (dict(scales=u8(3, 4)), DEVICE),
}


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("what", list(QUANT_MSG))
def test_quantise_message(what, back):
    a = {**dict(X=z(300, 200), codes=e4(300, 256), scales=u8(300, 4), axis=1), **QUANT_MSG[what][0]}
    with pytest.raises(ValueError, match=QUANT_MSG[what][1]):
        if back:
            ba.fp8_dequantize(a["codes"], a["scales"], a["X"], axis=a["axis"])
        else:
            ba.fp8_quantize(**a)


GEMM_MSG = {
    "B shorter": (dict(B=e4(6, 128)), "shape mismatch"), "B's codes uint8": (dict(B=u8(6, 256)), TYPES), "A's scales of other rows": (dict(a_scales=u8(3, 4)), PACK),
    "B's scales wider": (dict(b_scales=u8(6, 8)), PACK), "C of other rows": (dict(C=z(3, 6)), "shape mismatch"), "C flat": (dict(C=z(24)), "shape mismatch"),
    "C fp64": (dict(C=z(4, 6, dt=torch.float64)), "unsupported tensor dtype"), "a short bias": (dict(bias=z(5)), "bias must have N = 6"),
    "Z of another type": (dict(Z=z(4, 6, dt=torch.float16)), "Z must match C"), "Z of another shape": (dict(Z=z(6, 4)), "Z must match C"),
    "no such activation": (dict(act="swish"), "unknown activation|must be a device tensor"), "on the host": ({}, DEVICE),
}


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("what", list(GEMM_MSG))
def test_product_message(what, residual):
    a = {**dict(A=e4(4, 256), a_scales=u8(4, 4), B=e4(6, 256), b_scales=u8(6, 4), bias=z(6), C=z(4, 6), act="relu"), **GEMM_MSG[what][0]}
    with pytest.raises(ValueError, match=GEMM_MSG[what][1]):
        if residual:
            ba.gemm_fp8_bias_add_act(R=torch.zeros_like(a["C"]), **a)
        else:
            ba.gemm_fp8_bias_act(**a)


def test_residual_message():
    a = dict(A=e4(4, 256), a_scales=u8(4, 4), B=e4(6, 256), b_scales=u8(6, 4), bias=None, C=z(4, 6))
    for R in (None, z(6, 4), z(4, 6, dt=torch.float16)):
        with pytest.raises(ValueError, match="residual, shaped and typed|R must match"):
            ba.gemm_fp8_bias_add_act(R=R, **a)


NORM_MSG = {
    "X of three": (dict(X=z(4, 2, 5)), "X must be 2-D"), "X int8": (dict(X=z(4, 10, dt=torch.float64)), "unsupported tensor dtype"),
    "weights of two types": (dict(beta=z(10, dt=torch.float16)), "beta must be torch.float32"), "Y of another shape": (dict(Y=z(10, 4)), "device tensor|Y must match"),
    "on the host": ({}, DEVICE),
}


@pytest.mark.parametrize("what", list(NORM_MSG))
def test_norm_message(what):
    a = {**dict(X=z(4, 10), gamma=z(10), beta=z(10), Y=z(4, 10)), **NORM_MSG[what][0]}
    with pytest.raises(ValueError, match=NORM_MSG[what][1]):
        ba.layer_norm(**a)


def test_shape_and_type_messages():
    v, n = ba._binding._vector, ba._binding._like
    with pytest.raises(ValueError, match="gamma must have 9 elements"):
        v(z(10), 9, "gamma")
    with pytest.raises(ValueError, match="mean must be torch.float32"):
        v(z(9, dt=torch.float16), 9, "mean", torch.float32)
    with pytest.raises(ValueError, match="dX must match X"):
        n(z(4, 9), z(4, 10), "dX", "X")
    with pytest.raises(ValueError, match="dX must match X"):
        n(z(4, 10, dt=torch.float16), z(4, 10), "dX", "X")
    with pytest.raises(ValueError, match="mean and rstd of the forward pass"):
        ba.layer_norm_grad(z(4, 10), z(4, 10), None, None, z(4), z(4, 10))
    with pytest.raises(ValueError, match="workspace .* is required"):
        ba.layer_norm_grad(z(4, 10), z(4, 10), None, z(4), z(4), z(4, 10), z(10))
    with pytest.raises(ValueError, match="dgamma must be torch.float32"):
        ba.layer_norm_grad(z(4, 10), z(4, 10), z(10), z(4), z(4), z(4, 10), z(10, dt=torch.float16))
    with pytest.raises(ValueError, match="workspace .* is required"):
        ba.bias_act_grad(z(4, 10), z(4, 10), z(4, 10), z(10))
    with pytest.raises(ValueError, match="dY must be 2-D"):
        ba.bias_act_grad(z(40), None, z(40))


# ---- a call that the library refuses is made once ----------------------------------------------------------

class Refuses:
    calls = 0

    def f8_quantize(self, *a):
        self.calls += 1
        return self.status

    f8_dequantize = f8_gemm = act_grad = norm = norm_grad = f8_quantize


@pytest.mark.parametrize("status,error", [(3, ba.BiasActError), (1, ValueError), (2, ValueError)])
@pytest.mark.parametrize("name,nargs", [("fp8_quantize", 3), ("fp8_dequantize", 3), ("gemm_fp8_bias_act", 6), ("gemm_fp8_bias_add_act", 7),
                                        ("bias_act_grad", 3), ("layer_norm", 4), ("layer_norm_grad", 6)])
def test_a_failed_call_is_not_made_again(monkeypatch, name, nargs, status, error):
    n = Refuses()
    n.status = status
    monkeypatch.setattr(ba._binding, "_native", n)
    with pytest.raises(error, match=name + ": "):
        getattr(ba, name)(*[object()] * nargs)
    assert n.calls == 1


# ---- the format's definition against torch's conversions -----------------------------------------------------

@pytest.mark.parametrize("fmt,t", [("f8e4m3", torch.float8_e4m3fn), ("f8e5m2", torch.float8_e5m2)])
def test_the_reference_has_the_formats_values_and_rounding(fmt, t):
    assert np.array_equal(torch.arange(256, dtype=torch.uint8).view(t).double().numpy(), f8.table(fmt), equal_nan=True)
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((130, 300)) * np.exp2(rng.integers(-20, 20, (130, 1)))).astype(np.float32)
    for block in (1, 128):
        c, s = f8.quantize(x.astype(np.float64), fmt, block)
        e = np.repeat(np.repeat(s[:, :3].astype(np.int64) - 127, 128, 1), block, 0)[:130]
        v = np.pad(x, ((0, 0), (0, 84))) * np.exp2(-e.astype(np.float64))
        assert np.array_equal(torch.from_numpy(v).float().to(t).view(torch.uint8).numpy(), c)
        big = np.abs(v.reshape(-1, 128) if block == 1 else np.pad(v, ((0, 126), (0, 0))).reshape(2, 128, 3, 128).transpose(0, 2, 1, 3).reshape(6, -1)).max(1)
        assert (big <= f8.FMT[fmt][2]).all() and (big > f8.FMT[fmt][2] / 2).all()
