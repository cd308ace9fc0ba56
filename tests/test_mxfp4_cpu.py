"""MXFP4 checks that need no GPU: the numpy form of the format against its
closed forms, and every refusal of the entry points and of the binding."""
import ctypes

import numpy as np
import pytest

import mxfp4_ref as mx

ba = pytest.importorskip("conv_bias_activation_amd")
torch = pytest.importorskip("torch")
L = ba.lib

F32, F16, BF16, I8, MX = 0, 1, 2, 3, 5
P = ctypes.c_void_p(0x1000)          # never dereferenced: every call fails its checks
ODD16 = ctypes.c_void_p(0x1008)      # 8-byte aligned only
ODD4 = ctypes.c_void_p(0x1002)
ODD2 = ctypes.c_void_p(0x1001)
NUL = ctypes.c_void_p(0)


def _dt(a, b, bias, out):
    return a | (b << 8) | (bias << 16) | (out << 24)


# ---- the format -----------------------------------------------------------------

def test_values_of_every_code():
    codes = np.arange(256, dtype=np.uint8).reshape(4, 64)
    v = mx.values(codes, np.full((4, 4), 128, np.uint8), 128).ravel()       # scale 2
    assert list(v[0:2]) == [0.0, 0.0] and v[2 * 0x7F] == -12.0 and v[2 * 0x7F + 1] == 12.0
    assert v[2 * 0x21] == 1.0 and v[2 * 0x21 + 1] == 2.0                    # low four bits first


@pytest.mark.parametrize("x,want", [
    (0.25, 0.0), (0.75, 1.0), (1.25, 1.0), (1.75, 2.0), (2.5, 2.0), (3.5, 4.0), (5.0, 4.0),   # ties to even codes
    (0.2500001, 0.5), (0.7499999, 0.5), (5.0001, 6.0), (6.0, 6.0), (7.99, 6.0), (-5.0, -4.0)])
def test_rounding_rule(x, want):
    row = np.zeros((1, 32))
    row[0, 0] = x
    row[0, 1] = 4.0                                     # block maximum in [4, 8): scale 1
    codes, scales = mx.quantize(row)
    assert scales[0, 0] == 127
    assert mx.values(codes, scales, 32)[0, 0] == want


def test_scale_rule():
    for top, byte in ((1.0, 125), (6.0, 127), (4.0, 127), (3.999, 126), (2.0 ** -126, 0), (2.0 ** -124, 1),
                      (2.0 ** 127, 252), (0.0, 0), (np.inf, 255), (np.nan, 255)):
        row = np.zeros((1, 32))
        row[0, 5] = top
        assert mx.quantize(row)[1][0, 0] == byte, top


def test_quantised_values_are_fixed_points():
    rng = np.random.default_rng(3)
    codes, scales = mx.random_packed(rng, 5, 300)
    v = mx.values(codes, scales, 300)
    c2, s2 = mx.quantize(v)
    assert np.array_equal(mx.values(c2, s2, 300), v)


# ---- sizes ------------------------------------------------------------------------

@pytest.mark.parametrize("rows,K,codes,scales", [(1, 1, 64, 4), (3, 128, 192, 12), (3, 129, 384, 24), (0, 5, 0, 0), (5, 0, 0, 0)])
def test_packed_size(rows, K, codes, scales):
    c, s = ctypes.c_size_t(9), ctypes.c_size_t(9)
    assert L.mxfp4_packed_size(rows, K, ctypes.byref(c), ctypes.byref(s)) == 0
    assert (c.value, s.value) == (codes, scales)
    (r1, c1), (r2, s1) = ba.mxfp4_shapes(rows, K)
    assert r1 == r2 == rows and r1 * c1 == codes and r2 * s1 == scales


def test_packed_size_refuses():
    c = ctypes.c_size_t()
    assert L.mxfp4_packed_size(-1, 1, ctypes.byref(c), ctypes.byref(c)) == 1
    assert L.mxfp4_packed_size(1, -1, ctypes.byref(c), ctypes.byref(c)) == 1
    assert L.mxfp4_packed_size(1, 1, None, ctypes.byref(c)) == 1
    assert L.mxfp4_packed_size(1 << 31, 1, ctypes.byref(c), ctypes.byref(c)) == 2


# ---- refusals of the C entry points -----------------------------------------------

QUANT_BAD = [
    (dict(X=NUL), 1), (dict(codes=NUL), 1), (dict(scales=NUL), 1),
    (dict(rows=-1), 1), (dict(K=-1), 1), (dict(axis=2), 1), (dict(axis=-1), 1),
    (dict(codes=ODD16), 1), (dict(scales=ODD4), 1), (dict(X=ODD2), 1), (dict(X=ODD4, dt=F32), 1),
    (dict(dt=I8), 2), (dict(dt=MX), 2), (dict(dt=256), 2),
    (dict(rows=1 << 31), 2), (dict(K=1 << 31), 2), (dict(rows=1 << 16, K=1 << 15), 2),
    (dict(rows=(1 << 25) + 1, K=1), 2),                # X is small, its padded codes are not
    (dict(rows=(1 << 31) - 1, K=(1 << 31) - 1, dt=F32), 2),
]


@pytest.mark.parametrize("kw,code", QUANT_BAD)
def test_quantize_rejects(kw, code):
    a = dict(X=P, codes=P, scales=P, rows=4, K=64, axis=1, dt=BF16)
    a.update(kw)
    assert L.mxfp4_quantize(a["X"], a["codes"], a["scales"], a["rows"], a["K"], a["axis"], a["dt"], NUL) == code
    assert L.mxfp4_dequantize(a["codes"], a["scales"], a["X"], a["rows"], a["K"], a["axis"], a["dt"], NUL) == code


def test_quantize_empty_is_ok_without_launch():
    for rows, K in ((0, 5), (5, 0), (0, 0)):
        assert L.mxfp4_quantize(NUL, NUL, NUL, rows, K, 1, F32, NUL) == 0
        assert L.mxfp4_dequantize(NUL, NUL, NUL, rows, K, 0, F32, NUL) == 0


def gemm(A=P, As=P, B=P, Bs=P, bias=P, C=P, M=4, N=4, K=64, dt=_dt(MX, MX, F32, BF16), act=1, R=None):
    if R is None:
        return L.gemm_mxfp4_bias_act(A, As, B, Bs, bias, C, M, N, K, dt, act, 0.1, NUL)
    return L.gemm_mxfp4_bias_add_act(A, As, B, Bs, bias, R, C, M, N, K, dt, act, 0.1, NUL)


GEMM_BAD = [
    (dict(A=NUL), 1), (dict(As=NUL), 1), (dict(B=NUL), 1), (dict(Bs=NUL), 1), (dict(C=NUL), 1),
    (dict(M=-1), 1), (dict(N=-1), 1), (dict(K=-1), 1), (dict(act=6), 1), (dict(act=-1), 1),
    (dict(A=ODD16), 1), (dict(B=ODD16), 1), (dict(As=ODD4), 1), (dict(Bs=ODD4), 1),
    (dict(C=ODD2), 1), (dict(bias=ODD4), 1), (dict(R=ODD2), 1), (dict(R=NUL), 1),
    (dict(dt=_dt(F16, MX, F32, F32)), 1),              # scales beside a 16-bit A
    (dict(dt=_dt(F16, MX, F32, F32), As=NUL, A=NUL), 1),
    (dict(dt=_dt(BF16, MX, F32, F32), As=NUL, A=ODD2), 1),
    (dict(dt=_dt(MX, BF16, F32, F32)), 2), (dict(dt=_dt(F32, MX, F32, F32), As=NUL), 2),
    (dict(dt=_dt(I8, MX, F32, F32), As=NUL), 2), (dict(dt=_dt(MX, MX, F32, 4)), 2),
    (dict(dt=_dt(MX, MX, F32, MX)), 2), (dict(dt=_dt(MX, MX, 4, F32)), 2), (dict(dt=_dt(MX, MX, 7, F32)), 2),
    (dict(M=1 << 31), 2), (dict(N=1 << 31), 2), (dict(K=1 << 31), 2),
    (dict(M=1 << 16, N=1 << 15), 2),                   # C is 2^32 bytes
    (dict(M=1 << 20, K=1 << 13), 2),                   # A's codes are 2^32 bytes
    (dict(N=1 << 20, K=1 << 13), 2),
    (dict(M=1 << 15, K=1 << 16, dt=_dt(BF16, MX, F32, F32), As=NUL), 2),
]


@pytest.mark.parametrize("kw,code", GEMM_BAD)
def test_gemm_rejects(kw, code):
    assert gemm(**kw) == code


def test_gemm_empty_is_ok_without_launch():
    assert gemm(M=0) == 0 and gemm(N=0) == 0
    assert gemm(M=0, A=NUL, As=NUL, R=NUL) == 0


def test_mxfp4_stays_out_of_the_other_entry_points():
    assert L.gemm_bias_act(P, P, P, P, 4, 4, 4, _dt(MX, MX, F32, F32), 1, 0.0, NUL) == 2
    assert L.gemm_bias_act(P, P, P, P, 4, 4, 4, _dt(F16, MX, F32, F32), 1, 0.0, NUL) == 2


# ---- refusals of the binding --------------------------------------------------------

def _u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def test_binding_refuses():
    x, c, s = torch.zeros(4, 200), _u8(4, 128), _u8(4, 8)
    bad = [
        lambda: ba.mxfp4_quantize(x[0], c, s), lambda: ba.mxfp4_quantize(x, c, s, axis=2),
        lambda: ba.mxfp4_quantize(x, _u8(4, 100), s), lambda: ba.mxfp4_quantize(x, c, _u8(4, 7)),
        lambda: ba.mxfp4_quantize(x, c.int(), s), lambda: ba.mxfp4_quantize(x, c[0], s[0]),
        lambda: ba.mxfp4_quantize(x, c, s, axis=0), lambda: ba.mxfp4_quantize(x.double(), c, s),
        lambda: ba.mxfp4_quantize(x, c, s),                                    # not a device tensor
        lambda: ba.mxfp4_dequantize(c, s, x.t()), lambda: ba.mxfp4_dequantize(c, s, x),
    ]
    w, ws, y = _u8(6, 128), _u8(6, 8), torch.zeros(4, 6)
    h = x.half()
    bad += [
        lambda: ba.gemm_mxfp4_bias_act(c, s, w, ws, None, torch.zeros(4, 5)),
        lambda: ba.gemm_mxfp4_bias_act(c, s, _u8(6, 64), _u8(6, 4), None, y),      # other K
        lambda: ba.gemm_mxfp4_bias_act(h, None, _u8(6, 64), _u8(6, 4), None, y),
        lambda: ba.gemm_mxfp4_bias_act(h, s, w, ws, None, y),                      # scales beside a 16-bit A
        lambda: ba.gemm_mxfp4_bias_act(h[0], None, w, ws, None, y),
        lambda: ba.gemm_mxfp4_bias_act(c, s, w, ws, torch.zeros(5), y),
        lambda: ba.gemm_mxfp4_bias_act(c, s, w, ws, None, y, act="swish"),
        lambda: ba.gemm_mxfp4_bias_act(c, s, w, ws, None, y),                      # not a device tensor
        lambda: ba.gemm_mxfp4_bias_add_act(c, s, w, ws, None, None, y),
        lambda: ba.gemm_mxfp4_bias_add_act(c, s, w, ws, None, y.half(), y),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was accepted")


# ---- the C++ way of the binding -------------------------------------------------------

def test_native_call_declines_what_it_does_not_take():
    n = ba._binding._native
    if n is None:
        pytest.skip("built without torch")
    x, c, s, w, ws, y = torch.zeros(4, 200), _u8(4, 128), _u8(4, 8), _u8(6, 128), _u8(6, 8), torch.zeros(4, 6)
    for args in ((), (x, c, s), (x, c, s, 1), (x, c, s, 1.0), (x, c, s, None), (None, c, s, 1), (x, 3, "s", 1),
                 (x[0], c, s, 1), (x, c[0], s[0], 1), (x, c, s, 1 << 80), (object(),) * 4):
        assert n.quantize(*args) is False and n.dequantize(*args) is False
    good = [c, s, w, ws, None, None, y, "relu", 0.0]
    assert n.gemm(*good) is False                          # host tensors
    for i, bad in [(i, b) for i in range(9) for b in (None, 7, "x", x[0], torch.zeros(4, 6).int())]:
        assert n.gemm(*good[:i], bad, *good[i + 1:]) is False
    assert n.gemm(*good[:8]) is False and n.gemm() is False
    with pytest.raises(TypeError):
        n.bind(1, 2)
    with pytest.raises(TypeError):
        n.bind(1, 2, 3, "x")
