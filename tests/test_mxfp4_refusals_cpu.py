"""Refusals of the MXFP4 binding's Python checks, each by its own message (a
host tensor is refused too, but only after the checks of shapes and types)."""
import os
import re

import pytest

ba = pytest.importorskip("conv_bias_activation_amd")
torch = pytest.importorskip("torch")

SHAPES, U8, MISMATCH = r"codes must be \[rows, 64 g\] and scales", "must be uint8", "shape mismatch"


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def z(*shape, dt=torch.float32):
    return torch.zeros(shape, dtype=dt)


# X [4, 200], codes [4, 128], scales [4, 8]
QUANT = {
    "X of one dimension": (dict(X=z(800)), "must be 2-D"), "X of three": (dict(X=z(4, 200, 1)), "must be 2-D"),
    "no such axis": (dict(axis=2), "axis must be 0 or 1"), "a negative axis": (dict(axis=-1), "axis must be 0 or 1"),
    "the other axis": (dict(axis=0), "codes and scales must be"), "X of more rows": (dict(X=z(5, 200)), "codes and scales must be"),
    "X of more groups": (dict(X=z(4, 257)), "codes and scales must be"), "X of fewer groups": (dict(X=z(4, 128)), "codes and scales must be"),
    "codes too narrow": (dict(codes=u8(4, 100)), SHAPES), "codes of fewer rows": (dict(codes=u8(3, 128)), SHAPES),
    "codes of one dimension": (dict(codes=u8(512)), SHAPES), "codes int32": (dict(codes=u8(4, 128).int()), U8),
    "scales too narrow": (dict(scales=u8(4, 4)), SHAPES), "scales of a broken group": (dict(scales=u8(4, 7), codes=u8(4, 112)), SHAPES),
    "scales of one dimension": (dict(scales=u8(32)), SHAPES), "scales int8": (dict(scales=z(4, 8, dt=torch.int8)), U8),
    "X fp64": (dict(X=z(4, 200, dt=torch.float64)), "unsupported tensor dtype"), "on the host": ({}, "must be a device tensor"),
}


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("what", list(QUANT))
def test_quantise(what, back):
    a = {**dict(X=z(4, 200), codes=u8(4, 128), scales=u8(4, 8), axis=1), **QUANT[what][0]}
    with pytest.raises(ValueError, match=QUANT[what][1]):
        if back:
            ba.mxfp4_dequantize(a["codes"], a["scales"], a["X"], axis=a["axis"])
        else:
            ba.mxfp4_quantize(**a)


HALF = torch.float16
# A codes [4, 128] with scales [4, 8] or fp16 [4, 200]; B codes [6, 128], scales [6, 8]; C [4, 6]
GEMM = {
    "B of a shorter K": (dict(B=u8(6, 64), b_scales=u8(6, 4)), MISMATCH), "B of a longer K": (dict(B=u8(6, 192), b_scales=u8(6, 12)), MISMATCH),
    "B of more rows": (dict(B=u8(7, 128), b_scales=u8(7, 8)), MISMATCH), "B's codes too narrow": (dict(B=u8(6, 64)), SHAPES),
    "B's scales of fewer rows": (dict(b_scales=u8(5, 8)), SHAPES), "B int8": (dict(B=z(6, 128, dt=torch.int8)), U8),
    "C of fewer rows": (dict(C=z(3, 6)), MISMATCH), "C wider": (dict(C=z(4, 7)), MISMATCH), "C flat": (dict(C=z(24)), MISMATCH),
    "C fp64": (dict(C=z(4, 6, dt=torch.float64)), "unsupported tensor dtype"),
    "a short bias": (dict(bias=z(5)), "bias must have N = 6"), "a bias of one": (dict(bias=z(1)), "bias must have N = 6"),
    "no such activation": (dict(act="swish"), "unknown activation|must be a device tensor"), "on the host": ({}, "must be a device tensor"),
}
MX_ONLY = {
    "A of a shorter K": (dict(A=u8(4, 64), a_scales=u8(4, 4)), MISMATCH), "A of more rows": (dict(A=u8(5, 128), a_scales=u8(5, 8)), MISMATCH),
    "A's scales of fewer rows": (dict(a_scales=u8(3, 8)), SHAPES), "A without its scales": (dict(a_scales=None), "unsupported tensor dtype"),
}
HALF_ONLY = {
    "A of a shorter K": (dict(A=z(4, 128, dt=HALF)), MISMATCH), "A of a longer K": (dict(A=z(4, 257, dt=HALF)), MISMATCH),
    "A of more rows": (dict(A=z(5, 200, dt=HALF)), MISMATCH), "A of one dimension": (dict(A=z(200, dt=HALF)), "A must be 2-D"),
    "scales beside a 16-bit A": (dict(a_scales=u8(4, 8)), U8),
}


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("kind,what", [("mxfp4", w) for w in (*GEMM, *MX_ONLY)] + [("f16", w) for w in (*GEMM, *HALF_ONLY)])
def test_product(kind, what, residual):
    change, message = GEMM.get(what) or (MX_ONLY if kind == "mxfp4" else HALF_ONLY)[what]
    a = dict(A=u8(4, 128), a_scales=u8(4, 8)) if kind == "mxfp4" else dict(A=z(4, 200, dt=HALF), a_scales=None)
    a = {**a, **dict(B=u8(6, 128), b_scales=u8(6, 8), bias=z(6), C=z(4, 6), act="relu"), **change}
    with pytest.raises(ValueError, match=message):
        if residual:
            ba.gemm_mxfp4_bias_add_act(R=torch.zeros_like(a["C"]), **a)
        else:
            ba.gemm_mxfp4_bias_act(**a)


# ---- one polynomial in two headers --------------------------------------------------------

def test_erfc_of_the_tail_has_the_coefficients_of_erfc_f32():
    csrc = os.path.join(os.path.dirname(ba.__file__), "csrc")

    def body(name, head):
        with open(os.path.join(csrc, name)) as f:
            text = f.read()
        text = text[text.index(head):]
        return text[:text.index("\n}")]

    numbers = lambda t: re.findall(r"-?\d\.\d{9}e[+-]\d\d", t)  # noqa: E731
    a, b = numbers(body("device_common.hpp", "float erfc_f32(")), numbers(body("mx_act.hpp", "float erfc_scaled("))
    assert len(a) == 10 and a == b
