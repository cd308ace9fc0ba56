"""Refusals of the MXFP4 calls with operands on the device: a call that is
taken, with one argument changed at a time.  The C++ way must decline it without
calling anything and the public call must raise; nothing is launched, so the
outputs keep what was in them."""
import ctypes

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ba():
    import conv_bias_activation_amd as m
    return m


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8, device="cuda")


def z(*shape, dt=torch.float32):
    return torch.zeros(shape, dtype=dt, device="cuda")


# X [5, 200] -> codes [5, 128], scales [5, 8]; name -> (position, replacement)
QUANT = {
    "a row more": (0, lambda: z(6, 200)), "a group more": (0, lambda: z(5, 257)), "a group less": (0, lambda: z(5, 128)),
    "transposed": (0, lambda: z(200, 5)), "one dimension": (0, lambda: z(1000)), "three dimensions": (0, lambda: z(5, 200, 1)),
    "fp64": (0, lambda: z(5, 200, dt=torch.float64)), "int8": (0, lambda: z(5, 200, dt=torch.int8)),
    "X not contiguous": (0, lambda: z(200, 5).t()), "X a wider tensor's columns": (0, lambda: z(5, 208)[:, :200]),
    "X on the host": (0, lambda: torch.zeros(5, 200)),
    "codes of fewer rows": (1, lambda: u8(4, 128)), "codes too narrow": (1, lambda: u8(5, 64)),
    "codes too wide": (1, lambda: u8(5, 192)), "codes of one dimension": (1, lambda: u8(640)), "codes of three dimensions": (1, lambda: u8(5, 128, 1)),
    "codes int8": (1, lambda: z(5, 128, dt=torch.int8)), "codes not contiguous": (1, lambda: u8(128, 5).t()),
    "codes every other column": (1, lambda: u8(5, 256)[:, ::2]), "codes on the host": (1, lambda: torch.zeros(5, 128, dtype=torch.uint8)),
    "scales of fewer rows": (2, lambda: u8(4, 8)), "scales too narrow": (2, lambda: u8(5, 4)), "scales too wide": (2, lambda: u8(5, 12)),
    "scales of a broken group": (2, lambda: u8(5, 7)), "scales of a group and a byte": (2, lambda: u8(5, 9)), "scales of three dimensions": (2, lambda: u8(5, 8, 1)), "scales int32": (2, lambda: z(5, 8, dt=torch.int32)),
    "scales not contiguous": (2, lambda: u8(8, 5).t()), "scales on the host": (2, lambda: torch.zeros(5, 8, dtype=torch.uint8)),
    "the other axis": (3, lambda: 0), "no such axis": (3, lambda: 2), "a negative axis": (3, lambda: -1),
}


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("what", list(QUANT))
def test_quantise(ba, what, back):
    n = ba._binding._native
    args = [z(5, 200), u8(5, 128), u8(5, 8), 1]
    native = n.dequantize if back else n.quantize

    def public(X, codes, scales, axis, **kw):
        if back:
            ba.mxfp4_dequantize(codes, scales, X, axis=axis, **kw)
        else:
            ba.mxfp4_quantize(X, codes, scales, axis=axis, **kw)

    assert native(*args) is True                         # the call as it should be
    torch.cuda.synchronize()
    at, bad = QUANT[what]
    args[at] = bad()
    outputs = [args[0]] if back else args[1:3]
    for t in outputs:
        t.fill_(7)
    assert native(*args) is False
    for kw in ({}, {"stream": torch.cuda.current_stream()}):
        with pytest.raises(ValueError):
            public(*args, **kw)
    torch.cuda.synchronize()
    assert all(bool((t == 7).all()) for t in outputs)


@pytest.mark.parametrize("axis", [2, -1, 1.0, None])
def test_axis_of_a_square(ba, axis):
    # rows and columns fit either way: the axis alone is wrong
    n = ba._binding._native
    args = [z(200, 200), u8(200, 128), u8(200, 8)]
    assert n.quantize(*args, 0) is True and n.quantize(*args, 1) is True
    assert n.quantize(*args, axis) is False and n.dequantize(*args, axis) is False
    if axis != 1:                                        # (1.0 equals 1 for the Python checks)
        with pytest.raises(ValueError):
            ba.mxfp4_quantize(*args, axis=axis)
        with pytest.raises(ValueError):
            ba.mxfp4_dequantize(*args[1:], args[0], axis=axis)


# A [5, 200] (codes [5, 128], scales [5, 8]), B codes [6, 128], scales [6, 8], C [5, 6]
def arguments(kind):
    A, As = (u8(5, 128), u8(5, 8)) if kind == "mxfp4" else (z(5, 200, dt=torch.bfloat16), None)
    return dict(A=A, a_scales=As, B=u8(6, 128), b_scales=u8(6, 8), bias=z(6), R=z(5, 6), C=z(5, 6), act="relu", alpha=0.0)


BOTH = {
    "B of another K": dict(B=lambda: u8(6, 64), b_scales=lambda: u8(6, 4)),
    "B of a longer K": dict(B=lambda: u8(6, 192), b_scales=lambda: u8(6, 12)),
    "B of more rows": dict(B=lambda: u8(7, 128), b_scales=lambda: u8(7, 8)),
    "B's codes of fewer rows": dict(B=lambda: u8(5, 128)), "B's codes too narrow": dict(B=lambda: u8(6, 64)),
    "B's scales of fewer rows": dict(b_scales=lambda: u8(5, 8)), "B's scales too narrow": dict(b_scales=lambda: u8(6, 4)),
    "B's scales of a broken group": dict(b_scales=lambda: u8(6, 9)), "B int8": dict(B=lambda: z(6, 128, dt=torch.int8)),
    "B not contiguous": dict(B=lambda: u8(128, 6).t()), "B on the host": dict(B=lambda: torch.zeros(6, 128, dtype=torch.uint8)),
    "B's scales not contiguous": dict(b_scales=lambda: u8(8, 6).t()),
    "C of fewer rows": dict(C=lambda: z(4, 6)), "C of more rows": dict(C=lambda: z(6, 6)), "C narrower": dict(C=lambda: z(5, 5)),
    "C wider": dict(C=lambda: z(5, 7)), "C of one dimension": dict(C=lambda: z(30)), "C of three dimensions": dict(C=lambda: z(5, 6, 1), R=lambda: z(5, 6, 1)), "C fp64": dict(C=lambda: z(5, 6, dt=torch.float64)),
    "C of another type than R": dict(C=lambda: z(5, 6, dt=torch.float16)), "C not contiguous": dict(C=lambda: z(6, 5).t()),
    "C on the host": dict(C=lambda: torch.zeros(5, 6)),
    "a short bias": dict(bias=lambda: z(5)), "a long bias": dict(bias=lambda: z(7)), "a bias of one": dict(bias=lambda: z(1)),
    "bias int32": dict(bias=lambda: z(6, dt=torch.int32)), "bias not contiguous": dict(bias=lambda: z(12)[::2]),
    "bias on the host": dict(bias=lambda: torch.zeros(6)),
    "R of fewer rows": dict(R=lambda: z(4, 6)), "R of one row": dict(R=lambda: z(1, 6)), "R flat": dict(R=lambda: z(30)),
    "R fp16": dict(R=lambda: z(5, 6, dt=torch.float16)), "R not contiguous": dict(R=lambda: z(6, 5).t()),
    "R on the host": dict(R=lambda: torch.zeros(5, 6)), "no such activation": dict(act=lambda: "swish"),
}
KIND = {
    "mxfp4": {
        "A of another K": dict(A=lambda: u8(5, 64), a_scales=lambda: u8(5, 4)), "A of more rows": dict(A=lambda: u8(6, 128), a_scales=lambda: u8(6, 8)),
        "A's codes of fewer rows": dict(A=lambda: u8(4, 128)), "A's scales of fewer rows": dict(a_scales=lambda: u8(4, 8)),
        "A's scales of a broken group": dict(a_scales=lambda: u8(5, 7)), "A's codes without scales": dict(a_scales=lambda: None),
        "A not contiguous": dict(A=lambda: u8(128, 5).t()), "A's scales on the host": dict(a_scales=lambda: torch.zeros(5, 8, dtype=torch.uint8)),
    },
    "bf16": {
        "A of a shorter K": dict(A=lambda: z(5, 128, dt=torch.bfloat16)), "A of a longer K": dict(A=lambda: z(5, 257, dt=torch.bfloat16)),
        "A of more rows": dict(A=lambda: z(6, 200, dt=torch.bfloat16)), "A fp32": dict(A=lambda: z(5, 200)),
        "A int8": dict(A=lambda: z(5, 200, dt=torch.int8)), "A of one dimension": dict(A=lambda: z(200, dt=torch.bfloat16)),
        "A not contiguous": dict(A=lambda: z(200, 5, dt=torch.bfloat16).t()), "scales beside a 16-bit A": dict(a_scales=lambda: u8(5, 8)),
        "A on the host": dict(A=lambda: torch.zeros(5, 200, dtype=torch.bfloat16)),
    },
}


@pytest.mark.parametrize("kind,what", [(k, w) for k in ("mxfp4", "bf16") for w in (*BOTH, *KIND[k])])
def test_product(ba, kind, what):
    n = ba._binding._native
    a = arguments(kind)
    assert n.gemm(*a.values()) is True                   # the call as it should be
    torch.cuda.synchronize()
    change = BOTH.get(what) or KIND[kind][what]
    a.update({k: f() for k, f in change.items()})
    a["C"].fill_(7)
    assert n.gemm(*a.values()) is False
    calls = [lambda **kw: ba.gemm_mxfp4_bias_add_act(*a.values(), **kw)]
    if "R" not in what:                                  # (those differ in R alone)
        b = {k: v for k, v in a.items() if k != "R"}
        calls.append(lambda **kw: ba.gemm_mxfp4_bias_act(*b.values(), **kw))
    for call in calls:
        for kw in ({}, {"stream": torch.cuda.current_stream()}):
            with pytest.raises(ValueError):
                call(**kw)
    torch.cuda.synchronize()
    assert bool((a["C"] == 7).all())


@pytest.mark.parametrize("what", ["codes", "scales", "B", "b_scales"])
def test_alignment(ba, what):
    # views off the 16 (codes) or 4 (scales) bytes that the kernels read at a time
    def off(by, *shape):
        m = shape[0] * shape[1]
        return u8(m + 16)[by:by + m].view(shape)

    if what in ("codes", "scales"):
        codes = off(8, 5, 128) if what == "codes" else u8(5, 128)
        scales = off(2, 5, 8) if what == "scales" else u8(5, 8)
        with pytest.raises(ValueError):
            ba.mxfp4_quantize(z(5, 200), codes, scales)
        with pytest.raises(ValueError):
            ba.mxfp4_dequantize(codes, scales, z(5, 200))
    else:
        a = arguments("bf16")
        a[what] = off(8, 6, 128) if what == "B" else off(2, 6, 8)
        with pytest.raises(ValueError):
            ba.gemm_mxfp4_bias_add_act(*a.values())


@pytest.mark.parametrize("status", [1, 2, 3])
def test_the_status_of_a_call_that_fails(ba, status):
    # entry points that only count and fail: one call each, its status comes back
    B = ba._binding
    names = ("mxfp4_quantize", "mxfp4_dequantize", "gemm_mxfp4_bias_act", "gemm_mxfp4_bias_add_act")
    seen = []

    def failing(name):
        return ctypes.CFUNCTYPE(ctypes.c_int, *getattr(B.lib, name).argtypes)(lambda *a: seen.append(name) or status)

    address = lambda f: ctypes.cast(f, ctypes.c_void_p).value  # noqa: E731
    fakes = [failing(name) for name in names]
    q = (z(5, 200), u8(5, 128), u8(5, 8), 1)
    a = arguments("bf16")
    try:
        B._native.bind(*map(address, fakes))
        got = [B._native.quantize(*q), B._native.dequantize(*q), B._native.gemm(*{**a, "R": None}.values()), B._native.gemm(*a.values())]
        assert got == [status] * 4 and not any(g is True for g in got)
        assert seen == list(names)
        with pytest.raises(ba.BiasActError if status == 3 else ValueError):
            ba.gemm_mxfp4_bias_add_act(*a.values())
        assert len(seen) == 5
    finally:
        B._native.bind(*(address(getattr(B.lib, name)) for name in names))
    assert B._native.gemm(*a.values()) is True
