"""ctypes marshalling for libbiasact.so (see include/biasact.h for the
contract of every entry point).  No arithmetic of the method happens here."""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_HERE, "libbiasact.so")

DTYPE_CODES = {"f32": 0, "f16": 1, "bf16": 2, "i8": 3, "i32": 4, "mxfp4": 5}
ACT_CODES = {"none": 0, "relu": 1, "leaky_relu": 2, "tanh": 3, "gelu": 4, "sigmoid": 5}
BA_OK, BA_ERR_INVALID, BA_ERR_UNSUPPORTED, BA_ERR_HIP = 0, 1, 2, 3


class BiasActError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


def _load():
    if not os.path.exists(lib_path):
        raise ImportError(f"{lib_path} is not built; run `python -m conv_bias_activation_amd.build` "
                          "(or __graft_entry__.build()) first")
    # The library and torch must share one HIP runtime: device pointers and
    # stream handles cross the boundary.  torch ships its own libamdhip64
    # with the same soname the library links against, so loading torch first
    # makes the dynamic linker bind the library to that instance; loading the
    # library first would bring in a second runtime beside torch's.
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    l = ctypes.CDLL(lib_path)
    vp, i64, u32, i32p = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint32, ctypes.POINTER(ctypes.c_int32)
    l.gemm_bias_act.argtypes = [vp, vp, vp, vp, i64, i64, i64, u32, ctypes.c_int, ctypes.c_float, vp]
    l.gemm_bias_act.restype = ctypes.c_int
    l.gemm_bias_act_2k.argtypes = [vp, vp, vp, vp, i64, i64, i64, u32, ctypes.c_int, ctypes.c_float,
                                   vp, ctypes.c_size_t, vp]
    l.gemm_bias_act_2k.restype = ctypes.c_int
    l.gemm_bias_act_2k_noalloc.argtypes = [vp, vp, vp, vp, i64, i64, i64, u32, ctypes.c_int,
                                           ctypes.c_float, vp]
    l.gemm_bias_act_2k_noalloc.restype = ctypes.c_int
    l.gemm_bias_act_workspace_size.argtypes = [i64, i64]
    l.gemm_bias_act_workspace_size.restype = ctypes.c_size_t
    conv = [vp, vp, vp, vp] + [i64] * 7 + [i32p, i32p, i32p, u32, ctypes.c_int]
    l.conv2d_bias_act.argtypes = conv + [vp]
    l.conv2d_bias_act.restype = ctypes.c_int
    l.conv2d_bias_act_2k.argtypes = conv + [vp, ctypes.c_size_t, vp]
    l.conv2d_bias_act_2k.restype = ctypes.c_int
    l.conv2d_bias_act_workspace_size.argtypes = [i64] * 7 + [i32p, i32p, i32p]
    gr = [vp, vp, vp, vp, vp, i64, i64, i64, u32, ctypes.c_int, ctypes.c_float]
    l.gemm_bias_add_act.argtypes = gr + [vp]
    l.gemm_bias_add_act.restype = ctypes.c_int
    l.gemm_bias_add_act_2k.argtypes = gr + [vp, ctypes.c_size_t, vp]
    l.gemm_bias_add_act_2k.restype = ctypes.c_int
    cr = [vp, vp, vp, vp, vp] + [i64] * 7 + [i32p, i32p, i32p, u32, ctypes.c_int]
    l.conv2d_bias_add_act.argtypes = cr + [vp]
    l.conv2d_bias_add_act.restype = ctypes.c_int
    l.conv2d_bias_add_act_2k.argtypes = cr + [vp, ctypes.c_size_t, vp]
    l.conv2d_bias_add_act_2k.restype = ctypes.c_int
    l.conv2d_bias_act_workspace_size.restype = ctypes.c_size_t
    l.biasact_status_string.argtypes = [ctypes.c_int]
    l.biasact_status_string.restype = ctypes.c_char_p
    ip = ctypes.POINTER(ctypes.c_int)
    l.biasact_gemm_path.argtypes = [i64, i64, i64, u32, ctypes.c_int]
    l.biasact_gemm_path.restype = ctypes.c_int
    l.biasact_conv_path.argtypes = [i64] * 7 + [i32p, i32p, i32p, u32, ctypes.c_int]
    l.biasact_conv_path.restype = ctypes.c_int
    l.biasact_set_gemm_path.argtypes = [i64, i64, i64, u32, ctypes.c_int, ctypes.c_int]
    l.biasact_set_gemm_path.restype = ctypes.c_int
    l.biasact_set_conv_path.argtypes = [i64] * 7 + [i32p, i32p, i32p, u32, ctypes.c_int, ctypes.c_int]
    l.biasact_set_conv_path.restype = ctypes.c_int
    l.biasact_gemm_static_path.argtypes = [vp, vp, vp, vp, i64, i64, i64, u32, ctypes.c_int, vp,
                                           ctypes.c_size_t]
    l.biasact_gemm_static_path.restype = ctypes.c_int
    i64p = ctypes.POINTER(ctypes.c_int64)
    l.conv2d_bias_act_out_dims.argtypes = [i64] * 4 + [i32p, i32p, i32p, i64p, i64p]
    l.conv2d_bias_act_out_dims.restype = ctypes.c_int
    l.biasact_tune_gemm.argtypes = ([vp, vp, vp, vp, i64, i64, i64, u32, ctypes.c_int, ctypes.c_float,
                                     vp, ctypes.c_size_t, ctypes.c_int, vp, ip])
    l.biasact_tune_gemm.restype = ctypes.c_int
    l.biasact_tune_conv.argtypes = conv + [vp, ctypes.c_size_t, ctypes.c_int, vp, ip]
    l.biasact_tune_conv.restype = ctypes.c_int
    l.gemm_bias_act_auto.argtypes = l.gemm_bias_act_2k.argtypes
    l.gemm_bias_act_auto.restype = ctypes.c_int
    l.conv2d_bias_act_auto.argtypes = l.conv2d_bias_act_2k.argtypes
    l.conv2d_bias_act_auto.restype = ctypes.c_int
    l.biasact_last_tile_config.argtypes = [ctypes.c_char_p, ctypes.c_size_t]
    l.biasact_last_tile_config.restype = ctypes.c_int
    l.biasact_last_hip_error.argtypes = []
    l.biasact_last_hip_error.restype = ctypes.c_int
    l.biasact_last_hip_error_string.argtypes = []
    l.biasact_last_hip_error_string.restype = ctypes.c_char_p
    l.biasact_num_tile_configs.argtypes = []
    l.biasact_num_tile_configs.restype = ctypes.c_int
    l.biasact_tile_config_name.argtypes = [ctypes.c_int, ctypes.c_char_p, ctypes.c_size_t]
    l.biasact_tile_config_name.restype = ctypes.c_int
    l.biasact_gemm_tile_config.argtypes = [i64, i64, i64, u32]
    l.biasact_gemm_tile_config.restype = ctypes.c_int
    l.biasact_conv_tile_config.argtypes = [i64] * 5 + [u32]
    l.biasact_conv_tile_config.restype = ctypes.c_int
    l.biasact_force_tile_config.argtypes = [ctypes.c_int]
    l.biasact_force_tile_config.restype = ctypes.c_int
    l.biasact_force_halo_variant.argtypes = [ctypes.c_int]
    l.biasact_force_halo_variant.restype = ctypes.c_int
    u64p = ctypes.POINTER(ctypes.c_size_t)
    l.mxfp4_packed_size.argtypes = [i64, i64, u64p, u64p]
    l.mxfp4_packed_size.restype = ctypes.c_int
    l.mxfp4_quantize.argtypes = [vp, vp, vp, i64, i64, ctypes.c_int, u32, vp]
    l.mxfp4_quantize.restype = ctypes.c_int
    l.mxfp4_dequantize.argtypes = l.mxfp4_quantize.argtypes
    l.mxfp4_dequantize.restype = ctypes.c_int
    l.gemm_mxfp4_bias_act.argtypes = [vp] * 6 + [i64, i64, i64, u32, ctypes.c_int, ctypes.c_float, vp]
    l.gemm_mxfp4_bias_act.restype = ctypes.c_int
    l.gemm_mxfp4_bias_add_act.argtypes = [vp] * 7 + [i64, i64, i64, u32, ctypes.c_int, ctypes.c_float, vp]
    l.gemm_mxfp4_bias_add_act.restype = ctypes.c_int
    return l


lib = _load()


def _load_native():
    """The C++ way from torch tensors to the MXFP4 calls (native_call.cpp), or
    None where torch or the module is missing, or where the module does not
    load (built for another torch or Python; a warning says why): the calls
    below then marshal through ctypes, to the same entry points."""
    import importlib.machinery
    import importlib.util
    import warnings
    path = os.path.join(_HERE, "_native.so")
    try:
        import torch  # noqa: F401  (its libraries have to be there first)
    except ImportError:
        return None
    if not os.path.exists(path):
        return None
    loader = importlib.machinery.ExtensionFileLoader(__package__ + "._native", path)
    try:
        m = importlib.util.module_from_spec(importlib.util.spec_from_loader(loader.name, loader))
        loader.exec_module(m)
    except ImportError as e:
        warnings.warn(f"{path} does not load ({e}); the MXFP4 calls go through ctypes, which costs them up to "
                      "3 us of host time. Rebuild with `python conv_bias_activation_amd/build.py`.", RuntimeWarning,
                      stacklevel=2)
        return None
    m.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
        lib.mxfp4_quantize, lib.mxfp4_dequantize, lib.gemm_mxfp4_bias_act, lib.gemm_mxfp4_bias_add_act)))
    return m


_native = _load_native()


def status_string(status: int) -> str:
    return lib.biasact_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status == BA_OK:
        return
    msg = f"{what}: {status_string(status)}"
    if status in (BA_ERR_INVALID, BA_ERR_UNSUPPORTED):
        raise ValueError(msg)
    if status == BA_ERR_HIP:
        msg += (f" (hipError {lib.biasact_last_hip_error()}: "
                f"{lib.biasact_last_hip_error_string().decode()})")
    raise BiasActError(status, msg)


@functools.lru_cache(maxsize=None)
def dtypes_code(a: str, b: str, bias: Optional[str], out: str) -> int:
    try:
        codes = [DTYPE_CODES[a], DTYPE_CODES[b], DTYPE_CODES[bias or "f32"], DTYPE_CODES[out]]
    except KeyError as e:
        raise ValueError(f"unknown element type {e}; supported: {sorted(DTYPE_CODES)}") from None
    return codes[0] | (codes[1] << 8) | (codes[2] << 16) | (codes[3] << 24)


def _act(act) -> int:
    code = ACT_CODES.get(act)
    if code is not None:
        return code
    if isinstance(act, int):
        return act
    raise ValueError(f"unknown activation {act!r}; supported: {sorted(ACT_CODES)}")


# -- torch marshalling ------------------------------------------------------

def _torch():
    import torch  # device memory and streams only
    return torch


_TNAMES = None      # torch dtype -> element type name, built on first use


def _tname(t) -> str:
    global _TNAMES
    if _TNAMES is None:
        torch = _torch()
        _TNAMES = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16", torch.int8: "i8",
                   torch.int32: "i32"}
    name = _TNAMES.get(t.dtype)
    if name is None:
        raise ValueError(f"unsupported tensor dtype {t.dtype}; supported: float32, float16, "
                         "bfloat16, int8 and int32 (int8 GEMMs)")
    return name


def _dev(t, name):
    if t is None:
        return None
    if t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    raise ValueError(f"{name} must be contiguous (packed, row-major)")


def _current_stream():
    """() -> handle of the current device's current stream.  torch's public
    call builds a Stream object each time (2.6 us of host time, as much as a
    launch); the raw form that its own generated code uses takes 0.1 us."""
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    dev = getattr(torch._C, "_cuda_getDevice", None)
    if raw is None or dev is None:
        return lambda: torch.cuda.current_stream().cuda_stream
    return lambda: raw(dev())


_current = None      # set on first use: torch's device state must exist by then


def _stream(stream):
    global _current
    if stream is None:
        if _current is None:
            _torch().cuda.current_stream()
            _current = _current_stream()
        return _current()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _i32x(vals: Sequence[int], n: int, name: str):
    vals = [int(v) for v in vals]
    if len(vals) != n:
        raise ValueError(f"{name} needs {n} values")
    return (ctypes.c_int32 * n)(*vals)


# -- GEMM ------------------------------------------------------------------

def _gemm_args(A, B, bias, C):
    if A.dim() != 2 or B.dim() != 2 or C.dim() != 2:
        raise ValueError("A, B, C must be 2-D")
    M, K = A.shape
    K2, N = B.shape
    if K2 != K or tuple(C.shape) != (M, N):
        raise ValueError(f"shape mismatch: A{tuple(A.shape)} B{tuple(B.shape)} C{tuple(C.shape)}")
    if bias is not None and bias.numel() != N:
        raise ValueError(f"bias must have N = {N} elements")
    dt = dtypes_code(_tname(A), _tname(B), _tname(bias) if bias is not None else None, _tname(C))
    return M, N, K, dt


def gemm_bias_act(A, B, bias, C, act="none", alpha: float = 0.0, stream=None):
    """C = act(A @ B + bias) on the GPU, C written in place."""
    M, N, K, dt = _gemm_args(A, B, bias, C)
    rc = lib.gemm_bias_act(_dev(A, "A"), _dev(B, "B"), _dev(bias, "bias"), _dev(C, "C"),
                           M, N, K, dt, _act(act), float(alpha), _stream(stream))
    _check(rc, "gemm_bias_act")
    return C


def gemm_bias_act_workspace_size(M: int, N: int) -> int:
    return int(lib.gemm_bias_act_workspace_size(M, N))


def gemm_bias_act_2k(A, B, bias, C, act="none", alpha: float = 0.0, workspace=None, stream=None):
    M, N, K, dt = _gemm_args(A, B, bias, C)
    if workspace is None:
        raise ValueError("workspace (device buffer of gemm_bias_act_workspace_size bytes) is required")
    nbytes = workspace.numel() * workspace.element_size()
    rc = lib.gemm_bias_act_2k(_dev(A, "A"), _dev(B, "B"), _dev(bias, "bias"), _dev(C, "C"),
                              M, N, K, dt, _act(act), float(alpha), _dev(workspace, "workspace"),
                              nbytes, _stream(stream))
    _check(rc, "gemm_bias_act_2k")
    return C


def gemm_bias_act_2k_noalloc(A, B, bias, C, act="none", alpha: float = 0.0, stream=None):
    """The two-kernel GEMM with the library's own fixed workspace (no
    allocation; M * N * 4 <= 64 MiB; calls overlapping on one GPU race)."""
    M, N, K, dt = _gemm_args(A, B, bias, C)
    rc = lib.gemm_bias_act_2k_noalloc(_dev(A, "A"), _dev(B, "B"), _dev(bias, "bias"), _dev(C, "C"),
                                      M, N, K, dt, _act(act), float(alpha), _stream(stream))
    _check(rc, "gemm_bias_act_2k_noalloc")
    return C


def _residual(R, out, name="R"):
    if R is None:
        raise ValueError(f"{name} (the residual, shaped and typed like the output) is required")
    if tuple(R.shape) != tuple(out.shape) or R.dtype != out.dtype:
        raise ValueError(f"{name} must match the output: {tuple(out.shape)} {out.dtype}, "
                         f"got {tuple(R.shape)} {R.dtype}")
    return _dev(R, name)


def gemm_bias_add_act(A, B, bias, R, C, act="none", alpha: float = 0.0, stream=None):
    """C = act(A @ B + bias + R); R like C (may be C itself)."""
    M, N, K, dt = _gemm_args(A, B, bias, C)
    rc = lib.gemm_bias_add_act(_dev(A, "A"), _dev(B, "B"), _dev(bias, "bias"), _residual(R, C),
                               _dev(C, "C"), M, N, K, dt, _act(act), float(alpha), _stream(stream))
    _check(rc, "gemm_bias_add_act")
    return C


def gemm_bias_add_act_2k(A, B, bias, R, C, act="none", alpha: float = 0.0, workspace=None,
                         stream=None):
    M, N, K, dt = _gemm_args(A, B, bias, C)
    if workspace is None:
        raise ValueError("workspace (device buffer of gemm_bias_act_workspace_size bytes) is required")
    nbytes = workspace.numel() * workspace.element_size()
    rc = lib.gemm_bias_add_act_2k(_dev(A, "A"), _dev(B, "B"), _dev(bias, "bias"), _residual(R, C),
                                  _dev(C, "C"), M, N, K, dt, _act(act), float(alpha),
                                  _dev(workspace, "workspace"), nbytes, _stream(stream))
    _check(rc, "gemm_bias_add_act_2k")
    return C


# -- conv2d ----------------------------------------------------------------

def conv_out_hw(H, W, kh, kw, strides, pads, dilations):
    """(Ho, Wo) from the library's own output-size rule (None when the
    output would be empty or the attributes are invalid)."""
    ho, wo = ctypes.c_int64(0), ctypes.c_int64(0)
    rc = lib.conv2d_bias_act_out_dims(int(H), int(W), int(kh), int(kw), _i32x(strides, 2, "strides"),
                                      _i32x(pads, 4, "pads"), _i32x(dilations, 2, "dilations"),
                                      ctypes.byref(ho), ctypes.byref(wo))
    if rc != BA_OK:
        return None
    return ho.value, wo.value


def _conv_args(x, w, bias, y, strides, pads, dilations):
    if x.dim() != 4 or w.dim() != 4 or y.dim() != 4:
        raise ValueError("x, w, y must be 4-D (NCHW, OIHW, NCHW)")
    N, C, H, W = x.shape
    Co, C2, kh, kw = w.shape
    if C2 != C:
        raise ValueError("x and w disagree on the channel count")
    hw = conv_out_hw(H, W, kh, kw, strides, pads, dilations)
    if hw is not None and tuple(y.shape) != (N, Co, hw[0], hw[1]):
        raise ValueError(f"y must be {(N, Co, hw[0], hw[1])}, got {tuple(y.shape)}")
    if bias is not None and bias.numel() != Co:
        raise ValueError(f"bias must have Co = {Co} elements")
    dt = dtypes_code(_tname(x), _tname(w), _tname(bias) if bias is not None else None, _tname(y))
    return (N, C, H, W, Co, kh, kw), dt


def conv2d_bias_act(x, w, bias, y, strides=(1, 1), pads=(0, 0, 0, 0), dilations=(1, 1),
                    act="tanh", stream=None):
    """y = act(conv2d(x, w) + bias); pads = (top, bottom, left, right)."""
    dims, dt = _conv_args(x, w, bias, y, strides, pads, dilations)
    rc = lib.conv2d_bias_act(_dev(x, "x"), _dev(w, "w"), _dev(bias, "bias"), _dev(y, "y"), *dims,
                             _i32x(strides, 2, "strides"), _i32x(pads, 4, "pads"),
                             _i32x(dilations, 2, "dilations"), dt, _act(act), _stream(stream))
    _check(rc, "conv2d_bias_act")
    return y


def conv2d_bias_act_workspace_size(N, C, H, W, Co, kh, kw, strides, pads, dilations) -> int:
    return int(lib.conv2d_bias_act_workspace_size(N, C, H, W, Co, kh, kw,
                                                  _i32x(strides, 2, "strides"), _i32x(pads, 4, "pads"),
                                                  _i32x(dilations, 2, "dilations")))


def conv2d_bias_act_2k(x, w, bias, y, strides=(1, 1), pads=(0, 0, 0, 0), dilations=(1, 1),
                       act="tanh", workspace=None, stream=None):
    dims, dt = _conv_args(x, w, bias, y, strides, pads, dilations)
    if workspace is None:
        raise ValueError("workspace (device buffer of conv2d_bias_act_workspace_size bytes) is required")
    nbytes = workspace.numel() * workspace.element_size()
    rc = lib.conv2d_bias_act_2k(_dev(x, "x"), _dev(w, "w"), _dev(bias, "bias"), _dev(y, "y"), *dims,
                                _i32x(strides, 2, "strides"), _i32x(pads, 4, "pads"),
                                _i32x(dilations, 2, "dilations"), dt, _act(act),
                                _dev(workspace, "workspace"), nbytes, _stream(stream))
    _check(rc, "conv2d_bias_act_2k")
    return y


def conv2d_bias_add_act(x, w, bias, R, y, strides=(1, 1), pads=(0, 0, 0, 0), dilations=(1, 1),
                        act="tanh", stream=None):
    """y = act(conv2d(x, w) + bias + R); R like y (may be y itself)."""
    dims, dt = _conv_args(x, w, bias, y, strides, pads, dilations)
    rc = lib.conv2d_bias_add_act(_dev(x, "x"), _dev(w, "w"), _dev(bias, "bias"), _residual(R, y),
                                 _dev(y, "y"), *dims, _i32x(strides, 2, "strides"),
                                 _i32x(pads, 4, "pads"), _i32x(dilations, 2, "dilations"), dt,
                                 _act(act), _stream(stream))
    _check(rc, "conv2d_bias_add_act")
    return y


def conv2d_bias_add_act_2k(x, w, bias, R, y, strides=(1, 1), pads=(0, 0, 0, 0), dilations=(1, 1),
                           act="tanh", workspace=None, stream=None):
    dims, dt = _conv_args(x, w, bias, y, strides, pads, dilations)
    if workspace is None:
        raise ValueError("workspace (device buffer of conv2d_bias_act_workspace_size bytes) is required")
    nbytes = workspace.numel() * workspace.element_size()
    rc = lib.conv2d_bias_add_act_2k(_dev(x, "x"), _dev(w, "w"), _dev(bias, "bias"), _residual(R, y),
                                    _dev(y, "y"), *dims, _i32x(strides, 2, "strides"),
                                    _i32x(pads, 4, "pads"), _i32x(dilations, 2, "dilations"), dt,
                                    _act(act), _dev(workspace, "workspace"), nbytes,
                                    _stream(stream))
    _check(rc, "conv2d_bias_add_act_2k")
    return y


# -- fused or two-kernel, per problem -------------------------------------------

PATH_NAMES = {0: "fused", 1: "2k"}


def gemm_path(M, N, K, dtypes: int, act="none") -> str:
    return PATH_NAMES[int(lib.biasact_gemm_path(M, N, K, dtypes, _act(act)))]


def conv_path(N, C, H, W, Co, kh, kw, strides, pads, dilations, dtypes: int, act="tanh") -> str:
    rc = int(lib.biasact_conv_path(N, C, H, W, Co, kh, kw, _i32x(strides, 2, "strides"),
                                   _i32x(pads, 4, "pads"), _i32x(dilations, 2, "dilations"), dtypes,
                                   _act(act)))
    if rc < 0:
        _check(-rc, "conv_path")
    return PATH_NAMES[rc]


def set_gemm_path(M, N, K, dtypes: int, act="none", path="fused"):
    """Record the path for a GEMM problem (None forgets the record)."""
    code = -1 if path is None else {v: k for k, v in PATH_NAMES.items()}[path]
    _check(lib.biasact_set_gemm_path(M, N, K, dtypes, _act(act), code), "set_gemm_path")


def set_conv_path(N, C, H, W, Co, kh, kw, strides, pads, dilations, dtypes: int, act="tanh",
                  path="fused"):
    code = -1 if path is None else {v: k for k, v in PATH_NAMES.items()}[path]
    _check(lib.biasact_set_conv_path(N, C, H, W, Co, kh, kw, _i32x(strides, 2, "strides"),
                                     _i32x(pads, 4, "pads"), _i32x(dilations, 2, "dilations"),
                                     dtypes, _act(act), code), "set_conv_path")


def gemm_static_path(A, B, bias, C, act="none", workspace=None) -> str:
    """The library's static choice for these buffers (no launch)."""
    M, N, K, dt = _gemm_args(A, B, bias, C)
    ws, nbytes = _ws(workspace)
    return PATH_NAMES[int(lib.biasact_gemm_static_path(_dev(A, "A"), _dev(B, "B"), _dev(bias, "bias"),
                                                        _dev(C, "C"), M, N, K, dt, _act(act), ws,
                                                        nbytes))]


def _ws(workspace):
    if workspace is None:
        return None, 0
    return _dev(workspace, "workspace"), workspace.numel() * workspace.element_size()


def tune_gemm(A, B, bias, C, act="none", alpha: float = 0.0, workspace=None, reps: int = 20,
              stream=None) -> str:
    """Times both paths on these buffers (synchronising the stream; C is
    overwritten) and records the faster for this problem."""
    M, N, K, dt = _gemm_args(A, B, bias, C)
    ws, nbytes = _ws(workspace)
    path = ctypes.c_int(-1)
    rc = lib.biasact_tune_gemm(_dev(A, "A"), _dev(B, "B"), _dev(bias, "bias"), _dev(C, "C"), M, N,
                               K, dt, _act(act), float(alpha), ws, nbytes, int(reps),
                               _stream(stream), ctypes.byref(path))
    _check(rc, "tune_gemm")
    return PATH_NAMES[path.value]


def tune_conv(x, w, bias, y, strides=(1, 1), pads=(0, 0, 0, 0), dilations=(1, 1), act="tanh",
              workspace=None, reps: int = 20, stream=None) -> str:
    dims, dt = _conv_args(x, w, bias, y, strides, pads, dilations)
    ws, nbytes = _ws(workspace)
    path = ctypes.c_int(-1)
    rc = lib.biasact_tune_conv(_dev(x, "x"), _dev(w, "w"), _dev(bias, "bias"), _dev(y, "y"), *dims,
                               _i32x(strides, 2, "strides"), _i32x(pads, 4, "pads"),
                               _i32x(dilations, 2, "dilations"), dt, _act(act), ws, nbytes,
                               int(reps), _stream(stream), ctypes.byref(path))
    _check(rc, "tune_conv")
    return PATH_NAMES[path.value]


def gemm_bias_act_auto(A, B, bias, C, act="none", alpha: float = 0.0, workspace=None, stream=None):
    """The recorded path for this problem, else the library's static rule
    (the two-kernel path only with a large enough workspace)."""
    M, N, K, dt = _gemm_args(A, B, bias, C)
    ws, nbytes = _ws(workspace)
    rc = lib.gemm_bias_act_auto(_dev(A, "A"), _dev(B, "B"), _dev(bias, "bias"), _dev(C, "C"), M, N,
                                K, dt, _act(act), float(alpha), ws, nbytes, _stream(stream))
    _check(rc, "gemm_bias_act_auto")
    return C


def conv2d_bias_act_auto(x, w, bias, y, strides=(1, 1), pads=(0, 0, 0, 0), dilations=(1, 1),
                         act="tanh", workspace=None, stream=None):
    dims, dt = _conv_args(x, w, bias, y, strides, pads, dilations)
    ws, nbytes = _ws(workspace)
    rc = lib.conv2d_bias_act_auto(_dev(x, "x"), _dev(w, "w"), _dev(bias, "bias"), _dev(y, "y"),
                                  *dims, _i32x(strides, 2, "strides"), _i32x(pads, 4, "pads"),
                                  _i32x(dilations, 2, "dilations"), dt, _act(act), ws, nbytes,
                                  _stream(stream))
    _check(rc, "conv2d_bias_act_auto")
    return y


# -- MXFP4 ---------------------------------------------------------------------

def mxfp4_shapes(rows: int, K: int):
    """Shapes of the uint8 codes and scales of `rows` rows of K values."""
    g = -(-int(K) // 128)
    return (int(rows), 64 * g), (int(rows), 4 * g)


_U8 = None           # torch.uint8, set on first use


def _packed(codes, scales, name):
    """(rows, groups of 128 values per row) of an MXFP4 operand, checked."""
    global _U8
    if _U8 is None:
        _U8 = _torch().uint8
    shape = scales.shape
    if (len(shape) == 2 and codes.shape == (shape[0], 16 * shape[1]) and not shape[1] & 3
            and codes.dtype is _U8 and scales.dtype is _U8):
        return shape[0], shape[1] >> 2
    if codes.dtype is not _U8 or scales.dtype is not _U8:
        raise ValueError(f"{name}: codes and scales must be uint8")
    raise ValueError(f"{name}: codes must be [rows, 64 g] and scales [rows, 4 g], got "
                     f"{tuple(codes.shape)} and {tuple(shape)}")


def _mx_quant_args(X, codes, scales, axis, name):
    shape = X.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D")
    if axis == 1:
        rows, K = shape
    elif axis == 0:
        K, rows = shape
    else:
        raise ValueError("axis must be 0 or 1")
    if _packed(codes, scales, "mxfp4") != (rows, (K + 127) >> 7):
        raise ValueError(f"codes and scales must be {mxfp4_shapes(rows, K)}, got "
                         f"{tuple(codes.shape)} and {tuple(scales.shape)}")
    return rows, K, DTYPE_CODES[_tname(X)]


def mxfp4_quantize(X, codes, scales, axis: int = 1, stream=None):
    """Quantises X to MXFP4 with blocks of 32 along `axis`: the rows of
    X[rows, K] (axis 1) or the columns of X[K, rows] (axis 0).  codes and
    scales (uint8, mxfp4_shapes(rows, K)) are written and returned."""
    if stream is None and _native is not None:
        rc = _native.quantize(X, codes, scales, axis)
        if rc is True:
            return codes, scales
        if rc:                                   # the library's status; False: not called
            _check(rc, "mxfp4_quantize")
    rows, K, dt = _mx_quant_args(X, codes, scales, axis, "X")
    rc = lib.mxfp4_quantize(_dev(X, "X"), _dev(codes, "codes"), _dev(scales, "scales"), rows, K, axis,
                            dt, _stream(stream))
    if rc:
        _check(rc, "mxfp4_quantize")
    return codes, scales


def mxfp4_dequantize(codes, scales, Y, axis: int = 1, stream=None):
    """The values that codes and scales stand for, in Y's type and in Y's
    layout ([rows, K] with axis 1, [K, rows] with axis 0)."""
    if stream is None and _native is not None:
        rc = _native.dequantize(Y, codes, scales, axis)
        if rc is True:
            return Y
        if rc:
            _check(rc, "mxfp4_dequantize")
    rows, K, dt = _mx_quant_args(Y, codes, scales, axis, "Y")
    rc = lib.mxfp4_dequantize(_dev(codes, "codes"), _dev(scales, "scales"), _dev(Y, "Y"), rows, K, axis,
                              dt, _stream(stream))
    if rc:
        _check(rc, "mxfp4_dequantize")
    return Y


def _gemm_mx_args(A, a_scales, B, b_scales, bias, C):
    N, g = _packed(B, b_scales, "B")
    if a_scales is not None:
        M, ga = _packed(A, a_scales, "A")
        K, ta = 128 * ga, "mxfp4"
    elif A.dim() == 2:
        (M, K), ta = A.shape, _tname(A)
    else:
        raise ValueError("A must be 2-D")
    if (K + 127) >> 7 != g or C.shape != (M, N):
        raise ValueError(f"shape mismatch: A{tuple(A.shape)} B{tuple(B.shape)} C{tuple(C.shape)}")
    if bias is None:
        tb = None
    elif bias.numel() == N:
        tb = _tname(bias)
    else:
        raise ValueError(f"bias must have N = {N} elements")
    return M, N, K, dtypes_code(ta, "mxfp4", tb, _tname(C))


def gemm_mxfp4_bias_act(A, a_scales, B, b_scales, bias, C, act="none", alpha: float = 0.0, stream=None):
    """C = act(A @ B.T + bias), B in MXFP4 (codes and b_scales of its N rows);
    A in MXFP4 (codes and a_scales), or fp16 / bf16 with a_scales None."""
    if stream is None and _native is not None:
        rc = _native.gemm(A, a_scales, B, b_scales, bias, None, C, act, alpha)
        if rc is True:
            return C
        if rc:
            _check(rc, "gemm_mxfp4_bias_act")
    M, N, K, dt = _gemm_mx_args(A, a_scales, B, b_scales, bias, C)
    rc = lib.gemm_mxfp4_bias_act(_dev(A, "A"), _dev(a_scales, "a_scales"), _dev(B, "B"),
                                 _dev(b_scales, "b_scales"), _dev(bias, "bias"), _dev(C, "C"), M, N, K, dt,
                                 _act(act), float(alpha), _stream(stream))
    if rc:
        _check(rc, "gemm_mxfp4_bias_act")
    return C


def gemm_mxfp4_bias_add_act(A, a_scales, B, b_scales, bias, R, C, act="none", alpha: float = 0.0,
                            stream=None):
    """C = act(A @ B.T + bias + R); R like C (may be C itself)."""
    if stream is None and _native is not None and R is not None:
        rc = _native.gemm(A, a_scales, B, b_scales, bias, R, C, act, alpha)
        if rc is True:
            return C
        if rc:
            _check(rc, "gemm_mxfp4_bias_add_act")
    M, N, K, dt = _gemm_mx_args(A, a_scales, B, b_scales, bias, C)
    rc = lib.gemm_mxfp4_bias_add_act(_dev(A, "A"), _dev(a_scales, "a_scales"), _dev(B, "B"),
                                     _dev(b_scales, "b_scales"), _dev(bias, "bias"), _residual(R, C),
                                     _dev(C, "C"), M, N, K, dt, _act(act), float(alpha), _stream(stream))
    if rc:
        _check(rc, "gemm_mxfp4_bias_add_act")
    return C


# -- tile configs ------------------------------------------------------------

def num_tile_configs() -> int:
    return int(lib.biasact_num_tile_configs())


def tile_config_name(i: int) -> str:
    buf = ctypes.create_string_buffer(64)
    _check(lib.biasact_tile_config_name(i, buf, 64), "tile_config_name")
    return buf.value.decode()


def gemm_tile_config(M, N, K, dtypes: int) -> int:
    return int(lib.biasact_gemm_tile_config(M, N, K, dtypes))


def conv_tile_config(N, Co, Ho, Wo, K, dtypes: int) -> int:
    return int(lib.biasact_conv_tile_config(N, Co, Ho, Wo, K, dtypes))


def force_tile_config(i: int):
    _check(lib.biasact_force_tile_config(int(i)), "force_tile_config")


def last_tile_config() -> str:
    """The kernel and tile the calling thread's last launching call queued."""
    buf = ctypes.create_string_buffer(128)
    _check(lib.biasact_last_tile_config(buf, len(buf)), "last_tile_config")
    return buf.value.decode()


def force_halo_variant(v: int):
    """-1 automatic; 0 widest conv-halo tile; 1, 2 the two-per-CU variants; 3, 4 eight waves."""
    _check(lib.biasact_force_halo_variant(int(v)), "force_halo_variant")
