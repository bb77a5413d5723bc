"""ctypes binding of libharp.so (include/harp.h).

Argument marshalling, and for the 8-bit operators checks of the tensors: every
step of the path runs in the library's HIP kernels.  torch is used for device memory and the current stream.  The
functions carry the C names; tensors are passed by ``data_ptr()`` on
``torch.cuda.current_stream()`` unless a stream handle is given.

If libharp.so is missing this module raises on import: there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import c_char_p, c_float, c_int32, c_size_t, c_void_p

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libharp.so")

HARP_OK = 0
HARP_ERR_NULL = 1
HARP_ERR_SHAPE = 2
HARP_ERR_DTYPE = 3
HARP_ERR_ALIGN = 4
HARP_ERR_WORKSPACE = 5
HARP_ERR_UNSUPPORTED = 6
HARP_ERR_HIP = 7

HARP_F32 = 0
HARP_BF16 = 1

EXPORTED = (
    "harp_rotate_in", "harp_rotate_out", "harp_deq_gemv", "harp_deq_gemv_ws",
    "harp_deq_gemv_workspace_bytes", "harp_rotate_in_deq_gemv",
    "harp_deq_gemm",
    "harp_deq_gemm_workspace_bytes", "harp_linear_workspace_bytes", "harp_linear_fused",
    "harp_linear_fused_noalloc", "harp_linear_chain", "harp_linear_chain_workspace_bytes",
    "harp_dequant",
    "harp_rotate_weight", "harp_rotate_weight_workspace_bytes", "harp_quantize_pack",
    "harp_mixed_expand", "harp_rotate_in_mixed", "harp_rotate_out_mixed",
    "harp_rotate_mixed_workspace_bytes",
    "harp_linear_fused_mixed", "harp_linear_mixed_workspace_bytes",
    "harp_rmsnorm", "harp_rmsnorm_fp8", "harp_silu_mul_fp8", "harp_fp8_gemm",
    "harp_fp8_gemm_grouped",
    "harp_status_string", "harp_last_hip_error",
)


class HarpError(RuntimeError):
    def __init__(self, status: int, where: str, hip_error: int = 0):
        self.status = status
        self.hip_error = hip_error
        msg = f"{where}: {status_string(status)}"
        if status == HARP_ERR_HIP:
            msg += f" (hipError_t {hip_error})"
        super().__init__(msg)


class harp_rotation(ctypes.Structure):
    _fields_ = [("dim", c_int32), ("block", c_int32),
                ("cs", c_void_p), ("sign_bits", c_void_p),
                ("phi_codes", c_void_p), ("phi_step", c_float)]


HARP_MAX_STAGES = 16


class harp_mixed_rotation(ctypes.Structure):
    _fields_ = [("dim", c_int32), ("n_stages", c_int32), ("radix", c_int32 * HARP_MAX_STAGES),
                ("blocks", c_void_p), ("sign_bits", c_void_p)]


class harp_qweight(ctypes.Structure):
    _fields_ = [("N", c_int32), ("K", c_int32), ("bits", c_int32),
                ("group", c_int32), ("qweight", c_void_p), ("scale", c_void_p),
                ("zero", c_void_p)]


class harp_fp8_weight(ctypes.Structure):
    _fields_ = [("N", c_int32), ("K", c_int32), ("experts", c_int32), ("w", c_void_p),
                ("scale", c_void_p)]


class harp_chain_layer(ctypes.Structure):
    _fields_ = [("V", harp_rotation), ("W", harp_qweight), ("U", harp_rotation),
                ("y", c_void_p)]


def _load() -> ctypes.CDLL:
    # torch first: its bundled HIP runtime (soname libamdhip64.so.7) must be
    # the one loaded, so that torch's streams and allocations and this
    # library's kernels live in a single runtime.
    import torch  # noqa: F401
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; run `python rotated_bit_amd/build.py` "
            "(or __graft_entry__.build()). There is no fallback path.")
    lib = ctypes.CDLL(LIB_PATH)
    R = ctypes.POINTER(harp_rotation)
    Q = ctypes.POINTER(harp_qweight)
    MR = ctypes.POINTER(harp_mixed_rotation)
    F8 = ctypes.POINTER(harp_fp8_weight)
    sig = {
        "harp_rotate_in": (c_int32, [R, c_void_p, c_int32, c_void_p, c_int32, c_int32, c_void_p]),
        "harp_rotate_out": (c_int32, [R, c_void_p, c_void_p, c_int32, c_int32, c_void_p]),
        "harp_deq_gemv": (c_int32, [Q, c_void_p, c_void_p, c_int32, c_void_p]),
        "harp_deq_gemv_ws": (c_int32, [Q, c_void_p, c_void_p, c_int32, c_void_p, c_size_t,
                                       c_void_p]),
        "harp_deq_gemv_workspace_bytes": (c_size_t, [c_int32, c_int32, c_int32]),
        "harp_rotate_in_deq_gemv": (c_int32, [R, Q, c_void_p, c_int32, c_void_p, c_int32,
                                               c_void_p]),
        "harp_deq_gemm": (c_int32, [Q, c_void_p, c_void_p, c_int32, c_void_p, c_size_t,
                                    c_void_p]),
        "harp_deq_gemm_workspace_bytes": (c_size_t, [c_int32, c_int32, c_int32]),
        "harp_linear_workspace_bytes": (c_size_t, [c_int32, c_int32, c_int32]),
        "harp_linear_fused": (c_int32, [R, Q, R, c_void_p, c_int32, c_void_p, c_int32,
                                        c_int32, c_void_p, c_size_t, c_void_p]),
        "harp_linear_fused_noalloc": (c_int32, [R, Q, R, c_void_p, c_int32, c_void_p, c_int32,
                                                c_int32, c_void_p]),
        "harp_linear_chain": (c_int32, [ctypes.POINTER(harp_chain_layer), c_int32, c_void_p,
                                        c_int32, c_int32, c_int32, c_void_p, c_size_t,
                                        c_void_p]),
        "harp_linear_chain_workspace_bytes": (c_size_t, [c_int32]),
        "harp_dequant": (c_int32, [Q, c_void_p, c_int32, c_void_p]),
        "harp_rotate_weight": (c_int32, [R, R, c_void_p, c_void_p, c_int32, c_int32, c_void_p,
                                          c_size_t, c_void_p]),
        "harp_rotate_weight_workspace_bytes": (c_size_t, [c_int32, c_int32]),
        "harp_mixed_expand": (c_int32, [c_int32, c_void_p, c_void_p, c_void_p, c_void_p]),
        "harp_rotate_in_mixed": (c_int32, [MR, c_void_p, c_int32, c_void_p, c_int32, c_int32,
                                            c_void_p, c_size_t, c_void_p]),
        "harp_rotate_out_mixed": (c_int32, [MR, c_void_p, c_void_p, c_int32, c_int32, c_void_p,
                                             c_size_t, c_void_p]),
        "harp_rotate_mixed_workspace_bytes": (c_size_t, [c_int32, c_int32, c_int32]),
        "harp_linear_fused_mixed": (c_int32, [MR, Q, MR, c_void_p, c_int32, c_void_p, c_int32,
                                              c_int32, c_void_p, c_size_t, c_void_p]),
        "harp_linear_mixed_workspace_bytes": (c_size_t, [c_int32, c_int32, c_int32]),
        "harp_quantize_pack": (c_int32, [c_void_p, c_int32, c_int32, c_int32, c_void_p, c_void_p,
                                          c_void_p, c_void_p]),
        "harp_rmsnorm": (c_int32, [c_void_p, c_int32, c_void_p, c_void_p, c_void_p, c_int32,
                                   c_float, c_void_p, c_int32, c_int32, c_int32, c_void_p]),
        "harp_rmsnorm_fp8": (c_int32, [c_void_p, c_int32, c_void_p, c_void_p, c_void_p, c_int32,
                                       c_float, c_void_p, c_void_p, c_int32, c_int32,
                                       c_void_p]),
        "harp_silu_mul_fp8": (c_int32, [c_void_p, c_int32, c_void_p, c_void_p, c_int32, c_int32,
                                        c_void_p]),
        "harp_fp8_gemm": (c_int32, [F8, c_void_p, c_void_p, c_void_p, c_int32, c_int32,
                                    c_void_p]),
        "harp_fp8_gemm_grouped": (c_int32, [F8, c_void_p, c_void_p, c_int32, c_void_p, c_void_p,
                                            c_void_p, c_int32, c_int32, c_void_p]),
        "harp_status_string": (c_char_p, [c_int32]),
        "harp_last_hip_error": (c_int32, []),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


lib = _load()


def status_string(status: int) -> str:
    return lib.harp_status_string(status).decode()


# ---------------------------------------------------------------------------
# torch-facing marshalling
# ---------------------------------------------------------------------------

def _torch():
    import torch
    return torch


def _ptr(t):
    return None if t is None else c_void_p(t.data_ptr())


def _dtype_of(dtype) -> int:
    torch = _torch()
    if dtype == torch.float32:
        return HARP_F32
    if dtype == torch.bfloat16:
        return HARP_BF16
    raise TypeError(f"unsupported dtype {dtype} (float32 or bfloat16)")


def _dtype_code(t) -> int:
    return _dtype_of(t.dtype)


def _stream(stream):
    if stream is None:
        return c_void_p(_torch().cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return c_void_p(stream)
    return c_void_p(stream.cuda_stream)


def _check(status: int, where: str):
    if status != HARP_OK:
        raise HarpError(status, where, lib.harp_last_hip_error())


class Rotation:
    """One side: sign_bits int32/uint32 [ceil(dim/32)] and the angles, either
    cs float32 [dim/b][log2 b][b/2][2] (cos t, sin t) or, with cs None,
    phi_codes int8 [dim/b][log2 b][b/2] and phi_step (t = pi/4 + code*step)."""

    def __init__(self, cs, sign_bits, dim: int, block: int, phi_codes=None,
                 phi_step: float = 0.0):
        self.cs, self.sign_bits, self.dim, self.block = cs, sign_bits, dim, block
        self.phi_codes, self.phi_step = phi_codes, phi_step
        self.c = harp_rotation(dim, block, None if cs is None else cs.data_ptr(),
                               sign_bits.data_ptr(),
                               None if phi_codes is None else phi_codes.data_ptr(),
                               float(phi_step))


class MixedRotation:
    """A mixed-radix side: blocks float32 (stages concatenated, stage t
    [dim/b_t][b_t][b_t] row-major), sign_bits int32/uint32 [ceil(dim/32)]."""

    def __init__(self, blocks, sign_bits, radices):
        radices = [int(b) for b in radices]
        if len(radices) > HARP_MAX_STAGES:
            raise ValueError("too many stages")
        self.blocks, self.sign_bits, self.radices = blocks, sign_bits, radices
        self.dim = 1
        for b in radices:
            self.dim *= b
        arr = (c_int32 * HARP_MAX_STAGES)(*(radices + [0] * (HARP_MAX_STAGES - len(radices))))
        self.c = harp_mixed_rotation(self.dim, len(radices), arr, blocks.data_ptr(),
                                     sign_bits.data_ptr())


class QWeight:
    """Packed weight: qweight int32 [N][K*bits/32], scale/zero int16 or fp16 [N][K/64]."""

    def __init__(self, qweight, scale, zero, N: int, K: int, bits: int, group: int = 64):
        self.qweight, self.scale, self.zero = qweight, scale, zero
        self.N, self.K, self.bits, self.group = N, K, bits, group
        self.c = harp_qweight(N, K, bits, group, qweight.data_ptr(),
                              scale.data_ptr(), zero.data_ptr())


def harp_rotate_in(V: Rotation, x, xt, M: int | None = None, stream=None) -> None:
    M = x.shape[0] if M is None else M
    _check(lib.harp_rotate_in(ctypes.byref(V.c), _ptr(x), _dtype_code(x), _ptr(xt),
                              _dtype_code(xt), M, _stream(stream)), "harp_rotate_in")


def harp_rotate_out(U: Rotation, yt, y, M: int | None = None, stream=None) -> None:
    M = yt.shape[0] if M is None else M
    _check(lib.harp_rotate_out(ctypes.byref(U.c), _ptr(yt), _ptr(y), _dtype_code(y), M,
                               _stream(stream)), "harp_rotate_out")


def harp_deq_gemv(W: QWeight, xt, yt, M: int | None = None, stream=None) -> None:
    M = xt.shape[0] if M is None else M
    _check(lib.harp_deq_gemv(ctypes.byref(W.c), _ptr(xt), _ptr(yt), M, _stream(stream)),
           "harp_deq_gemv")


def harp_deq_gemv_ws(W: QWeight, xt, yt, workspace=None, M: int | None = None,
                     stream=None) -> None:
    M = xt.shape[0] if M is None else M
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.harp_deq_gemv_ws(ctypes.byref(W.c), _ptr(xt), _ptr(yt), M, _ptr(workspace),
                                ws_bytes, _stream(stream)), "harp_deq_gemv_ws")


def harp_deq_gemv_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib.harp_deq_gemv_workspace_bytes(M, N, K))


def harp_rotate_in_deq_gemv(V: Rotation, W: QWeight, x, yt, M: int | None = None,
                            stream=None) -> None:
    M = x.shape[0] if M is None else M
    _check(lib.harp_rotate_in_deq_gemv(ctypes.byref(V.c), ctypes.byref(W.c), _ptr(x),
                                       _dtype_code(x), _ptr(yt), M, _stream(stream)),
           "harp_rotate_in_deq_gemv")


def harp_deq_gemm(W: QWeight, xt_bf16, yt, workspace=None, M: int | None = None,
                  stream=None) -> None:
    M = xt_bf16.shape[0] if M is None else M
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.harp_deq_gemm(ctypes.byref(W.c), _ptr(xt_bf16), _ptr(yt), M,
                             _ptr(workspace), ws_bytes, _stream(stream)), "harp_deq_gemm")


def harp_deq_gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib.harp_deq_gemm_workspace_bytes(M, N, K))


def harp_linear_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib.harp_linear_workspace_bytes(M, N, K))


def harp_linear_fused(V: Rotation, W: QWeight, U: Rotation, x, y, workspace,
                      M: int | None = None, stream=None) -> None:
    M = x.shape[0] if M is None else M
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.harp_linear_fused(ctypes.byref(V.c), ctypes.byref(W.c), ctypes.byref(U.c),
                                 _ptr(x), _dtype_code(x), _ptr(y), _dtype_code(y), M,
                                 _ptr(workspace), ws_bytes, _stream(stream)),
           "harp_linear_fused")


def harp_linear_fused_noalloc(V: Rotation, W: QWeight, U: Rotation, x, y,
                              M: int | None = None, stream=None) -> None:
    M = x.shape[0] if M is None else M
    _check(lib.harp_linear_fused_noalloc(ctypes.byref(V.c), ctypes.byref(W.c), ctypes.byref(U.c),
                                         _ptr(x), _dtype_code(x), _ptr(y), _dtype_code(y), M,
                                         _stream(stream)),
           "harp_linear_fused_noalloc")


def harp_linear_chain_workspace_bytes(dim: int) -> int:
    return int(lib.harp_linear_chain_workspace_bytes(dim))


def harp_linear_chain(layers, x, workspace, M: int | None = None, stream=None) -> None:
    """layers: sequence of (V, W, U, y) with y the layer's output tensor
    [M][dim] (float32 or bfloat16, the same for every layer)."""
    layers = list(layers)
    M = x.shape[0] if M is None else M
    arr = (harp_chain_layer * max(1, len(layers)))()
    y_dt = HARP_F32
    for i, (V, W, U, y) in enumerate(layers):
        arr[i] = harp_chain_layer(V.c, W.c, U.c, y.data_ptr())
        y_dt = _dtype_code(y)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.harp_linear_chain(arr, len(layers), _ptr(x), _dtype_code(x), y_dt, M,
                                 _ptr(workspace), ws_bytes, _stream(stream)),
           "harp_linear_chain")


def harp_dequant(W: QWeight, out, stream=None) -> None:
    _check(lib.harp_dequant(ctypes.byref(W.c), _ptr(out), _dtype_code(out), _stream(stream)),
           "harp_dequant")


def _ws(workspace):
    if workspace is None:
        return None, 0
    return _ptr(workspace), workspace.numel() * workspace.element_size()


def harp_rotate_mixed_workspace_bytes(dim: int, M: int, out_dtype) -> int:
    return int(lib.harp_rotate_mixed_workspace_bytes(dim, M, _dtype_of(out_dtype)))


def harp_mixed_expand(radices, params, gaussians=None):
    """Host expansion of a mixed-radix side (numpy in, numpy out).

    params: per stage an array of shape (dim / b_t, b_t (b_t - 1) / 2);
    gaussians: per stage a (b_t, b_t) array for radices that are not powers
    of two (None entries, or None, for powers of two).  Returns the float32
    blocks, stages concatenated, ready for MixedRotation.
    """
    import numpy as np
    radices = [int(b) for b in radices]
    dim = 1
    for b in radices:
        dim *= b
    rad = np.ascontiguousarray(radices, dtype=np.int32)
    p = np.ascontiguousarray(np.concatenate([np.asarray(a, dtype=np.float64).ravel()
                                             for a in params]))
    gl = [np.asarray(g, dtype=np.float64).ravel()
          for g, b in zip(gaussians or [None] * len(radices), radices)
          if b & (b - 1) and g is not None]
    g = np.ascontiguousarray(np.concatenate(gl)) if gl else None
    out = np.empty(dim * sum(radices), dtype=np.float32)
    _check(lib.harp_mixed_expand(len(radices), rad.ctypes.data, p.ctypes.data,
                                 None if g is None else g.ctypes.data, out.ctypes.data),
           "harp_mixed_expand")
    return out


def harp_rotate_in_mixed(R: MixedRotation, x, xt, workspace=None, M: int | None = None,
                         stream=None) -> None:
    M = x.shape[0] if M is None else M
    wp, wb = _ws(workspace)
    _check(lib.harp_rotate_in_mixed(ctypes.byref(R.c), _ptr(x), _dtype_code(x), _ptr(xt),
                                    _dtype_code(xt), M, wp, wb, _stream(stream)),
           "harp_rotate_in_mixed")


def harp_rotate_out_mixed(R: MixedRotation, yt, y, workspace=None, M: int | None = None,
                          stream=None) -> None:
    M = yt.shape[0] if M is None else M
    wp, wb = _ws(workspace)
    _check(lib.harp_rotate_out_mixed(ctypes.byref(R.c), _ptr(yt), _ptr(y), _dtype_code(y), M,
                                     wp, wb, _stream(stream)), "harp_rotate_out_mixed")


def harp_linear_mixed_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib.harp_linear_mixed_workspace_bytes(M, N, K))


def harp_linear_fused_mixed(V: MixedRotation, W: QWeight, U: MixedRotation, x, y, workspace,
                            M: int | None = None, stream=None) -> None:
    M = x.shape[0] if M is None else M
    wp, wb = _ws(workspace)
    _check(lib.harp_linear_fused_mixed(ctypes.byref(V.c), ctypes.byref(W.c), ctypes.byref(U.c),
                                       _ptr(x), _dtype_code(x), _ptr(y), _dtype_code(y), M,
                                       wp, wb, _stream(stream)), "harp_linear_fused_mixed")


def harp_rotate_weight_workspace_bytes(N: int, K: int) -> int:
    return int(lib.harp_rotate_weight_workspace_bytes(N, K))


def harp_rotate_weight(V: Rotation, U: Rotation, W, Wp, workspace, stream=None) -> None:
    """Wp = F_U W F_V^T for W, Wp float32 [N][K]."""
    N, K = W.shape
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.harp_rotate_weight(ctypes.byref(V.c), ctypes.byref(U.c), _ptr(W), _ptr(Wp), N, K,
                                  _ptr(workspace), ws_bytes, _stream(stream)),
           "harp_rotate_weight")


def harp_quantize_pack(Wp, bits: int, qweight, scale, zero, stream=None) -> None:
    """Quantize float32 Wp [N][K] into qweight [N][K*bits/32] and fp16-bit
    scale / zero [N][K/64] (int32 / int16 tensors)."""
    N, K = Wp.shape
    _check(lib.harp_quantize_pack(_ptr(Wp), N, K, bits, _ptr(qweight), _ptr(scale), _ptr(zero),
                                  _stream(stream)), "harp_quantize_pack")


# 8-bit operators.  Their tensors are checked here as well (device, type,
# shape, contiguous rows): the C entry points see plain addresses.  A call
# at decode sizes takes 2 to 6 us on the GPU and its launch 3 us on the host,
# so the checks are one expression per tensor, only a tensor that fails one
# is looked at for the message, and the handle of the current stream is read
# without a Stream object around it (torch.cuda.current_stream(): 2.7 us).

def _runs(n: int) -> int:
    return (n + 127) >> 7


def _reject(name: str, t, shape, dtypes, index):
    """Raises for a tensor that is not what its call needs."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: not contiguous")
    if index < 0:
        raise ValueError(f"{name}: expected tensors on a GPU")
    raise ValueError(f"{name}: on {t.device}, expected GPU {index}")


def _expect(name: str, t, shape, dtypes, index):
    if not (t.shape == shape and t.dtype in dtypes and t.is_contiguous()
            and t.get_device() == index):
        _reject(name, t, shape, dtypes, index)


def _accessors():
    torch = _torch()
    device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                     lambda index: torch.cuda.current_stream(index).cuda_stream)
    return (device, stream, {torch.float32: HARP_F32, torch.bfloat16: HARP_BF16},
            (torch.float8_e4m3fn, torch.uint8), (torch.float32,), (torch.int32,))


_current_device, _current_stream, _FLOATS, _CODES, _F32, _I32 = _accessors()


def _call(where, f, index, stream, args):
    """f on the tensors' device (made current for the call) and stream."""
    if index < 0:
        raise ValueError(f"{where}: expected tensors on a GPU")
    if stream is None:
        stream = _current_stream(index)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if index == _current_device():
        status = f(*args, stream)
    else:
        with _torch().cuda.device(index):
            status = f(*args, stream)
    if status != HARP_OK:
        _check(status, where)


class FP8Weight:
    """e4m3 weight: w float8_e4m3fn (or uint8 codes) [N][K] or [experts][N][K]
    and scale float32 [ceil(N/128)][ceil(K/128)], with experts in front where
    w has them."""

    def __init__(self, w, scale):
        if w.dim() not in (2, 3):
            raise ValueError("w: [N][K] or [experts][N][K]")
        self.experts = w.shape[0] if w.dim() == 3 else 1
        self.N, self.K = w.shape[-2:]
        self.runs = _runs(self.K)
        self.index = w.get_device()
        _expect("w", w, w.shape, _CODES, self.index)
        _expect("scale", scale, (*w.shape[:-2], _runs(self.N), self.runs), _F32, self.index)
        self.w, self.scale = w, scale
        self.c = harp_fp8_weight(self.N, self.K, self.experts, w.data_ptr(), scale.data_ptr())
        self.ref = ctypes.byref(self.c)


def _norm_inputs(x, weight, residual, residual_out):
    """(M, D, x's device, its first six arguments of the C call)."""
    shape, index, dtype = x.shape, x.get_device(), x.dtype
    if len(shape) != 2:
        raise ValueError("x: [M][D]")
    if not (dtype in _FLOATS and x.is_contiguous()):
        _reject("x", x, shape, _FLOATS, index)
    M, D = shape
    if not (weight.shape == (D,) and weight.dtype in _FLOATS and weight.is_contiguous()
            and weight.get_device() == index):
        _reject("weight", weight, (D,), _FLOATS, index)
    r = ro = None
    if residual is not None:
        if not (residual.shape == shape and residual.dtype == dtype
                and residual.is_contiguous() and residual.get_device() == index):
            _reject("residual", residual, shape, (dtype,), index)
        r = residual.data_ptr()
    if residual_out is not None:
        if not (residual_out.shape == shape and residual_out.dtype == dtype
                and residual_out.is_contiguous() and residual_out.get_device() == index):
            _reject("residual_out", residual_out, shape, (dtype,), index)
        ro = residual_out.data_ptr()
    return M, D, index, (x.data_ptr(), _FLOATS[dtype], r, ro, weight.data_ptr(),
                         _FLOATS[weight.dtype])


def harp_rmsnorm(x, weight, y, eps: float = 1e-6, residual=None, residual_out=None,
                 stream=None) -> None:
    """y = norm(x + residual) * weight for x [M][D], and residual_out = x + residual."""
    M, D, index, args = _norm_inputs(x, weight, residual, residual_out)
    _expect("y", y, (M, D), _FLOATS, index)
    _call("harp_rmsnorm", lib.harp_rmsnorm, index, stream,
          (*args, eps, y.data_ptr(), _FLOATS[y.dtype], M, D))


def harp_rmsnorm_fp8(x, weight, q, q_scale, eps: float = 1e-6, residual=None, residual_out=None,
                     stream=None) -> None:
    """harp_rmsnorm with its output as codes q [M][D] and q_scale [M][ceil(D/128)]."""
    M, D, index, args = _norm_inputs(x, weight, residual, residual_out)
    _expect("q", q, (M, D), _CODES, index)
    _expect("q_scale", q_scale, (M, (D + 127) >> 7), _F32, index)
    _call("harp_rmsnorm_fp8", lib.harp_rmsnorm_fp8, index, stream,
          (*args, eps, q.data_ptr(), q_scale.data_ptr(), M, D))


def harp_silu_mul_fp8(gate_up, q, q_scale, stream=None) -> None:
    """Codes of silu(gate) * up for gate_up [M][2 D] (gates first)."""
    M, D = q.shape
    index = q.get_device()
    _expect("q", q, (M, D), _CODES, index)
    _expect("gate_up", gate_up, (M, 2 * D), _FLOATS, index)
    _expect("q_scale", q_scale, (M, (D + 127) >> 7), _F32, index)
    _call("harp_silu_mul_fp8", lib.harp_silu_mul_fp8, index, stream,
          (gate_up.data_ptr(), _FLOATS[gate_up.dtype], q.data_ptr(), q_scale.data_ptr(), M, D))


def harp_fp8_gemm(W: FP8Weight, a, a_scale, y, stream=None) -> None:
    """y [M][N] = W a for codes a [M][K] with a_scale [M][ceil(K/128)]."""
    M, index = a.shape[0], W.index
    _expect("a", a, (M, W.K), _CODES, index)
    _expect("a_scale", a_scale, (M, W.runs), _F32, index)
    _expect("y", y, (M, W.N), _FLOATS, index)
    _call("harp_fp8_gemm", lib.harp_fp8_gemm, index, stream,
          (W.ref, a.data_ptr(), a_scale.data_ptr(), y.data_ptr(), _FLOATS[y.dtype], M))


def harp_fp8_gemm_grouped(W: FP8Weight, a, a_scale, offsets, y, rows=None, stream=None) -> None:
    """y[i] = W_e a[rows[i]] for offsets[e] <= i < offsets[e + 1] (int32 device tensors)."""
    a_rows, M, index = a.shape[0], y.shape[0], W.index
    _expect("a", a, (a_rows, W.K), _CODES, index)
    _expect("a_scale", a_scale, (a_rows, W.runs), _F32, index)
    _expect("offsets", offsets, (W.experts + 1,), _I32, index)
    _expect("y", y, (M, W.N), _FLOATS, index)
    r = None
    if rows is not None:
        _expect("rows", rows, (M,), _I32, index)
        r = rows.data_ptr()
    _call("harp_fp8_gemm_grouped", lib.harp_fp8_gemm_grouped, index, stream,
          (W.ref, a.data_ptr(), a_scale.data_ptr(), a_rows, r, offsets.data_ptr(),
           y.data_ptr(), _FLOATS[y.dtype], M))


def harp_last_hip_error() -> int:
    return int(lib.harp_last_hip_error())
