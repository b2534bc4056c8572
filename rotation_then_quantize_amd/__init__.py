"""Python binding of librtq, the MI355X (gfx950) rotate-then-quantize linear layer.

Argument marshalling only: every step of the computation runs in librtq's HIP kernels behind the
C ABI declared in ``include/rtq.h``.  torch supplies device memory and the current stream.  There
is no CPU or PyTorch fallback: if ``librtq.so`` is missing, every call raises.

The method (OrbitQuant article, hotelren.com/news/3376620, sections 2.1-2.3): weights are rotated
offline, W' = W Pi^T, and quantised per row; activations are rotated online, x' = Pi x, quantised
per token and multiplied against the quantised weights, where Pi^T Pi = I cancels.
"""
from __future__ import annotations

import ctypes
import functools
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "librtq.so")

RTQ_OK, RTQ_ERR_INVALID_ARG, RTQ_ERR_UNSUPPORTED, RTQ_ERR_MISALIGNED, RTQ_ERR_HIP = 0, -1, -2, -3, -4
RTQ_F32, RTQ_BF16, RTQ_I32 = 0, 1, 2
RTQ_E4M3, RTQ_E5M2, RTQ_E8M0 = 3, 4, 5
RTQ_FP8_ROWS, RTQ_FP8_BLOCKS = 0, 1
RTQ_ACT_GELU_TANH, RTQ_ACT_GELU, RTQ_ACT_SILU = 1, 2, 3
FP8_BLOCK = 128   # elements per scale of 8-bit floating point codes
RTQ_INT8, RTQ_CODEBOOK, RTQ_CODEBOOK_I8, RTQ_INT8_TILED = 0, 1, 2, 3
RTQ_CODEBOOK_TILED, RTQ_CODEBOOK_I8_TILED = 4, 5
TILE_ROWS, TILE_K = 256, 64   # the tiled layouts: 256-row tiles, K slices of 64 elements
_CODEBOOK_MODES = (RTQ_CODEBOOK, RTQ_CODEBOOK_I8, RTQ_CODEBOOK_TILED, RTQ_CODEBOOK_I8_TILED)


def tiled_rows(rows: int) -> int:
    """Rows a codes buffer in a tiled layout holds (rows padded to a multiple of 256)."""
    return -(-rows // TILE_ROWS) * TILE_ROWS


def tiled_code_bytes(rows: int, d: int, mode: int, bits: int = 8) -> int:
    """Bytes of a codes buffer in the tiled layout of `mode` (0 for the row-major modes)."""
    if mode in (RTQ_INT8_TILED, RTQ_CODEBOOK_I8_TILED):
        return tiled_rows(rows) * d
    if mode == RTQ_CODEBOOK_TILED:
        return tiled_rows(rows) * d * bits // 8
    return 0

EXPORTS = ("rtq_rpbh_make", "rtq_lloyd_max", "rtq_rpbh_rotate", "rtq_quantize_rows", "rtq_qgemm",
           "rtq_qgemm_ws", "rtq_qgemm_workspace", "rtq_rotated_qlinear", "rtq_rotated_qlinear_workspace",
           "rtq_quantize_rows_asym", "rtq_qgemm_asym", "rtq_rotated_qlinear_asym",
           "rtq_rotated_qlinear_asym_workspace", "rtq_rotated_qlinear_noalloc", "rtq_fp8_quantize",
           "rtq_fp8_dequantize", "rtq_fp8_qgemm", "rtq_fp8_qgemm_workspace", "rtq_fp8_dgrad",
           "rtq_fp8_dgrad_workspace", "rtq_fp8_linear", "rtq_fp8_linear_workspace", "rtq_fp8_linear_dgrad",
           "rtq_fp8_linear_dgrad_workspace", "rtq_fp8_wgrad", "rtq_fp8_wgrad_workspace", "rtq_act_fp8_forward",
           "rtq_act_fp8_backward", "rtq_rmsnorm_forward", "rtq_rmsnorm_backward", "rtq_rmsnorm_backward_workspace",
           "rtq_fp8_glu", "rtq_fp8_glu_workspace", "rtq_glu_fp8_backward", "rtq_grad_norm", "rtq_grad_norm_workspace",
           "rtq_grad_clip", "rtq_last_error")

NOALLOC_SCRATCH_BYTES = 96 << 20   # RTQ_NOALLOC_SCRATCH_BYTES


class RtqError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"librtq status {status}: {message}")
        self.status = status


class _Rpbh(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("h", ctypes.c_int32), ("perm", ctypes.c_void_p), ("signs", ctypes.c_void_p)]


class _Tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("n", ctypes.c_int64), ("type", ctypes.c_int)]


class _Codebook(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int32), ("centroids", ctypes.c_void_p), ("boundaries", ctypes.c_void_p)]


_lib = None


def load_library():
    """Load librtq.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                           f"(hipcc --offload-arch=gfx950); there is no fallback path")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, u64, f32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64,
                                  ctypes.c_float, ctypes.c_size_t)
    R = ctypes.POINTER(_Rpbh)
    C = ctypes.POINTER(_Codebook)
    lib.rtq_rpbh_make.argtypes = [u64, i32, i32, vp, vp]
    lib.rtq_lloyd_max.argtypes = [i32, i32, vp, vp]
    lib.rtq_rpbh_rotate.argtypes = [vp, i32, vp, i32, i64, R, i32, vp]
    lib.rtq_quantize_rows.argtypes = [vp, i32, i64, i32, R, i32, C, f32, vp, vp, i32, vp]
    lib.rtq_qgemm.argtypes = [vp, vp, i64, vp, vp, i32, i64, i32, i32, C, C, vp, i32, vp]
    lib.rtq_qgemm_ws.argtypes = [vp, vp, i64, vp, vp, i32, i64, i32, i32, C, C, vp, i32, vp, sz, vp]
    lib.rtq_qgemm_workspace.argtypes = []
    lib.rtq_qgemm_workspace.restype = sz
    lib.rtq_rotated_qlinear.argtypes = [vp, i32, i64, R, vp, vp, i32, i64, i32, C, C, vp, i32, vp, sz, vp]
    lib.rtq_rotated_qlinear_noalloc.argtypes = [vp, i32, i64, R, vp, vp, i32, i64, i32, C, C, vp, i32, vp]
    lib.rtq_rotated_qlinear_workspace.argtypes = [i64, i32, i32, i32]
    lib.rtq_rotated_qlinear_workspace.restype = sz
    lib.rtq_quantize_rows_asym.argtypes = [vp, i32, i64, i32, R, vp, vp, i32, vp, vp, vp]
    lib.rtq_qgemm_asym.argtypes = [vp, vp, vp, vp, i64, vp, vp, i32, vp, vp, i64, i32, vp, i32, vp, sz, vp]
    lib.rtq_rotated_qlinear_asym.argtypes = [vp, i32, i64, R, vp, vp, i32, vp, vp, i64, vp, i32, vp, sz, vp]
    lib.rtq_rotated_qlinear_asym_workspace.argtypes = [i64, i32]
    lib.rtq_rotated_qlinear_asym_workspace.restype = sz
    lib.rtq_fp8_quantize.argtypes = [vp, i32, i64, i32, i32, vp, i32, vp, i32, vp]
    lib.rtq_fp8_dequantize.argtypes = [vp, i32, vp, i32, i64, i32, i32, vp, i32, vp]
    lib.rtq_fp8_qgemm.argtypes = [vp, i32, vp, i64, vp, vp, i32, i64, i32, vp, i32, vp, sz, vp]
    lib.rtq_fp8_dgrad.argtypes = [vp, i32, vp, i64, vp, vp, i32, i32, i32, vp, i32, vp, sz, vp]
    lib.rtq_fp8_linear.argtypes = [vp, i32, i64, vp, vp, i32, i64, i32, vp, vp, vp, i32, vp, sz, vp]
    lib.rtq_fp8_linear_dgrad.argtypes = [vp, i32, i32, i64, vp, vp, i32, i32, i32, vp, i32, vp, sz, vp]
    lib.rtq_fp8_wgrad.argtypes = [vp, i64, vp, vp, i32, i32, i32, vp, i32, i32, vp, sz, vp]
    lib.rtq_act_fp8_forward.argtypes = [vp, i32, i64, i32, i32, vp, vp, vp, vp, vp, i32, vp]
    lib.rtq_act_fp8_backward.argtypes = [vp, i32, vp, vp, i32, i64, i32, i32, vp, vp]
    for name, n in (("rtq_fp8_qgemm_workspace", i64), ("rtq_fp8_linear_workspace", i64),
                    ("rtq_fp8_dgrad_workspace", i32), ("rtq_fp8_linear_dgrad_workspace", i32),
                    ("rtq_fp8_wgrad_workspace", i32)):
        getattr(lib, name).argtypes = [i64, n, i32]
        getattr(lib, name).restype = sz
    lib.rtq_rmsnorm_forward.argtypes = [vp, i32, vp, i32, i64, i32, vp, i32, f32, vp, vp, vp, vp, i32, vp]
    lib.rtq_rmsnorm_backward.argtypes = [vp, i32, vp, i32, vp, i64, i32, vp, i32, f32, vp, vp, i32, i32, vp, sz, vp]
    lib.rtq_rmsnorm_backward_workspace.argtypes = [i64, i32]
    lib.rtq_rmsnorm_backward_workspace.restype = sz
    lib.rtq_fp8_glu.argtypes = [vp, vp, i64, vp, vp, i32, i32, i32, i32, vp, vp, vp, i32, vp, vp, vp, sz, vp]
    lib.rtq_fp8_glu_workspace.argtypes = [i64, i32, i32]
    lib.rtq_fp8_glu_workspace.restype = sz
    lib.rtq_glu_fp8_backward.argtypes = [vp, i32, vp, vp, i32, i64, i32, i32, vp, vp, i32, vp, vp]
    lib.rtq_grad_norm.argtypes = [vp, i32, vp, vp, sz, vp]
    lib.rtq_grad_norm_workspace.argtypes = [vp, i32]
    lib.rtq_grad_norm_workspace.restype = sz
    lib.rtq_grad_clip.argtypes = [vp, vp, i32, vp, f32, vp]
    lib.rtq_last_error.argtypes = []
    lib.rtq_last_error.restype = ctypes.c_char_p
    for name in ("rtq_rpbh_make", "rtq_lloyd_max", "rtq_rpbh_rotate", "rtq_quantize_rows", "rtq_qgemm",
                 "rtq_qgemm_ws", "rtq_rotated_qlinear", "rtq_quantize_rows_asym", "rtq_qgemm_asym",
                 "rtq_rotated_qlinear_asym", "rtq_rotated_qlinear_noalloc", "rtq_fp8_quantize", "rtq_fp8_dequantize",
                 "rtq_fp8_qgemm", "rtq_fp8_dgrad", "rtq_fp8_linear", "rtq_fp8_linear_dgrad", "rtq_fp8_wgrad",
                 "rtq_act_fp8_forward", "rtq_act_fp8_backward", "rtq_rmsnorm_forward", "rtq_rmsnorm_backward",
                 "rtq_fp8_glu", "rtq_glu_fp8_backward", "rtq_grad_norm", "rtq_grad_clip"):
        getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def last_error() -> str:
    return load_library().rtq_last_error().decode()


def _check(status: int):
    if status != RTQ_OK:
        raise RtqError(status, last_error())


# ------------------------------------------------------------------ host helpers

def rpbh_make(seed: int, d: int, h: int = 64):
    """Seeded RPBH descriptor as host arrays (perm int32[d], signs int8[d])."""
    perm = np.empty(d, np.int32)
    signs = np.empty(d, np.int8)
    _check(load_library().rtq_rpbh_make(seed & 0xFFFFFFFFFFFFFFFF, d, h, perm.ctypes.data, signs.ctypes.data))
    return perm, signs


def lloyd_max(d: int, bits: int):
    """Lloyd-Max codebook for N(0, 1/d): (centroids fp32[2^bits], boundaries fp32[2^bits-1])."""
    c = np.empty(1 << bits, np.float32)
    t = np.empty((1 << bits) - 1, np.float32)
    _check(load_library().rtq_lloyd_max(d, bits, c.ctypes.data, t.ctypes.data))
    return c, t


# ------------------------------------------------------------------ device objects

def _torch():
    import torch
    return torch


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return RTQ_F32
    if t.dtype == torch.bfloat16:
        return RTQ_BF16
    if t.dtype == torch.int32:
        return RTQ_I32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t) -> int:
    return 0 if t is None else int(t.data_ptr())


def _stream_local_workspace(torch, nbytes: int, device, stream):
    """A temporary workspace for one call.  torch's caching allocator may hand its memory to other
    work once it is freed; recording the launch stream makes that wait for the call's kernels when
    they run on a stream other than the current one."""
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    if stream is not None:
        ws.record_stream(stream)
    return ws


def _stream(stream) -> int:
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


class Rpbh:
    """A rotation descriptor on the device (perm int32[d], signs int8[d], h = 64)."""

    def __init__(self, perm, signs, h: int = 64):
        torch = _torch()
        self.perm = perm if isinstance(perm, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(perm))
        self.signs = signs if isinstance(signs, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(signs))
        self.d = int(self.perm.numel())
        self.h = h
        self._c = _Rpbh(self.d, h, _ptr(self.perm), _ptr(self.signs))

    @classmethod
    def from_seed(cls, seed: int, d: int, device="cuda"):
        perm, signs = rpbh_make(seed, d)
        torch = _torch()
        return cls(torch.from_numpy(perm).to(device), torch.from_numpy(signs).to(device))

    @classmethod
    def without_permutation(cls, seed: int, d: int, device="cuda"):
        """Block Hadamard with the seeded signs and no permutation (perm = identity): the ablation
        of the permutation step (OrbitQuant article, sections 2.3 and 3.3)."""
        _, signs = rpbh_make(seed, d)
        torch = _torch()
        return cls(torch.arange(d, dtype=torch.int32, device=device), torch.from_numpy(signs).to(device))

    @property
    def c(self):
        return ctypes.byref(self._c)


class Codebook:
    """A Lloyd-Max codebook on the device (centroids fp32[2^bits], boundaries fp32[2^bits - 1])."""

    def __init__(self, bits: int, centroids, boundaries):
        self.bits = bits
        self.centroids = centroids
        self.boundaries = boundaries
        self._c = _Codebook(bits, _ptr(centroids), _ptr(boundaries))

    @classmethod
    def for_dim(cls, d: int, bits: int, device="cuda"):
        c, t = lloyd_max(d, bits)
        torch = _torch()
        return cls(bits, torch.from_numpy(c).to(device), torch.from_numpy(t).to(device))

    @property
    def c(self):
        return ctypes.byref(self._c)


def _cb(cb):
    return None if cb is None else cb.c


# ------------------------------------------------------------------ device calls

def rpbh_rotate(x, y, R: Rpbh, inverse: bool = False, stream=None):
    """y = Pi x (or x = Pi^T y when inverse) row by row."""
    rows = x.shape[0] if x.dim() > 1 else 0
    _check(load_library().rtq_rpbh_rotate(_ptr(x), _dtype_code(x), _ptr(y), _dtype_code(y), rows, R.c,
                                          1 if inverse else 0, _stream(stream)))
    return y


def quantize_rows(x, codes, scale, R: Rpbh | None = None, mode: int = RTQ_INT8, cb: Codebook | None = None,
                  eps: float = 0.0, stream=None):
    """Rotate (if R) and quantise each row of x into codes + per-row scale/norm."""
    rows, d = x.shape
    need = tiled_code_bytes(rows, d, mode, cb.bits if cb is not None else 8)
    if codes.numel() * codes.element_size() < need:
        raise ValueError(f"tiled codes need {need} bytes (rows padded to a multiple of 256)")
    _check(load_library().rtq_quantize_rows(_ptr(x), _dtype_code(x), rows, d, None if R is None else R.c, mode,
                                            _cb(cb), ctypes.c_float(eps), _ptr(codes), _ptr(scale),
                                            _dtype_code(scale), _stream(stream)))
    return codes, scale


def qgemm(a_codes, a_scale, w_codes, w_scale, y, d: int, mode: int = RTQ_INT8, cb_a: Codebook | None = None,
          cb_w: Codebook | None = None, stream=None, workspace=None, n_tokens: int | None = None,
          n_out: int | None = None):
    """y = dequantised product of activation and weight codes (rotation already cancelled).
    With a workspace (qgemm_workspace() bytes) this is rtq_qgemm_ws: a partial last round of tiles
    is shared along d (stream-K runs after a full round, equal K ranges otherwise).
    T and N default to the codes' first dimensions; pass n_tokens / n_out for tiled codes (whose
    buffers hold rows padded to a multiple of 256), or take them from y."""
    T = a_codes.shape[0] if n_tokens is None else n_tokens
    N = w_codes.shape[0] if n_out is None else n_out
    lib = load_library()
    if workspace is None:
        _check(lib.rtq_qgemm(_ptr(a_codes), _ptr(a_scale), T, _ptr(w_codes), _ptr(w_scale), _dtype_code(w_scale), N,
                             d, mode, _cb(cb_a), _cb(cb_w), _ptr(y), _dtype_code(y), _stream(stream)))
    else:
        _check(lib.rtq_qgemm_ws(_ptr(a_codes), _ptr(a_scale), T, _ptr(w_codes), _ptr(w_scale), _dtype_code(w_scale),
                                N, d, mode, _cb(cb_a), _cb(cb_w), _ptr(y), _dtype_code(y), _ptr(workspace),
                                workspace.numel() * workspace.element_size(), _stream(stream)))
    return y


def qgemm_workspace() -> int:
    """Bytes of workspace qgemm(..., workspace=...) uses on the current device."""
    return int(load_library().rtq_qgemm_workspace())


def new_qgemm_workspace(device="cuda"):
    """A zero-filled workspace for qgemm(..., workspace=...): its arrival counters must start at
    zero, and every product that completes leaves them zero again, so it can be reused as is."""
    return _torch().zeros(qgemm_workspace(), dtype=_torch().uint8, device=device)


def rotated_qlinear_workspace(T: int, d: int, mode: int = RTQ_INT8, bits_a: int = 8) -> int:
    return int(load_library().rtq_rotated_qlinear_workspace(T, d, mode, bits_a))


def rotated_qlinear(x, R: Rpbh, w_codes, w_scale, y, mode: int = RTQ_INT8, cb_a: Codebook | None = None,
                    cb_w: Codebook | None = None, workspace=None, stream=None):
    """The online layer: rotate + quantise x, then the quantised product, on one stream."""
    torch = _torch()
    T = x.shape[0]
    bits_a = cb_a.bits if (mode in _CODEBOOK_MODES and cb_a is not None) else 8
    N = y.shape[1]
    need = rotated_qlinear_workspace(T, R.d, mode, bits_a)
    if workspace is None:
        workspace = _stream_local_workspace(torch, max(need, 16), x.device, stream)
    _check(load_library().rtq_rotated_qlinear(_ptr(x), _dtype_code(x), T, R.c, _ptr(w_codes), _ptr(w_scale),
                                              _dtype_code(w_scale), N, mode, _cb(cb_a), _cb(cb_w),
                                              _ptr(y), _dtype_code(y), _ptr(workspace), workspace.numel(),
                                              _stream(stream)))
    return y


def rotated_qlinear_noalloc(x, R: Rpbh, w_codes, w_scale, y, mode: int = RTQ_INT8, cb_a: Codebook | None = None,
                            cb_w: Codebook | None = None, stream=None):
    """The online layer with no workspace: the activation codes and scales go to the library's
    static device scratch (NOALLOC_SCRATCH_BYTES per GPU; calls on one GPU must not overlap)."""
    T = x.shape[0]
    _check(load_library().rtq_rotated_qlinear_noalloc(_ptr(x), _dtype_code(x), T, R.c, _ptr(w_codes), _ptr(w_scale),
                                                      _dtype_code(w_scale), y.shape[1], mode, _cb(cb_a),
                                                      _cb(cb_w), _ptr(y), _dtype_code(y), _stream(stream)))
    return y


# ------------------------------------------------------------------ asymmetric INT8

def quantize_rows_asym(x, codes, scale, zero, code_sum, R: Rpbh, stream=None):
    """Rotate and quantise each row with a scale and a zero point (int8 codes, scale, int32 zero
    point, int32 code sum per row)."""
    rows, d = x.shape
    _check(load_library().rtq_quantize_rows_asym(_ptr(x), _dtype_code(x), rows, d, R.c, _ptr(codes), _ptr(scale),
                                                 _dtype_code(scale), _ptr(zero), _ptr(code_sum), _stream(stream)))
    return codes, scale, zero, code_sum


def qgemm_asym(a_codes, a_scale, a_zero, a_sum, w_codes, w_scale, w_zero, w_sum, y, d: int, stream=None,
               workspace=None):
    """y = a_scale * w_scale * sum_j (qa - za)(qw - zw)."""
    T, N = a_codes.shape[0], w_codes.shape[0]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().rtq_qgemm_asym(_ptr(a_codes), _ptr(a_scale), _ptr(a_zero), _ptr(a_sum), T, _ptr(w_codes),
                                         _ptr(w_scale), _dtype_code(w_scale), _ptr(w_zero), _ptr(w_sum), N, d, _ptr(y),
                                         _dtype_code(y), _ptr(workspace), ws_bytes, _stream(stream)))
    return y


def rotated_qlinear_asym_workspace(T: int, d: int) -> int:
    return int(load_library().rtq_rotated_qlinear_asym_workspace(T, d))


def rotated_qlinear_asym(x, R: Rpbh, w_codes, w_scale, w_zero, w_sum, y, workspace=None, stream=None):
    """The online asymmetric layer: rotate + quantise x with zero points, then the zero-point product."""
    torch = _torch()
    T = x.shape[0]
    if workspace is None:
        workspace = _stream_local_workspace(torch, max(rotated_qlinear_asym_workspace(T, R.d), 16), x.device, stream)
    _check(load_library().rtq_rotated_qlinear_asym(_ptr(x), _dtype_code(x), T, R.c, _ptr(w_codes), _ptr(w_scale),
                                                   _dtype_code(w_scale), _ptr(w_zero), _ptr(w_sum), w_codes.shape[0],
                                                   _ptr(y), _dtype_code(y), _ptr(workspace), workspace.numel(),
                                                   _stream(stream)))
    return y


# ------------------------------------------------------------------ 8-bit floating point, scales for blocks of 128
#
# Codes are torch.float8_e4m3fn (gradients also float8_e5m2) tensors, scales float32 or
# float8_e8m0fnu.  Tensors are contiguous and on one device; the calls run on that device, on
# `stream` or its current stream.

def fp8_groups(d: int) -> int:
    """Scales along d elements (blocks of 128, the last one possibly shorter)."""
    return -(-d // FP8_BLOCK)


@functools.lru_cache(maxsize=None)
def _types():
    """Type codes of (float, 8-bit float, e4m3 only, scale) dtypes."""
    torch = _torch()
    e4m3 = {torch.float8_e4m3fn: RTQ_E4M3}
    return ({torch.float32: RTQ_F32, torch.bfloat16: RTQ_BF16}, {**e4m3, torch.float8_e5m2: RTQ_E5M2}, e4m3,
            {torch.float32: RTQ_F32, torch.float8_e8m0fnu: RTQ_E8M0})


def _operand(t, name: str, types: dict, shape=None, like=None) -> int:
    """Type code of a device tensor, after checking its type, shape, layout and device."""
    code = types.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    if t.dim() != 2 if shape is None else t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {'two dimensions' if shape is None else tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if like is None or like is t:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor")
    elif t.get_device() != like.get_device():
        raise ValueError(f"{name} must be a GPU tensor" if not t.is_cuda else
                         f"{name} is on {t.device}, expected {like.device}")
    return code


def _call(like, stream, fn, *args):
    """fn(*args, stream) on the device of `like`, on `stream` or that device's current one."""
    torch = _torch()
    index = like.get_device()
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(index)
    elif stream.device == like.device:
        handle = stream.cuda_stream
    else:
        raise ValueError(f"stream is on {stream.device}, the tensors on {like.device}")
    if index == torch._C._cuda_getDevice():
        status = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            status = fn(*args, handle)
    if status != RTQ_OK:
        raise RtqError(status, last_error())


def _workspace(given, like, stream, query, *sizes):
    """The caller's workspace, or a temporary one of the queried size for the call's stream."""
    if given is None:
        torch = _torch()
        if like.get_device() == torch._C._cuda_getDevice():
            need = query(*sizes)
        else:
            with torch.cuda.device(like.device):
                need = query(*sizes)
        return _stream_local_workspace(torch, need, like.device, stream)
    if given.get_device() != like.get_device():
        raise ValueError(f"workspace is on {given.device}, expected {like.device}")
    if not given.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return given


def fp8_quantize(x, codes, scale, blocks: bool = False, stream=None):
    """Codes and power-of-two scales of x [rows][d]: row groups of 128 (scale [groups][rows],
    group-major) or, with blocks, 128 x 128 blocks (scale [row blocks][column blocks])."""
    xt = _operand(x, "x", _types()[0])
    rows, d = x.shape
    ct = _operand(codes, "codes", _types()[1], x.shape, x)
    st = _operand(scale, "scale", _types()[3],
                  (fp8_groups(rows), fp8_groups(d)) if blocks else (fp8_groups(d), rows), x)
    _call(x, stream, load_library().rtq_fp8_quantize, _ptr(x), xt, rows, d,
          RTQ_FP8_BLOCKS if blocks else RTQ_FP8_ROWS, _ptr(codes), ct, _ptr(scale), st)
    return codes, scale


def fp8_dequantize(codes, scale, y, blocks: bool = False, stream=None):
    """y = code * scale, for codes and scales as fp8_quantize writes them."""
    ct = _operand(codes, "codes", _types()[1])
    rows, d = codes.shape
    st = _operand(scale, "scale", _types()[3],
                  (fp8_groups(rows), fp8_groups(d)) if blocks else (fp8_groups(d), rows), codes)
    yt = _operand(y, "y", _types()[0], codes.shape, codes)
    _call(codes, stream, load_library().rtq_fp8_dequantize, _ptr(codes), ct, _ptr(scale), st, rows, d,
          RTQ_FP8_BLOCKS if blocks else RTQ_FP8_ROWS, _ptr(y), yt)
    return y


def _fp8_weight(w_codes, w_scale, like):
    """(N, K, scale type code) of block-scaled weight codes."""
    _operand(w_codes, "w_codes", _types()[2], None, like)
    N, K = w_codes.shape
    return N, K, _operand(w_scale, "w_scale", _types()[3], (fp8_groups(N), fp8_groups(K)), like)


def _same_scale(a, name: str, w_scale):
    if a.dtype != w_scale.dtype:
        raise TypeError(f"{name} is {a.dtype}, w_scale {w_scale.dtype}: the scales of a product share one type")


def fp8_qgemm_workspace(T: int, N: int, K: int) -> int:
    return int(load_library().rtq_fp8_qgemm_workspace(T, N, K))


def fp8_qgemm(a_codes, a_scale, w_codes, w_scale, y, workspace=None, stream=None):
    """y [T][N] = a W^T of row-group codes a [T][K] and block codes W [N][K]."""
    N, K, st = _fp8_weight(w_codes, w_scale, a_codes)
    T = a_codes.shape[0]
    at = _operand(a_codes, "a_codes", _types()[1], (T, K))
    _operand(a_scale, "a_scale", _types()[3], (fp8_groups(K), T), a_codes)
    _same_scale(a_scale, "a_scale", w_scale)
    yt = _operand(y, "y", _types()[0], (T, N), a_codes)
    ws = _workspace(workspace, a_codes, stream, fp8_qgemm_workspace, T, N, K)
    _call(a_codes, stream, load_library().rtq_fp8_qgemm, _ptr(a_codes), at, _ptr(a_scale), T, _ptr(w_codes),
          _ptr(w_scale), st, N, K, _ptr(y), yt, _ptr(ws), ws.numel() * ws.element_size())
    return y


def fp8_dgrad_workspace(T: int, N: int, K: int) -> int:
    return int(load_library().rtq_fp8_dgrad_workspace(T, N, K))


def fp8_dgrad(g_codes, g_scale, w_codes, w_scale, dx, workspace=None, stream=None):
    """dx [T][K] = g W of row-group codes g [T][N] (quantised output gradients) and block codes W [N][K]."""
    N, K, st = _fp8_weight(w_codes, w_scale, g_codes)
    T = g_codes.shape[0]
    gt = _operand(g_codes, "g_codes", _types()[1], (T, N))
    _operand(g_scale, "g_scale", _types()[3], (fp8_groups(N), T), g_codes)
    _same_scale(g_scale, "g_scale", w_scale)
    dxt = _operand(dx, "dx", _types()[0], (T, K), g_codes)
    ws = _workspace(workspace, g_codes, stream, fp8_dgrad_workspace, T, N, K)
    _call(g_codes, stream, load_library().rtq_fp8_dgrad, _ptr(g_codes), gt, _ptr(g_scale), T, _ptr(w_codes),
          _ptr(w_scale), st, N, K, _ptr(dx), dxt, _ptr(ws), ws.numel() * ws.element_size())
    return dx


def fp8_linear_workspace(T: int, N: int, K: int) -> int:
    return int(load_library().rtq_fp8_linear_workspace(T, N, K))


def fp8_linear(x, w_codes, w_scale, y, x_codes=None, x_scale=None, workspace=None, stream=None):
    """y [T][N] = quantise(x) W^T for x [T][K] and block codes W [N][K].  With x_codes [T][K] (e4m3)
    and x_scale [groups][T] the codes the product read are kept: the checkpoint fp8_wgrad takes."""
    N, K, st = _fp8_weight(w_codes, w_scale, x)
    T = x.shape[0]
    xt = _operand(x, "x", _types()[0], (T, K))
    yt = _operand(y, "y", _types()[0], (T, N), x)
    if (x_codes is None) != (x_scale is None):
        raise ValueError("x_codes and x_scale are given together or not at all")
    if x_codes is not None:
        _operand(x_codes, "x_codes", _types()[2], (T, K), x)
        _operand(x_scale, "x_scale", _types()[3], (fp8_groups(K), T), x)
        _same_scale(x_scale, "x_scale", w_scale)
    ws = _workspace(workspace, x, stream, fp8_linear_workspace, T, N, K)
    _call(x, stream, load_library().rtq_fp8_linear, _ptr(x), xt, T, _ptr(w_codes), _ptr(w_scale), st, N, K,
          _ptr(x_codes), _ptr(x_scale), _ptr(y), yt, _ptr(ws), ws.numel() * ws.element_size())
    return y


def fp8_linear_dgrad_workspace(T: int, N: int, K: int) -> int:
    return int(load_library().rtq_fp8_linear_dgrad_workspace(T, N, K))


def fp8_linear_dgrad(dy, w_codes, w_scale, dx, grad_dtype=None, workspace=None, stream=None):
    """dx [T][K] = quantise(dy) W for dy [T][N] and block codes W [N][K]; grad_dtype is the format dy is
    quantised to, torch.float8_e5m2 (default) or torch.float8_e4m3fn."""
    torch = _torch()
    N, K, st = _fp8_weight(w_codes, w_scale, dy)
    T = dy.shape[0]
    dyt = _operand(dy, "dy", _types()[0], (T, N))
    dxt = _operand(dx, "dx", _types()[0], (T, K), dy)
    grad_dtype = torch.float8_e5m2 if grad_dtype is None else grad_dtype
    if grad_dtype not in _types()[1]:
        raise TypeError(f"grad_dtype: unsupported dtype {grad_dtype}")
    ws = _workspace(workspace, dy, stream, fp8_linear_dgrad_workspace, T, N, K)
    _call(dy, stream, load_library().rtq_fp8_linear_dgrad, _ptr(dy), dyt, _types()[1][grad_dtype], T, _ptr(w_codes),
          _ptr(w_scale), st, N, K, _ptr(dx), dxt, _ptr(ws), ws.numel() * ws.element_size())
    return dx


def fp8_wgrad_workspace(T: int, N: int, K: int) -> int:
    return int(load_library().rtq_fp8_wgrad_workspace(T, N, K))


def fp8_wgrad(dy, x_codes, x_scale, dw, accumulate: bool = False, workspace=None, stream=None):
    """dw [N][K] = dy^T x^ (added to dw with accumulate) for dy [T][N] (bf16) and the checkpoint x^ of the
    layer's input: codes [T][K] (e4m3) and scales [groups][T]."""
    torch = _torch()
    _operand(dy, "dy", {torch.bfloat16: RTQ_BF16})
    T, N = dy.shape
    _operand(x_codes, "x_codes", _types()[2], (T, x_codes.shape[-1]), dy)
    K = x_codes.shape[1]
    st = _operand(x_scale, "x_scale", _types()[3], (fp8_groups(K), T), dy)
    dwt = _operand(dw, "dw", _types()[0], (N, K), dy)
    ws = _workspace(workspace, dy, stream, fp8_wgrad_workspace, T, N, K)
    _call(dy, stream, load_library().rtq_fp8_wgrad, _ptr(dy), T, _ptr(x_codes), _ptr(x_scale), st, N, K, _ptr(dw),
          dwt, 1 if accumulate else 0, _ptr(ws), ws.numel() * ws.element_size())
    return dw


def act_fp8_forward(h, act: int, h_codes, h_scale, y=None, y_codes=None, y_scale=None, stream=None):
    """y = f(h) with h kept as codes [rows][d] (e4m3) and scales [groups][rows]; f is RTQ_ACT_GELU_TANH,
    RTQ_ACT_GELU or RTQ_ACT_SILU.  y comes back as y (h's type), or quantised as y_codes, y_scale."""
    e4m3 = _types()[2]
    ht = _operand(h, "h", _types()[0])
    rows, d = h.shape
    _operand(h_codes, "h_codes", e4m3, h.shape, h)
    st = _operand(h_scale, "h_scale", _types()[3], (fp8_groups(d), rows), h)
    if (y_codes is None) != (y_scale is None) or (y is None) == (y_codes is None):
        raise ValueError("give either y, or y_codes and y_scale")
    if y is not None:
        _operand(y, "y", {h.dtype: ht}, h.shape, h)
    else:
        _operand(y_codes, "y_codes", e4m3, h.shape, h)
        _operand(y_scale, "y_scale", {h_scale.dtype: st}, (fp8_groups(d), rows), h)
    _call(h, stream, load_library().rtq_act_fp8_forward, _ptr(h), ht, rows, d, act, _ptr(h_codes), _ptr(h_scale),
          _ptr(y), _ptr(y_codes), _ptr(y_scale), st)
    return y if y is not None else (y_codes, y_scale)


def act_fp8_backward(dy, h_codes, h_scale, act: int, dh, stream=None):
    """dh = dy f'(h^) from the checkpoint of h (act_fp8_forward).  dh may be dy."""
    dyt = _operand(dy, "dy", _types()[0])
    rows, d = dy.shape
    _operand(h_codes, "h_codes", _types()[2], dy.shape, dy)
    st = _operand(h_scale, "h_scale", _types()[3], (fp8_groups(d), rows), dy)
    _operand(dh, "dh", {dy.dtype: dyt}, dy.shape, dy)
    _call(dy, stream, load_library().rtq_act_fp8_backward, _ptr(dy), dyt, _ptr(h_codes), _ptr(h_scale), st, rows, d,
          act, _ptr(dh))
    return dh


# ------------------------------------------------------------------ around the 8-bit layers of an MLP block

@functools.lru_cache(maxsize=None)
def _bound():
    """The compiled binding (csrc/bind.cpp): it checks the tensors and calls the library.  Raises if it has not been built."""
    load_library()
    _torch()
    try:
        import importlib
        native = importlib.import_module("._native", __package__)
    except ImportError as e:
        raise RuntimeError(f"{os.path.join(_PKG, '_native.so')} cannot be loaded ({e}): build it with __graft_entry__.build(); "
                           f"there is no fallback path") from e
    native.load(LIB_PATH)
    return native


def rmsnorm_forward(x, gamma, eps: float, residual=None, h=None, codes=None, scale=None, y=None, stream=None):
    """n = h / sqrt(mean h^2 + eps) gamma for rows of h = x, or of h = x + residual, which is written to h [rows][d]
    (residual's type; h may be residual).  n comes back quantised, as codes [rows][d] (e4m3) and scale [groups][rows],
    as y [rows][d] (x's type), or as both.  Returns the residual stream: h, or x without a residual."""
    status = _bound().rmsnorm_forward(x, gamma, eps, residual, h, codes, scale, y, stream)
    if status:
        _check(status)
    return x if h is None else h


def rmsnorm_backward_workspace(rows: int, d: int) -> int:
    return int(load_library().rtq_rmsnorm_backward_workspace(rows, d))


def rmsnorm_backward(dn, h, gamma, eps: float, dh, dgamma=None, dresidual=None, accumulate: bool = False, workspace=None,
                     stream=None):
    """dh [rows][d] (h's type), the gradient of h and thus of x and residual, from the gradient dn [rows][d] of
    rmsnorm_forward's n and the residual stream's own, dresidual (h's type, or None); dh may be dresidual, or dn if their
    types agree.  dgamma [d] (float32 or bfloat16) is written, or added to with accumulate."""
    if workspace is None and dgamma is not None:
        _operand(dn, "dn", _types()[0])
        workspace = _workspace(None, dn, stream, rmsnorm_backward_workspace, *dn.shape)
    status = _bound().rmsnorm_backward(dn, h, gamma, eps, dh, dgamma, dresidual, accumulate, workspace, stream)
    if status:
        _check(status)
    return dh


def fp8_glu_workspace(T: int, N: int, K: int) -> int:
    return int(load_library().rtq_fp8_glu_workspace(T, N, K))


def fp8_glu(x_codes, x_scale, w_codes, w_scale, act: int, y=None, y_codes=None, y_scale=None, h_codes=None, h_scale=None,
            workspace=None, stream=None):
    """y = f(g) u with [g u] = x W^T of row-group codes x [T][K] and block codes W [2 N][K], the gate's N rows first (N a
    multiple of 128); f is RTQ_ACT_GELU_TANH, RTQ_ACT_GELU or RTQ_ACT_SILU.  y [T][N] comes back as y (float32 or
    bfloat16), or quantised as y_codes, y_scale.  With h_codes [T][2 N] and h_scale, [g u] is kept in 8 bits, for
    glu_fp8_backward."""
    if workspace is None:
        _operand(x_codes, "x_codes", _types()[2])
        _operand(w_codes, "w_codes", _types()[2], None, x_codes)
        workspace = _workspace(None, x_codes, stream, fp8_glu_workspace, x_codes.shape[0], w_codes.shape[0] // 2, x_codes.shape[1])
    status = _bound().fp8_glu(x_codes, x_scale, w_codes, w_scale, act, y, y_codes, y_scale, h_codes, h_scale, workspace, stream)
    if status:
        _check(status)
    return y if y is not None else (y_codes, y_scale)


def glu_fp8_backward(dy, h_codes, h_scale, act: int, dh=None, dh_codes=None, dh_scale=None, stream=None):
    """[dg du] = [dy u^ f'(g^), dy f(g^)] from dy [T][N] and fp8_glu's checkpoint, as dh [T][2 N] (dy's type; fp8_wgrad
    takes it in bfloat16) and/or quantised, as dh_codes [T][2 N] (e4m3 or e5m2) and dh_scale, for fp8_dgrad."""
    status = _bound().glu_fp8_backward(dy, h_codes, h_scale, act, dh, dh_codes, dh_scale, stream)
    if status:
        _check(status)
    return dh if dh is not None else (dh_codes, dh_scale)


def _overlap(reads, writes) -> bool:
    """Whether any of the address ranges (begin, end) of writes overlaps another one, of reads or of writes."""
    read_end = write_end = 0
    for begin, end, written in sorted([(b, e, False) for b, e in reads if b < e] + [(b, e, True) for b, e in writes if b < e]):
        if begin < write_end or (written and begin < read_end):
            return True
        if written:
            write_end = max(write_end, end)
        else:
            read_end = max(read_end, end)
    return False


class TensorList:
    """Tensors (float32 or bfloat16, contiguous, on one GPU) as grad_norm and grad_clip take them, and where grad_clip puts
    its results: outs, of the same shapes and types, or the tensors themselves; no out may overlap another out or another
    tensor.  It holds them; a program that replaces tensors, or their memory, needs a new list."""

    def __init__(self, tensors, outs=None):
        self.tensors = tuple(tensors)
        if not self.tensors:
            raise ValueError("no tensors")
        self.outs = self.tensors if outs is None else tuple(outs)
        if len(self.outs) != len(self.tensors):
            raise ValueError(f"{len(self.outs)} outs for {len(self.tensors)} tensors")
        for t in self.tensors + self.outs:
            if not isinstance(t, _torch().Tensor):
                raise TypeError(f"tensors are expected, not {type(t).__name__}")
        floats, like, n = _types()[0], self.tensors[0], len(self.tensors)
        self._c, self._outs = (_Tensor * n)(), (ctypes.c_void_p * n)()
        reads, writes = [], []
        for i, (t, o) in enumerate(zip(self.tensors, self.outs)):
            code = _operand(t, f"tensors[{i}]", floats, t.shape, like)
            _operand(o, f"outs[{i}]", {t.dtype: code}, t.shape, like)
            self._c[i] = _Tensor(t.data_ptr(), t.numel(), code)
            self._outs[i] = o.data_ptr()
            writes.append((o.data_ptr(), o.data_ptr() + o.nbytes))
            if t.data_ptr() != o.data_ptr():
                reads.append((t.data_ptr(), t.data_ptr() + t.nbytes))
        if _overlap(reads, writes):
            raise ValueError("an out overlaps another out or another tensor")
        self._like, self._at, self._outs_at = like, ctypes.addressof(self._c), ctypes.addressof(self._outs)


def grad_norm_workspace(tensors: TensorList) -> int:
    return int(load_library().rtq_grad_norm_workspace(tensors._c, len(tensors.tensors)))


def grad_norm(tensors: TensorList, norm, workspace=None, stream=None):
    """norm (one float32 on the GPU) = the 2-norm of all tensors together."""
    if workspace is None:
        workspace = _workspace(None, tensors._like, stream, grad_norm_workspace, tensors)
    status = _bound().grad_norm(tensors.tensors, tensors._at, norm, workspace, stream)
    if status:
        _check(status)
    return norm


def grad_clip(tensors: TensorList, norm, most: float, stream=None):
    """Each tensor times min(1, most / (norm + 1e-6)), to the list's outs."""
    status = _bound().grad_clip(tensors.tensors, tensors._at, tensors.outs, tensors._outs_at, norm, most, stream)
    if status:
        _check(status)
    return tensors.outs
