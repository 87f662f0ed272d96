"""Python binding of libbc.so, the B200 fused group-wise dequant matmul.

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in ``include/bc.h``.  PyTorch supplies the
device memory and the current stream.  There is no CPU fallback: importing
this package on a machine without the built library raises.

Functions (same names as the C entry points, without the ``bc_`` prefix):
    group_params, quantize_codes, pack_int4, matmul_q, matmul_q_batched,
    workspace_size, workspace_size_batched
and, around the projections:
    add_rmsnorm, add_rmsnorm_q8   residual addition and norm before a projection
    lora_add, lora_add_batched    adapters of many requests beside it
    beam_select, matmul_q_beam, beam_reorder   beam search after the LM head
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbc.so")

BC_OK, BC_ERR_INVALID_ARG, BC_ERR_UNSUPPORTED, BC_ERR_ALIGNMENT, \
    BC_ERR_WORKSPACE, BC_ERR_CUDA = range(6)
BC_F32, BC_F16, BC_BF16 = 0, 1, 2
BC_MODE_RUNTIME, BC_MODE_PACKED_INT4, BC_MODE_RUNTIME_RANGE = 0, 1, 2
BC_MODE_PACKED = BC_MODE_PACKED_INT4
GROUP_PER_CHANNEL = 0
BC_FLAG_STATIC_WEIGHTS = 1

# Every symbol include/bc.h declares.
EXPORTS = ("bc_group_params", "bc_group_minmax", "bc_quantize_codes", "bc_pack_int4",
           "bc_pack_codes",
           "bc_matmul_q", "bc_workspace_size", "bc_matmul_q_batched",
           "bc_matmul_q_batched_ex",
           "bc_workspace_size_batched", "bc_matmul_q_noalloc",
           "bc_matmul_q_argmax", "bc_workspace_size_argmax",
           "bc_add_rmsnorm", "bc_add_rmsnorm_q8", "bc_lora_add", "bc_lora_add_batched",
           "bc_workspace_size_lora", "bc_beam_select", "bc_workspace_size_beam", "bc_matmul_q_beam",
           "bc_workspace_size_matmul_beam", "bc_beam_reorder",
           "bc_device_timeouts", "bc_set_wait_limit",
           "bc_status_string", "bc_version")


class BCError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} (status {status})")
        self.status = status


class MatmulDesc(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("W_or_packed", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("zeros", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("N", ctypes.c_int64),
                ("K", ctypes.c_int64)]


class LoraDesc(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("A", ctypes.c_void_p), ("B", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


class BeamState(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("row_bytes", ctypes.c_int64), ("row_stride", ctypes.c_int64),
                ("beam_stride", ctypes.c_int64)]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with "
            "`python quantized_matmul_02_b200/build.py` (nvcc, sm_100a)")
    lib = ctypes.CDLL(LIB_PATH)
    P, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    lib.bc_group_params.argtypes = [P, i64, i64, i32, i64, i32, P, P, P]
    lib.bc_quantize_codes.argtypes = [P, P, P, i32, i64, i64, i32, i64, P, P]
    lib.bc_group_minmax.argtypes = [P, i64, i64, i64, P, P]
    lib.bc_group_minmax.restype = i32
    lib.bc_pack_int4.argtypes = [P, P, P, i64, i64, P, P]
    lib.bc_pack_codes.argtypes = [P, P, P, i64, i64, i32, P, P]
    lib.bc_pack_codes.restype = i32
    lib.bc_matmul_q.argtypes = [P, i32, P, P, P, i64, i64, i64, i32, i64, i32,
                                P, P, sz, P]
    lib.bc_workspace_size.argtypes = [i64, i64, i64, i32]
    lib.bc_workspace_size.restype = sz
    lib.bc_matmul_q_batched.argtypes = [ctypes.POINTER(MatmulDesc), i32, i64,
                                        i32, i64, i32, i32, P, sz, P]
    lib.bc_matmul_q_batched_ex.argtypes = [ctypes.POINTER(MatmulDesc), i32, i64,
                                           i32, i64, i32, i32, P, sz, ctypes.c_uint, P]
    lib.bc_workspace_size_batched.argtypes = [ctypes.POINTER(MatmulDesc), i32,
                                              i64, i32, i32]
    lib.bc_workspace_size_batched.restype = sz
    lib.bc_matmul_q_noalloc.argtypes = [P, P, P, P, i64, i64, i64, i32, i64,
                                        i32, P, P]
    lib.bc_matmul_q_noalloc.restype = i32
    lib.bc_matmul_q_argmax.argtypes = [P, i32, P, P, P, i64, i64, i64, i32, i64, i32,
                                       P, P, sz, P]
    lib.bc_matmul_q_argmax.restype = i32
    lib.bc_workspace_size_argmax.argtypes = [i64, i64, i64, i32, i32]
    lib.bc_workspace_size_argmax.restype = sz
    f32 = ctypes.c_float
    lib.bc_add_rmsnorm.argtypes = [P, i32, P, i32, P, i32, i64, i64, f32, P, i32, P]
    lib.bc_add_rmsnorm_q8.argtypes = [P, i32, P, i32, P, i32, i64, i64, f32, P, P, P, P]
    lib.bc_lora_add.argtypes = [P, i32, P, P, i32, i64, i64, i64, i64, i64, P, P, i64, P, P,
                                P, P, sz, P]
    lib.bc_lora_add_batched.argtypes = [P, i32, i64, i64, i64, i32, i32,
                                        P, P, i64, P, P, P, sz, P]
    lib.bc_workspace_size_lora.argtypes = [P, i32, i64, i64, i64, i64, i32]
    lib.bc_workspace_size_lora.restype = sz
    lib.bc_beam_select.argtypes = [P, P, P, i64, i64, i64, i64, i32, i32, P, P, P, P, P, sz, P]
    lib.bc_workspace_size_beam.argtypes = [i64, i64, i64, i64]
    lib.bc_workspace_size_beam.restype = sz
    lib.bc_matmul_q_beam.argtypes = [P, i32, P, P, P, i64, i64, i64, i64, i32, i64, i32, P, P,
                                     i64, i32, i32, P, P, P, P, P, sz, P]
    lib.bc_workspace_size_matmul_beam.argtypes = [i64, i64, i64, i64, i64, i32, i32]
    lib.bc_workspace_size_matmul_beam.restype = sz
    lib.bc_beam_reorder.argtypes = [P, i32, P, i64, i64, i64, P]
    for name in ("bc_add_rmsnorm", "bc_add_rmsnorm_q8", "bc_lora_add", "bc_lora_add_batched",
                 "bc_beam_select", "bc_matmul_q_beam", "bc_beam_reorder"):
        getattr(lib, name).restype = i32
    lib.bc_set_wait_limit.argtypes = [ctypes.c_uint64]
    lib.bc_set_wait_limit.restype = i32
    lib.bc_device_timeouts.argtypes = [ctypes.POINTER(ctypes.c_uint)]
    lib.bc_device_timeouts.restype = i32
    lib.bc_status_string.argtypes = [i32]
    lib.bc_status_string.restype = ctypes.c_char_p
    lib.bc_version.restype = i32
    for name in ("bc_group_params", "bc_quantize_codes", "bc_pack_int4",
                 "bc_matmul_q", "bc_matmul_q_batched", "bc_matmul_q_batched_ex"):
        getattr(lib, name).restype = i32
    return lib


lib = _load()


def status_string(status: int) -> str:
    return lib.bc_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != BC_OK:
        raise BCError(status, what)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _stream(stream: Optional[torch.cuda.Stream]) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


_DT = {torch.float32: BC_F32, torch.float16: BC_F16, torch.bfloat16: BC_BF16}


def group_params(W: torch.Tensor, bits: int, group: int, out_dtype=torch.float32,
                 scales: Optional[torch.Tensor] = None,
                 zeros: Optional[torch.Tensor] = None, stream=None):
    """Per-group scale/zero of fp16 W [N][K]; returns (scales, zeros)."""
    N, K = W.shape
    g = K if group in (0, K) else group
    if scales is None:
        scales = torch.empty((N, K // g), dtype=out_dtype, device=W.device)
    if zeros is None:
        zeros = torch.empty((N, K // g), dtype=out_dtype, device=W.device)
    _check(lib.bc_group_params(_ptr(W), N, K, bits, group, _DT[out_dtype],
                               _ptr(scales), _ptr(zeros), _stream(stream)),
           "bc_group_params")
    return scales, zeros


def group_minmax(W: torch.Tensor, group: int, ranges: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """Per-group range of fp16 W [N][K] as int32 words [N][K/group] (fp16 min
    in the low half, fp16 max in the high half), for BC_MODE_RUNTIME_RANGE."""
    N, K = W.shape
    g = K if group in (0, K) else group
    if ranges is None:
        ranges = torch.empty((N, K // g), dtype=torch.int32, device=W.device)
    _check(lib.bc_group_minmax(_ptr(W), N, K, group, _ptr(ranges), _stream(stream)),
           "bc_group_minmax")
    return ranges


def quantize_codes(W: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                   bits: int, group: int, codes: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    N, K = W.shape
    if codes is None:
        codes = torch.empty((N, K), dtype=torch.uint8, device=W.device)
    _check(lib.bc_quantize_codes(_ptr(W), _ptr(scales), _ptr(zeros),
                                 _DT[scales.dtype], N, K, bits, group,
                                 _ptr(codes), _stream(stream)),
           "bc_quantize_codes")
    return codes


def pack_int4(W: torch.Tensor, scales_f16: torch.Tensor, zeros_f16: torch.Tensor,
              packed: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    N, K = W.shape
    if packed is None:
        packed = torch.empty((N, K // 2), dtype=torch.uint8, device=W.device)
    _check(lib.bc_pack_int4(_ptr(W), _ptr(scales_f16), _ptr(zeros_f16), N, K,
                            _ptr(packed), _stream(stream)), "bc_pack_int4")
    return packed


def pack_codes(W: torch.Tensor, scales_f16: torch.Tensor, zeros_f16: torch.Tensor,
               bits: int, packed: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Packed codes of `bits` (2, 3, 4, 8) bits: uint8 [N][K*bits/8]."""
    N, K = W.shape
    if packed is None:
        packed = torch.empty((N, K * bits // 8), dtype=torch.uint8, device=W.device)
    _check(lib.bc_pack_codes(_ptr(W), _ptr(scales_f16), _ptr(zeros_f16), N, K, bits,
                             _ptr(packed), _stream(stream)), "bc_pack_codes")
    return packed


def workspace_size(M: int, N: int, K: int, mode: int) -> int:
    return int(lib.bc_workspace_size(M, N, K, mode))


def matmul_q(x: torch.Tensor, W: torch.Tensor, scales: Optional[torch.Tensor],
             zeros: Optional[torch.Tensor], bits: int, group: int, mode: int,
             y: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y = x . deq(W)^T.  W is fp16 [N][K] (runtime) or packed uint8 [N][K/2]."""
    M, K = x.shape
    N = W.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    need = workspace_size(M, N, K, mode) if x.dtype == torch.float32 else 0
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    wsp = _ptr(workspace) if workspace is not None else None
    wsb = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.bc_matmul_q(_ptr(x), _DT[x.dtype], _ptr(W), _ptr(scales),
                           _ptr(zeros), M, N, K, bits, group, mode, _ptr(y),
                           wsp, wsb, _stream(stream)), "bc_matmul_q")
    return y


def make_descs(items: Sequence[tuple]) -> ctypes.Array:
    """items: (x, W_or_packed, scales, zeros, y) tensors per matrix."""
    arr = (MatmulDesc * len(items))()
    for i, (x, W, s, z, y) in enumerate(items):
        arr[i] = MatmulDesc(_ptr(x), _ptr(W), _ptr(s), _ptr(z), _ptr(y),
                            y.shape[1], x.shape[1])
    return arr


def workspace_size_batched(descs, M: int, mode: int, x_dtype: int) -> int:
    return int(lib.bc_workspace_size_batched(descs, len(descs), M, mode, x_dtype))


def matmul_q_batched(descs, M: int, bits: int, group: int, mode: int,
                     x_dtype: int = BC_F32, workspace: Optional[torch.Tensor] = None,
                     stream=None, static_weights: bool = False) -> None:
    """One grouped launch over the matrices in `descs` (from make_descs).
    Without `workspace`, split-K scratch (if any) is taken from torch.
    static_weights: BC_FLAG_STATIC_WEIGHTS (no pending work writes the
    weights, scales or zeros; the decode kernel may then start before the
    previous kernel on the stream has finished)."""
    if workspace is None:
        need = workspace_size_batched(descs, M, mode, x_dtype)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device="cuda")
    wsp = _ptr(workspace) if workspace is not None else None
    wsb = workspace.numel() * workspace.element_size() if workspace is not None else 0
    flags = BC_FLAG_STATIC_WEIGHTS if static_weights else 0
    _check(lib.bc_matmul_q_batched_ex(descs, len(descs), M, bits, group, mode,
                                      x_dtype, wsp, wsb, flags, _stream(stream)),
           "bc_matmul_q_batched_ex")


def device_timeouts() -> int:
    """Bounded in-kernel waits that ran out on this device (0 when healthy)."""
    c = ctypes.c_uint(0)
    _check(lib.bc_device_timeouts(ctypes.byref(c)), "bc_device_timeouts")
    return int(c.value)


def set_wait_limit(cycles: int) -> None:
    """bc_set_wait_limit: the in-kernel wait limit in cycles (0 = default)."""
    _check(lib.bc_set_wait_limit(int(cycles)), "bc_set_wait_limit")


def matmul_q_noalloc(x: torch.Tensor, W: torch.Tensor,
                     scales: Optional[torch.Tensor], zeros: Optional[torch.Tensor],
                     bits: int, group: int, mode: int, y: torch.Tensor,
                     stream=None) -> torch.Tensor:
    """bc_matmul_q_noalloc: the fp32-x decode matmul using the library's own
    fixed scratch instead of a workspace (for callers that cannot allocate).
    `y` must be supplied; nothing is allocated by this call."""
    M, K = x.shape
    N = W.shape[0]
    # The C call reads x as fp32 [M][K] and writes y as fp32 [M][N]: anything
    # else would be read or written out of bounds, so refuse it here.
    if x.dtype != torch.float32 or y.dtype != torch.float32:
        raise ValueError("matmul_q_noalloc: x and y must be float32")
    if tuple(y.shape) != (M, N):
        raise ValueError(f"matmul_q_noalloc: y must have shape {(M, N)}")
    devs = {t.device for t in (x, W, y, scales, zeros) if t is not None}
    if len(devs) != 1 or not next(iter(devs)).type == "cuda":
        raise ValueError("matmul_q_noalloc: all tensors must be on one CUDA device")
    _check(lib.bc_matmul_q_noalloc(_ptr(x), _ptr(W), _ptr(scales), _ptr(zeros),
                                   M, N, K, bits, group, mode, _ptr(y),
                                   _stream(stream)), "bc_matmul_q_noalloc")
    return y


def workspace_size_argmax(M: int, N: int, K: int, mode: int, x_dtype: int = BC_F32) -> int:
    return int(lib.bc_workspace_size_argmax(M, N, K, mode, x_dtype))


def matmul_q_argmax(x: torch.Tensor, W: torch.Tensor, scales: Optional[torch.Tensor],
                    zeros: Optional[torch.Tensor], bits: int, group: int, mode: int,
                    token: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """bc_matmul_q_argmax: int32 [M], per row of x the index of the largest
    output of x . deq(W)^T (lowest index among equal values)."""
    M, K = x.shape
    N = W.shape[0]
    if token is None:
        token = torch.empty((M,), dtype=torch.int32, device=x.device)
    need = workspace_size_argmax(M, N, K, mode, _DT[x.dtype])
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=x.device)
    _check(lib.bc_matmul_q_argmax(_ptr(x), _DT[x.dtype], _ptr(W), _ptr(scales), _ptr(zeros),
                                  M, N, K, bits, group, mode, _ptr(token), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(),
                                  _stream(stream)), "bc_matmul_q_argmax")
    return token


# ---------------------------------------------------------------------------
# Around the projections: norm, adapters, beam search.  These calls take
# tensors of one device, run there (also when it is not the current one), and
# check shapes and types before the C call sees pointers.  A decode step makes
# hundreds of them, so the checks are kept to a few attribute reads a tensor.
# ---------------------------------------------------------------------------
_F32, _F16, _BF16 = torch.float32, torch.float16, torch.bfloat16
_I32, _U8 = torch.int32, torch.uint8
_FLOATS = (_F32, _F16, _BF16)
# The calls behind torch.cuda.current_device and current_stream, without their
# wrappers' cost; a torch that lacks them (one without CUDA does) has the latter.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _one_device(what: str, first: torch.Tensor, *tensors: Optional[torch.Tensor]) -> int:
    """Index of the device that holds all of them, contiguous."""
    dev = first.get_device()
    if dev < 0:
        raise ValueError(f"{what}: expected CUDA tensors")
    _same_device(what, dev, first, *tensors)
    return dev


def _same_device(what: str, dev: int, *tensors: Optional[torch.Tensor]) -> None:
    for t in tensors:
        if t is not None:
            if t.get_device() != dev:
                raise ValueError(f"{what}: all tensors must be on one CUDA device")
            if not t.is_contiguous():
                raise ValueError(f"{what}: expected contiguous tensors")


def _bad(what: str, name: str, t: torch.Tensor, shape, *dtypes) -> None:
    raise ValueError(f"{what}: {name} must be {' or '.join(map(str, dtypes))} {tuple(shape)}, "
                     f"got {t.dtype} {tuple(t.shape)}")


def _want(what: str, name: str, t: torch.Tensor, shape: tuple, *dtypes) -> None:
    if t.dtype not in dtypes or t.shape != shape:
        _bad(what, name, t, shape, *dtypes)


def _elsewhere(what: str, dev: int, stream: Optional[torch.cuda.Stream]):
    """None when the call runs on the current device's current stream; else
    the context that makes its device and stream current, so that outputs and
    scratch made inside belong to that stream."""
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError(f"{what}: the stream belongs to another device than the tensors")
        return torch.cuda.stream(stream)
    return None if dev == _current_device() else torch.cuda.device(dev)


def _scratch(nbytes: int, device) -> torch.Tensor:
    return torch.empty_strided((nbytes,), (1,), dtype=_U8, device=device)


def _p(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _norm_args(what, x, weight, residual):
    if x.dtype not in _FLOATS or x.dim() < 1 or x.numel() == 0:
        raise ValueError(f"{what}: x must be a float tensor [..., D] with elements")
    shape = x.shape
    D = shape[-1]
    if weight is not None and (weight.dtype not in _FLOATS or weight.shape != (D,)):
        _bad(what, "weight", weight, (D,), *_FLOATS)
    if residual is not None and (residual.dtype not in _FLOATS or residual.shape != shape):
        _bad(what, "residual", residual, shape, *_FLOATS)
    return x.numel() // D, D


def add_rmsnorm(x: torch.Tensor, weight: Optional[torch.Tensor], eps: float = 1e-6,
                residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                out_dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """h = x + residual; residual <- h; returns h / rms(h) * weight over the
    last dimension, in `out_dtype` (default: x's).  `residual` is updated in
    place; `out` may be x."""
    what = "add_rmsnorm"
    M, D = _norm_args(what, x, weight, residual)
    if out is not None:
        _want(what, "out", out, x.shape, *_FLOATS)
    elif out_dtype is not None and out_dtype not in _FLOATS:
        raise ValueError(f"{what}: out_dtype must be float32, float16 or bfloat16")
    dev = _one_device(what, x, weight, residual, out)
    other = _elsewhere(what, dev, stream)
    if other is not None:
        with other:
            return add_rmsnorm(x, weight, eps, residual, out, out_dtype)
    if out is None:
        out = torch.empty_like(x, dtype=out_dtype)
    _check(lib.bc_add_rmsnorm(x.data_ptr(), _DT[x.dtype], _p(residual),
                              BC_F32 if residual is None else _DT[residual.dtype], _p(weight),
                              BC_F32 if weight is None else _DT[weight.dtype], M, D, eps,
                              out.data_ptr(), _DT[out.dtype], _raw_stream(dev)), "bc_add_rmsnorm")
    return out


def add_rmsnorm_q8(x: torch.Tensor, weight: Optional[torch.Tensor], eps: float = 1e-6,
                   residual: Optional[torch.Tensor] = None,
                   codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                   zeros: Optional[torch.Tensor] = None, stream=None):
    """add_rmsnorm with the output as (codes uint8 [..., D], scales, zeros fp16
    [..., D/64]): what matmul_q reads as packed weights of 8 bits."""
    what = "add_rmsnorm_q8"
    M, D = _norm_args(what, x, weight, residual)
    if D % 64:
        raise ValueError(f"{what}: D must be a multiple of 64")
    gs = (*x.shape[:-1], D // 64)
    if codes is not None:
        _want(what, "codes", codes, x.shape, _U8)
    if scales is not None:
        _want(what, "scales", scales, gs, _F16)
    if zeros is not None:
        _want(what, "zeros", zeros, gs, _F16)
    dev = _one_device(what, x, weight, residual, codes, scales, zeros)
    other = _elsewhere(what, dev, stream)
    if other is not None:
        with other:
            return add_rmsnorm_q8(x, weight, eps, residual, codes, scales, zeros)
    if codes is None:
        codes = torch.empty_like(x, dtype=_U8)
    if scales is None:
        scales = torch.empty(gs, dtype=_F16, device=x.device)
    if zeros is None:
        zeros = torch.empty(gs, dtype=_F16, device=x.device)
    _check(lib.bc_add_rmsnorm_q8(x.data_ptr(), _DT[x.dtype], _p(residual),
                                 BC_F32 if residual is None else _DT[residual.dtype], _p(weight),
                                 BC_F32 if weight is None else _DT[weight.dtype], M, D, eps,
                                 codes.data_ptr(), scales.data_ptr(), zeros.data_ptr(),
                                 _raw_stream(dev)), "bc_add_rmsnorm_q8")
    return codes, scales, zeros


class LoraDescs:
    """The projections of one lora_add_batched call (from make_lora_descs);
    holds their tensors, whatever becomes of the list that it was made from.  Keep it for the steps that use the same buffers."""
    __slots__ = ("array", "count", "M", "R", "n_adapters", "x_dtype", "w_dtype", "device", "tensors")


def make_lora_descs(items: Sequence[tuple]) -> LoraDescs:
    """items: (x, A, B, y) per projection: x [M][K] fp32 or bf16, A
    [n_adapters][R][K] and B [n_adapters][N][R] fp16 or bf16, y fp32 [M][N].
    Neighbours that read the same x share a pass over it."""
    what = "make_lora_descs"
    if not items:
        raise ValueError(f"{what}: no projections")
    x0, A0 = items[0][0], items[0][1]
    xt, wt = x0.dtype, A0.dtype
    if x0.dim() != 2 or A0.dim() != 3:
        raise ValueError(f"{what}: x must be [M][K] and A [n_adapters][R][K]")
    if xt not in (_F32, _BF16) or wt not in (_F16, _BF16):
        raise ValueError(f"{what}: x must be float32 or bfloat16, adapters float16 or bfloat16")
    M, (n, R, _) = x0.shape[0], A0.shape
    dev = x0.get_device()
    if dev < 0:
        raise ValueError(f"{what}: expected CUDA tensors")
    fields, seen = [], None
    for x, A, B, y in items:
        if x is not seen:                                   # projections in a row share their x
            K = x.shape[-1]
            if x.dtype != xt or x.shape != (M, K):
                _bad(what, "x", x, (M, K), xt)
            _same_device(what, dev, x)
            xp, seen = x.data_ptr(), x
        N = y.shape[-1]
        if A.dtype is not wt or A.shape != (n, R, K):
            _bad(what, "A", A, (n, R, K), wt)
        if B.dtype is not wt or B.shape != (n, N, R):
            _bad(what, "B", B, (n, N, R), wt)
        if y.dtype is not _F32 or y.shape != (M, N):
            _bad(what, "y", y, (M, N), _F32)
        if not (A.get_device() == B.get_device() == y.get_device() == dev and A.is_contiguous()
                and B.is_contiguous() and y.is_contiguous()):
            _same_device(what, dev, A, B, y)
        fields += (xp, A.data_ptr(), B.data_ptr(), y.data_ptr(), N, K)
    d = LoraDescs()
    d.M, d.n_adapters, d.R, d.count, d.device = M, n, R, len(items), dev
    d.x_dtype, d.w_dtype, d.tensors = _DT[xt], _DT[wt], tuple(map(tuple, items))
    d.array = struct.pack(f"{len(fields)}q", *fields)       # bc_lora_desc: six 8-byte fields
    return d


def workspace_size_lora(descs: LoraDescs, n_segments: int) -> int:
    return lib.bc_workspace_size_lora(descs.array, descs.count, descs.M, descs.R,
                                      descs.n_adapters, n_segments, descs.x_dtype)


def lora_add_batched(descs: LoraDescs, seg_start: torch.Tensor, seg_adapter: torch.Tensor,
                     ranks: Optional[torch.Tensor] = None,
                     scaling: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """y[m] += scaling[a] * B[a] (A[a] x[m]) for every projection of `descs`:
    the rows seg_start[i] .. seg_start[i+1]-1 use adapter a = seg_adapter[i]
    (outside 0..n_adapters-1: none).  seg_start int32 [S+1], seg_adapter int32
    [S]; ranks int32 and scaling fp32 [n_adapters], or None."""
    what = "lora_add_batched"
    S, n = seg_adapter.numel(), descs.n_adapters
    if seg_adapter.dtype != _I32 or seg_adapter.dim() != 1:
        _bad(what, "seg_adapter", seg_adapter, (S,), _I32)
    if seg_start.dtype != _I32 or seg_start.shape != (S + 1,):
        _bad(what, "seg_start", seg_start, (S + 1,), _I32)
    if ranks is not None and (ranks.dtype != _I32 or ranks.shape != (n,)):
        _bad(what, "ranks", ranks, (n,), _I32)
    if scaling is not None and (scaling.dtype != _F32 or scaling.shape != (n,)):
        _bad(what, "scaling", scaling, (n,), _F32)
    dev = descs.device
    _same_device(what, dev, seg_start, seg_adapter, ranks, scaling, workspace)
    other = None if stream is None and dev == _current_device() else _elsewhere(what, dev, stream)
    if other is not None:
        with other:
            return lora_add_batched(descs, seg_start, seg_adapter, ranks, scaling, workspace)
    if workspace is None:
        workspace = _scratch(workspace_size_lora(descs, S), seg_start.device)
    _check(lib.bc_lora_add_batched(descs.array, descs.count, descs.M, descs.R, n, descs.x_dtype,
                                   descs.w_dtype, seg_start.data_ptr(), seg_adapter.data_ptr(), S,
                                   _p(ranks), _p(scaling), workspace.data_ptr(), workspace.nbytes,
                                   _raw_stream(dev)), "bc_lora_add_batched")


def lora_add(x: torch.Tensor, A: torch.Tensor, B: torch.Tensor, y: torch.Tensor,
             seg_start: torch.Tensor, seg_adapter: torch.Tensor,
             ranks: Optional[torch.Tensor] = None, scaling: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """lora_add_batched for one projection; returns y."""
    lora_add_batched(make_lora_descs([(x, A, B, y)]), seg_start, seg_adapter, ranks, scaling,
                     workspace, stream)
    return y


def workspace_size_beam(batch: int, beams: int, V: int, n_out: int) -> int:
    return lib.bc_workspace_size_beam(batch, beams, V, n_out)


def _beam_out(what, device, batch, n_out, out):
    shape = (batch, n_out)
    if out is None:
        if batch <= 0 or n_out <= 0:
            raise ValueError(f"{what}: nothing to select")
        parent = torch.empty_strided(shape, (n_out, 1), dtype=_I32, device=device)
        return (torch.empty_like(parent, dtype=_F32), parent, torch.empty_like(parent),
                torch.empty_like(parent, dtype=_U8))
    for t, name, dt in zip(out, ("out scores", "parent", "token", "out finished"),
                           (_F32, _I32, _I32, _U8)):
        _want(what, name, t, shape, dt)
    return tuple(out)


def beam_select(logits: torch.Tensor, scores: torch.Tensor, n_out: int,
                finished: Optional[torch.Tensor] = None, eos: int = -1, pad: int = 0,
                out: Optional[Sequence[torch.Tensor]] = None,
                workspace: Optional[torch.Tensor] = None, stream=None):
    """The n_out best continuations of each request: logits fp32
    [batch * beams][V], scores fp32 [batch][beams], finished uint8 (or bool)
    [batch][beams].  Returns (scores fp32, parent int32, token int32, finished
    uint8), each [batch][n_out], in descending order of total."""
    what = "beam_select"
    if scores.dim() != 2 or logits.dim() != 2:
        raise ValueError(f"{what}: logits must be [batch * beams][V], scores [batch][beams]")
    batch, beams = scores.shape
    V = logits.shape[1]
    if logits.dtype is not _F32 or logits.shape[0] != batch * beams:
        _bad(what, "logits", logits, (batch * beams, V), _F32)
    if scores.dtype is not _F32:
        _bad(what, "scores", scores, (batch, beams), _F32)
    if finished is not None:
        _want(what, "finished", finished, (batch, beams), _U8, torch.bool)
    dev = _one_device(what, logits, scores, finished, workspace, *(out or ()))
    other = None if stream is None and dev == _current_device() else _elsewhere(what, dev, stream)
    if other is not None:
        with other:
            return beam_select(logits, scores, n_out, finished, eos, pad, out, workspace)
    o = _beam_out(what, logits.device, batch, n_out, out)
    if workspace is None:
        workspace = _scratch(lib.bc_workspace_size_beam(batch, beams, V, n_out), logits.device)
    _check(lib.bc_beam_select(logits.data_ptr(), scores.data_ptr(), _p(finished), batch, beams, V,
                              n_out, eos, pad, o[0].data_ptr(), o[1].data_ptr(), o[2].data_ptr(),
                              o[3].data_ptr(), workspace.data_ptr(), workspace.nbytes,
                              _raw_stream(dev)), "bc_beam_select")
    return o


def workspace_size_matmul_beam(batch: int, beams: int, N: int, K: int, n_out: int, mode: int,
                               x_dtype: int = BC_F32) -> int:
    return lib.bc_workspace_size_matmul_beam(batch, beams, N, K, n_out, mode, x_dtype)


def matmul_q_beam(x: torch.Tensor, W: torch.Tensor, scales: Optional[torch.Tensor],
                  zeros: Optional[torch.Tensor], bits: int, group: int, mode: int,
                  beam_scores: torch.Tensor, n_out: int,
                  finished: Optional[torch.Tensor] = None, eos: int = -1, pad: int = 0,
                  out: Optional[Sequence[torch.Tensor]] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None):
    """The LM head's matmul_q on x [batch * beams][K] and beam_select over its
    logits, in one call; returns what beam_select returns."""
    what = "matmul_q_beam"
    if beam_scores.dim() != 2 or x.dim() != 2 or x.shape[0] != beam_scores.numel():
        raise ValueError(f"{what}: x must be [batch * beams][K], beam_scores [batch][beams]")
    if x.dtype not in (_F32, _BF16):
        raise ValueError(f"{what}: x must be float32 or bfloat16")
    batch, beams = beam_scores.shape
    K, N = x.shape[1], W.shape[0]
    packed = mode == BC_MODE_PACKED
    _want(what, "W", W, (N, K * bits // 8) if packed else (N, K), _U8 if packed else _F16)
    if packed or bits != 16:
        groups = K // 64 if group == 64 else 1
        sz = _F16 if packed else _I32 if mode == BC_MODE_RUNTIME_RANGE else _F32
        if scales is None or (zeros is None and mode != BC_MODE_RUNTIME_RANGE):
            raise ValueError(f"{what}: this mode needs scales and zeros")
        _want(what, "scales", scales, (N, groups), sz)
        if mode != BC_MODE_RUNTIME_RANGE:
            _want(what, "zeros", zeros, (N, groups), sz)
    _want(what, "beam_scores", beam_scores, (batch, beams), _F32)
    if finished is not None:
        _want(what, "finished", finished, (batch, beams), _U8, torch.bool)
    dev = _one_device(what, x, W, scales, zeros, beam_scores, finished, workspace, *(out or ()))
    other = _elsewhere(what, dev, stream)
    if other is not None:
        with other:
            return matmul_q_beam(x, W, scales, zeros, bits, group, mode, beam_scores, n_out,
                                 finished, eos, pad, out, workspace)
    o = _beam_out(what, x.device, batch, n_out, out)
    if workspace is None:
        need = workspace_size_matmul_beam(batch, beams, N, K, n_out, mode, _DT[x.dtype])
        workspace = _scratch(need, x.device)
    _check(lib.bc_matmul_q_beam(x.data_ptr(), _DT[x.dtype], W.data_ptr(), _p(scales), _p(zeros),
                                batch, beams, N, K, bits, group, mode, beam_scores.data_ptr(),
                                _p(finished), n_out, eos, pad, o[0].data_ptr(), o[1].data_ptr(),
                                o[2].data_ptr(), o[3].data_ptr(), workspace.data_ptr(),
                                workspace.nbytes, _raw_stream(dev)), "bc_matmul_q_beam")
    return o


class BeamStates:
    """States of beam_reorder (from make_beam_states); holds their tensors,
    whatever becomes of the list that it was made from."""
    __slots__ = ("array", "count", "beams_total", "device", "tensors")


def make_beam_states(tensors: Sequence[torch.Tensor]) -> BeamStates:
    """tensors: views [batch * beams, ...] of caches or histories, of any type.
    Dimension 0 counts the beams; the others have to be runs of contiguous
    elements at one stride (a cache [batch * beams, heads, room, width] cut to
    its first `len` places is heads runs of len * width elements)."""
    what = "make_beam_states"
    if not tensors:
        raise ValueError(f"{what}: no states")
    dev, total = tensors[0].get_device(), tensors[0].shape[0]
    if dev < 0:
        raise ValueError(f"{what}: expected CUDA tensors")
    fields = []
    for i, t in enumerate(tensors):
        shape, strides, size = t.shape, t.stride(), t.element_size()
        if t.get_device() != dev:
            raise ValueError(f"{what}: all states must be on one CUDA device")
        if shape[0] != total or t.numel() == 0:
            raise ValueError(f"{what}: every state must be [batch * beams, ...] with elements")
        run, rows, row_stride = 1, 1, 0
        for k in range(len(shape) - 1, 0, -1):
            n, s = shape[k], strides[k]
            if n == 1:
                continue
            if rows == 1 and s == run:
                run *= n
            elif rows == 1:
                rows, row_stride = n, s
            elif s == row_stride * rows:
                rows *= n
            else:
                raise ValueError(f"{what}: state {i} is not runs of contiguous elements at one stride")
        if rows > 1 and row_stride < run:
            raise ValueError(f"{what}: state {i} overlaps itself")
        beam = strides[0] if total > 1 else max(strides[0], run)
        fields += (t.data_ptr(), rows, run * size, row_stride * size, beam * size)
    st = BeamStates()
    st.beams_total, st.device, st.tensors, st.count = total, dev, tuple(tensors), len(tensors)
    st.array = struct.pack(f"{len(fields)}q", *fields)      # bc_beam_state: five 8-byte fields
    return st


def beam_reorder(states, parent: torch.Tensor, stream=None) -> None:
    """new[i][w] = old[i][parent[i][w]] in place for every state: `states` are
    tensors as make_beam_states takes them, or its result; parent int32
    [batch][beams] (a view of wider rows is fine)."""
    what = "beam_reorder"
    if not isinstance(states, BeamStates):
        states = make_beam_states(states)
    if parent.dtype != _I32 or parent.dim() != 2 or (parent.stride(1) != 1 and parent.shape[1] > 1):
        raise ValueError(f"{what}: parent must be int32 [batch][beams]")
    batch, beams = parent.shape
    dev = states.device
    if parent.get_device() != dev:
        raise ValueError(f"{what}: all tensors must be on one CUDA device")
    if batch * beams != states.beams_total:
        raise ValueError(f"{what}: the states have {states.beams_total} beams, parent {batch} x {beams}")
    other = _elsewhere(what, dev, stream)
    if other is not None:
        with other:
            return beam_reorder(states, parent)
    _check(lib.bc_beam_reorder(states.array, states.count, parent.data_ptr(),
                               parent.stride(0) if batch > 1 else beams, batch, beams,
                               _raw_stream(dev)), "bc_beam_reorder")
