"""Python binding of libmoegmm.so: the routed-expert W4A16 grouped matmul for
MI355X (gfx950).

Thin ctypes marshalling over the C ABI in include/moe_gmm.h: every function
takes torch CUDA tensors, passes their device pointers and the current HIP
stream, allocates outputs with torch, and raises on a non-zero status.  All
arithmetic runs in the library's HIP kernels; there is no fallback path.  The
library is loaded on first use and its absence is an error.
"""

import ctypes
import os

import torch

__all__ = [
    "MXFP4", "NVFP4", "W_BF16", "F32", "BF16", "GMM_AUTO", "GMM_STREAM", "GMM_TILED", "ACT_NONE", "ACT_SILU_MUL",
    "MoeGmmError", "library", "route_sort", "route_sort_workspace_bytes", "packed_weight_bytes", "mxfp4_encode",
    "moe_gmm", "moe_combine", "mxfp4_to_nvfp4", "debug_decode", "bf16_encode",
    "mxfp4_quantize", "moe_gmm_w4a4",
    "GATE_SOFTMAX", "GATE_SIGMOID", "topk_gate", "topk_gate_bwd", "moe_dispatch", "moe_dispatch_bwd",
    "moe_combine_bwd", "silu_mul", "moe_gmm_dgrad",
    "w4_gemv", "gate_up", "gate_up_bwd", "gate_up_bwd_workspace_bytes",
]

MXFP4, NVFP4, W_BF16 = 0, 1, 2
F32, BF16 = 0, 1
GMM_AUTO, GMM_STREAM, GMM_TILED = 0, 1, 2
ACT_NONE, ACT_SILU_MUL = 0, 1
GATE_SOFTMAX, GATE_SIGMOID = 0, 1

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoegmm.so")
_lib = None

_vp, _i32, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
_SIGNATURES = {
    "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "moe_route_sort_workspace_bytes": (_sz, [_i32, _i32, _i32]),
    "moe_route_sort": (ctypes.c_int, [_vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_route_sort_noalloc": (ctypes.c_int, [_vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp]),
    "moe_packed_weight_bytes": (_sz, [ctypes.c_int, _i32, _i32, _i32]),
    "mxfp4_encode": (ctypes.c_int, [ctypes.c_int, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp]),
    "moe_bf16_encode": (ctypes.c_int, [_vp, _i32, _i32, _i32, _vp, _vp]),
    "moe_mxfp4_quantize": (ctypes.c_int, [_vp, _i32, _i32, _vp, _vp, _vp]),
    "moe_gmm_w4a4": (ctypes.c_int, [_vp, ctypes.c_int, _i32, _i32, _i32, _vp, _vp, _i32, _vp, _vp, _i32, _vp,
                                    ctypes.c_int, ctypes.c_int, _vp, _vp]),
    "moe_gmm": (ctypes.c_int, [_vp, ctypes.c_int, _i32, _i32, _i32, _vp, _i32, _vp, _vp, _i32,
                               _vp, ctypes.c_int, _vp]),
    "moe_gmm_ex": (ctypes.c_int, [_vp, ctypes.c_int, _i32, _i32, _i32, _vp, _i32, _vp, _vp, _i32,
                                  _vp, ctypes.c_int, ctypes.c_int, _vp]),
    "moe_gmm_act": (ctypes.c_int, [_vp, ctypes.c_int, _i32, _i32, _i32, _vp, _i32, _vp, _vp, _i32,
                                   _vp, ctypes.c_int, ctypes.c_int, ctypes.c_int, _vp]),
    "moe_combine": (ctypes.c_int, [_vp, ctypes.c_int, _vp, _vp, _i32, _i32, _i32, _vp,
                                   ctypes.c_int, _vp]),
    "moe_mxfp4_to_nvfp4": (ctypes.c_int, [_vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp]),
    "moe_topk_gate": (ctypes.c_int, [_vp, ctypes.c_int, _vp, _i32, _i32, _i32, ctypes.c_int, ctypes.c_int,
                                     ctypes.c_float, _vp, _vp, _vp]),
    "moe_topk_gate_bwd": (ctypes.c_int, [_vp, ctypes.c_int, _vp, _vp, _i32, _i32, _i32, ctypes.c_int, ctypes.c_int,
                                         ctypes.c_float, _vp, _vp]),
    "moe_dispatch": (ctypes.c_int, [_vp, ctypes.c_int, _vp, _i32, _i32, _i32, _i32, _vp, _vp]),
    "moe_dispatch_bwd": (ctypes.c_int, [_vp, ctypes.c_int, _vp, _i32, _i32, _i32, _i32, _vp, ctypes.c_int, _vp]),
    "moe_combine_bwd": (ctypes.c_int, [_vp, ctypes.c_int, _vp, ctypes.c_int, _vp, _vp, _i32, _i32, _i32, _i32,
                                       _vp, ctypes.c_int, _vp, _vp]),
    "moe_silu_mul": (ctypes.c_int, [_vp, ctypes.c_int, _i32, _i32, _vp, _vp, ctypes.c_int, _vp]),
    "moe_gmm_dgrad": (ctypes.c_int, [_vp, ctypes.c_int, _i32, _i32, _i32, _vp, _vp, _i32, _vp, ctypes.c_int, _vp,
                                     ctypes.c_int, ctypes.c_int, _vp]),
    "moe_w4_gemv": (ctypes.c_int, [_vp, _vp, ctypes.c_int, _vp, _i32, _i32, _i32, _i32, _vp, _i32, _i32, _vp, _vp,
                                   _i32, _vp, ctypes.c_int, ctypes.c_int, _vp]),
    "moe_gate_up": (ctypes.c_int, [_vp, _vp, _i32, _i32, _i32, _vp, ctypes.c_int, _vp, ctypes.c_int, _vp]),
    "moe_gate_up_bwd": (ctypes.c_int, [_vp, ctypes.c_int, _vp, _vp, _vp, ctypes.c_int, _i32, _i32, _i32, _vp,
                                       ctypes.c_int, _vp, ctypes.c_int, _vp, _sz, _vp]),
    "moe_gate_up_bwd_workspace_bytes": (_sz, [_i32, _i32, _i32, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                              ctypes.c_int]),
    "moe_debug_decode": (ctypes.c_int, [_vp, ctypes.c_int, _i32, _i32, _i32, _vp, _vp]),
    "moe_calib_mfma_bf16": (ctypes.c_int, [_vp, _vp, _i32, _i32, _vp, _vp]),
    "moe_calib_hbm_read": (ctypes.c_int, [_vp, _sz, _i32, _vp, _vp]),
    "moe_calib_mfma_parts": (ctypes.c_int, [_i32, _i32, _vp, _vp, _vp, _sz, _vp, _sz, ctypes.c_float, _i32, _i32,
                                            _vp, _vp]),
}


class MoeGmmError(RuntimeError):
    pass


def library():
    """The loaded libmoegmm.so (ctypes.CDLL).  torch is imported first so the
    library binds to the HIP runtime torch already loaded."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise MoeGmmError(
                "libmoegmm.so is not built (%s); run python -m moe_grouped_gemm_route_amd.build"
                % _LIB_PATH)
        lib = ctypes.CDLL(_LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _check(status):
    if status != 0:
        msg = library().moe_status_string(status).decode()
        raise MoeGmmError("libmoegmm status %d: %s" % (status, msg))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    """The current stream of the current device, as a pointer value."""
    return _raw_stream(torch.cuda.current_device())


# the pointer without a Stream object around it (2.7 us of a call otherwise)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _dev(t, dtype, name, ndim=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise MoeGmmError("%s must be a CUDA (HIP) tensor" % name)
    if t.dtype != dtype:
        raise MoeGmmError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise MoeGmmError("%s must be contiguous" % name)
    if ndim is not None and t.dim() != ndim:
        raise MoeGmmError("%s must have %d dims" % (name, ndim))
    return t


def _bits16(t, name):
    """bf16 tensors (or their uint16/int16 bit views) as a 16-bit view."""
    if t.dtype == torch.bfloat16:
        t = t.view(torch.int16)
    if t.dtype == torch.uint16:
        t = t.view(torch.int16)
    return _dev(t, torch.int16, name)


def route_sort_workspace_bytes(T, k, E):
    """moe_route_sort_workspace_bytes: device workspace bytes of a route sort
    of T tokens x k slots over E experts (0 when none is needed)."""
    return int(library().moe_route_sort_workspace_bytes(T, k, E))


def route_sort(topk_ids, E, ws=None):
    """moe_route_sort.  topk_ids [T, k] int32 -> dict of int32 tensors
    group_offsets [E+1], sorted_token, sorted_pair, pair_row [T*k] and
    err_count [1].  ws: a device tensor of at least
    route_sort_workspace_bytes(T, k, E) bytes, or None to allocate one."""
    _dev(topk_ids, torch.int32, "topk_ids", 2)
    T, k = topk_ids.shape
    dev = topk_ids.device
    out = {
        "group_offsets": torch.empty(E + 1, dtype=torch.int32, device=dev),
        "sorted_token": torch.empty(T * k, dtype=torch.int32, device=dev),
        "sorted_pair": torch.empty(T * k, dtype=torch.int32, device=dev),
        "pair_row": torch.empty(T * k, dtype=torch.int32, device=dev),
        "err_count": torch.empty(1, dtype=torch.int32, device=dev),
    }
    need = route_sort_workspace_bytes(T, k, E)
    if ws is None and need > 0:
        ws = torch.empty((need + 3) // 4, dtype=torch.int32, device=dev)
    if ws is not None:
        if not isinstance(ws, torch.Tensor) or not ws.is_cuda or not ws.is_contiguous():
            raise MoeGmmError("ws must be a contiguous CUDA (HIP) tensor")
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(library().moe_route_sort(
        _ptr(topk_ids), T, k, E, _ptr(out["group_offsets"]), _ptr(out["sorted_token"]),
        _ptr(out["sorted_pair"]), _ptr(out["pair_row"]), _ptr(out["err_count"]), _ptr(ws), ws_bytes,
        _stream()))
    return out


def packed_weight_bytes(fmt, E, N, K):
    n = library().moe_packed_weight_bytes(fmt, E, N, K)
    if n == 0 or (fmt | E | N | K) >> 31:   # (ctypes passes the low 32 bits)
        raise MoeGmmError("unsupported weight shape E=%d N=%d K=%d" % (E, N, K))
    return n


def mxfp4_encode(codes, scales, tensor_scale=None, fmt=MXFP4, err_count=None):
    """mxfp4_encode.  codes [E, N, K/2] uint8, scales [E, N, K/32] (MXFP4) or
    [E, N, K/16] (NVFP4) uint8, tensor_scale [E] float32 (NVFP4 only).
    Returns the packed uint8 buffer.  err_count: an optional [1] int32 device
    tensor that receives the number of scale values outside the exact-decode
    domain."""
    _dev(codes, torch.uint8, "codes", 3)
    _dev(scales, torch.uint8, "scales", 3)
    E, N, K2 = codes.shape
    K = 2 * K2
    per = 32 if fmt == MXFP4 else 16
    if tuple(scales.shape) != (E, N, K // per):
        raise MoeGmmError("scales must be [E, N, K/%d]" % per)
    if fmt == NVFP4:
        _dev(tensor_scale, torch.float32, "tensor_scale", 1)
    packed = torch.empty(packed_weight_bytes(fmt, E, N, K), dtype=torch.uint8, device=codes.device)
    if err_count is not None:
        _dev(err_count, torch.int32, "err_count", 1)
    _check(library().mxfp4_encode(fmt, _ptr(codes), _ptr(scales), _ptr(tensor_scale), E, N, K,
                                  _ptr(packed), _ptr(err_count), _stream()))
    return packed


def bf16_encode(weights):
    """moe_bf16_encode.  weights [E, N, K] bfloat16 (or its int16/uint16 bit
    view) -> the packed uint8 buffer of the bf16 comparison arm."""
    wb = _bits16(weights, "weights")
    if wb.dim() != 3:
        raise MoeGmmError("weights must be [E, N, K]")
    E, N, K = wb.shape
    packed = torch.empty(packed_weight_bytes(W_BF16, E, N, K), dtype=torch.uint8, device=wb.device)
    _check(library().moe_bf16_encode(_ptr(wb), E, N, K, _ptr(packed), _stream()))
    return packed


def moe_gmm(packed, fmt, E, N, K, x, group_offsets, M, row_index=None, out_dtype=F32,
            kernel=GMM_AUTO, out=None, act=ACT_NONE):
    """moe_gmm_act.  x: bf16 [T, K] (gathered through row_index) or [M, K].
    Returns y [M, N] (act=ACT_NONE) or [M, N/2] (act=ACT_SILU_MUL), float32 or
    bfloat16."""
    _dev(packed, torch.uint8, "packed", 1)
    xb = _bits16(x, "x")
    _dev(group_offsets, torch.int32, "group_offsets", 1)
    if group_offsets.numel() != E + 1:
        raise MoeGmmError("group_offsets must have E+1 entries")
    if xb.dim() != 2 or xb.shape[1] != K:
        raise MoeGmmError("x must be [rows, K]")
    if row_index is None:
        if xb.shape[0] < M:
            raise MoeGmmError("x must have M rows when row_index is None")
    else:
        _dev(row_index, torch.int32, "row_index", 1)
        if row_index.numel() < M:
            raise MoeGmmError("row_index must have M entries")
    if packed.numel() < packed_weight_bytes(fmt, E, N, K):
        raise MoeGmmError("packed buffer too small")
    dt = torch.float32 if out_dtype == F32 else torch.bfloat16
    cols = N // 2 if act == ACT_SILU_MUL else N
    if out is None:
        out = torch.empty((M, cols), dtype=dt, device=packed.device)
    else:
        _dev(out, dt, "out", 2)
        if tuple(out.shape) != (M, cols):
            raise MoeGmmError("out must be [M, %d]" % cols)
    _check(library().moe_gmm_act(_ptr(packed), fmt, E, N, K, _ptr(xb), xb.shape[0], _ptr(row_index),
                                 _ptr(group_offsets), M, _ptr(out), out_dtype, act, kernel,
                                 _stream()))
    return out


def mxfp4_quantize(x):
    """moe_mxfp4_quantize.  x bf16 [R, K] -> (codes [R, K/2] uint8, scales
    [R, K/32] uint8)."""
    xb = _bits16(x, "x")
    if xb.dim() != 2 or xb.shape[1] % 32:
        raise MoeGmmError("x must be [R, K] with K a multiple of 32")
    R, K = xb.shape
    codes = torch.empty((R, K // 2), dtype=torch.uint8, device=xb.device)
    scales = torch.empty((R, K // 32), dtype=torch.uint8, device=xb.device)
    _check(library().moe_mxfp4_quantize(_ptr(xb), R, K, _ptr(codes), _ptr(scales), _stream()))
    return codes, scales


def moe_gmm_w4a4(packed, E, N, K, xq_codes, xq_scales, group_offsets, M, row_index=None,
                 out_dtype=F32, act=ACT_NONE, out=None, fmt=MXFP4, err_count=None):
    """moe_gmm_w4a4.  xq_codes [rows, K/2], xq_scales [rows, K/32] from
    mxfp4_quantize; packed MXFP4 or NVFP4 (power-of-two block scales)
    weights.  Returns y [M, N] or [M, N/2].  err_count: an optional [1] int32
    device tensor that receives the NVFP4 weight blocks whose scales do not
    qualify."""
    _dev(packed, torch.uint8, "packed", 1)
    _dev(xq_codes, torch.uint8, "xq_codes", 2)
    _dev(xq_scales, torch.uint8, "xq_scales", 2)
    _dev(group_offsets, torch.int32, "group_offsets", 1)
    rows = xq_codes.shape[0]
    if tuple(xq_codes.shape) != (rows, K // 2) or tuple(xq_scales.shape) != (rows, K // 32):
        raise MoeGmmError("xq_codes must be [rows, K/2] and xq_scales [rows, K/32]")
    if group_offsets.numel() != E + 1:
        raise MoeGmmError("group_offsets must have E+1 entries")
    if row_index is None:
        if rows < M:
            raise MoeGmmError("the activations must have M rows when row_index is None")
    else:
        _dev(row_index, torch.int32, "row_index", 1)
        if row_index.numel() < M:
            raise MoeGmmError("row_index must have M entries")
    if packed.numel() < packed_weight_bytes(fmt, E, N, K):
        raise MoeGmmError("packed buffer too small")
    dt = torch.float32 if out_dtype == F32 else torch.bfloat16
    cols = N // 2 if act == ACT_SILU_MUL else N
    if out is None:
        out = torch.empty((M, cols), dtype=dt, device=packed.device)
    else:
        _dev(out, dt, "out", 2)
        if tuple(out.shape) != (M, cols):
            raise MoeGmmError("out must be [M, %d]" % cols)
    if err_count is not None:
        _dev(err_count, torch.int32, "err_count", 1)
    _check(library().moe_gmm_w4a4(_ptr(packed), fmt, E, N, K, _ptr(xq_codes), _ptr(xq_scales), rows,
                                  _ptr(row_index), _ptr(group_offsets), M, _ptr(out), out_dtype, act,
                                  _ptr(err_count), _stream()))
    return out


def moe_combine(y, topk_weights, pair_row, out_dtype=F32):
    """moe_combine.  y [rows, N] float32/bfloat16, topk_weights [T, k] float32,
    pair_row [T*k] int32 -> out [T, N]."""
    if y.dtype not in (torch.float32, torch.bfloat16):
        raise MoeGmmError("y must be float32 or bfloat16")
    _dev(y, y.dtype, "y", 2)
    _dev(topk_weights, torch.float32, "topk_weights", 2)
    _dev(pair_row, torch.int32, "pair_row", 1)
    T, k = topk_weights.shape
    N = y.shape[1]
    if pair_row.numel() != T * k:
        raise MoeGmmError("pair_row must have T*k entries")
    dt = torch.float32 if out_dtype == F32 else torch.bfloat16
    out = torch.empty((T, N), dtype=dt, device=y.device)
    _check(library().moe_combine(_ptr(y), F32 if y.dtype == torch.float32 else BF16,
                                 _ptr(topk_weights), _ptr(pair_row), T, k, N, _ptr(out),
                                 out_dtype, _stream()))
    return out


_FLOATS = {torch.float32: F32, torch.bfloat16: BF16}
_OUT = {F32: torch.float32, BF16: torch.bfloat16}
_Tensor = torch.Tensor
_I32_MIN, _I32_MAX = -(1 << 31), (1 << 31) - 1


def _float(t, name, ndim):
    """A contiguous float32 or bfloat16 device tensor; returns its dtype enum."""
    dt = _FLOATS.get(getattr(t, "dtype", None))
    if dt is None:
        raise MoeGmmError("%s must be a float32 or bfloat16 tensor" % name)
    if not (t.is_cuda and t.is_contiguous() and t.dim() == ndim):
        _dev(t, t.dtype, name, ndim)
    return dt


def _out(out, shape, dtype, name, like):
    """out checked, or a new tensor beside `like`; dtype is an F32/BF16 enum or
    its torch dtype."""
    dtype = _OUT.get(dtype, dtype)
    if dtype not in _FLOATS:
        raise MoeGmmError("the type of %s must be F32 or BF16" % name)
    if out is None:
        return like.new_empty(shape, dtype=dtype)
    _dev(out, dtype, name, len(shape))
    if tuple(out.shape) != tuple(shape):
        raise MoeGmmError("%s must be %s" % (name, list(shape)))
    return out


def _too_wide(a):
    """A whole number that the C entry's int32 does not hold (ctypes would pass
    its low 32 bits)."""
    raise MoeGmmError("%d does not fit 32 bits" % a)


def _launch(fn, tensors, *args):
    """fn(*args, stream) on the device that holds every tensor of tensors (None
    skipped), on that device's current stream.  A tensor in args stands for its
    pointer; whole numbers are int32."""
    index = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise MoeGmmError("the tensors must be on one device, got %s and %s" % (tensors[0].device, t.device))
    args = [(a if _I32_MIN <= a <= _I32_MAX else _too_wide(a)) if type(a) is int else
            a.data_ptr() if isinstance(a, _Tensor) else a for a in args]
    if index == torch.cuda.current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status:
        _check(status)


def topk_gate(logits, k, score=GATE_SOFTMAX, bias=None, renormalize=True, scale=1.0):
    """moe_topk_gate.  logits [T, E] float32 or bfloat16, bias [E] float32 or
    None -> (topk_ids [T, k] int32, topk_weights [T, k] float32), as
    route_sort and moe_combine take them."""
    dt = _float(logits, "logits", 2)
    T, E = logits.shape
    if bias is not None:
        _dev(bias, torch.float32, "bias", 1)
        if bias.numel() != E:
            raise MoeGmmError("bias must have E entries")
    if not 1 <= k <= E:
        raise MoeGmmError("k must be 1 to E")
    ids = logits.new_empty((T, k), dtype=torch.int32)
    weights = logits.new_empty((T, k), dtype=torch.float32)
    _launch(library().moe_topk_gate, (logits, bias), logits, dt, bias, T, E, k, score,
            int(bool(renormalize)), float(scale), ids, weights)
    return ids, weights


def topk_gate_bwd(logits, topk_ids, dweights, score=GATE_SOFTMAX, renormalize=True, scale=1.0):
    """moe_topk_gate_bwd.  logits [T, E] and the score, renormalize and scale
    given to topk_gate, its topk_ids [T, k], dweights [T, k] float32 ->
    dlogits [T, E] of the logits' type."""
    dt = _float(logits, "logits", 2)
    _dev(topk_ids, torch.int32, "topk_ids", 2)
    _dev(dweights, torch.float32, "dweights", 2)
    T, E = logits.shape
    if topk_ids.shape[0] != T or dweights.shape != topk_ids.shape:
        raise MoeGmmError("topk_ids and dweights must be [T, k]")
    out = torch.empty_like(logits)
    _launch(library().moe_topk_gate_bwd, (logits, topk_ids, dweights), logits, dt, topk_ids,
            dweights, T, E, topk_ids.shape[1], score, int(bool(renormalize)), float(scale), out)
    return out


def _pairs(pair_row, k):
    """pair_row checked against k slots per token; returns T."""
    _dev(pair_row, torch.int32, "pair_row", 1)
    if k < 1 or pair_row.numel() % k:
        raise MoeGmmError("pair_row must have T*k entries")
    return pair_row.numel() // k


def moe_dispatch(x, pair_row, k, out=None):
    """moe_dispatch.  x [T, N] float32 or bfloat16, pair_row [T*k] int32 (no
    row twice) -> xs [T*k, N] of x's type (or out, [rows, N]); rows no pair
    names are left as they were."""
    dt = _float(x, "x", 2)
    T, N = x.shape
    if _pairs(pair_row, k) != T:
        raise MoeGmmError("pair_row must have T*k entries")
    rows = T * k
    if out is not None:
        _dev(out, x.dtype, "out", 2)
        rows = out.shape[0]
    out = _out(out, (rows, N), x.dtype, "out", x)
    _launch(library().moe_dispatch, (x, pair_row, out), x, dt, pair_row, T, k, N, rows, out)
    return out


def moe_dispatch_bwd(dxs, pair_row, k, out_dtype=F32):
    """moe_dispatch_bwd.  dxs [rows, N] float32 or bfloat16, pair_row [T*k]
    int32 -> dx [T, N]."""
    dt = _float(dxs, "dxs", 2)
    T = _pairs(pair_row, k)
    rows, N = dxs.shape
    dx = _out(None, (T, N), out_dtype, "dx", dxs)
    _launch(library().moe_dispatch_bwd, (dxs, pair_row), dxs, dt, pair_row, T, k, N, rows, dx,
            _FLOATS[dx.dtype])
    return dx


def moe_combine_bwd(dout, y, topk_weights, pair_row, out_dtype=F32, out=None):
    """moe_combine_bwd.  dout [T, N] and y [rows, N] float32 or bfloat16,
    topk_weights [T, k] float32, pair_row [T*k] int32 (no row twice) ->
    (dy [rows, N], dweights [T, k] float32).  out: a [rows, N] tensor for dy
    whose rows no pair names are left as they were."""
    gdt = _float(dout, "dout", 2)
    ydt = _float(y, "y", 2)
    _dev(topk_weights, torch.float32, "topk_weights", 2)
    T, k = topk_weights.shape
    rows, N = y.shape
    if _pairs(pair_row, k) != T or tuple(dout.shape) != (T, N):
        raise MoeGmmError("dout must be [T, N] and pair_row must have T*k entries")
    dy = _out(out, (rows, N), out_dtype, "out", y)
    dweights = torch.empty_like(topk_weights)
    _launch(library().moe_combine_bwd, (dout, y, topk_weights, pair_row, dy), dout, gdt, y, ydt,
            topk_weights, pair_row, T, k, N, rows, dy, _FLOATS[dy.dtype], dweights)
    return dy, dweights


def silu_mul(y, group_offsets=None, out_dtype=F32, out=None):
    """moe_silu_mul.  y [M, N] float32 or bfloat16 -> h [M, N/2].  With
    group_offsets [E+1] int32 only the rows of its bands are read and
    written."""
    dt = _float(y, "y", 2)
    M, N = y.shape
    n_rows = None
    if group_offsets is not None:
        _dev(group_offsets, torch.int32, "group_offsets", 1)
        if group_offsets.numel() < 2:
            raise MoeGmmError("group_offsets must have E+1 entries")
        n_rows = _vp(group_offsets.data_ptr() + 4 * (group_offsets.numel() - 1))
    h = _out(out, (M, N // 2), out_dtype, "out", y)
    _launch(library().moe_silu_mul, (y, group_offsets, h), y, dt, M, N, n_rows, h, _FLOATS[h.dtype])
    return h


def moe_gmm_dgrad(packed, fmt, E, N, K, dy, group_offsets, M, out_dtype=F32, act=ACT_NONE, preact=None, out=None):
    """moe_gmm_dgrad.  dy bf16 [M, N] in band order -> dx [M, K], the gradient
    of moe_gmm's input (act=ACT_NONE), or with act=ACT_SILU_MUL and preact
    [M, 2K] float32 or bfloat16 the gradient [M, 2K] of the gate/up sums whose
    activation that input was."""
    _dev(packed, torch.uint8, "packed", 1)
    db = _bits16(dy, "dy")
    _dev(group_offsets, torch.int32, "group_offsets", 1)
    if group_offsets.numel() != E + 1:
        raise MoeGmmError("group_offsets must have E+1 entries")
    if tuple(db.shape) != (M, N):
        raise MoeGmmError("dy must be [M, N]")
    if packed.numel() < packed_weight_bytes(fmt, E, N, K):
        raise MoeGmmError("packed buffer too small")
    pdt = F32
    if preact is not None:
        pdt = _float(preact, "preact", 2)
        if tuple(preact.shape) != (M, 2 * K):
            raise MoeGmmError("preact must be [M, 2K]")
    dx = _out(out, (M, 2 * K if act == ACT_SILU_MUL else K), out_dtype, "out", packed)
    _launch(library().moe_gmm_dgrad, (packed, db, group_offsets, preact, dx), packed, fmt, E, N, K, db,
            group_offsets, M, preact, pdt, dx, _FLOATS[dx.dtype], act)
    return dx


# What a small call costs is its checks: these read each property once.
_U8, _I32, _F32T, _BF16T, _I16, _U16 = (torch.uint8, torch.int32, torch.float32, torch.bfloat16, torch.int16,
                                        torch.uint16)
_WANTED = {None, F32, BF16}
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _is(t, dtype, ndim, name):
    """t checked as a contiguous device tensor."""
    if not (isinstance(t, _Tensor) and t.dtype is dtype and t.is_cuda and t.dim() == ndim and t.is_contiguous()):
        _dev(t, dtype, name, ndim)


def _is_bits16(t, name):
    """t checked as a contiguous 2-d device tensor of bfloat16 or its 16-bit views."""
    if not (isinstance(t, _Tensor) and t.dtype is _BF16T and t.is_cuda and t.dim() == 2 and t.is_contiguous()):
        _dev(t, t.dtype if getattr(t, "dtype", None) in (_BF16T, _I16, _U16) else _BF16T, name, 2)


def _one_device(index, *tensors):
    for t in tensors:
        if t is not None and not (isinstance(t, _Tensor) and t.get_device() == index):
            raise MoeGmmError("the tensors must be on one device, got cuda:%d and %s"
                              % (index, getattr(t, "device", type(t))))


def _enqueue(fn, index, args):
    """fn(*args, stream) on device index, on its current stream."""
    if index == _current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status:
        _check(status)


def w4_gemv(codes, scales, x, zeros=None, topk_ids=None, topk_weights=None, out_dtype=F32, act=ACT_NONE, out=None):
    """moe_w4_gemv: a few rows times 4-bit integer weights with group scales.
    Dense: codes [N, K/2] uint8, scales [N, K/G] float32 or bfloat16, zeros
    [N, K/G] uint8 or None (8 everywhere), x bf16 [T, K] -> y [T, N].
    With topk_ids [T, k] int32: codes [E, N, K/2], scales and zeros [E, N, K/G],
    x [T, K] or [T*k, K] -> y [T*k, N], a row per pair (zeros for an id outside
    [0, E)); with topk_weights [T, k] float32 -> y [T, N], a token's rows summed.
    act=ACT_SILU_MUL: N/2 columns (not with topk_weights).  out: a tensor of
    out_dtype to write."""
    nd = 2 if topk_ids is None else 3
    _is(codes, _U8, nd, "codes")
    sdt = _float(scales, "scales", nd)
    _is_bits16(x, "x")
    lead, slead = codes.shape, scales.shape
    N, K2 = lead[-2:]
    rows, K = x.shape
    groups = slead[-1]
    if K != 2 * K2 or slead[:-1] != lead[:-1] or groups < 1 or K % groups:
        raise MoeGmmError("codes must be [.., N, K/2] and scales [.., N, K/G] for x [rows, K]")
    if zeros is not None:
        _is(zeros, _U8, nd, "zeros")
        if zeros.shape != slead:
            raise MoeGmmError("zeros must have the shape of scales")
    E, T, k, out_rows = 1, rows, 1, rows
    ids = weights = None
    if topk_ids is not None:
        _is(topk_ids, _I32, 2, "topk_ids")
        E = lead[0]
        T, k = topk_ids.shape
        out_rows = T * k
        ids = topk_ids.data_ptr()
        if rows != T and rows != out_rows:
            raise MoeGmmError("x must have T or T*k rows")
    if topk_weights is not None:
        if ids is None:
            raise MoeGmmError("topk_weights go with topk_ids")
        _is(topk_weights, _F32T, 2, "topk_weights")
        if topk_weights.shape != topk_ids.shape:
            raise MoeGmmError("topk_weights must be [T, k]")
        out_rows = T
        weights = topk_weights.data_ptr()
    if (E | N | K | rows | T | k) >> 31:
        _too_wide(max(E, N, K, rows, T, k))
    index = codes.get_device()
    _one_device(index, scales, x, zeros, topk_ids, topk_weights, out)
    y = _out(out, (out_rows, N // 2 if act == ACT_SILU_MUL else N), out_dtype, "out", scales)
    _enqueue(library().moe_w4_gemv, index,
             (codes.data_ptr(), scales.data_ptr(), sdt, None if zeros is None else zeros.data_ptr(), K // groups, E, N,
              K, x.data_ptr(), rows, T, ids, weights, k, y.data_ptr(), _FLOATS[y.dtype], act))
    return y


def _gate_up_shape(x, w13):
    """M, N, K of x [M, K] and w13 [N, K] bf16."""
    _is_bits16(x, "x")
    _is_bits16(w13, "w13")
    M, K = x.shape
    N, K1 = w13.shape
    if K != K1 or N % 2:
        raise MoeGmmError("x must be [M, K] and w13 [N, K] with N even")
    if (M | N | K) >> 31:
        _too_wide(max(M, N, K))
    return M, N, K


def gate_up(x, w13, out_dtype=F32, preact_dtype=None, out=None, preact=None):
    """moe_gate_up.  x bf16 [M, K], w13 bf16 [N, K] (gate rows, then up rows) ->
    h [M, N/2]; with preact_dtype (F32 or BF16), or a preact tensor [M, N] to
    write, (h, preact): the sums that gate_up_bwd takes.  out: a tensor of
    out_dtype to write."""
    M, N, K = _gate_up_shape(x, w13)
    index = x.get_device()
    _one_device(index, w13, out, preact)
    h = _out(out, (M, N // 2), out_dtype, "out", x)
    pre, pdt = None, F32
    if preact is not None or preact_dtype is not None:
        preact = _out(preact, (M, N), preact.dtype if preact_dtype is None else preact_dtype, "preact", x)
        pre, pdt = preact.data_ptr(), _FLOATS[preact.dtype]
    _enqueue(library().moe_gate_up, index,
             (x.data_ptr(), w13.data_ptr(), M, N, K, h.data_ptr(), _FLOATS[h.dtype], pre, pdt))
    return h if preact is None else (h, preact)


def gate_up_bwd_workspace_bytes(M, N, K, dx_dtype=F32, dw_dtype=F32):
    """moe_gate_up_bwd_workspace_bytes; a dtype of None: that gradient is not
    wanted."""
    dx_dtype, dw_dtype = _FLOATS.get(dx_dtype, dx_dtype), _FLOATS.get(dw_dtype, dw_dtype)
    if (M | N | K) >> 31 or not {dx_dtype, dw_dtype} <= _WANTED:   # (ctypes passes the low 32 bits)
        return 0
    return library().moe_gate_up_bwd_workspace_bytes(M, N, K, dx_dtype is not None, dx_dtype or 0,
                                                     dw_dtype is not None, dw_dtype or 0)


def gate_up_bwd(dh, x, w13, preact, dx_dtype=F32, dw_dtype=F32, dx=None, dw13=None, ws=None):
    """moe_gate_up_bwd.  dh [M, N/2] float32 or bfloat16, x and w13 as given to
    gate_up, the preact it kept -> (dx [M, K], dw13 [N, K]); a dtype of None
    leaves that gradient out (None in its place).  dx, dw13: tensors to write, whose
    types stand for dx_dtype and dw_dtype.
    ws: a device tensor of at least gate_up_bwd_workspace_bytes, 256-byte
    aligned, or None to allocate one."""
    hdt = _float(dh, "dh", 2)
    pdt = _float(preact, "preact", 2)
    M, N, K = _gate_up_shape(x, w13)
    if dh.shape != (M, N // 2) or preact.shape != (M, N):
        raise MoeGmmError("dh must be [M, N/2] and preact [M, N]")
    index = x.get_device()
    _one_device(index, dh, w13, preact, dx, dw13, ws)
    if dx is not None or dx_dtype is not None:
        dx = _out(dx, (M, K), dx_dtype if dx is None else dx.dtype, "dx", x)
    if dw13 is not None or dw_dtype is not None:
        dw13 = _out(dw13, (N, K), dw_dtype if dw13 is None else dw13.dtype, "dw13", x)
    xdt, wdt = (None if t is None else _FLOATS[t.dtype] for t in (dx, dw13))
    if ws is None:
        ws = x.new_empty(gate_up_bwd_workspace_bytes(M, N, K, xdt, wdt) or 1, dtype=_U8)
    elif not isinstance(ws, _Tensor) or not ws.is_cuda or not ws.is_contiguous():
        raise MoeGmmError("ws must be a contiguous CUDA (HIP) tensor")
    _enqueue(library().moe_gate_up_bwd, index,
             (dh.data_ptr(), hdt, x.data_ptr(), w13.data_ptr(), preact.data_ptr(), pdt, M, N, K,
              None if dx is None else dx.data_ptr(), xdt or 0, None if dw13 is None else dw13.data_ptr(), wdt or 0,
              ws.data_ptr(), ws.numel() * ws.element_size()))
    return dx, dw13


def mxfp4_to_nvfp4(scales):
    """moe_mxfp4_to_nvfp4.  scales [E, N, K/32] uint8 E8M0 ->
    (block_scales [E, N, K/16] uint8 E4M3, tensor_scale [E] float32,
    err_count [1] int32)."""
    _dev(scales, torch.uint8, "scales", 3)
    E, N, KB = scales.shape
    bs = torch.empty((E, N, 2 * KB), dtype=torch.uint8, device=scales.device)
    ts = torch.empty(E, dtype=torch.float32, device=scales.device)
    err = torch.empty(1, dtype=torch.int32, device=scales.device)
    _check(library().moe_mxfp4_to_nvfp4(_ptr(scales), E, N, 32 * KB, _ptr(bs), _ptr(ts),
                                        _ptr(err), _stream()))
    return bs, ts, err


def debug_decode(packed, fmt, E, N, K):
    """moe_debug_decode -> dense bf16 bit patterns [E, N, K] (int16 view)."""
    _dev(packed, torch.uint8, "packed", 1)
    w = torch.empty((E, N, K), dtype=torch.int16, device=packed.device)
    _check(library().moe_debug_decode(_ptr(packed), fmt, E, N, K, _ptr(w), _stream()))
    return w


def calib_mfma_bf16(a, b, blocks, iters):
    """moe_calib_mfma_bf16: blocks workgroups of 4 waves, each wave issuing
    iters * 128 bf16 MFMAs (16x16x32) on register-resident fragments taken
    from a ([blocks*256*8*8] bf16 bits) and b ([blocks*256*4*8]).  Returns the
    [blocks*256] f32 sums; FLOPs = blocks * 4 * iters * 128 * 16384."""
    a = _bits16(a, "a")
    b = _bits16(b, "b")
    lanes = blocks * 256
    if a.numel() < lanes * 64 or b.numel() < lanes * 32:
        raise MoeGmmError("calib_mfma_bf16: a needs %d and b %d bf16 values" % (lanes * 64, lanes * 32))
    out = torch.empty(lanes, dtype=torch.float32, device=a.device)
    _check(library().moe_calib_mfma_bf16(_ptr(a), _ptr(b), blocks, iters, _ptr(out), _stream()))
    return out


PARTS_LDS_A, PARTS_CODES, PARTS_STAGE, PARTS_BARRIER, PARTS_REG_DECODE, PARTS_CODES_XOR = 1, 2, 4, 8, 16, 32


def calib_mfma_parts(parts, rows16, a, b, codes, x, scale, blocks, chunks):
    """moe_calib_mfma_parts: the tiled kernel's wave tile (rows16 row subtiles
    x 4 column subtiles) over chunks 128-deep chunks per wave, with the data
    movement named by parts (PARTS_* bits).  a and b as for calib_mfma_bf16;
    codes and x are device buffers (any dtype) of the code stream and the
    staging source.  Returns the [blocks*256] f32 sums; FLOPs = blocks * 4 *
    chunks * 4 * rows16 * 4 * 16384."""
    a = _bits16(a, "a")
    b = _bits16(b, "b")
    lanes = blocks * 256
    if a.numel() < lanes * 64 or b.numel() < lanes * 32:
        raise MoeGmmError("calib_mfma_parts: a needs %d and b %d bf16 values" % (lanes * 64, lanes * 32))
    for name, t in (("codes", codes), ("x", x)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
            raise MoeGmmError("%s must be a contiguous CUDA (HIP) tensor" % name)
    out = torch.empty(lanes, dtype=torch.float32, device=a.device)
    _check(library().moe_calib_mfma_parts(parts, rows16, _ptr(a), _ptr(b), _ptr(codes),
                                          codes.numel() * codes.element_size(), _ptr(x),
                                          x.numel() * x.element_size(), float(scale), blocks, chunks, _ptr(out),
                                          _stream()))
    return out


def calib_hbm_read(src, blocks):
    """moe_calib_hbm_read: blocks workgroups of 256 threads stream the device
    buffer src (16-byte aligned, a multiple of 16 bytes) with 16-byte loads.
    Returns the [blocks * 256] uint32 XOR partials (as int32 bits)."""
    if not isinstance(src, torch.Tensor) or not src.is_cuda or not src.is_contiguous():
        raise MoeGmmError("src must be a contiguous CUDA (HIP) tensor")
    nbytes = src.numel() * src.element_size()
    out = torch.empty(blocks * 256, dtype=torch.int32, device=src.device)
    _check(library().moe_calib_hbm_read(_ptr(src), nbytes, blocks, _ptr(out), _stream()))
    return out
