"""ctypes declarations of ``include/moe.h`` and thin wrappers over torch tensors."""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Dict, Optional, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_HERE, "libmoe_b200.so")

WDTYPE = {"bf16": 0, "mxfp4": 1, "nvfp4": 2, "int4": 3}
_BLOCK = {"bf16": 1, "mxfp4": 32, "nvfp4": 16, "int4": 128}

MOE_OK = 0


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({moe_status_string(status)})")


class LayerDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d_model", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("d_ff", ctypes.c_int32), ("n_shared", ctypes.c_int32),
                ("wdtype", ctypes.c_int32), ("router_fp32", ctypes.c_int32)]


class Weights(ctypes.Structure):
    _fields_ = [("w13", ctypes.c_void_p), ("s13", ctypes.c_void_p), ("w2", ctypes.c_void_p),
                ("s2", ctypes.c_void_p), ("g13", ctypes.c_void_p), ("g2", ctypes.c_void_p),
                ("stride_w13", ctypes.c_int64), ("stride_s13", ctypes.c_int64),
                ("stride_w2", ctypes.c_int64), ("stride_s2", ctypes.c_int64),
                ("slot_map", ctypes.c_void_p), ("n_physical", ctypes.c_int32)]


class GemmDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("n_experts", ctypes.c_int32), ("N", ctypes.c_int32),
                ("K", ctypes.c_int32), ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("n_physical", ctypes.c_int32), ("ld_x", ctypes.c_int64), ("ld_y", ctypes.c_int64),
                ("ld_w", ctypes.c_int64), ("stride_w", ctypes.c_int64)]


class WorkspaceLayout(ctypes.Structure):
    _fields_ = [("topk_idx", ctypes.c_size_t), ("topk_w", ctypes.c_size_t), ("offsets", ctypes.c_size_t),
                ("row_token", ctypes.c_size_t), ("inv", ctypes.c_size_t), ("total", ctypes.c_size_t)]


class CacheDesc(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("slots_per_layer", ctypes.c_int32), ("expert_bytes", ctypes.c_int64),
                ("host_bank", ctypes.c_void_p), ("device", ctypes.c_int32)]


class ProfileEntry(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 32), ("launches", ctypes.c_int64), ("total_ms", ctypes.c_double)]


class CacheStats(ctypes.Structure):
    _fields_ = [("lookups", ctypes.c_int64), ("hits", ctypes.c_int64), ("misses", ctypes.c_int64),
                ("evictions", ctypes.c_int64), ("prefetch_issued", ctypes.c_int64),
                ("prefetch_used", ctypes.c_int64), ("bytes_h2d", ctypes.c_int64), ("copy_ms", ctypes.c_double)]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


_LIB = None

_P = ctypes.c_void_p
_DP = ctypes.POINTER(LayerDesc)
_WP = ctypes.POINTER(Weights)
_GP = _P  # a GemmDesc by its address
_I32, _I64 = ctypes.c_int32, ctypes.c_int64

_SIGS = {
    "moe_workspace_size": [_DP, ctypes.POINTER(ctypes.c_size_t)],
    "moe_workspace_layout_of": [_DP, ctypes.POINTER(WorkspaceLayout)],
    "moe_route_topk": [_DP, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
    "moe_route_topk_noalloc": [_DP, _P, _P, _P, _P, _P, _P],
    "moe_permute": [_DP, _P, _P, _P, _P, _P, _P, _P],
    "moe_grouped_ffn": [_DP, _WP, _WP, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
    "moe_combine": [_DP, _P, _P, _P, _P, _P, _P],
    "moe_layer_forward": [_DP, _P, _P, _P, _WP, _WP, _P, _P, ctypes.c_size_t, _P],
    "moe_grouped_gemm": [_GP, _P, _P, _P, _P, _P, _P],
    "moe_grouped_gemm_grad_x": [_GP, _P, _P, _P, _P, _P, _P],
    "moe_grouped_gemm_grad_w": [_GP, _P, _P, _P, _P, ctypes.c_int, _P],
    "moe_grouped_gemm_i8": [_GP, _P, _P, _P, _P, _P, _P, _P, _P],
    "moe_quant_rows_i8": [_I32, _I32, _I32, _P, _I64, _P, _I32, _P, _I64, _P, _P],
    "moe_swiglu": [_I32, _I32, _I32, _P, _I64, _P, _I64, _P],
    "moe_swiglu_quant_i8": [_I32, _I32, _I32, _P, _I64, _P, _I64, _P, _P],
    "moe_swiglu_grad": [_I32, _I32, _I32, _P, _I64, _P, _I64, _P, _I64, _P],
    "moe_cache_init": [ctypes.POINTER(_P), ctypes.POINTER(CacheDesc)],
    "moe_cache_prefetch": [_P, ctypes.c_int32, ctypes.POINTER(ctypes.c_int32), ctypes.c_int32],
    "moe_cache_lookup": [_P, ctypes.c_int32, ctypes.POINTER(ctypes.c_int32), ctypes.c_int32, _P, _P],
    "moe_cache_release": [_P, ctypes.c_int32, _P],
    "moe_cache_slot_map": [_P, ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)],
    "moe_cache_stats": [_P, ctypes.POINTER(CacheStats)],
    "moe_cache_destroy": [_P],
    "moe_get_last_error": [],
    "moe_profile_enable": [ctypes.c_int],
    "moe_diag_wait_timeout": [ctypes.c_uint64, _P, _P],
    "moe_diag_wait_moving": [ctypes.c_uint64, _I32, _I32, _P, _P],
    "moe_profile_collect": [ctypes.POINTER(ProfileEntry), ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)],
}
_PTR_RET = {"moe_cache_host_expert": [_P, ctypes.c_int32, ctypes.c_int32],
            "moe_cache_slot_base": [_P, ctypes.c_int32]}

EXPORTS = sorted(list(_SIGS) + list(_PTR_RET) + ["moe_status_string"])


def lib() -> ctypes.CDLL:
    """The loaded CUDA library; raises if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(lib_path):
            raise ImportError(f"{lib_path} is missing: build it with `python -m expert_ffn_layer_route_b200.build`")
        L = ctypes.CDLL(lib_path)
        for name, args in _SIGS.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        for name, args in _PTR_RET.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_void_p
        L.moe_status_string.argtypes = [ctypes.c_int]
        L.moe_status_string.restype = ctypes.c_char_p
        _LIB = L
    return _LIB


def moe_status_string(status: int) -> str:
    try:
        return lib().moe_status_string(status).decode()
    except ImportError:
        return "?"


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoeError(status, where)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    import torch

    return torch.cuda.current_stream().cuda_stream


def router_sum_depth(d: int) -> int:
    """MOE_ROUTER_SUM_DEPTH(d) of the header."""
    return 8 * ((d + 2047) // 2048) + 12


def make_desc(shape, T: int) -> LayerDesc:
    """LayerDesc from a ``moe_inputs.LayerShape``-like object."""
    return LayerDesc(int(T), shape.d_model, shape.n_experts, shape.top_k, shape.d_ff, shape.n_shared,
                     WDTYPE[shape.wdtype], 1 if shape.router_fp32 else 0)


def make_weights(experts: Dict[str, object], slot_map=None, n_physical: int = 0,
                 strides: Optional[Sequence[int]] = None) -> Weights:
    """Weights from a dict of device tensors w13/s13/w2/s2/g13/g2 (missing = NULL)."""
    w = Weights()
    for key in ("w13", "s13", "w2", "s2", "g13", "g2"):
        setattr(w, key, _ptr(experts.get(key)))
    if strides is not None:
        w.stride_w13, w.stride_s13, w.stride_w2, w.stride_s2 = strides
    w.slot_map = _ptr(slot_map)
    w.n_physical = n_physical
    return w


def moe_workspace_size(desc: LayerDesc) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_workspace_size(ctypes.byref(desc), ctypes.byref(n)), "moe_workspace_size")
    return n.value


def moe_workspace_layout_of(desc: LayerDesc) -> WorkspaceLayout:
    out = WorkspaceLayout()
    _check(lib().moe_workspace_layout_of(ctypes.byref(desc), ctypes.byref(out)), "moe_workspace_layout_of")
    return out


def moe_route_topk(desc, x, w_router, logit_bias, topk_idx, topk_w, workspace, stream=None):
    _check(lib().moe_route_topk(ctypes.byref(desc), _ptr(x), _ptr(w_router), _ptr(logit_bias), _ptr(topk_idx),
                                _ptr(topk_w), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                _stream(stream)), "moe_route_topk")


def moe_route_topk_noalloc(desc, x, w_router, logit_bias, topk_idx, topk_w, stream=None):
    """moe_route_topk with the library's fixed scratch (for callers that cannot allocate)."""
    _check(lib().moe_route_topk_noalloc(ctypes.byref(desc), _ptr(x), _ptr(w_router), _ptr(logit_bias),
                                        _ptr(topk_idx), _ptr(topk_w), _stream(stream)), "moe_route_topk_noalloc")


def moe_permute(desc, topk_idx, offsets, row_token, inv, stream=None, x=None, x_perm=None):
    """Grouping; with ``x`` also gathers x_perm[r] = x[row_token[r]]."""
    _check(lib().moe_permute(ctypes.byref(desc), _ptr(topk_idx), _ptr(x), _ptr(offsets), _ptr(row_token),
                             _ptr(inv), _ptr(x_perm), _stream(stream)), "moe_permute")


def moe_grouped_ffn(desc, routed: Weights, shared: Optional[Weights], offsets, row_token, x, y_perm, y_shared,
                    workspace, stream=None):
    _check(lib().moe_grouped_ffn(ctypes.byref(desc), ctypes.byref(routed),
                                 ctypes.byref(shared) if shared is not None else None, _ptr(offsets),
                                 _ptr(row_token), _ptr(x), _ptr(y_perm), _ptr(y_shared), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(stream)),
           "moe_grouped_ffn")


def moe_combine(desc, y_perm, inv, topk_w, y_shared, out, stream=None):
    _check(lib().moe_combine(ctypes.byref(desc), _ptr(y_perm), _ptr(inv), _ptr(topk_w), _ptr(y_shared), _ptr(out),
                             _stream(stream)), "moe_combine")


def moe_layer_forward(desc, x, w_router, logit_bias, routed: Weights, shared: Optional[Weights], out, workspace,
                      stream=None):
    _check(lib().moe_layer_forward(ctypes.byref(desc), _ptr(x), _ptr(w_router), _ptr(logit_bias),
                                   ctypes.byref(routed), ctypes.byref(shared) if shared is not None else None,
                                   _ptr(out), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                   _stream(stream)), "moe_layer_forward")


# ---------------------------------------------------------------------------
# Expert operators.  These take whole tensors and read sizes, types and pitches
# off them, so they also check them: the C entry points see only pointers.  A
# single-token call takes the GPU a few microseconds, so what depends on sizes,
# pitches and types alone is checked once for each combination of them (the
# cached functions below; a refusal raises and is not kept).

_TYPE = {}  # torch dtype -> moe_dtype, filled on first use (torch is imported late)
_torch = _raw_stream = _current = None


def _setup():
    global _torch, _raw_stream, _current
    import torch

    lib()
    _TYPE.update({torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, torch.int8: 3})
    _raw_stream, _current = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    _torch = torch


def _refuse(where: str, why: str):
    raise MoeError(1, f"{where}: {why}")


def _pitch(shape, stride, rows, cols, where, name) -> int:
    """Row pitch of what has to be a [rows][cols] matrix of contiguous rows."""
    if shape != (rows, cols):
        _refuse(where, f"{name} has shape {tuple(shape)}, ({rows}, {cols}) is wanted")
    if stride[1] != 1 and cols > 1:
        _refuse(where, f"{name}'s rows are not contiguous")
    if rows > 1 and stride[0] < cols:  # (an expanded tensor: 0, which C would read as "not given")
        _refuse(where, f"{name}'s rows overlap (a copy by contiguous() would not)")
    return stride[0] if rows > 1 else (cols + 15) & -16


def _vector(t, n, dtype, where, name):
    if t.dim() != 1 or t.shape[0] < n or t.dtype != dtype or (t.shape[0] > 1 and t.stride(0) != 1):
        _refuse(where, f"{name} has to be a contiguous {dtype} vector of at least {n} values")


@functools.lru_cache(maxsize=1024)
def _gemm_desc(where, w_name, w, w_stride, w_type, x_name, x, x_stride, x_type, y_name, y, y_stride, y_type, off,
               off_stride, off_type, by_slots, a_type, b_type, out_type):
    """(description, its address, rows, experts, matrices, N) of a grouped product.  The caller holds the description
    itself until its call is over (two threads may both make one, and only one of them is kept).  w [M][N][K], x [R][K],
    y [R][N] and offsets [E + 1], by their shapes, strides and types; a_type, b_type, out_type: the types of the
    two operands and of the result."""
    if len(w) != 3:
        _refuse(where, f"{w_name} has {len(w)} dimensions, 3 are wanted")
    M, N, K = w
    if len(off) != 1 or off[0] < 2 or off_type != _torch.int32 or off_stride[0] != 1:
        _refuse(where, "offsets has to be a contiguous int32 vector of E + 1 values")
    E = off[0] - 1
    if not by_slots and M != E:
        _refuse(where, f"{M} matrices for {E} experts (a slot_map would say which is whose)")
    R = x[0] if len(x) else -1
    int8 = where == "moe_grouped_gemm_i8"
    t, to = _TYPE.get(a_type, 9), _TYPE.get(out_type, 9)
    if a_type != b_type or to > 2 or (t != 3 if int8 else t > 1):
        _refuse(where, f"types {a_type}, {b_type} -> {out_type}")
    ld_x = _pitch(x, x_stride, R, K, where, x_name)
    ld_y = _pitch(y, y_stride, R, N, where, y_name)
    if w_stride[2] != 1 and K > 1:
        _refuse(where, f"{w_name}'s rows are not contiguous")
    if N > 1 and w_stride[1] < K:
        _refuse(where, f"{w_name}'s rows overlap (a copy by contiguous() would not)")
    ld_w = w_stride[1] if N > 1 else (K + 15) & -16
    if M > 1 and w_stride[0] < (N - 1) * ld_w + K:
        _refuse(where, f"{w_name}'s matrices overlap (a slot_map says which experts share a matrix)")
    d = GemmDesc(R, E, N, K, t, to, M, ld_x, ld_y, ld_w, w_stride[0] if M > 1 else N * ld_w)
    return d, ctypes.addressof(d), R, E, M, N


def _call(where, index, f, stream, *args):
    """f(*args, stream) on GPU `index`; stream None: the current one there."""
    if stream is None:
        stream = _raw_stream(index)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if _current() == index:
        status = f(*args, stream)
    else:
        with _torch.cuda.device(index):
            status = f(*args, stream)
    if status != MOE_OK:
        raise MoeError(status, where)


def _one_gpu(where, *tensors) -> int:
    """Index of the GPU that all of the tensors lie on."""
    index = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != index:
            index = -1
    if index < 0:
        _refuse(where, "the tensors have to be on one CUDA device")
    return index


def moe_grouped_gemm(x, w, offsets, out, slot_map=None, stream=None):
    """out[r] = x[r] w[e]^T for the rows r of each expert e (x [R][K], w [E][N][K], out [R][N])."""
    where = "moe_grouped_gemm"
    if _torch is None:
        _setup()
    desc, d, _, E, _, _ = _gemm_desc(where, "w", w.shape, w.stride(), w.dtype, "x", x.shape, x.stride(), x.dtype,
                                     "out", out.shape, out.stride(), out.dtype, offsets.shape, offsets.stride(),
                                     offsets.dtype, slot_map is not None, x.dtype, w.dtype, out.dtype)
    if slot_map is not None:
        _vector(slot_map, E, _torch.int32, where, "slot_map")
    _call(where, _one_gpu(where, x, w, offsets, out, slot_map), _LIB.moe_grouped_gemm, stream, d, x.data_ptr(),
          w.data_ptr(), _ptr(slot_map), offsets.data_ptr(), out.data_ptr())


def moe_grouped_gemm_grad_x(dy, w, offsets, dx, slot_map=None, stream=None):
    """dx[r] = dy[r] w[e] for the rows r of each expert e (dy [R][N], w [E][N][K], dx [R][K])."""
    where = "moe_grouped_gemm_grad_x"
    if _torch is None:
        _setup()
    desc, d, _, E, _, _ = _gemm_desc(where, "w", w.shape, w.stride(), w.dtype, "dx", dx.shape, dx.stride(), dx.dtype,
                                     "dy", dy.shape, dy.stride(), dy.dtype, offsets.shape, offsets.stride(),
                                     offsets.dtype, slot_map is not None, dy.dtype, w.dtype, dx.dtype)
    if slot_map is not None:
        _vector(slot_map, E, _torch.int32, where, "slot_map")
    _call(where, _one_gpu(where, dy, w, offsets, dx, slot_map), _LIB.moe_grouped_gemm_grad_x, stream, d,
          dy.data_ptr(), w.data_ptr(), _ptr(slot_map), offsets.data_ptr(), dx.data_ptr())


def moe_grouped_gemm_grad_w(dy, x, offsets, dw, accumulate=False, stream=None):
    """dw[e] (+)= dy[rows of e]^T x[rows of e] (dy [R][N], x [R][K], dw [E][N][K])."""
    where = "moe_grouped_gemm_grad_w"
    if _torch is None:
        _setup()
    desc, d, _, _, _, _ = _gemm_desc(where, "dw", dw.shape, dw.stride(), dw.dtype, "x", x.shape, x.stride(), x.dtype,
                                     "dy", dy.shape, dy.stride(), dy.dtype, offsets.shape, offsets.stride(),
                                     offsets.dtype, False, dy.dtype, x.dtype, dw.dtype)
    _call(where, _one_gpu(where, dy, x, offsets, dw), _LIB.moe_grouped_gemm_grad_w, stream, d, dy.data_ptr(),
          x.data_ptr(), offsets.data_ptr(), dw.data_ptr(), 1 if accumulate else 0)


def moe_grouped_gemm_i8(x, x_scale, w, w_scale, offsets, out, slot_map=None, stream=None):
    """out[r][n] = x_scale[r] w_scale[e][n] sum_k x[r][k] w[e][n][k] over int8 codes x [R][K], w [E][N][K]."""
    where = "moe_grouped_gemm_i8"
    if _torch is None:
        _setup()
    desc, d, R, E, M, N = _gemm_desc(where, "w", w.shape, w.stride(), w.dtype, "x", x.shape, x.stride(), x.dtype,
                                     "out", out.shape, out.stride(), out.dtype, offsets.shape, offsets.stride(),
                                     offsets.dtype, slot_map is not None, x.dtype, w.dtype, out.dtype)
    _vector(x_scale, R, _torch.float32, where, "x_scale")
    if w_scale.shape != (M, N) or w_scale.dtype != _torch.float32 or not w_scale.is_contiguous():
        _refuse(where, f"w_scale has to be a contiguous float32 tensor of shape ({M}, {N})")
    if slot_map is not None:
        _vector(slot_map, E, _torch.int32, where, "slot_map")
    _call(where, _one_gpu(where, x, x_scale, w, w_scale, offsets, out, slot_map), _LIB.moe_grouped_gemm_i8, stream, d,
          x.data_ptr(), x_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(), _ptr(slot_map), offsets.data_ptr(),
          out.data_ptr())


@functools.lru_cache(maxsize=1024)
def _quant_sizes(where, x, x_stride, x_type, q, q_stride, q_type, gather):
    """(rows, K, type, pitch of x, rows of x, pitch of q)"""
    if len(x) != 2 or len(q) != 2:
        _refuse(where, "x and q have to be matrices")
    t = _TYPE.get(x_type, 9)
    if t > 1 or q_type != _torch.int8:
        _refuse(where, f"types {x_type} -> {q_type}")
    if not gather and x[0] != q[0]:
        _refuse(where, f"{x[0]} rows of x, {q[0]} of q")
    K = x[1]
    return q[0], K, t, _pitch(x, x_stride, x[0], K, where, "x"), x[0], _pitch(q, q_stride, q[0], K, where, "q")


def moe_quant_rows_i8(x, q, scale, row_token=None, stream=None):
    """int8 codes q [R][K] and scale [R] of the rows of x, or of x[row_token[r]] (a dropped row: zeros)."""
    where = "moe_quant_rows_i8"
    if _torch is None:
        _setup()
    R, K, t, ld_x, T, ld_q = _quant_sizes(where, x.shape, x.stride(), x.dtype, q.shape, q.stride(), q.dtype,
                                          row_token is not None)
    if row_token is not None:
        _vector(row_token, R, _torch.int32, where, "row_token")
    _vector(scale, R, _torch.float32, where, "scale")
    _call(where, _one_gpu(where, x, q, scale, row_token), _LIB.moe_quant_rows_i8, stream, R, K, t, x.data_ptr(), ld_x,
          _ptr(row_token), T, q.data_ptr(), ld_q, scale.data_ptr())


@functools.lru_cache(maxsize=1024)
def _swiglu_sizes(where, gu, gu_stride, gu_type, *others):
    """(rows, F, type, pitch of gate_up, pitches of the others); others: name, factor of F, shape, stride, type."""
    t = _TYPE.get(gu_type, 9)
    if len(gu) != 2 or gu[1] & 1 or t > 1:
        _refuse(where, "gate_up has to be a bf16 or fp16 matrix [R][2F]")
    R, F = gu[0], gu[1] >> 1
    out = [R, F, t, _pitch(gu, gu_stride, R, 2 * F, where, "gate_up")]
    for i in range(0, len(others), 5):
        name, factor, shape, stride, dtype = others[i: i + 5]
        if dtype != (_torch.int8 if name == "q" else gu_type):
            _refuse(where, f"types {gu_type} -> {dtype}")
        out.append(_pitch(shape, stride, R, factor * F, where, name))
    return out


def moe_swiglu(gate_up, h, stream=None):
    """h = silu(gate_up[:, :F]) * gate_up[:, F:] (h [R][F])."""
    where = "moe_swiglu"
    if _torch is None:
        _setup()
    R, F, t, ld, ld_h = _swiglu_sizes(where, gate_up.shape, gate_up.stride(), gate_up.dtype, "h", 1, h.shape,
                                      h.stride(), h.dtype)
    _call(where, _one_gpu(where, gate_up, h), _LIB.moe_swiglu, stream, R, F, t, gate_up.data_ptr(), ld, h.data_ptr(),
          ld_h)


def moe_swiglu_quant_i8(gate_up, q, scale, stream=None):
    """int8 codes q [R][F] and scale [R] of silu(gate_up[:, :F]) * gate_up[:, F:]."""
    where = "moe_swiglu_quant_i8"
    if _torch is None:
        _setup()
    R, F, t, ld, ld_q = _swiglu_sizes(where, gate_up.shape, gate_up.stride(), gate_up.dtype, "q", 1, q.shape,
                                      q.stride(), q.dtype)
    _vector(scale, R, _torch.float32, where, "scale")
    _call(where, _one_gpu(where, gate_up, q, scale), _LIB.moe_swiglu_quant_i8, stream, R, F, t, gate_up.data_ptr(),
          ld, q.data_ptr(), ld_q, scale.data_ptr())


def moe_swiglu_grad(gate_up, dh, dgate_up, stream=None):
    """dgate_up [R][2F], the gradient of moe_swiglu at gate_up for a given dh [R][F]; it may be gate_up itself."""
    where = "moe_swiglu_grad"
    if _torch is None:
        _setup()
    R, F, t, ld, ld_h, ld_d = _swiglu_sizes(where, gate_up.shape, gate_up.stride(), gate_up.dtype, "dh", 1, dh.shape,
                                            dh.stride(), dh.dtype, "dgate_up", 2, dgate_up.shape, dgate_up.stride(),
                                            dgate_up.dtype)
    _call(where, _one_gpu(where, gate_up, dh, dgate_up), _LIB.moe_swiglu_grad, stream, R, F, t, gate_up.data_ptr(), ld,
          dh.data_ptr(), ld_h, dgate_up.data_ptr(), ld_d)


def moe_get_last_error() -> int:
    return lib().moe_get_last_error()


def moe_diag_wait_timeout(limit_ns: int, finished, stream=None):
    _check(lib().moe_diag_wait_timeout(int(limit_ns), _ptr(finished), _stream(stream)), "moe_diag_wait_timeout")


def moe_diag_wait_moving(limit_ns: int, moves: int, complete: bool, finished, stream=None):
    _check(lib().moe_diag_wait_moving(int(limit_ns), moves, int(complete), _ptr(finished), _stream(stream)),
           "moe_diag_wait_moving")


def moe_profile_enable(on: bool = True):
    _check(lib().moe_profile_enable(1 if on else 0), "moe_profile_enable")


def moe_profile_collect() -> dict:
    """{kernel name: (launches, total ms)} recorded since the last collect."""
    cap = 64
    arr = (ProfileEntry * cap)()
    n = ctypes.c_int32()
    _check(lib().moe_profile_collect(arr, cap, ctypes.byref(n)), "moe_profile_collect")
    return {arr[i].name.decode(): (arr[i].launches, arr[i].total_ms) for i in range(min(n.value, cap))}


class ExpertCache:
    """Owner of one ``moe_cache`` (per-layer LRU over HBM slots + pinned host bank)."""

    def __init__(self, n_layers: int, n_experts: int, slots_per_layer: int, expert_bytes: int, device: int = 0,
                 host_bank: Optional[int] = None):
        self.desc = CacheDesc(n_layers, n_experts, slots_per_layer, expert_bytes, host_bank, device)
        h = ctypes.c_void_p()
        _check(lib().moe_cache_init(ctypes.byref(h), ctypes.byref(self.desc)), "moe_cache_init")
        self.handle = h
        self.n_experts = n_experts

    def host_expert(self, layer: int, e: int) -> int:
        return lib().moe_cache_host_expert(self.handle, layer, e)

    def slot_base(self, layer: int) -> int:
        return lib().moe_cache_slot_base(self.handle, layer)

    @staticmethod
    def _ints(xs):
        xs = [int(v) for v in xs]
        return (ctypes.c_int32 * max(len(xs), 1))(*xs), len(xs)

    def prefetch(self, layer: int, experts):
        arr, n = self._ints(experts)
        _check(lib().moe_cache_prefetch(self.handle, layer, arr, n), "moe_cache_prefetch")

    def lookup(self, layer: int, experts, slot_map_dev, stream=None):
        """slot_map_dev may be None for a policy-only cache (device < 0)."""
        arr, n = self._ints(experts)
        st = _stream(stream) if self.desc.device >= 0 else None
        _check(lib().moe_cache_lookup(self.handle, layer, arr, n, _ptr(slot_map_dev), st), "moe_cache_lookup")

    def release(self, layer: int, stream=None):
        st = _stream(stream) if self.desc.device >= 0 else None
        _check(lib().moe_cache_release(self.handle, layer, st), "moe_cache_release")

    def slot_map(self, layer: int):
        out = (ctypes.c_int32 * self.n_experts)()
        _check(lib().moe_cache_slot_map(self.handle, layer, out), "moe_cache_slot_map")
        return list(out)

    def stats(self) -> dict:
        s = CacheStats()
        _check(lib().moe_cache_stats(self.handle, ctypes.byref(s)), "moe_cache_stats")
        return s.as_dict()

    def close(self):
        if self.handle:
            _check(lib().moe_cache_destroy(self.handle), "moe_cache_destroy")
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
