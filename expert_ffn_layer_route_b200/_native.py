"""ctypes declarations of ``include/moe.h`` and thin wrappers over torch tensors."""
from __future__ import annotations

import ctypes
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
_GP = ctypes.POINTER(GemmDesc)
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
# off them, so they also check them: the C entry points see only pointers.

_DTYPE = {}  # torch dtype -> moe_dtype, filled on first use (torch is imported late)


def _dtypes():
    if not _DTYPE:
        import torch

        _DTYPE.update({torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, torch.int8: 3})
    return _DTYPE


def _refuse(where: str, why: str):
    raise MoeError(1, f"{where}: {why}")


def _rows_of(t, rows, cols, where, name) -> int:
    """Pitch of a [rows][cols] tensor whose rows are contiguous."""
    if t.dim() != 2:
        _refuse(where, f"{name} has {t.dim()} dimensions, 2 are wanted")
    if tuple(t.shape) != (rows, cols):
        _refuse(where, f"{name} has shape {tuple(t.shape)}, ({rows}, {cols}) is wanted")
    s = t.stride()
    if s[1] != 1 and cols > 1:
        _refuse(where, f"{name}'s rows are not contiguous")
    return s[0] if rows > 1 else (cols + 15) // 16 * 16


def _matrices_of(t, E, N, K, where, name):
    """(row pitch, distance of the matrices) of an [E][N][K] tensor."""
    if t.dim() != 3 or t.shape[1] != N or t.shape[2] != K or (E is not None and t.shape[0] != E):
        _refuse(where, f"{name} has shape {tuple(t.shape)}, ({'E' if E is None else E}, {N}, {K}) is wanted")
    s = t.stride()
    if s[2] != 1 and K > 1:
        _refuse(where, f"{name}'s rows are not contiguous")
    ld = s[1] if N > 1 else (K + 15) // 16 * 16
    return ld, (s[0] if t.shape[0] > 1 else N * ld)


def _vector(t, n, dtype, where, name):
    if t.dim() != 1 or t.shape[0] < n or t.dtype != dtype or (t.shape[0] > 1 and t.stride(0) != 1):
        _refuse(where, f"{name} has to be a contiguous {dtype} vector of at least {n} values")


def _place(where, stream, *tensors):
    """(device index, raw stream) of a call on these tensors, which have to lie on one GPU."""
    import torch

    dev = tensors[0].device
    for t in tensors:
        if t is not None and (not t.is_cuda or t.device != dev):
            _refuse(where, "the tensors have to be on one CUDA device")
    if stream is None:
        return dev.index, torch._C._cuda_getCurrentRawStream(dev.index)
    return dev.index, stream if isinstance(stream, int) else stream.cuda_stream


def _launch(where, index, call, *args):
    """call(*args) with device `index` current."""
    import torch

    if torch._C._cuda_getDevice() == index:
        status = call(*args)
    else:
        with torch.cuda.device(index):
            status = call(*args)
    if status != MOE_OK:
        raise MoeError(status, where)


def _groups(offsets, slot_map, E_w, where):
    """Number of experts of a grouped product (E from offsets, checked against the matrices)."""
    import torch

    if offsets.dim() != 1 or offsets.shape[0] < 2 or offsets.dtype != torch.int32 or offsets.stride(0) != 1:
        _refuse(where, "offsets has to be a contiguous int32 vector of E + 1 values")
    E = offsets.shape[0] - 1
    if slot_map is not None:
        _vector(slot_map, E, torch.int32, where, "slot_map")
    elif E_w != E:
        _refuse(where, f"{E_w} matrices for {E} experts (a slot_map would say which is whose)")
    return E


def moe_grouped_gemm(x, w, offsets, out, slot_map=None, stream=None):
    """out[r] = x[r] w[e]^T for the rows r of each expert e (x [R][K], w [E][N][K], out [R][N])."""
    where = "moe_grouped_gemm"
    types = _dtypes()
    if w.dim() != 3:
        _refuse(where, "w has to be [E][N][K]")
    Ew, N, K = w.shape
    E = _groups(offsets, slot_map, Ew, where)
    R = x.shape[0]
    if x.dtype != w.dtype or types.get(x.dtype, 9) > 1 or types.get(out.dtype, 9) > 2:
        _refuse(where, f"types {x.dtype}, {w.dtype} -> {out.dtype}")
    ldx = _rows_of(x, R, K, where, "x")
    ldy = _rows_of(out, R, N, where, "out")
    ldw, sw = _matrices_of(w, None, N, K, where, "w")
    d = GemmDesc(R, E, N, K, types[x.dtype], types[out.dtype], Ew, ldx, ldy, ldw, sw)
    dev, st = _place(where, stream, x, w, offsets, out, slot_map)
    _launch(where, dev, lib().moe_grouped_gemm, d, x.data_ptr(), w.data_ptr(), _ptr(slot_map), offsets.data_ptr(),
            out.data_ptr(), st)


def moe_grouped_gemm_grad_x(dy, w, offsets, dx, slot_map=None, stream=None):
    """dx[r] = dy[r] w[e] for the rows r of each expert e (dy [R][N], w [E][N][K], dx [R][K])."""
    where = "moe_grouped_gemm_grad_x"
    types = _dtypes()
    if w.dim() != 3:
        _refuse(where, "w has to be [E][N][K]")
    Ew, N, K = w.shape
    E = _groups(offsets, slot_map, Ew, where)
    R = dy.shape[0]
    if dy.dtype != w.dtype or types.get(dy.dtype, 9) > 1 or types.get(dx.dtype, 9) > 2:
        _refuse(where, f"types {dy.dtype}, {w.dtype} -> {dx.dtype}")
    ldy = _rows_of(dy, R, N, where, "dy")
    ldx = _rows_of(dx, R, K, where, "dx")
    ldw, sw = _matrices_of(w, None, N, K, where, "w")
    d = GemmDesc(R, E, N, K, types[dy.dtype], types[dx.dtype], Ew, ldx, ldy, ldw, sw)
    dev, st = _place(where, stream, dy, w, offsets, dx, slot_map)
    _launch(where, dev, lib().moe_grouped_gemm_grad_x, d, dy.data_ptr(), w.data_ptr(), _ptr(slot_map),
            offsets.data_ptr(), dx.data_ptr(), st)


def moe_grouped_gemm_grad_w(dy, x, offsets, dw, accumulate=False, stream=None):
    """dw[e] (+)= dy[rows of e]^T x[rows of e] (dy [R][N], x [R][K], dw [E][N][K])."""
    where = "moe_grouped_gemm_grad_w"
    types = _dtypes()
    if dw.dim() != 3:
        _refuse(where, "dw has to be [E][N][K]")
    E, N, K = dw.shape
    _groups(offsets, None, E, where)
    R = x.shape[0]
    if x.dtype != dy.dtype or types.get(x.dtype, 9) > 1 or types.get(dw.dtype, 9) > 2:
        _refuse(where, f"types {dy.dtype}, {x.dtype} -> {dw.dtype}")
    ldx = _rows_of(x, R, K, where, "x")
    ldy = _rows_of(dy, R, N, where, "dy")
    ldw, sw = _matrices_of(dw, E, N, K, where, "dw")
    d = GemmDesc(R, E, N, K, types[x.dtype], types[dw.dtype], 0, ldx, ldy, ldw, sw)
    dev, st = _place(where, stream, dw, x, dy, offsets)
    _launch(where, dev, lib().moe_grouped_gemm_grad_w, d, dy.data_ptr(), x.data_ptr(), offsets.data_ptr(),
            dw.data_ptr(), 1 if accumulate else 0, st)


def moe_grouped_gemm_i8(x, x_scale, w, w_scale, offsets, out, slot_map=None, stream=None):
    """out[r][n] = x_scale[r] w_scale[e][n] sum_k x[r][k] w[e][n][k] over int8 codes x [R][K], w [E][N][K]."""
    import torch

    where = "moe_grouped_gemm_i8"
    types = _dtypes()
    if w.dim() != 3:
        _refuse(where, "w has to be [E][N][K]")
    Ew, N, K = w.shape
    E = _groups(offsets, slot_map, Ew, where)
    R = x.shape[0]
    if x.dtype != torch.int8 or w.dtype != torch.int8 or types.get(out.dtype, 9) > 2:
        _refuse(where, f"types {x.dtype}, {w.dtype} -> {out.dtype}")
    ldx = _rows_of(x, R, K, where, "x")
    ldy = _rows_of(out, R, N, where, "out")
    ldw, sw = _matrices_of(w, None, N, K, where, "w")
    _vector(x_scale, R, torch.float32, where, "x_scale")
    if tuple(w_scale.shape) != (Ew, N) or w_scale.dtype != torch.float32 or not w_scale.is_contiguous():
        _refuse(where, f"w_scale has to be a contiguous float32 tensor of shape ({Ew}, {N})")
    d = GemmDesc(R, E, N, K, 3, types[out.dtype], Ew, ldx, ldy, ldw, sw)
    dev, st = _place(where, stream, x, x_scale, w, w_scale, offsets, out, slot_map)
    _launch(where, dev, lib().moe_grouped_gemm_i8, d, x.data_ptr(), x_scale.data_ptr(), w.data_ptr(),
            w_scale.data_ptr(), _ptr(slot_map), offsets.data_ptr(), out.data_ptr(), st)


def moe_quant_rows_i8(x, q, scale, row_token=None, stream=None):
    """int8 codes q [R][K] and scale [R] of the rows of x, or of x[row_token[r]] (a dropped row: zeros)."""
    import torch

    where = "moe_quant_rows_i8"
    types = _dtypes()
    if x.dim() != 2 or q.dim() != 2:
        _refuse(where, "x and q have to be matrices")
    T, K = x.shape
    R = q.shape[0]
    if types.get(x.dtype, 9) > 1 or q.dtype != torch.int8:
        _refuse(where, f"types {x.dtype} -> {q.dtype}")
    if row_token is None:
        if T != R:
            _refuse(where, f"{T} rows of x, {R} of q")
    else:
        _vector(row_token, R, torch.int32, where, "row_token")
    ldx = _rows_of(x, T, K, where, "x")
    ldq = _rows_of(q, R, K, where, "q")
    _vector(scale, R, torch.float32, where, "scale")
    dev, st = _place(where, stream, x, q, scale, row_token)
    _launch(where, dev, lib().moe_quant_rows_i8, R, K, types[x.dtype], x.data_ptr(), ldx, _ptr(row_token), T,
            q.data_ptr(), ldq, scale.data_ptr(), st)


def _gate_up(gate_up, where):
    if gate_up.dim() != 2 or gate_up.shape[1] % 2 or _dtypes().get(gate_up.dtype, 9) > 1:
        _refuse(where, "gate_up has to be a bf16 or fp16 matrix [R][2F]")
    R, F2 = gate_up.shape
    return R, F2 // 2, _rows_of(gate_up, R, F2, where, "gate_up")


def moe_swiglu(gate_up, h, stream=None):
    """h = silu(gate_up[:, :F]) * gate_up[:, F:] (h [R][F])."""
    where = "moe_swiglu"
    R, F, ldg = _gate_up(gate_up, where)
    if h.dtype != gate_up.dtype:
        _refuse(where, f"types {gate_up.dtype} -> {h.dtype}")
    ldh = _rows_of(h, R, F, where, "h")
    dev, st = _place(where, stream, gate_up, h)
    _launch(where, dev, lib().moe_swiglu, R, F, _DTYPE[h.dtype], gate_up.data_ptr(), ldg, h.data_ptr(), ldh, st)


def moe_swiglu_quant_i8(gate_up, q, scale, stream=None):
    """int8 codes q [R][F] and scale [R] of silu(gate_up[:, :F]) * gate_up[:, F:]."""
    import torch

    where = "moe_swiglu_quant_i8"
    R, F, ldg = _gate_up(gate_up, where)
    if q.dtype != torch.int8:
        _refuse(where, f"types {gate_up.dtype} -> {q.dtype}")
    ldq = _rows_of(q, R, F, where, "q")
    _vector(scale, R, torch.float32, where, "scale")
    dev, st = _place(where, stream, gate_up, q, scale)
    _launch(where, dev, lib().moe_swiglu_quant_i8, R, F, _DTYPE[gate_up.dtype], gate_up.data_ptr(), ldg,
            q.data_ptr(), ldq, scale.data_ptr(), st)


def moe_swiglu_grad(gate_up, dh, dgate_up, stream=None):
    """dgate_up [R][2F], the gradient of moe_swiglu at gate_up for a given dh [R][F]; it may be gate_up itself."""
    where = "moe_swiglu_grad"
    R, F, ldg = _gate_up(gate_up, where)
    if dh.dtype != gate_up.dtype or dgate_up.dtype != gate_up.dtype:
        _refuse(where, f"types {gate_up.dtype}, {dh.dtype} -> {dgate_up.dtype}")
    ldh = _rows_of(dh, R, F, where, "dh")
    ldd = _rows_of(dgate_up, R, 2 * F, where, "dgate_up")
    dev, st = _place(where, stream, gate_up, dh, dgate_up)
    _launch(where, dev, lib().moe_swiglu_grad, R, F, _DTYPE[dh.dtype], gate_up.data_ptr(), ldg, dh.data_ptr(), ldh,
            dgate_up.data_ptr(), ldd, st)


def moe_get_last_error() -> int:
    return lib().moe_get_last_error()


def moe_diag_wait_timeout(limit_ns: int, finished, stream=None):
    _check(lib().moe_diag_wait_timeout(int(limit_ns), _ptr(finished), _stream(stream)), "moe_diag_wait_timeout")


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
