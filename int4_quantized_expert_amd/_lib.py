"""ctypes binding of libmoe.so (include/moe.h), same names as the C entry points.

Argument marshalling only: tensors are passed as raw device pointers, the HIP
stream as its handle; every step runs in the library's HIP kernels. There is
no fallback: if libmoe.so is missing the import fails.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_OK, MOE_E_NULL, MOE_E_SHAPE, MOE_E_WORKSPACE, MOE_E_HIP, MOE_E_NOMEM, MOE_E_UNSUPPORTED, MOE_E_ARG = (
    0, -1, -2, -3, -4, -5, -6, -7)
MOE_TIE_EXPERT, MOE_TIE_GROUP, MOE_TIE_ORDER = 1, 2, 4
MOE_DTYPE_F32, MOE_DTYPE_BF16, MOE_DTYPE_F16 = 0, 1, 2
MOE_SCORE_SIGMOID, MOE_SCORE_SOFTMAX = 0, 1
MOE_GROUP_TOP2, MOE_GROUP_MAX = 0, 1
(MOE_ACT_NONE, MOE_ACT_RELU, MOE_ACT_SILU, MOE_ACT_GELU, MOE_ACT_GELU_TANH, MOE_ACT_SWIGLU) = range(6)
MOE_N_STAGES = 9
STAGES = ("router", "topk", "dispatch", "q8_x", "gateup_gemv", "down_gemv", "gateup_mfma", "down_mfma",
          "combine")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build()")
# torch ships its own HIP runtime under the same soname as the system one; the
# library must bind to the runtime torch uses (tensors and streams come from
# torch), so torch is loaded first whenever it is installed.
try:
    import torch
except ImportError:
    torch = None
_lib = ctypes.CDLL(LIB_PATH)

P, I32, I64, SZ, F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float


class moe_config(ctypes.Structure):
    _fields_ = [("hidden", I32), ("n_experts", I32), ("n_group", I32), ("topk_group", I32), ("top_k", I32),
                ("inter", I32), ("n_shared", I32), ("routed_scaling_factor", F32), ("gemm_min_tokens", I32),
                ("weight_bits", I32), ("group_size", I32), ("topp", F32)]


class moe_layer_weights(ctypes.Structure):
    _fields_ = [(n, P) for n in ("router_w", "router_bias", "w13", "s13", "w2", "s2", "sh_w13", "sh_s13", "sh_w2",
                                 "sh_s2")]


class moe_route_config(ctypes.Structure):
    _fields_ = [("n_experts", I32), ("n_group", I32), ("topk_group", I32), ("top_k", I32), ("score", I32),
                ("group_score", I32), ("renorm", I32), ("scale", F32)]


class moe_linear_config(ctypes.Structure):
    _fields_ = [("rows", I32), ("cols", I32), ("weight_bits", I32), ("group_size", I32), ("act", I32)]


class moe_adapters(ctypes.Structure):
    _fields_ = [("n_adapters", I32), ("rank", I32), ("a", P), ("b", P), ("scale", P)]


class moe_grad(ctypes.Structure):
    _fields_ = [("g", P), ("out", P), ("n", I64), ("dtype", I32)]


class moe_grads(ctypes.Structure):
    _fields_ = [("count", I32), ("chunks", I64), ("table", P)]


class moe_taps(ctypes.Structure):
    _fields_ = [("topk_ids", P), ("topk_w", P), ("near_tie", P), ("qx", P), ("dx", P), ("h", P), ("qh", P),
                ("dh", P), ("e_out", P), ("sum_slot", I32), ("gateup_sums", P), ("down_sums", P), ("counts", P),
                ("offsets", P), ("sorted_slots", P), ("slot_pos", P), ("unique_ids", P), ("n_unique", P)]


class moe_host_experts(ctypes.Structure):
    _fields_ = [("w13", P), ("s13", P), ("w2", P), ("s2", P)]


class moe_cache_stats(ctypes.Structure):
    _fields_ = [("hits", I64), ("misses", I64), ("evictions", I64), ("bytes_h2d", I64), ("steps", I64),
                ("h2d_ms", ctypes.c_double), ("pinned", I64)]


def _sig(name, res, args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = args
    return f


_sig("moe_version", I32, [])
_sig("moe_strerror", ctypes.c_char_p, [I32])
_sig("moe_last_hip_error", I32, [])
_sig("moe_workspace_bytes", SZ, [P, I32])
_sig("moe_quantize_int4", I32, [P, I32, I32, P, P, P])
_sig("moe_quantize_int8", I32, [P, I32, I32, P, P, P])
_sig("moe_quantize_int4_grouped", I32, [P, I32, I32, I32, P, P, P])
_sig("moe_quantize_q8_0", I32, [P, I64, P, P, P])
_sig("moe_tile_int4", I32, [P, I32, I32, P, P])
_sig("moe_tile_int8", I32, [P, I32, I32, P, P])
_sig("moe_tile_group_scales", I32, [P, I32, I32, P, P])
_sig("moe_router", I32, [P, P, I32, P, P, P, P, P, P, SZ, P])
_sig("moe_dispatch", I32, [P, P, I32, P, P, P, P, P, P, P, SZ, P])
_sig("moe_layer_forward", I32, [P, P, P, I32, P, P, SZ, P, P])
_sig("moe_layer_forward_noalloc", I32, [P, P, P, I32, P, P, P])
_sig("moe_layer_forward_routed", I32, [P, P, P, I32, P, P, P, P, SZ, P, P])
_sig("moe_route_workspace_bytes", SZ, [P, I32])
_sig("moe_route", I32, [P, P, I32, I64, I32, P, P, P, P, P, P, P, SZ, P])
_sig("moe_route_backward", I32, [P, P, I32, I64, I32, P, P, P, P, P, I64, P])
_sig("moe_slot_weight_grad", I32, [P, P, P, I32, I32, I32, P, P])
_sig("moe_slot_weight_grad_experts", I32, [P, P, P, I32, I32, I32, I32, P, P])
_sig("moe_linear_workspace_bytes", SZ, [P, I32])
_sig("moe_linear", I32, [P, P, P, P, P, I64, I32, I32, P, I64, P, I64, P, SZ, P])
_sig("moe_linear_adapted_workspace_bytes", SZ, [P, P, I32])
_sig("moe_linear_adapted", I32, [P, P, P, P, P, P, P, I64, I32, I32, P, I64, P, I64, P, I64, P, SZ, P])
_sig("moe_linear_backward_workspace_bytes", SZ, [P, P, I32])
_sig("moe_linear_backward", I32, [P, P, P, P, P, P, I64, I32, I32, P, I64, P, I64, P, I64, P, I64, P, P, P, SZ, P])
_sig("moe_grad_table_bytes", SZ, [P, I32])
_sig("moe_grad_table", I32, [P, I32, P, SZ, P, P])
_sig("moe_grad_clip", I32, [P, F32, P, P])
_sig("moe_expert_cache_create", I32, [P, I32, I32, ctypes.POINTER(P)])
_sig("moe_expert_cache_forward", I32, [P, P, P, P, I32, P, P, SZ, P, P, P, P])
_sig("moe_expert_cache_stats", I32, [P, P])
_sig("moe_expert_cache_usage", I32, [P, P])
_sig("moe_expert_cache_set_usage", I32, [P, P])
_sig("moe_expert_cache_pin_hottest", I32, [P, I32, P, P])
_sig("moe_expert_cache_destroy", None, [P])
_sig("moe_prof_enable", I32, [I32, ctypes.c_uint32])
_sig("moe_prof_read", I32, [P, I32, P])
_sig("moe_prof_disable", None, [])
_sig("moe_membench_read", I32, [P, SZ, I32, I32, P, P])
_sig("moe_membench_copy", I32, [P, P, SZ, I32, P])
_sig("moe_peakbench_mfma_i8", I32, [I32, I32, I32, P, P])
_sig("moe_peakbench_valu_fma", I32, [I32, I32, ctypes.c_float, ctypes.c_float, P, P])

EXPORTED = ("moe_version", "moe_strerror", "moe_last_hip_error", "moe_workspace_bytes", "moe_quantize_int4",
            "moe_quantize_int8", "moe_quantize_int4_grouped", "moe_quantize_q8_0",
            "moe_tile_int4", "moe_tile_int8", "moe_tile_group_scales", "moe_router", "moe_dispatch", "moe_layer_forward",
            "moe_layer_forward_noalloc", "moe_layer_forward_routed", "moe_route_workspace_bytes", "moe_route",
            "moe_route_backward", "moe_slot_weight_grad", "moe_slot_weight_grad_experts",
            "moe_linear_workspace_bytes", "moe_linear",
            "moe_linear_adapted_workspace_bytes", "moe_linear_adapted", "moe_linear_backward_workspace_bytes",
            "moe_linear_backward", "moe_grad_table_bytes", "moe_grad_table", "moe_grad_clip",
            "moe_expert_cache_create",
            "moe_expert_cache_forward", "moe_expert_cache_stats", "moe_expert_cache_usage", "moe_expert_cache_set_usage",
            "moe_expert_cache_pin_hottest", "moe_expert_cache_destroy", "moe_prof_enable",
            "moe_prof_read", "moe_prof_disable", "moe_membench_read", "moe_membench_copy",
            "moe_peakbench_mfma_i8", "moe_peakbench_valu_fma")


class MoeError(RuntimeError):
    def __init__(self, fn, rc):
        msg = _lib.moe_strerror(rc).decode()
        if rc == MOE_E_HIP:
            msg += f" (hipError {_lib.moe_last_hip_error()})"
        super().__init__(f"{fn}: {msg} [{rc}]")
        self.rc = rc


def _check(fn, rc):
    if rc != MOE_OK:
        raise MoeError(fn, rc)
    return rc


def _ptr(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


class ArgError(ValueError):
    """A tensor handed to the binding does not match what the C entry point will read or write."""


_DT = {}


def _dtype(name):
    import torch
    if not _DT:
        _DT.update(f32=torch.float32, i32=torch.int32, i8=torch.int8, u8=torch.uint8)
    return _DT[name]


def _need(t, name, dtype=None, numel=None, rows=None, cols=None):
    """Checks a device tensor before its raw pointer reaches the library: on the GPU, contiguous, of the element
    type the entry point reads, and at least as large as the call will touch (the library only sees pointers,
    so a short or strided buffer would become out-of-bounds device accesses)."""
    if t is None:
        raise ArgError(f"{name}: a device tensor is required")
    if not getattr(t, "is_cuda", False):
        raise ArgError(f"{name}: must be a GPU tensor")
    if not t.is_contiguous():
        raise ArgError(f"{name}: must be contiguous")
    if dtype is not None and t.dtype != _dtype(dtype):
        raise ArgError(f"{name}: dtype {t.dtype}, expected {_dtype(dtype)}")
    if numel is not None and t.numel() < numel:
        raise ArgError(f"{name}: {t.numel()} elements, the call touches {numel}")
    if rows is not None and (t.dim() != 2 or t.shape[0] < rows or (cols is not None and t.shape[1] != cols)):
        raise ArgError(f"{name}: shape {tuple(t.shape)}, expected [>= {rows}, {cols}]")
    return t


def _opt(t, name, dtype, numel):
    return None if t is None else _need(t, name, dtype, numel)


def _stream(stream):
    if stream is None:
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


@dataclass
class Config:
    hidden: int
    n_experts: int
    n_group: int
    topk_group: int
    top_k: int
    inter: int
    n_shared: int
    routed_scaling_factor: float
    gemm_min_tokens: int = 0
    weight_bits: int = 4
    group_size: int = 0
    topp: float = 0.0

    def c(self):
        return moe_config(self.hidden, self.n_experts, self.n_group, self.topk_group, self.top_k, self.inter,
                          self.n_shared, self.routed_scaling_factor, self.gemm_min_tokens, self.weight_bits,
                          self.group_size, self.topp)


def moe_version():
    return _lib.moe_version()


def moe_workspace_bytes(cfg: Config, max_tokens: int) -> int:
    c = cfg.c()
    return int(_lib.moe_workspace_bytes(ctypes.byref(c), int(max_tokens)))


def _quant_args(w, out, scales, out_numel, sc_numel, names):
    _need(w, "w", "f32")
    if w.dim() != 2:
        raise ArgError(f"w: 2-D [rows][cols] expected, got {tuple(w.shape)}")
    _need(out, names[0], None, None)
    if out.numel() * out.element_size() < out_numel:
        raise ArgError(f"{names[0]}: {out.numel() * out.element_size()} bytes, the call writes {out_numel}")
    _need(scales, "scales", "f32", sc_numel)


def moe_quantize_int4(w, packed, scales, stream=None):
    rows, cols = w.shape
    _quant_args(w, packed, scales, rows * cols // 2, rows, ("packed",))
    return _check("moe_quantize_int4",
                  _lib.moe_quantize_int4(_ptr(w), rows, cols, _ptr(packed), _ptr(scales), _stream(stream)))


def moe_quantize_int8(w, codes, scales, stream=None):
    rows, cols = w.shape
    _quant_args(w, codes, scales, rows * cols, rows, ("codes",))
    return _check("moe_quantize_int8",
                  _lib.moe_quantize_int8(_ptr(w), rows, cols, _ptr(codes), _ptr(scales), _stream(stream)))


def moe_quantize_int4_grouped(w, group, packed, scales, stream=None):
    rows, cols = w.shape
    g = int(group)
    # an invalid group size is the library's to reject (MOE_E_ARG / MOE_E_SHAPE); size the scales only for a valid one
    _quant_args(w, packed, scales, rows * cols // 2, rows * (cols // g) if g > 0 and cols % g == 0 else 0, ("packed",))
    return _check("moe_quantize_int4_grouped",
                  _lib.moe_quantize_int4_grouped(_ptr(w), rows, cols, int(group), _ptr(packed), _ptr(scales),
                                                 _stream(stream)))


def moe_quantize_q8_0(x, q, d, stream=None):
    _need(x, "x", "f32")
    _need(q, "q", "i8", x.numel())
    _need(d, "d", "f32", x.numel() // 32)
    return _check("moe_quantize_q8_0", _lib.moe_quantize_q8_0(_ptr(x), x.numel(), _ptr(q), _ptr(d), _stream(stream)))


def _tile_args(src, dst, nbytes, src_dtype, names):
    """Both buffers on the GPU, contiguous, of the element type, and holding the `nbytes` the call reads and writes."""
    _need(src, names[0], src_dtype)
    _need(dst, names[1], "u8")
    for t, n in ((src, names[0]), (dst, names[1])):
        if t.numel() * t.element_size() < nbytes:
            raise ArgError(f"{n}: {t.numel() * t.element_size()} bytes, the call touches {nbytes}")


def moe_tile_int4(rowmajor, tiled, stream=None):
    """Canonical row-major packed int4 [rows][cols/2] bytes -> the row-tiled layout (byte permutation)."""
    _need(rowmajor, "rowmajor", "u8")
    if rowmajor.dim() != 2:
        raise ArgError(f"rowmajor: 2-D [rows][cols/2] expected, got {tuple(rowmajor.shape)}")
    rows, cols = rowmajor.shape[0], 2 * rowmajor.shape[1]
    _tile_args(rowmajor, tiled, rows * cols // 2, "u8", ("rowmajor", "tiled"))
    return _check("moe_tile_int4", _lib.moe_tile_int4(_ptr(rowmajor), rows, cols, _ptr(tiled), _stream(stream)))


def moe_tile_int8(rowmajor, tiled, stream=None):
    """Canonical row-major int8 codes [rows][cols] -> the row-tiled int8 layout (byte permutation)."""
    _need(rowmajor, "rowmajor", "i8")
    if rowmajor.dim() != 2:
        raise ArgError(f"rowmajor: 2-D [rows][cols] expected, got {tuple(rowmajor.shape)}")
    rows, cols = rowmajor.shape
    _tile_args(rowmajor, tiled, rows * cols, "i8", ("rowmajor", "tiled"))
    return _check("moe_tile_int8", _lib.moe_tile_int8(_ptr(rowmajor), rows, cols, _ptr(tiled), _stream(stream)))


def moe_tile_group_scales(rowmajor, tiled, stream=None):
    """Group scales [rows][n_groups] fp32 -> the tiled group-scale layout [rows/64][n_groups][64]."""
    _need(rowmajor, "rowmajor", "f32")
    if rowmajor.dim() != 2:
        raise ArgError(f"rowmajor: 2-D [rows][n_groups] expected, got {tuple(rowmajor.shape)}")
    rows, ng = rowmajor.shape
    _need(tiled, "tiled", "f32", rows * ng)
    return _check("moe_tile_group_scales", _lib.moe_tile_group_scales(_ptr(rowmajor), rows, ng, _ptr(tiled),
                                                                      _stream(stream)))


def moe_router(cfg: Config, x, router_w, router_bias, topk_ids, topk_w, near_tie, ws, stream=None):
    c = cfg.c()
    _need(x, "x", "f32")
    _need(ws, "ws")
    if _lib.moe_workspace_bytes(ctypes.byref(c), 1) > 0:  # an invalid configuration is the library's to reject
        _need(x, "x", "f32", rows=1, cols=cfg.hidden)
        T, E, K = x.shape[0], cfg.n_experts, cfg.top_k
        _need(router_w, "router_w", "f32", E * cfg.hidden)
        _need(router_bias, "router_bias", "f32", E)
        _need(topk_ids, "topk_ids", "i32", T * K)
        _need(topk_w, "topk_w", "f32", T * K)
        _opt(near_tie, "near_tie", "u8", T)
    return _check("moe_router", _lib.moe_router(ctypes.byref(c), _ptr(x), x.shape[0], _ptr(router_w),
                                                _ptr(router_bias), _ptr(topk_ids), _ptr(topk_w), _ptr(near_tie),
                                                _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_dispatch(cfg: Config, topk_ids, counts, offsets, sorted_slots, slot_pos, unique_ids, n_unique, ws,
                 stream=None):
    c = cfg.c()
    _need(topk_ids, "topk_ids", "i32")
    _need(ws, "ws")
    if _lib.moe_workspace_bytes(ctypes.byref(c), 1) > 0:  # an invalid configuration is the library's to reject
        _need(topk_ids, "topk_ids", "i32", rows=1, cols=cfg.top_k)
        T, E, K = topk_ids.shape[0], cfg.n_experts, cfg.top_k
        for t, n, k in ((counts, "counts", E), (offsets, "offsets", E + 1), (sorted_slots, "sorted_slots", T * K),
                        (slot_pos, "slot_pos", T * K), (unique_ids, "unique_ids", E), (n_unique, "n_unique", 1)):
            _need(t, n, "i32", k)
    return _check("moe_dispatch", _lib.moe_dispatch(ctypes.byref(c), _ptr(topk_ids), topk_ids.shape[0], _ptr(counts),
                                                    _ptr(offsets), _ptr(sorted_slots), _ptr(slot_pos),
                                                    _ptr(unique_ids), _ptr(n_unique), _ptr(ws),
                                                    ws.numel() * ws.element_size(), _stream(stream)))


def layer_weights(router_w, router_bias, w13, s13, w2, s2, sh_w13=None, sh_s13=None, sh_w2=None, sh_s2=None,
                  cfg: Config | None = None):
    """moe_layer_weights from device tensors. With cfg, every tensor is checked against the sizes the layer reads
    (routed arrays for E experts, shared arrays for n_shared): element type, device, contiguity, size."""
    if cfg is not None:
        E, H, I, NS = cfg.n_experts, cfg.hidden, cfg.inter, cfg.n_shared
        wb = cfg.weight_bits if cfg.weight_bits > 0 else 4
        G = cfg.group_size if cfg.group_size > 0 else 0
        b13, b2 = I * H * wb // 4, H * I * wb // 8
        n13, n2 = (2 * I * H // G, H * I // G) if G else (2 * I, H)
        _need(router_w, "router_w", "f32", E * H)
        _need(router_bias, "router_bias", "f32", E)
        for t, n, dt, k in ((w13, "w13", "u8", E * b13), (s13, "s13", "f32", E * n13), (w2, "w2", "u8", E * b2),
                            (s2, "s2", "f32", E * n2)):
            _need(t, n, dt, k)
        if NS:
            for t, n, dt, k in ((sh_w13, "sh_w13", "u8", NS * b13), (sh_s13, "sh_s13", "f32", NS * n13),
                                (sh_w2, "sh_w2", "u8", NS * b2), (sh_s2, "sh_s2", "f32", NS * n2)):
                _need(t, n, dt, k)
    return moe_layer_weights(*[_ptr(t) for t in (router_w, router_bias, w13, s13, w2, s2, sh_w13, sh_s13, sh_w2,
                                                 sh_s2)])


# element type and size (in terms of T, K, H, I, E, R = T*K + n_shared*T) of each tap buffer
_TAP_SPEC = {
    "topk_ids": ("i32", lambda T, K, H, I, E, R: T * K), "topk_w": ("f32", lambda T, K, H, I, E, R: T * K),
    "near_tie": ("u8", lambda T, K, H, I, E, R: T), "qx": ("i8", lambda T, K, H, I, E, R: T * H),
    "dx": ("f32", lambda T, K, H, I, E, R: T * H // 32), "h": ("f32", lambda T, K, H, I, E, R: R * I),
    "qh": ("i8", lambda T, K, H, I, E, R: R * I), "dh": ("f32", lambda T, K, H, I, E, R: R * I // 32),
    "e_out": ("f32", lambda T, K, H, I, E, R: R * H),
    "gateup_sums": ("i32", lambda T, K, H, I, E, R: 2 * I * (H // 32)),
    "down_sums": ("i32", lambda T, K, H, I, E, R: H * (I // 32)),
    "counts": ("i32", lambda T, K, H, I, E, R: E), "offsets": ("i32", lambda T, K, H, I, E, R: E + 1),
    "sorted_slots": ("i32", lambda T, K, H, I, E, R: T * K), "slot_pos": ("i32", lambda T, K, H, I, E, R: T * K),
    "unique_ids": ("i32", lambda T, K, H, I, E, R: E), "n_unique": ("i32", lambda T, K, H, I, E, R: 1),
}


def taps(sum_slot=-1, **bufs):
    """moe_taps from device tensors; moe_layer_forward checks each one's type and size against the call."""
    t = moe_taps()
    t.sum_slot = sum_slot
    for k, v in bufs.items():
        if k not in _TAP_SPEC:
            raise ArgError(f"unknown tap {k}")
        setattr(t, k, None if v is None else v.data_ptr())
    t._bufs = {k: v for k, v in bufs.items() if v is not None}
    return t


def _check_forward_args(cfg: Config, x, y, T, ws, tap):
    """What the library cannot see behind its raw pointers: x and y hold T rows of H fp32 on the GPU, the
    workspace and tap buffers are device tensors of the right type and size. An invalid configuration or T < 1
    is left to the library, which rejects it with its own code before any device work."""
    _need(x, "x", "f32")
    _need(y, "y", "f32")
    if T > x.shape[0] or T > y.shape[0]:
        raise ArgError(f"T = {T} above the rows of x ({x.shape[0]}) or y ({y.shape[0]})")
    if ws is not None:
        _need(ws, "ws")
    c = cfg.c()
    if T < 1 or _lib.moe_workspace_bytes(ctypes.byref(c), 1) == 0:
        return
    _need(x, "x", "f32", rows=T, cols=cfg.hidden)
    _need(y, "y", "f32", rows=T, cols=cfg.hidden)
    if tap is not None:
        K, H, I, E = cfg.top_k, cfg.hidden, cfg.inter, cfg.n_experts
        R = T * K + cfg.n_shared * T
        for k, v in getattr(tap, "_bufs", {}).items():
            dt, size = _TAP_SPEC[k]
            _need(v, k, dt, size(T, K, H, I, E, R))


def moe_layer_forward(cfg: Config, weights: moe_layer_weights, x, y, ws, tap: moe_taps | None = None, stream=None,
                      T: int | None = None):
    c = cfg.c()
    T = x.shape[0] if T is None else T
    _check_forward_args(cfg, x, y, T, ws, tap)
    return _check("moe_layer_forward",
                  _lib.moe_layer_forward(ctypes.byref(c), ctypes.byref(weights), _ptr(x), T, _ptr(y), _ptr(ws),
                                         ws.numel() * ws.element_size(), ctypes.byref(tap) if tap else None,
                                         _stream(stream)))


NOALLOC_WORKSPACE_BYTES = 128 << 20  # MOE_NOALLOC_WORKSPACE_BYTES


def moe_layer_forward_noalloc(cfg: Config, weights: moe_layer_weights, x, y, tap: moe_taps | None = None,
                              stream=None, T: int | None = None):
    c = cfg.c()
    T = x.shape[0] if T is None else T
    _check_forward_args(cfg, x, y, T, None, tap)
    return _check("moe_layer_forward_noalloc",
                  _lib.moe_layer_forward_noalloc(ctypes.byref(c), ctypes.byref(weights), _ptr(x), T, _ptr(y),
                                                 ctypes.byref(tap) if tap else None, _stream(stream)))


_FLOAT_DT = {}


def _float_types():
    """{torch dtype: MOE_DTYPE_*} of the tensors that may be fp32, bf16 or fp16."""
    _FLOAT_DT.update({torch.float32: MOE_DTYPE_F32, torch.bfloat16: MOE_DTYPE_BF16, torch.float16: MOE_DTYPE_F16})
    return _FLOAT_DT


def _matrix(t, name, cols):
    """A [rows][cols] device tensor of one of the three float types, rows possibly strided: (dtype code, rows,
    elements between rows)."""
    if t is None or not getattr(t, "is_cuda", False):
        raise ArgError(f"{name}: must be a GPU tensor")
    dt = (_FLOAT_DT or _float_types()).get(t.dtype)
    if dt is None:
        raise ArgError(f"{name}: dtype {t.dtype}, expected float32, bfloat16 or float16")
    shape = t.shape
    if len(shape) != 2 or shape[1] != cols or shape[0] < 1:
        raise ArgError(f"{name}: shape {tuple(shape)}, expected [>= 1, {cols}]")
    rows, (ld, step) = shape[0], t.stride()
    if rows == 1 and ld < cols:
        ld = cols
    if ld < cols or (step != 1 and cols > 1):
        raise ArgError(f"{name}: strides {t.stride()}, expected rows of adjacent elements")
    return dt, rows, ld


def _dev_ptr(t, name, dtype, numel, dev):
    """Address of a device tensor after _need's checks, which this repeats only for the message; the tensors of one
    call share a device, since the library would read another GPU's pointer through the wrong one."""
    if (getattr(t, "is_cuda", False) and t.numel() >= numel and t.is_contiguous()
            and (dtype is None or t.dtype == (_DT.get(dtype) or _dtype(dtype)))):
        if t.get_device() != dev:
            raise ArgError(f"{name}: on {t.device}, the other tensors on cuda:{dev}")
        return t.data_ptr()
    _need(t, name, dtype, numel)


def _same_dev(t, name, dev):
    if t.get_device() != dev:
        raise ArgError(f"{name}: on {t.device}, the other tensors on cuda:{dev}")
    return t.data_ptr()


def _opt_ptr(t, name, dtype, numel, dev):
    return None if t is None else _dev_ptr(t, name, dtype, numel, dev)


def _launch(fn, dev, stream, *args):
    """Calls C entry fn with the tensors' device current (kernels launch on the current device) on the given
    stream, else on that device's current stream."""
    # torch's own accessors behind torch.cuda.current_device and current_stream: the handle alone, without the Stream
    # object around it, saves 1.2 us of an 8 us call
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return _launch(fn, dev, stream, *args)
    st = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)
    rc = fn(*args, st)
    return rc if rc == MOE_OK else _check(fn.__name__, rc)


def moe_layer_forward_routed(cfg: Config, weights: moe_layer_weights, x, ids, w, y, ws, tap: moe_taps | None = None,
                             stream=None, T: int | None = None):
    """moe_layer_forward under a given routing: ids [T][K] int32 (outside [0, E): slot dropped), w [T][K] fp32."""
    c = cfg.c()
    T = x.shape[0] if T is None else T
    _check_forward_args(cfg, x, y, T, ws, tap)
    dev, n = x.get_device(), max(T, 0) * max(cfg.top_k, 0)
    return _launch(_lib.moe_layer_forward_routed, dev, stream, ctypes.byref(c), ctypes.byref(weights), x.data_ptr(), T,
                   _dev_ptr(ids, "ids", "i32", n, dev), _dev_ptr(w, "w", "f32", n, dev),
                   _dev_ptr(y, "y", None, 0, dev), _dev_ptr(ws, "ws", None, 0, dev), ws.numel() * ws.element_size(),
                   ctypes.byref(tap) if tap else None)


class _CStruct:
    """Keeps the C struct that c() builds until a field changes (building it takes 0.5 us of a 6 us call)."""

    def __setattr__(self, name, value):
        self.__dict__.pop("_struct", None)
        self.__dict__[name] = value

    def __getstate__(self):  # copies and pickles carry the fields only
        return {k: v for k, v in self.__dict__.items() if k != "_struct"}

    def ref(self):
        r = self.__dict__.get("_struct")
        if r is None:
            r = self.__dict__["_struct"] = ctypes.byref(self.c())
        return r


@dataclass
class RouteConfig(_CStruct):
    """moe_route_config: softmax or sigmoid scores, group limiting, renormalised weights."""
    n_experts: int
    top_k: int
    n_group: int = 1
    topk_group: int = 1
    score: int = MOE_SCORE_SIGMOID
    group_score: int = MOE_GROUP_TOP2
    renorm: bool = True
    scale: float = 1.0

    def c(self):
        return moe_route_config(self.n_experts, self.n_group, self.topk_group, self.top_k, self.score,
                                self.group_score, int(self.renorm), self.scale)


def moe_route_workspace_bytes(cfg: RouteConfig, max_tokens: int) -> int:
    c = cfg.c()
    return int(_lib.moe_route_workspace_bytes(ctypes.byref(c), int(max_tokens)))


def moe_route(cfg: RouteConfig, logits, ids, w, bias=None, valid=None, load=None, importance=None, ws=None,
              stream=None):
    """Top-K routing of logits [T][E] (fp32, bf16 or fp16; rows may be strided) into ids and w [T][K]. load [E] int32
    and importance [E] fp32 need the workspace ws of moe_route_workspace_bytes."""
    E, K = cfg.n_experts, max(cfg.top_k, 0)
    dt, T, ld = _matrix(logits, "logits", E)
    dev = logits.get_device()
    return _launch(_lib.moe_route, dev, stream, cfg.ref(), logits.data_ptr(), dt, ld, T,
                   _opt_ptr(bias, "bias", "f32", E, dev), _opt_ptr(valid, "valid", "u8", T, dev),
                   _dev_ptr(ids, "ids", "i32", T * K, dev), _dev_ptr(w, "w", "f32", T * K, dev),
                   _opt_ptr(load, "load", "i32", E, dev), _opt_ptr(importance, "importance", "f32", E, dev),
                   _opt_ptr(ws, "ws", None, 0, dev), 0 if ws is None else ws.numel() * ws.element_size())


def moe_route_backward(cfg: RouteConfig, logits, ids, d_logits, d_w=None, d_importance=None, valid=None, stream=None):
    """Gradient of the logits from those of moe_route's weights and importance sums (one of the two may be None)."""
    E, K = cfg.n_experts, max(cfg.top_k, 0)
    dt, T, ld = _matrix(logits, "logits", E)
    dt_d, T_d, ld_d = _matrix(d_logits, "d_logits", E)
    if dt_d != dt or T_d < T:
        raise ArgError(f"d_logits: {d_logits.dtype} {tuple(d_logits.shape)}, expected {logits.dtype} [>= {T}, {E}]")
    dev = logits.get_device()
    return _launch(_lib.moe_route_backward, dev, stream, cfg.ref(), logits.data_ptr(), dt, ld, T,
                   _opt_ptr(valid, "valid", "u8", T, dev), _dev_ptr(ids, "ids", "i32", T * K, dev),
                   _opt_ptr(d_w, "d_w", "f32", T * K, dev), _opt_ptr(d_importance, "d_importance", "f32", E, dev),
                   _same_dev(d_logits, "d_logits", dev), ld_d)


def moe_slot_weight_grad(e_out, ids, dy, d_w, stream=None, n_experts=None):
    """d_w [T][K] = <dy[t], e_out[t*K + k]>, 0 for dropped slots; e_out is the layer's tap (its first T*K rows). With
    n_experts every id outside [0, n_experts) drops its slot, as in moe_layer_forward_routed; without it only negative
    ids do."""
    _need(ids, "ids", "i32")
    _need(dy, "dy", "f32")
    if ids.dim() != 2 or dy.dim() != 2 or dy.shape[0] < ids.shape[0]:
        raise ArgError(f"ids {tuple(ids.shape)}, dy {tuple(dy.shape)}: expected [T, K] and [>= T, H]")
    (T, K), H = ids.shape, dy.shape[1]
    _need(e_out, "e_out", "f32", rows=T * K, cols=H)
    dev = e_out.get_device()
    fn, limit = (_lib.moe_slot_weight_grad, ()) if n_experts is None else (_lib.moe_slot_weight_grad_experts, (n_experts,))
    return _launch(fn, dev, stream, e_out.data_ptr(), _same_dev(ids, "ids", dev), _same_dev(dy, "dy", dev), T, K, H,
                   *limit, _dev_ptr(d_w, "d_w", "f32", T * K, dev))


@dataclass
class LinearConfig(_CStruct):
    """moe_linear_config: weight codes [rows][cols] and the activation of the epilogue."""
    rows: int
    cols: int
    weight_bits: int = 4
    group_size: int = 0
    act: int = MOE_ACT_NONE

    def c(self):
        return moe_linear_config(self.rows, self.cols, self.weight_bits, self.group_size, self.act)


def moe_linear_workspace_bytes(cfg: LinearConfig, max_tokens: int) -> int:
    c = cfg.c()
    return int(_lib.moe_linear_workspace_bytes(ctypes.byref(c), int(max_tokens)))


def moe_linear(cfg: LinearConfig, codes, scales, x, y, ws, bias=None, residual=None, stream=None):
    """y [T][N] = act(W x + bias) + residual (N = rows / 2 with MOE_ACT_SWIGLU) over row-tiled codes; x, y and
    residual of one type (fp32, bf16 or fp16), rows possibly strided. residual may be y."""
    rows, cols, G = cfg.rows, cfg.cols, cfg.group_size
    out = rows // 2 if cfg.act == MOE_ACT_SWIGLU else rows
    dt, T, ldx = _matrix(x, "x", cols)
    dt_y, T_y, ldy = _matrix(y, "y", out)
    if dt_y != dt or T_y < T:
        raise ArgError(f"y: {y.dtype} {tuple(y.shape)}, expected {x.dtype} [>= {T}, {out}]")
    dev = x.get_device()
    res, ldr = None, 0
    if residual is not None:
        dt_r, T_r, ldr = _matrix(residual, "residual", out)
        if dt_r != dt or T_r < T:
            raise ArgError(f"residual: {residual.dtype} {tuple(residual.shape)}, expected {x.dtype} [>= {T}, {out}]")
        res = _same_dev(residual, "residual", dev)
    # an invalid configuration is the library's to reject, before it looks at the data: sizes as if it were valid
    n_codes = rows * cols * (8 if cfg.weight_bits == 8 else 4) // 8
    n_scales = rows * (cols // G) if G > 0 else rows
    return _launch(_lib.moe_linear, dev, stream, cfg.ref(), _dev_ptr(codes, "codes", "u8", n_codes, dev),
                   _dev_ptr(scales, "scales", "f32", n_scales, dev), _opt_ptr(bias, "bias", "f32", rows, dev),
                   x.data_ptr(), ldx, T, dt, res, ldr, _same_dev(y, "y", dev), ldy, _dev_ptr(ws, "ws", None, 0, dev),
                   ws.numel() * ws.element_size())


class Adapters:
    """moe_adapters: a [n][R][cols] and b [n][rows][R] of the activations' type, scale [n] fp32, on one GPU (kept alive
    here)."""

    def __init__(self, a, b, scale):
        for t, name in ((a, "a"), (b, "b")):
            _need(t, name)
            if t.dim() != 3 or t.dtype not in _float_types():
                raise ArgError(f"{name}: {t.dtype} {tuple(t.shape)}, expected three dimensions of float32, bfloat16 or float16")
        n, R, cols = a.shape
        if b.shape[0] != n or b.shape[2] != R or b.dtype != a.dtype:
            raise ArgError(f"b: {b.dtype} {tuple(b.shape)}, expected {a.dtype} [{n}, rows, {R}]")
        _need(scale, "scale", "f32", n)
        self.device, self.dtype, self.n, self.rank, self.cols, self.rows = a.get_device(), _FLOAT_DT[a.dtype], n, R, cols, b.shape[1]
        self._keep = (a, b, scale)
        self.c = moe_adapters(n, R, a.data_ptr(), _same_dev(b, "b", self.device), _same_dev(scale, "scale", self.device))
        self._ref = ctypes.byref(self.c)

    def ref(self):
        return self._ref


def _adapters_ref(adapters, ids, cfg, T, dt, dev):
    """References to the adapters and the tokens' ids, or (None, None)."""
    if adapters is None:
        return None, None
    if adapters.device != dev or adapters.dtype != dt or adapters.cols != cfg.cols or adapters.rows != cfg.rows:
        raise ArgError(f"adapters: [{adapters.rows}, {adapters.cols}] of type {adapters.dtype} on cuda:{adapters.device}, "
                       f"the call's [{cfg.rows}, {cfg.cols}] of type {dt} on cuda:{dev}")
    return adapters._ref, _opt_ptr(ids, "ids", "i32", T, dev)


def moe_linear_adapted_workspace_bytes(cfg: LinearConfig, adapters, max_tokens: int) -> int:
    return int(_lib.moe_linear_adapted_workspace_bytes(cfg.ref(), adapters and adapters.ref(), int(max_tokens)))


def _rows_like(t, name, dt, T, cols, dev):
    """(address, elements between rows) of an optional matrix of the call's type and tokens."""
    if t is None:
        return None, 0
    dt_t, rows, ld = _matrix(t, name, cols)
    if dt_t != dt or rows < T:
        raise ArgError(f"{name}: {t.dtype} {tuple(t.shape)}, expected the call's type and [>= {T}, {cols}]")
    return _same_dev(t, name, dev), ld


def _code_ptrs(cfg, codes, scales, dev):
    # an invalid configuration is the library's to reject, before it looks at the data: sizes as if it were valid
    rows, cols, G = cfg.rows, cfg.cols, cfg.group_size
    return (_dev_ptr(codes, "codes", "u8", rows * cols * (8 if cfg.weight_bits == 8 else 4) // 8, dev),
            _dev_ptr(scales, "scales", "f32", rows * (cols // G) if G > 0 else rows, dev))


def moe_linear_adapted(cfg: LinearConfig, codes, scales, adapters, ids, x, y, ws, bias=None, residual=None, pre=None,
                       stream=None):
    """moe_linear with a low-rank adapter by token: ids [T] int32 (outside [0, n): none; None: adapter 0 for all). pre
    [T][rows] takes the values in front of the activation, for moe_linear_backward."""
    rows = cfg.rows
    out = rows // 2 if cfg.act == MOE_ACT_SWIGLU else rows
    dt, T, ldx = _matrix(x, "x", cfg.cols)
    dev = x.get_device()
    ad, ids = _adapters_ref(adapters, ids, cfg, T, dt, dev)
    if y is None:
        raise ArgError("y: a device tensor is required")
    return _launch(_lib.moe_linear_adapted, dev, stream, cfg.ref(), *_code_ptrs(cfg, codes, scales, dev),
                   _opt_ptr(bias, "bias", "f32", rows, dev), ad, ids, x.data_ptr(), ldx, T, dt,
                   *_rows_like(residual, "residual", dt, T, out, dev), *_rows_like(y, "y", dt, T, out, dev),
                   *_rows_like(pre, "pre", dt, T, rows, dev), _dev_ptr(ws, "ws", None, 0, dev),
                   ws.numel() * ws.element_size())


def moe_linear_backward_workspace_bytes(cfg: LinearConfig, adapters, max_tokens: int) -> int:
    return int(_lib.moe_linear_backward_workspace_bytes(cfg.ref(), adapters and adapters.ref(), int(max_tokens)))


def moe_linear_backward(cfg: LinearConfig, codes, scales, dy, dx, ws, pre=None, adapters=None, ids=None, x=None, d_a=None,
                        d_b=None, residual=None, stream=None):
    """Gradients of moe_linear_adapted (without adapters: of moe_linear) from dy: dx [T][cols] (+ residual, which may be dx
    itself), d_a and d_b like the adapters' a and b. pre is what the forward call saved (not needed without an activation),
    x its activations (needed for d_a and d_b). dx, d_a or d_b may be None."""
    rows, cols = cfg.rows, cfg.cols
    dt, T, ldd = _matrix(dy, "dy", rows // 2 if cfg.act == MOE_ACT_SWIGLU else rows)
    dev = dy.get_device()
    ad, ids = _adapters_ref(adapters, ids, cfg, T, dt, dev)
    grads = []
    for t, name, k in ((d_a, "d_a", cols), (d_b, "d_b", rows)):
        if t is not None and ad is None:
            raise ArgError(f"{name}: there are no adapters")
        if t is not None and t.dtype != dy.dtype:
            raise ArgError(f"{name}: dtype {t.dtype}, expected {dy.dtype}")
        grads.append(None if t is None else _dev_ptr(t, name, None, adapters.n * adapters.rank * k, dev))
    return _launch(_lib.moe_linear_backward, dev, stream, cfg.ref(), *_code_ptrs(cfg, codes, scales, dev), ad, ids,
                   *_rows_like(x, "x", dt, T, cols, dev), T, dt, *_rows_like(pre, "pre", dt, T, rows, dev),
                   dy.data_ptr(), ldd, *_rows_like(residual, "residual", dt, T, cols, dev),
                   *_rows_like(dx, "dx", dt, T, cols, dev), *grads, _dev_ptr(ws, "ws", None, 0, dev),
                   ws.numel() * ws.element_size())


class GradTable:
    """moe_grad_table of a list of contiguous gradients (kept alive here) and where they go: `out`, as many tensors of the
    same sizes and types, or None for in place. It holds their addresses: gradients that a program allocates anew each step
    need a table each step. Building it waits for the current stream."""

    def __init__(self, grads, out=None):
        grads = list(grads)
        out = grads if out is None else list(out)
        if not grads or len(out) != len(grads):
            raise ArgError(f"{len(grads)} gradients, {len(out)} outputs")
        self.device = _need(grads[0], "grads").get_device()
        types = _float_types()
        c = (moe_grad * len(grads))()
        for i, (g, o) in enumerate(zip(grads, out)):
            for t, name in ((g, f"grads[{i}]"), (o, f"out[{i}]")):
                _need(t, name)
                _same_dev(t, name, self.device)
            if g.dtype not in types or o.dtype != g.dtype or o.numel() != g.numel():
                raise ArgError(f"grads[{i}]: {g.dtype} {tuple(g.shape)} to {o.dtype} {tuple(o.shape)}")
            c[i] = moe_grad(g.data_ptr(), o.data_ptr(), g.numel(), types[g.dtype])
        self._keep = (grads, out)
        with torch.cuda.device(self.device):
            size = int(_lib.moe_grad_table_bytes(c, len(grads)))
            self._table = torch.empty((max(size, 1),), dtype=torch.uint8, device=f"cuda:{self.device}")
            self.c = moe_grads()
            _launch(_lib.moe_grad_table, self.device, None, c, len(grads), self._table.data_ptr(), size, ctypes.byref(self.c))
            torch.cuda.current_stream().synchronize()
        self._ref = ctypes.byref(self.c)


def moe_grad_clip(table: GradTable, max_norm: float, norm, stream=None):
    """norm [1] = the 2-norm over all gradients of the table; out = gradient * min(1, max_norm / norm)."""
    dev = table.device
    return _launch(_lib.moe_grad_clip, dev, stream, table._ref, max_norm, _dev_ptr(norm, "norm", "f32", 1, dev))


def moe_prof_enable(max_calls: int, stages=None):
    """Time the named stages (names from STAGES; None = all) of the next max_calls forwards."""
    mask = 0 if stages is None else sum(1 << STAGES.index(n) for n in stages)
    return _check("moe_prof_enable", _lib.moe_prof_enable(int(max_calls), mask))


def moe_prof_read(max_calls: int):
    import numpy as np
    out = np.zeros((max_calls, MOE_N_STAGES), np.float32)
    n = ctypes.c_int32(0)
    _check("moe_prof_read", _lib.moe_prof_read(out.ctypes.data, max_calls, ctypes.byref(n)))
    return out[:n.value]


def moe_prof_disable():
    _lib.moe_prof_disable()


def moe_membench_read(buf, blocks: int, unroll: int, sink, stream=None):
    _need(buf, "buf")
    _need(sink, "sink", None, 1)
    return _check("moe_membench_read", _lib.moe_membench_read(_ptr(buf), buf.numel() * buf.element_size(), blocks,
                                                              unroll, _ptr(sink), _stream(stream)))


def moe_membench_copy(src, dst, blocks: int, stream=None):
    _need(src, "src")
    _need(dst, "dst")
    if dst.numel() * dst.element_size() < src.numel() * src.element_size():
        raise ArgError("dst: smaller than src")
    return _check("moe_membench_copy", _lib.moe_membench_copy(_ptr(src), _ptr(dst), src.numel() * src.element_size(),
                                                              blocks, _stream(stream)))


def moe_peakbench_mfma_i8(blocks: int, iters: int, value: int, out, stream=None):
    _need(out, "out", "i32", int(blocks) * 256)
    return _check("moe_peakbench_mfma_i8", _lib.moe_peakbench_mfma_i8(int(blocks), int(iters), int(value), _ptr(out),
                                                                      _stream(stream)))


def moe_peakbench_valu_fma(blocks: int, iters: int, m: float, c: float, out, stream=None):
    _need(out, "out", "f32", int(blocks) * 256)
    return _check("moe_peakbench_valu_fma", _lib.moe_peakbench_valu_fma(int(blocks), int(iters), float(m), float(c),
                                                                        _ptr(out), _stream(stream)))


class HostExperts:
    """Pointer arrays of moe_host_experts: per expert, pinned host pointers (int) or pinned host tensors (kept
    alive here) for w13, s13, w2, s2."""

    def __init__(self, w13, s13, w2, s2):
        self._keep = (list(w13), list(s13), list(w2), list(s2))
        E = len(self._keep[0])
        arr = ctypes.c_void_p * E
        self._arrs = [arr(*[t if isinstance(t, int) else t.data_ptr() for t in lst]) for lst in self._keep]
        self.c = moe_host_experts(*[ctypes.cast(a, P) for a in self._arrs])


class ExpertCache:
    """moe_expert_cache_* of one layer; destroy() (or garbage collection) releases the slot pool."""

    def __init__(self, cfg: Config, n_slots: int, max_tokens: int):
        self._h = P()
        c = cfg.c()
        _check("moe_expert_cache_create", _lib.moe_expert_cache_create(ctypes.byref(c), int(n_slots),
                                                                        int(max_tokens), ctypes.byref(self._h)))
        self.E = cfg.n_experts

    def forward(self, resident, host: HostExperts, x, y, ws, compute, copy, T=None, trace=False):
        import numpy as np
        T = x.shape[0] if T is None else T
        _need(x, "x", "f32", rows=T)
        _need(y, "y", "f32", rows=T, cols=x.shape[1])
        _need(ws, "ws")
        hit = np.zeros(self.E, np.int8) if trace else None
        slot = np.zeros(self.E, np.int32) if trace else None
        _check("moe_expert_cache_forward",
               _lib.moe_expert_cache_forward(self._h, ctypes.byref(resident), ctypes.byref(host.c), _ptr(x), T,
                                             _ptr(y), _ptr(ws), ws.numel() * ws.element_size(), _stream(compute),
                                             _stream(copy), hit.ctypes.data if trace else None,
                                             slot.ctypes.data if trace else None))
        return (hit, slot) if trace else None

    def stats(self):
        s = moe_cache_stats()
        _check("moe_expert_cache_stats", _lib.moe_expert_cache_stats(self._h, ctypes.byref(s)))
        return dict(hits=s.hits, misses=s.misses, evictions=s.evictions, bytes_h2d=s.bytes_h2d, steps=s.steps,
                    h2d_ms=s.h2d_ms, pinned=s.pinned)

    def usage(self):
        """Positions routed to each expert over every forward (host int64 [E])."""
        import numpy as np
        out = np.zeros(self.E, np.int64)
        _check("moe_expert_cache_usage", _lib.moe_expert_cache_usage(self._h, out.ctypes.data))
        return out

    def set_usage(self, usage):
        import numpy as np
        u = np.ascontiguousarray(usage, dtype=np.int64)
        assert u.shape == (self.E,)
        _check("moe_expert_cache_set_usage", _lib.moe_expert_cache_set_usage(self._h, u.ctypes.data))

    def pin_hottest(self, n_pin: int, host: HostExperts, copy):
        _check("moe_expert_cache_pin_hottest",
               _lib.moe_expert_cache_pin_hottest(self._h, int(n_pin), ctypes.byref(host.c), _stream(copy)))

    def destroy(self):
        if self._h:
            _lib.moe_expert_cache_destroy(self._h)
            self._h = P()

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass
