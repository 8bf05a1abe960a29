"""GB300 (sm_103a) row-wise RMSNorm: plain, fused residual-add, and
reduce + residual-add.

Thin Python binding over the C ABI in ``include/rarn.h`` (``librarn.so``,
built in-tree by ``residual_add_rmsnorm_gb300.build``).  This module only
checks and marshals arguments -- tensors to device pointers, the current CUDA
stream -- and raises on a non-OK status.  Every step of the computation runs
in the library's CUDA kernels; there is no CPU or PyTorch fallback: if the
library is missing or fails to load, every call raises.

    y = rms_norm(x, gamma, eps)                         # x: [..., H]
    y = fused_add_rms_norm(x, residual, gamma, eps)     # residual updated in place
    y = reduce_add_rms_norm(partials, residual, gamma, eps)   # partials: [R, ..., H]

Attention side (per-head norm and rotation, an 8-bit paged key / value cache,
attention of drafted tokens over it):

    qk_norm_rope(q, k, q_gamma, k_gamma, eps, cos_sin, positions)
    cache = KVCache.empty(pages, page_size, heads, head_dim)
    qk_norm_rope_kv_write(q, k, v, q_gamma, k_gamma, eps, cos_sin, positions, cache, slots)
    kv_cache_write(k, v, cache, slots)
    kv_cache_read(cache, page_table, starts, k_out, v_out)
    tree_attention(q, cache, page_table, context_lens, starts, mask=mask)

A step of drafted tokens (pages, slots and positions from the sequences' lengths;
the drafts' verification; the cache's tidying after it):

    pages = KVPages.empty(sequences, width, num_pages, page_size)
    starts, slots, positions, served = kv_step(pages, context_lens, new_lens, tokens)
    positions += (depths - rows) * (slots >= 0)     # a tree's; a chain's as they are
    new_tokens, path, lengths = verify_drafts(probs, tokens, starts, uniforms, final_uniforms, most)
    kv_cache_compact(cache, pages.page_table, context_lens, path, lengths)
    kv_trim(pages, kept_lens)

8-bit output (e4m3 / e5m2 codes with a per-tensor or per-row scale):

    rms_norm_fp8(x, gamma, eps, out, scale, fmt="e4m3", scale_mode="tensor")
    fused_add_rms_norm_fp8(x, residual, gamma, eps, out, scale, ...)
    reduce_add_rms_norm_fp8(partials, residual, gamma, eps, out, scale, ...)

The norms after and before a block, with its gate and the residual between them:

    gated_add_rms_norm(x, residual, x_gamma, gamma, eps, gate=gate, scale=0.5)
"""
from __future__ import annotations

import ctypes
import os

__all__ = ["rms_norm", "fused_add_rms_norm", "reduce_add_rms_norm", "rms_norm_host",
           "fused_add_rms_norm_host", "reduce_add_rms_norm_host", "RarnError", "library",
           "set_path", "get_path", "set_pdl", "get_pdl", "plan", "watchdog", "PATHS",
           "DTYPE_CODES", "rms_norm_ex", "fused_add_rms_norm_ex", "reduce_add_rms_norm_ex",
           "rms_norm_fp8", "fused_add_rms_norm_fp8", "reduce_add_rms_norm_fp8", "plan_fp8",
           "FP8_FORMATS", "SCALE_MODES", "gemm_add_rms_norm", "plan_gemm", "plan_fp8in", "plan_tp",
           "gemm_workspace_bytes", "gemm_add_rms_norm_noalloc", "reduce_add_rms_norm_fp8in",
           "TUNING", "set_tuning", "get_tuning", "reset_tuning", "tuning", "gemm_noalloc_rows",
           "launch_floor", "tp_rows", "tp_reduce_add_rms_norm", "tp_reduce_add_rms_norm_world",
           "ipc_export", "ipc_import", "ipc_close", "TP_MAX_RANKS", "TP_SIGNAL_BYTES",
           "IPC_HANDLE_BYTES", "qk_norm_rope", "KVCache", "kv_cache_write",
           "qk_norm_rope_kv_write", "kv_cache_read", "tree_attention",
           "tree_attention_workspace_bytes", "plan_tree_attention", "ROTATION_STYLES",
           "SECTION_ORDERS", "gated_add_rms_norm", "KVPages", "kv_step", "kv_trim",
           "kv_cache_compact", "MAX_STEP_SEQUENCES", "verify_drafts"]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "librarn.so")

DTYPE_CODES = {"f32": 0, "f16": 1, "bf16": 2}
OP_CODES = {"rms_norm": 0, "fused_add_rms_norm": 1, "reduce_add_rms_norm": 2}
PATHS = {"auto": 0, "rows": 1, "stream": 2, "cluster": 3}
FP8_FORMATS = {"e4m3": 0, "e5m2": 1}
SCALE_MODES = {"tensor": 0, "row": 1}
ROTATION_STYLES = {"half": 0, "interleaved": 1}
SECTION_ORDERS = ("blocks", "cyclic")
# rarn_tuning knobs (planner overrides; -1 is the planner's own choice)
TUNING = {"rows_per_thread": 0, "rows_grid": 1, "rows_pipeline": 2, "l2_rows": 3,
          "stream_packs": 4, "stream_groups": 5, "gemm_cols": 6, "gemm_slab": 7,
          "gemm_ctas_per_sm": 8, "gemm_persistent": 9, "gemm_pair": 10,
          "gemm_norm_in_epilogue": 11, "gemm_tail_split": 12, "gemm_split_k": 13,
          "fp8in_ring": 14, "fp8in_pack16": 15, "tp_prefetch": 16}
STATUS = {0: "RARN_OK", 1: "RARN_ERR_INVALID_ARG", 2: "RARN_ERR_UNSUPPORTED",
          3: "RARN_ERR_ALIAS", 4: "RARN_ERR_CUDA"}


class RarnError(RuntimeError):
    """A non-OK status from the C ABI."""

    def __init__(self, status: int, what: str, cuda_error: int = 0):
        self.status = status
        self.cuda_error = cuda_error
        msg = f"{what}: {STATUS.get(status, status)}"
        if status == 4:
            msg += f" (cudaError {cuda_error})"
        super().__init__(msg)


class Rows(ctypes.Structure):
    """``rarn_rows``: data pointer, row stride in elements, storage type."""
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int)]


MAX_STEP_SEQUENCES = 8192
MAX_PAGE_SIZE = 1 << 20
TP_MAX_RANKS = 8
TP_SIGNAL_BYTES = 1024 * TP_MAX_RANKS * 4
IPC_HANDLE_BYTES = 96


class TpGroup(ctypes.Structure):
    """``rarn_tp_group``: world size, rank, every rank's buffer and signal pad
    as this process addresses them."""
    _fields_ = [("world_size", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("buffers", ctypes.c_void_p * TP_MAX_RANKS),
                ("signals", ctypes.c_void_p * TP_MAX_RANKS)]


class Fp8Rows(ctypes.Structure):
    """``rarn_fp8_rows``: code matrix (row stride in bytes), format, scale
    mode and the scale's device pointer."""
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64),
                ("format", ctypes.c_int), ("scale_mode", ctypes.c_int),
                ("scale", ctypes.c_void_p)]


class Gate(ctypes.Structure):
    """``rarn_gate``: data pointer, row stride in elements, rows, index."""
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("index", ctypes.c_void_p)]


class Heads(ctypes.Structure):
    """``rarn_heads``: data pointer, token and head strides in elements, heads,
    storage type."""
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("heads", ctypes.c_int32),
                ("dtype", ctypes.c_int)]


class Rotation(ctypes.Structure):
    """``rarn_rotation``: table, positions, table rows, rotated elements, style."""
    _fields_ = [("cos_sin", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("table_rows", ctypes.c_int64), ("rot_dim", ctypes.c_int32),
                ("style", ctypes.c_int)]


class RotationAxes(ctypes.Structure):
    """``rarn_rotation_axes``: the rotation, axes, elements between two axes'
    positions, each pair's axis (host memory)."""
    _fields_ = [("rotation", Rotation), ("axes", ctypes.c_int32),
                ("position_stride", ctypes.c_int64), ("axis_of_pair", ctypes.c_void_p)]


class KvCacheDesc(ctypes.Structure):
    """``rarn_kv_cache``."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("slot_stride", ctypes.c_int64),
                ("scale_page_stride", ctypes.c_int64), ("scale_head_stride", ctypes.c_int64),
                ("scale_slot_stride", ctypes.c_int64), ("num_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("format", ctypes.c_int),
                ("scale_mode", ctypes.c_int)]


class KvPagesDesc(ctypes.Structure):
    """``rarn_kv_pages``."""
    _fields_ = [("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("table_width", ctypes.c_int64), ("held", ctypes.c_void_p),
                ("free_pages", ctypes.c_void_p), ("free_count", ctypes.c_void_p),
                ("ticket", ctypes.c_void_p), ("sequences", ctypes.c_int64),
                ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int32)]


_lib = None


def library() -> ctypes.CDLL:
    """The loaded ``librarn.so`` with its argument types declared."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m residual_add_rmsnorm_gb300.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i64, i32, f32, c_int = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32,
                                ctypes.c_float, ctypes.c_int)
    lib.rarn_rms_norm.argtypes = [vp, vp, vp, i64, i64, f32, c_int, vp]
    lib.rarn_fused_add_rms_norm.argtypes = [vp, vp, vp, vp, i64, i64, f32, c_int, vp]
    lib.rarn_reduce_add_rms_norm.argtypes = [vp, vp, i32, vp, vp, i64, i64, f32, c_int, vp]
    lib.rarn_rms_norm_host.argtypes = [vp, vp, vp, i64, i64, f32, c_int, vp]
    lib.rarn_fused_add_rms_norm_host.argtypes = [vp, vp, vp, vp, i64, i64, f32, c_int, vp]
    lib.rarn_reduce_add_rms_norm_host.argtypes = [vp, vp, i32, vp, vp, i64, i64, f32, c_int, vp]
    for f in (lib.rarn_rms_norm, lib.rarn_fused_add_rms_norm, lib.rarn_reduce_add_rms_norm,
              lib.rarn_rms_norm_host, lib.rarn_fused_add_rms_norm_host,
              lib.rarn_reduce_add_rms_norm_host):
        f.restype = c_int
    lib.rarn_status_string.argtypes = [c_int]
    lib.rarn_status_string.restype = ctypes.c_char_p
    lib.rarn_last_cuda_error.argtypes = []
    lib.rarn_last_cuda_error.restype = c_int
    lib.rarn_set_path.argtypes = [c_int]
    lib.rarn_set_path.restype = c_int
    lib.rarn_get_path.argtypes = []
    lib.rarn_get_path.restype = c_int
    lib.rarn_plan.argtypes = [c_int, i64, i64, i32, c_int, c_int, c_int, ctypes.c_char_p,
                              ctypes.c_size_t]
    lib.rarn_plan.restype = c_int
    lib.rarn_watchdog.argtypes = [ctypes.POINTER(ctypes.c_uint32), c_int]
    lib.rarn_watchdog.restype = c_int
    lib.rarn_version.argtypes = []
    lib.rarn_version.restype = c_int
    lib.rarn_host_access.argtypes = []
    lib.rarn_host_access.restype = c_int
    lib.rarn_rms_norm_ex.argtypes = [Rows, Rows, vp, i64, i64, f32, vp]
    lib.rarn_fused_add_rms_norm_ex.argtypes = [Rows, Rows, Rows, vp, i64, i64, f32, vp]
    lib.rarn_reduce_add_rms_norm_ex.argtypes = [Rows, Rows, i64, i32, Rows, vp, i64, i64, f32,
                                                vp]
    for f in (lib.rarn_rms_norm_ex, lib.rarn_fused_add_rms_norm_ex,
              lib.rarn_reduce_add_rms_norm_ex):
        f.restype = c_int
    lib.rarn_plan_ex.argtypes = [c_int, i64, i64, i32, c_int, c_int, c_int, c_int,
                                 ctypes.c_char_p, ctypes.c_size_t]
    lib.rarn_plan_ex.restype = c_int
    fp = ctypes.POINTER(Fp8Rows)
    lib.rarn_rms_norm_fp8.argtypes = [fp, Rows, vp, i64, i64, f32, vp]
    lib.rarn_fused_add_rms_norm_fp8.argtypes = [fp, Rows, Rows, vp, i64, i64, f32, vp]
    lib.rarn_reduce_add_rms_norm_fp8.argtypes = [fp, Rows, i64, i32, Rows, vp, i64, i64, f32, vp]
    for f in (lib.rarn_rms_norm_fp8, lib.rarn_fused_add_rms_norm_fp8,
              lib.rarn_reduce_add_rms_norm_fp8):
        f.restype = c_int
    lib.rarn_plan_fp8.argtypes = [c_int, i64, i64, i32, c_int, c_int, c_int, ctypes.c_char_p,
                                  ctypes.c_size_t]
    lib.rarn_plan_fp8.restype = c_int
    lib.rarn_gated_add_rms_norm.argtypes = [Rows, Rows, Rows, Rows, vp, vp, ctypes.POINTER(Gate),
                                            f32, f32, i64, i64, f32, vp]
    lib.rarn_gated_add_rms_norm.restype = c_int
    lib.rarn_gemm_add_rms_norm.argtypes = [Rows, Rows, Rows, Rows, vp, i64, i64, i64, f32, vp,
                                           ctypes.c_size_t, vp]
    lib.rarn_gemm_add_rms_norm.restype = c_int
    lib.rarn_gemm_add_rms_norm_noalloc.argtypes = [Rows, Rows, Rows, Rows, vp, i64, i64, i64,
                                                   f32, vp]
    lib.rarn_gemm_add_rms_norm_noalloc.restype = c_int
    lib.rarn_reduce_add_rms_norm_fp8in.argtypes = [vp, vp, i32, c_int, vp, vp, vp, i64, i64, f32,
                                                   c_int, vp]
    lib.rarn_reduce_add_rms_norm_fp8in.restype = c_int
    lib.rarn_gemm_workspace_bytes.argtypes = [i64, i64]
    lib.rarn_gemm_workspace_bytes.restype = i64
    lib.rarn_plan_gemm.argtypes = [i64, i64, i64, c_int, ctypes.c_int32, ctypes.c_char_p,
                                   ctypes.c_size_t]
    lib.rarn_plan_gemm.restype = c_int
    lib.rarn_plan_tree_attention.argtypes = [i64] * 6 + [ctypes.c_char_p, ctypes.c_size_t]
    lib.rarn_plan_tree_attention.restype = c_int
    lib.rarn_plan_fp8in.argtypes = [i64, i64, ctypes.c_int32, c_int, c_int, ctypes.c_int32,
                                    ctypes.c_int32, ctypes.c_char_p, ctypes.c_size_t]
    lib.rarn_plan_fp8in.restype = c_int
    lib.rarn_plan_tp.argtypes = [i64, i64, ctypes.c_int32, c_int, c_int, ctypes.c_int32,
                                 ctypes.c_int32, ctypes.c_char_p, ctypes.c_size_t]
    lib.rarn_plan_tp.restype = c_int
    lib.rarn_set_pdl.argtypes = [c_int]
    lib.rarn_set_pdl.restype = c_int
    lib.rarn_get_pdl.argtypes = []
    lib.rarn_get_pdl.restype = c_int
    lib.rarn_test_stall.argtypes = [ctypes.c_longlong, ctypes.c_ulonglong]
    lib.rarn_test_stall.restype = c_int
    lib.rarn_set_tuning.argtypes = [c_int, i64]
    lib.rarn_set_tuning.restype = c_int
    lib.rarn_get_tuning.argtypes = [c_int, ctypes.POINTER(i64)]
    lib.rarn_get_tuning.restype = c_int
    lib.rarn_reset_tuning.argtypes = []
    lib.rarn_reset_tuning.restype = c_int
    tg = ctypes.POINTER(TpGroup)
    lib.rarn_tp_rows.argtypes = [i64, i32, i32, ctypes.POINTER(i64), ctypes.POINTER(i64)]
    lib.rarn_tp_rows.restype = c_int
    lib.rarn_tp_reduce_add_rms_norm.argtypes = [tg, vp, vp, i64, i64, f32, c_int, vp]
    lib.rarn_tp_reduce_add_rms_norm.restype = c_int
    lib.rarn_tp_reduce_add_rms_norm_world.argtypes = [tg, vp, vp, i64, i64, f32, c_int, vp]
    lib.rarn_tp_reduce_add_rms_norm_world.restype = c_int
    lib.rarn_ipc_export.argtypes = [vp, vp]
    lib.rarn_ipc_export.restype = c_int
    lib.rarn_ipc_import.argtypes = [vp, ctypes.POINTER(vp)]
    lib.rarn_ipc_import.restype = c_int
    lib.rarn_ipc_close.argtypes = [vp]
    lib.rarn_ipc_close.restype = c_int
    lib.rarn_launch_floor.argtypes = [vp, i64, i32, i32, vp]
    lib.rarn_launch_floor.restype = c_int
    lib.rarn_gemm_noalloc_rows.argtypes = [i64]
    lib.rarn_gemm_noalloc_rows.restype = i64
    rot, kc = ctypes.POINTER(Rotation), ctypes.POINTER(KvCacheDesc)
    lib.rarn_qk_norm_rope.argtypes = [Heads, Heads, Heads, Heads, vp, vp, rot, i64, i64, f32, vp]
    lib.rarn_kv_cache_write.argtypes = [kc, Heads, Heads, vp, i64, vp]
    lib.rarn_qk_norm_rope_kv_write.argtypes = [Heads, kc, Heads, Heads, Heads, vp, vp, rot, vp,
                                               i64, f32, vp]
    ra = ctypes.POINTER(RotationAxes)
    lib.rarn_qk_norm_rope_axes.argtypes = [Heads, Heads, Heads, Heads, vp, vp, ra, i64, i64, f32,
                                           vp]
    lib.rarn_qk_norm_rope_axes_kv_write.argtypes = [Heads, kc, Heads, Heads, Heads, vp, vp, ra, vp,
                                                    i64, f32, vp]
    lib.rarn_kv_cache_read.argtypes = [Heads, Heads, kc, vp, i64, i64, vp, i64, i64, vp]
    lib.rarn_tree_attention.argtypes = [Heads, Heads, kc, vp, i64, i64, vp, vp, vp, i64, i64, i64,
                                        f32, vp, ctypes.c_size_t, vp]
    for f in (lib.rarn_qk_norm_rope, lib.rarn_kv_cache_write, lib.rarn_qk_norm_rope_kv_write,
              lib.rarn_qk_norm_rope_axes, lib.rarn_qk_norm_rope_axes_kv_write,
              lib.rarn_kv_cache_read, lib.rarn_tree_attention):
        f.restype = c_int
    kp = ctypes.POINTER(KvPagesDesc)
    lib.rarn_kv_step.argtypes = [kp, vp, vp, vp, vp, vp, vp, i64, vp]
    lib.rarn_kv_trim.argtypes = [kp, vp, vp]
    lib.rarn_kv_cache_compact.argtypes = [kc, vp, i64, i64, vp, vp, vp, i64, i64, vp]
    lib.rarn_verify_drafts.argtypes = [vp, vp, vp, Rows, ctypes.POINTER(Rows), vp, vp, vp, vp, vp,
                                       i64, i64, i64, i64, vp]
    for f in (lib.rarn_kv_step, lib.rarn_kv_trim, lib.rarn_kv_cache_compact,
              lib.rarn_verify_drafts):
        f.restype = c_int
    lib.rarn_tree_attention_workspace_bytes.argtypes = [i64, i64, i64, i64, i64]
    lib.rarn_tree_attention_workspace_bytes.restype = i64
    _lib = lib
    return lib


def _check(status: int, what: str):
    if status != 0:
        raise RarnError(status, what, library().rarn_last_cuda_error() if status == 4 else 0)


def _dtype_code(t) -> int:
    import torch
    codes = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
    if t.dtype not in codes:
        raise TypeError(f"unsupported dtype {t.dtype}: expected float32, float16 or bfloat16")
    return codes[t.dtype]


def _check_tensor(name, t, dtype, device):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _stream(device):
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def rms_norm(x, gamma, eps: float, out=None):
    """y = x * rsqrt(mean(x^2, -1) + eps) * gamma over the last dimension.

    x: [..., H] CUDA tensor (float32 / float16 / bfloat16, contiguous);
    gamma: [H].  ``out`` may be given (it may be ``x`` itself).  Runs on the
    current stream of x's device.
    """
    import torch
    H = x.shape[-1]
    _check_tensor("x", x, x.dtype, x.device)
    _check_tensor("gamma", gamma, x.dtype, x.device)
    if gamma.numel() != H:
        raise ValueError(f"gamma has {gamma.numel()} elements, expected {H}")
    y = torch.empty_like(x) if out is None else out
    _check_tensor("out", y, x.dtype, x.device)
    if y.shape != x.shape:
        raise ValueError("out must have the shape of x")
    T = x.numel() // H if H else 0
    with torch.cuda.device(x.device):
        _check(library().rarn_rms_norm(y.data_ptr(), x.data_ptr(), gamma.data_ptr(), T, H,
                                       float(eps), _dtype_code(x), _stream(x.device)),
               "rarn_rms_norm")
    return y


def fused_add_rms_norm(x, residual, gamma, eps: float, out=None):
    """residual <- x + residual (in place); returns RMSNorm(residual) * gamma.

    x, residual: [..., H]; gamma: [H]; all one dtype, contiguous, on one CUDA
    device.  ``out`` may be ``x``.
    """
    import torch
    H = x.shape[-1]
    for n, t in (("x", x), ("residual", residual), ("gamma", gamma)):
        _check_tensor(n, t, x.dtype, x.device)
    if residual.shape != x.shape:
        raise ValueError("residual must have the shape of x")
    if gamma.numel() != H:
        raise ValueError(f"gamma has {gamma.numel()} elements, expected {H}")
    y = torch.empty_like(x) if out is None else out
    _check_tensor("out", y, x.dtype, x.device)
    if y.shape != x.shape:
        raise ValueError("out must have the shape of x")
    T = x.numel() // H if H else 0
    with torch.cuda.device(x.device):
        _check(library().rarn_fused_add_rms_norm(
            y.data_ptr(), x.data_ptr(), residual.data_ptr(), gamma.data_ptr(), T, H, float(eps),
            _dtype_code(x), _stream(x.device)), "rarn_fused_add_rms_norm")
    return y


def reduce_add_rms_norm(partials, residual, gamma, eps: float, out=None):
    """residual <- ((p_0 + p_1) + ... + p_{R-1}) + residual (binary32, one
    rounding, in place); returns RMSNorm(residual) * gamma.

    partials: [R, ..., H]; residual: [..., H]; gamma: [H].  ``out`` may be
    ``partials[0]``.
    """
    import torch
    R = partials.shape[0]
    H = residual.shape[-1]
    for n, t in (("partials", partials), ("residual", residual), ("gamma", gamma)):
        _check_tensor(n, t, residual.dtype, residual.device)
    if tuple(partials.shape[1:]) != tuple(residual.shape):
        raise ValueError("partials must have shape [R, *residual.shape]")
    if gamma.numel() != H:
        raise ValueError(f"gamma has {gamma.numel()} elements, expected {H}")
    y = torch.empty_like(residual) if out is None else out
    _check_tensor("out", y, residual.dtype, residual.device)
    if y.shape != residual.shape:
        raise ValueError("out must have the shape of residual")
    T = residual.numel() // H if H else 0
    with torch.cuda.device(residual.device):
        _check(library().rarn_reduce_add_rms_norm(
            y.data_ptr(), partials.data_ptr(), R, residual.data_ptr(), gamma.data_ptr(), T, H,
            float(eps), _dtype_code(residual), _stream(residual.device)),
            "rarn_reduce_add_rms_norm")
    return y


def _check_host(name, t, dtype):
    if t.is_cuda:
        raise ValueError(f"{name} must be a pinned host tensor")
    if not t.is_pinned():
        raise ValueError(f"{name} must be pinned (torch.Tensor.pin_memory())")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _host_call(fn, what, device):
    import torch
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    with torch.cuda.device(dev):
        _check(fn(_stream(dev)), what)


def rms_norm_host(x, gamma, eps: float, out=None, device=None):
    """rms_norm on pinned host tensors: the kernel on ``device`` (default:
    the current one) reads x and gamma and writes y through their device
    mapping; y is in host memory once that device's current stream reaches
    the call."""
    import torch
    H = x.shape[-1]
    for n, t in (("x", x), ("gamma", gamma)):
        _check_host(n, t, x.dtype)
    y = torch.empty_like(x).pin_memory() if out is None else out
    _check_host("out", y, x.dtype)
    if y.shape != x.shape or gamma.numel() != H:
        raise ValueError("shape mismatch")
    T = x.numel() // H if H else 0
    _host_call(lambda st: library().rarn_rms_norm_host(
        y.data_ptr(), x.data_ptr(), gamma.data_ptr(), T, H, float(eps), _dtype_code(x), st),
        "rarn_rms_norm_host", device)
    return y


def fused_add_rms_norm_host(x, residual, gamma, eps: float, out=None, device=None):
    """fused_add_rms_norm on pinned host tensors (see rms_norm_host)."""
    import torch
    H = x.shape[-1]
    for n, t in (("x", x), ("residual", residual), ("gamma", gamma)):
        _check_host(n, t, x.dtype)
    y = torch.empty_like(x).pin_memory() if out is None else out
    _check_host("out", y, x.dtype)
    if y.shape != x.shape or residual.shape != x.shape or gamma.numel() != H:
        raise ValueError("shape mismatch")
    T = x.numel() // H if H else 0
    _host_call(lambda st: library().rarn_fused_add_rms_norm_host(
        y.data_ptr(), x.data_ptr(), residual.data_ptr(), gamma.data_ptr(), T, H, float(eps),
        _dtype_code(x), st), "rarn_fused_add_rms_norm_host", device)
    return y


def reduce_add_rms_norm_host(partials, residual, gamma, eps: float, out=None, device=None):
    """reduce_add_rms_norm on pinned host tensors (see rms_norm_host)."""
    import torch
    R = partials.shape[0]
    H = residual.shape[-1]
    for n, t in (("partials", partials), ("residual", residual), ("gamma", gamma)):
        _check_host(n, t, residual.dtype)
    y = torch.empty_like(residual).pin_memory() if out is None else out
    _check_host("out", y, residual.dtype)
    if tuple(partials.shape[1:]) != tuple(residual.shape) or y.shape != residual.shape or \
            gamma.numel() != H:
        raise ValueError("shape mismatch")
    T = residual.numel() // H if H else 0
    _host_call(lambda st: library().rarn_reduce_add_rms_norm_host(
        y.data_ptr(), partials.data_ptr(), R, residual.data_ptr(), gamma.data_ptr(), T, H,
        float(eps), _dtype_code(residual), st), "rarn_reduce_add_rms_norm_host", device)
    return y


def set_path(name: str) -> None:
    """Force a kernel family ('auto', 'rows', 'stream', 'cluster'), process-wide."""
    _check(library().rarn_set_path(PATHS[name]), "rarn_set_path")


def _rows(name, t, device):
    """A 2-D CUDA tensor with unit element stride as a rarn_rows."""
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device}")
    if t.dim() != 2 or t.stride(1) != 1 or t.stride(0) < t.shape[1]:
        raise ValueError(f"{name} must be 2-D with unit stride along rows and a row stride "
                         f">= its row length")
    return Rows(t.data_ptr(), t.stride(0), _dtype_code(t))


def rms_norm_ex(x, gamma, eps: float, out):
    """rms_norm on row-strided 2-D views: x [T, H] and out [T, H] may be
    slices of wider tensors (unit stride within a row, any row stride >= H)."""
    import torch
    T, H = x.shape
    _check_tensor("gamma", gamma, x.dtype, x.device)
    if gamma.numel() != H or tuple(out.shape) != (T, H):
        raise ValueError("shape mismatch")
    with torch.cuda.device(x.device):
        _check(library().rarn_rms_norm_ex(_rows("out", out, x.device), _rows("x", x, x.device),
                                          gamma.data_ptr(), T, H, float(eps), _stream(x.device)),
               "rarn_rms_norm_ex")
    return out


def fused_add_rms_norm_ex(x, residual, gamma, eps: float, out):
    """fused_add_rms_norm on row-strided 2-D views; the residual may be
    float32 with float16 / bfloat16 x, gamma and out (an fp32 residual
    stream: the sum is kept in binary32)."""
    import torch
    T, H = x.shape
    _check_tensor("gamma", gamma, x.dtype, x.device)
    if gamma.numel() != H or tuple(out.shape) != (T, H) or tuple(residual.shape) != (T, H):
        raise ValueError("shape mismatch")
    with torch.cuda.device(x.device):
        _check(library().rarn_fused_add_rms_norm_ex(
            _rows("out", out, x.device), _rows("x", x, x.device),
            _rows("residual", residual, x.device), gamma.data_ptr(), T, H, float(eps),
            _stream(x.device)), "rarn_fused_add_rms_norm_ex")
    return out


def reduce_add_rms_norm_ex(partials, residual, gamma, eps: float, out):
    """reduce_add_rms_norm on strided views: partials [R, T, H] with unit
    stride within a row and any row / partial strides; residual and out are
    row-strided 2-D views; the residual may be float32 with 16-bit partials."""
    import torch
    R, T, H = partials.shape
    dev = partials.device
    if not partials.is_cuda or partials.stride(2) != 1 or partials.stride(1) < H:
        raise ValueError("partials must be [R, T, H] with unit stride within a row")
    _check_tensor("gamma", gamma, partials.dtype, dev)
    if gamma.numel() != H or tuple(out.shape) != (T, H) or tuple(residual.shape) != (T, H):
        raise ValueError("shape mismatch")
    pr = Rows(partials.data_ptr(), partials.stride(1), _dtype_code(partials))
    with torch.cuda.device(dev):
        _check(library().rarn_reduce_add_rms_norm_ex(
            _rows("out", out, dev), pr, partials.stride(0), R, _rows("residual", residual, dev),
            gamma.data_ptr(), T, H, float(eps), _stream(dev)), "rarn_reduce_add_rms_norm_ex")
    return out


def _fp8_out(out, scale, fmt, scale_mode, T, H, device):
    """The rarn_fp8_rows of an 8-bit output: ``out`` is a 2-D [T, H] view
    (unit stride within a row) of uint8 or a torch float8 type (whose format
    must then match ``fmt``); ``scale`` a float32 CUDA tensor of 1 (per
    tensor) or T (per row, contiguous) values."""
    import torch
    f8 = {torch.float8_e4m3fn: "e4m3", torch.float8_e5m2: "e5m2"}
    if out.dtype in f8:
        if f8[out.dtype] != fmt:
            raise ValueError(f"out is {out.dtype} but fmt is {fmt}")
    elif out.dtype != torch.uint8:
        raise TypeError("out must be uint8 or a float8 tensor")
    if not out.is_cuda or out.device != device:
        raise ValueError(f"out must be a CUDA tensor on {device}")
    if tuple(out.shape) != (T, H) or out.stride(1) != 1 or (T > 1 and out.stride(0) < H):
        raise ValueError("out must be [T, H] with unit stride within a row")
    n = 1 if scale_mode == "tensor" else T
    if (not scale.is_cuda or scale.device != device or scale.dtype != torch.float32 or
            scale.numel() != n or (n > 1 and scale.stride(0) != 1)):
        raise ValueError(f"scale must be a contiguous float32 CUDA tensor of {n} values")
    return Fp8Rows(out.data_ptr(), out.stride(0) if T > 1 else H, FP8_FORMATS[fmt],
                   SCALE_MODES[scale_mode], scale.data_ptr())


def rms_norm_fp8(x, gamma, eps: float, out, scale, fmt: str = "e4m3",
                 scale_mode: str = "tensor"):
    """RMSNorm with an 8-bit output: out[t, i] = code of v / s, v = x_i /
    RMS(x) * gamma_i, s = scale[0] (per tensor) or max|v| / maxf written to
    scale[t] (per row).  x: 2-D row-strided view."""
    import torch
    T, H = x.shape
    _check_tensor("gamma", gamma, x.dtype, x.device)
    if gamma.numel() != H:
        raise ValueError("shape mismatch")
    d = _fp8_out(out, scale, fmt, scale_mode, T, H, x.device)
    with torch.cuda.device(x.device):
        _check(library().rarn_rms_norm_fp8(ctypes.byref(d), _rows("x", x, x.device),
                                           gamma.data_ptr(), T, H, float(eps),
                                           _stream(x.device)), "rarn_rms_norm_fp8")
    return out


def fused_add_rms_norm_fp8(x, residual, gamma, eps: float, out, scale, fmt: str = "e4m3",
                           scale_mode: str = "tensor"):
    """fused_add_rms_norm with an 8-bit output (residual updated in place, of
    x's type)."""
    import torch
    T, H = x.shape
    _check_tensor("gamma", gamma, x.dtype, x.device)
    if gamma.numel() != H or tuple(residual.shape) != (T, H):
        raise ValueError("shape mismatch")
    d = _fp8_out(out, scale, fmt, scale_mode, T, H, x.device)
    with torch.cuda.device(x.device):
        _check(library().rarn_fused_add_rms_norm_fp8(
            ctypes.byref(d), _rows("x", x, x.device), _rows("residual", residual, x.device),
            gamma.data_ptr(), T, H, float(eps), _stream(x.device)), "rarn_fused_add_rms_norm_fp8")
    return out


def reduce_add_rms_norm_fp8(partials, residual, gamma, eps: float, out, scale,
                            fmt: str = "e4m3", scale_mode: str = "tensor"):
    """reduce_add_rms_norm with an 8-bit output: partials [R, T, H] with unit
    stride within a row (any row / partial strides)."""
    import torch
    R, T, H = partials.shape
    dev = partials.device
    if not partials.is_cuda or partials.stride(2) != 1 or partials.stride(1) < H:
        raise ValueError("partials must be [R, T, H] with unit stride within a row")
    _check_tensor("gamma", gamma, partials.dtype, dev)
    if gamma.numel() != H or tuple(residual.shape) != (T, H):
        raise ValueError("shape mismatch")
    d = _fp8_out(out, scale, fmt, scale_mode, T, H, dev)
    pr = Rows(partials.data_ptr(), partials.stride(1), _dtype_code(partials))
    with torch.cuda.device(dev):
        _check(library().rarn_reduce_add_rms_norm_fp8(
            ctypes.byref(d), pr, partials.stride(0), R, _rows("residual", residual, dev),
            gamma.data_ptr(), T, H, float(eps), _stream(dev)), "rarn_reduce_add_rms_norm_fp8")
    return out


def plan_fp8(op: str, T: int, H: int, R: int, dtype: str, vec_ok: bool = True,
             num_sms: int = 0) -> str:
    """The kernel the current path setting would launch for an 8-bit output."""
    buf = ctypes.create_string_buffer(256)
    st = library().rarn_plan_fp8(OP_CODES[op], T, H, R, DTYPE_CODES[dtype], int(vec_ok),
                                 num_sms, buf, 256)
    if st not in (0, 2):
        _check(st, "rarn_plan_fp8")
    return buf.value.decode()


def gemm_noalloc_rows(H: int) -> int:
    """Rows one launch sequence of gemm_add_rms_norm_noalloc covers at row
    length H (-1: H unsupported)."""
    return int(library().rarn_gemm_noalloc_rows(H))


def gemm_workspace_bytes(T: int, H: int) -> int:
    """Workspace bytes the GEMM form needs for T rows of H (-1: H unsupported)."""
    return int(library().rarn_gemm_workspace_bytes(T, H))


def gemm_add_rms_norm(a, w, residual, gamma, eps: float, out=None, workspace=None):
    """The fused form whose partial is a matrix product: P = a @ w.T
    (a [T, K], w [H, K], bfloat16 or float16; 2-D views with unit stride
    within a row), residual [T, H] <- RN(P + residual) in place,
    y = RMSNorm(residual) * gamma into ``out`` (allocated if None).
    ``workspace``: a CUDA tensor of at least gemm_workspace_bytes(T, H) bytes
    (allocated if None)."""
    import torch
    T, K = a.shape
    H = w.shape[0]
    dev = a.device
    if tuple(w.shape) != (H, K) or tuple(residual.shape) != (T, H) or gamma.numel() != H:
        raise ValueError("shape mismatch")
    _check_tensor("gamma", gamma, a.dtype, dev)
    if out is None:
        out = torch.empty(T, H, dtype=a.dtype, device=dev)
    if workspace is None:
        n = max(gemm_workspace_bytes(T, H), 4)
        workspace = torch.empty((n + 3) // 4, dtype=torch.float32, device=dev)
    if not workspace.is_cuda or workspace.device != dev:
        raise ValueError(f"workspace must be a CUDA tensor on {dev}")
    with torch.cuda.device(dev):
        _check(library().rarn_gemm_add_rms_norm(
            _rows("out", out, dev), _rows("a", a, dev), _rows("w", w, dev),
            _rows("residual", residual, dev), gamma.data_ptr(), T, H, K, float(eps),
            workspace.data_ptr(), workspace.numel() * workspace.element_size(),
            _stream(dev)), "rarn_gemm_add_rms_norm")
    return out


def gemm_add_rms_norm_noalloc(a, w, residual, gamma, eps: float, out=None):
    """gemm_add_rms_norm through the entry point that allocates nothing.

    For callers that cannot allocate device memory (a plug-in whose host
    program owns all device memory, a runtime that forbids allocation once it
    serves, code that cannot take cudaMalloc's implicit synchronisation): the
    partial sums live in a 4 MiB array the library reserves on each GPU when
    it is loaded.  The first call on a device looks up that array's address;
    make it before any stream capture.  Calls on one device share the array,
    so calls that overlap on the GPU race: keep them on one stream or
    synchronise the streams.  ``out`` is allocated here only when not given;
    pass it to keep the whole call allocation-free."""
    import torch
    T, K = a.shape
    H = w.shape[0]
    dev = a.device
    if tuple(w.shape) != (H, K) or tuple(residual.shape) != (T, H) or gamma.numel() != H:
        raise ValueError("shape mismatch")
    _check_tensor("gamma", gamma, a.dtype, dev)
    if out is None:
        out = torch.empty(T, H, dtype=a.dtype, device=dev)
    with torch.cuda.device(dev):
        _check(library().rarn_gemm_add_rms_norm_noalloc(
            _rows("out", out, dev), _rows("a", a, dev), _rows("w", w, dev),
            _rows("residual", residual, dev), gamma.data_ptr(), T, H, K, float(eps),
            _stream(dev)), "rarn_gemm_add_rms_norm_noalloc")
    return out


def reduce_add_rms_norm_fp8in(codes, scales, residual, gamma, eps: float, fmt: str = "e4m3",
                              out=None):
    """reduce_add_rms_norm over R partials stored as 8-bit codes: ``codes``
    [R, ...rows..., H] (uint8, or a torch float8 tensor of the format),
    ``scales`` [R] binary32 on the same device (partial r is code * scales[r]),
    ``residual`` [...rows..., H] updated in place; returns y like the
    residual."""
    import torch
    if codes.dtype in (getattr(torch, "float8_e4m3fn", None), getattr(torch, "float8_e5m2", None)):
        codes = codes.view(torch.uint8)
    if codes.dtype != torch.uint8:
        raise TypeError("codes must be uint8 or float8")
    R, H = codes.shape[0], residual.shape[-1]
    dev = residual.device
    if tuple(codes.shape[1:]) != tuple(residual.shape) or gamma.numel() != H:
        raise ValueError("shape mismatch")
    if scales.dtype != torch.float32 or scales.numel() != R or scales.device != dev:
        raise ValueError("scales must be R binary32 values on the residual's device")
    for n, t in (("codes", codes), ("residual", residual), ("scales", scales)):
        if t.device != dev or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous tensor on {dev}")
    _check_tensor("gamma", gamma, residual.dtype, dev)
    if out is None:
        out = torch.empty_like(residual)
    T = residual.numel() // H if H else 0
    with torch.cuda.device(dev):
        _check(library().rarn_reduce_add_rms_norm_fp8in(
            out.data_ptr(), codes.data_ptr(), R, FP8_FORMATS[fmt], scales.data_ptr(),
            residual.data_ptr(), gamma.data_ptr(), T, H, float(eps), _dtype_code(residual),
            _stream(dev)), "rarn_reduce_add_rms_norm_fp8in")
    return out


def plan_fp8in(T: int, H: int, R: int, dtype: str = "bf16", codes_aligned16: bool = True,
               num_sms: int = 152, max_smem: int = 232448) -> str:
    """The kernel reduce_add_rms_norm_fp8in takes for a problem on a device
    with `num_sms` SMs and `max_smem` bytes of opt-in shared memory per CTA
    (host logic only; the defaults are a GB300's)."""
    buf = ctypes.create_string_buffer(256)
    st = library().rarn_plan_fp8in(T, H, R, DTYPE_CODES[dtype], int(codes_aligned16), num_sms,
                                   max_smem, buf, 256)
    if st not in (0, 2):
        _check(st, "rarn_plan_fp8in")
    return buf.value.decode()


def plan_tp(T: int, H: int, N: int, dtype: str = "bf16", world: bool = True, num_sms: int = 152,
            blocks_per_sm: int = 0) -> str:
    """The launch a tensor-parallel call over N ranks makes (``world``: every
    rank's part in one launch) on a device with ``num_sms`` SMs that holds
    ``blocks_per_sm`` CTAs of the kernel per SM; 0 for either queries the
    current device (host logic only when both are given)."""
    buf = ctypes.create_string_buffer(256)
    st = library().rarn_plan_tp(T, H, N, DTYPE_CODES[dtype], int(world), num_sms, blocks_per_sm,
                                buf, 256)
    if st not in (0, 2):
        _check(st, "rarn_plan_tp")
    return buf.value.decode()


def plan_gemm(T: int, H: int, K: int, dtype: str = "bf16", num_sms: int = 152) -> str:
    """The GEMM kernel's tiling for a problem on a device with ``num_sms`` SMs
    (host logic only; the default is a GB300's; 0 queries the current
    device)."""
    buf = ctypes.create_string_buffer(256)
    st = library().rarn_plan_gemm(T, H, K, DTYPE_CODES[dtype], num_sms, buf, 256)
    if st not in (0, 2):
        _check(st, "rarn_plan_gemm")
    return buf.value.decode()


# What the attention side's calls keep at hand: a decode step makes several of
# them per layer, and Python is most of a short call's time.
_codes = {}       # torch dtype -> rarn_dtype
_get_device = _raw_stream = None


def _on(device, what, fn, *args):
    """fn(*args, stream) on ``device`` and its current stream; raises on a
    status other than OK."""
    global _get_device, _raw_stream
    if _get_device is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda i: torch.cuda.current_stream(i).cuda_stream)
        # last: another thread that sees it uses both
        _get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    i = device.index
    if _get_device() == i:
        status = fn(*args, _raw_stream(i))
    else:
        import torch
        with torch.cuda.device(i):
            status = fn(*args, _raw_stream(i))
    if status:
        _check(status, what)


def _heads(name, t, T, heads, D, dtype, device):
    """A [T, heads, D] CUDA tensor with unit stride inside a head as a
    rarn_heads (heads None: any number)."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[0] != T or shape[2] != D or \
            (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must be [{T}, {'heads' if heads is None else heads}, {D}], got "
                         f"{list(shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.get_device() != device.index:  # -1 and None for the CPU
        raise ValueError(f"{name} must be a CUDA tensor on {device}")
    if stride[2] != 1 and D > 1:
        raise ValueError(f"{name} must have unit stride inside a head")
    return Heads(t.data_ptr(), stride[0], stride[1], shape[1], _codes.get(dtype) or _code(t))


def _indices(name, t, dtype, n, device):
    """A contiguous CUDA index tensor of n values."""
    if t.dtype is not dtype or t.get_device() != device.index:
        raise TypeError(f"{name} must be a {dtype} CUDA tensor on {device}")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with {n} values")
    return t.data_ptr()


def _gamma(name, g, D, dtype, device):
    if g is None:
        return None
    if g.dtype is not dtype or g.get_device() != device.index or not g.is_contiguous():
        _check_tensor(name, g, dtype, device)
    if g.numel() != D:
        raise ValueError(f"{name} has {g.numel()} elements, expected {D}")
    return g.data_ptr()


def _code(t) -> int:
    """The rarn_dtype of a tensor."""
    dtype = t.dtype
    code = _codes.get(dtype)
    if code is None:
        code = _codes[dtype] = _dtype_code(t)
    return code


def _matrix(name, t, shape, dtype, code, device):
    """A CUDA tensor of ``shape`` [T, H] with unit stride within a row as a
    rarn_rows."""
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.get_device() != device.index:
        raise ValueError(f"{name} must be a CUDA tensor on {device}")
    row, one = t.stride()
    if one != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have unit stride within a row")
    return Rows(t.data_ptr(), row, code)


def gated_add_rms_norm(x, residual, x_gamma, gamma, eps: float, gate=None, gate_index=None,
                       scale: float = 1.0, residual_scale: float = 1.0, out=None,
                       residual_out=None):
    """The norms after and before a block with its gate and the residual between
    them:

        n = x * rsqrt(mean(x^2) + eps) * x_gamma          (x_gamma None: n = x)
        h = residual_scale * residual + scale * (gate * n)
        y = h * rsqrt(mean(h^2) + eps) * gamma

    x, residual [T, H]: CUDA tensors with unit stride within a row; the residual
    of x's type or float32; x_gamma, gamma [H].  gate: [H] (one for all tokens),
    [T, H], or [rows, H] with ``gate_index`` [T] int32 naming each token's row (a
    token whose index is outside keeps its output rows and sets watchdog bit 4);
    None: no gate.  h goes to ``residual_out``, or in place into the residual
    where that is None.  ``out`` may be x.  Returns y."""
    dev, dt, shape = x.device, x.dtype, x.shape
    if len(shape) != 2:
        raise ValueError("x must be [T, H]")
    T, H = shape
    code, rt = _code(x), residual.dtype
    rx = _matrix("x", x, shape, dt, code, dev)
    rr = rh = _matrix("residual", residual, shape, rt, _code(residual), dev)
    if residual_out is not None and residual_out is not residual:
        rh = _matrix("residual_out", residual_out, shape, rt, rr.dtype, dev)
    if out is None:
        import torch
        out = torch.empty(shape, dtype=dt, device=dev)
    ry = _matrix("out", out, shape, dt, code, dev)
    xg, g = _gamma("x_gamma", x_gamma, H, dt, dev), _gamma("gamma", gamma, H, dt, dev)
    pg = None
    if gate is not None:
        if gate.dim() == 1:
            gate = gate[None]
        n = gate.shape[0]
        rg = _matrix("gate", gate, (n, H), dt, code, dev)
        if gate_index is None:
            if n != 1 and n != T:
                raise ValueError(f"gate must have one row or {T}, or a gate_index")
            index = None
        else:
            import torch
            index = _indices("gate_index", gate_index, torch.int32, T, dev)
        pg = ctypes.byref(Gate(rg.data, rg.row_stride, n, index))
    elif gate_index is not None:
        raise ValueError("gate_index needs a gate")
    _on(dev, "rarn_gated_add_rms_norm", library().rarn_gated_add_rms_norm, ry, rh, rx, rr, xg, g,
        pg, scale, residual_scale, T, H, eps)
    return out


def _rotation(cos_sin, positions, style, T, device):
    """The rarn_rotation of a call, or None without a table."""
    import torch
    if cos_sin is None:
        return _rotation_at(cos_sin, None, style, device)
    if positions is None:
        raise ValueError("cos_sin needs positions")
    if not isinstance(positions, torch.Tensor):
        raise TypeError(f"positions must be an int64 CUDA tensor on {device}")
    return _rotation_at(cos_sin, _indices("positions", positions, torch.int64, T, device), style,
                        device)


def _rotation_at(cos_sin, address, style, device):
    """The same for positions that the caller has checked, by their address."""
    import torch
    code = ROTATION_STYLES.get(style)
    if code is None:
        raise ValueError(f"style must be one of {sorted(ROTATION_STYLES)}")
    if cos_sin is None:
        return None
    if cos_sin.dtype is not torch.float32 or cos_sin.get_device() != device.index or \
            not cos_sin.is_contiguous():
        _check_tensor("cos_sin", cos_sin, torch.float32, device)
    shape = cos_sin.shape
    if len(shape) != 2:
        raise ValueError("cos_sin must be [positions, rot_dim]")
    return Rotation(cos_sin.data_ptr(), address, shape[0], shape[1], code)


# axis_of_pair of a model's sections, as the C ABI takes it
_axis_maps = {}   # (pairs, sections, order) -> ctypes array


def _axis_map(pairs, sections, order):
    key = (pairs, sections, order)
    got = _axis_maps.get(key)
    if got is None:
        if order not in SECTION_ORDERS:
            raise ValueError(f"section_order must be one of {SECTION_ORDERS}")
        left = [int(n) for n in sections]
        if not left or min(left) < 0 or sum(left) != pairs:
            raise ValueError(f"sections must be pairs of each axis, {pairs} in all")
        if order == "blocks":
            axes = [a for a, n in enumerate(left) for _ in range(n)]
        else:
            axes = []
            while len(axes) < pairs:
                for a, n in enumerate(left):
                    if n:
                        axes.append(a)
                        left[a] = n - 1
        got = _axis_maps[key] = (ctypes.c_uint8 * max(pairs, 1))(*axes)
    return got


def _rotation_axes(cos_sin, positions, style, sections, order, T, device):
    """The rarn_rotation_axes of a call."""
    import torch
    if cos_sin is None or positions is None:
        raise ValueError("sections need cos_sin and positions")
    sections = sections if type(sections) is tuple else tuple(sections)
    A = len(sections)
    if not isinstance(positions, torch.Tensor) or positions.dtype is not torch.int64 or \
            positions.get_device() != device.index:
        raise TypeError(f"positions must be an int64 CUDA tensor on {device}")
    shape, stride = positions.shape, positions.stride()
    if len(shape) != 2 or shape[0] != A or shape[1] != T or (T > 1 and stride[1] != 1):
        raise ValueError(f"positions must be [{A}, {T}] with unit stride along the tokens")
    rot = _rotation_at(cos_sin, positions.data_ptr(), style, device)
    amap = _axis_map(rot.rot_dim // 2, sections, order)
    return RotationAxes(rot, A, stride[0], ctypes.addressof(amap))


def qk_norm_rope(q, k, q_gamma, k_gamma, eps: float, cos_sin=None, positions=None,
                 style: str = "half", q_out=None, k_out=None, sections=None,
                 section_order: str = "blocks"):
    """RMSNorm of every query and key head over its D elements, times gamma,
    then the position rotation; returns (q_out, k_out).

    q [T, Hq, D], k [T, Hk, D]: CUDA tensors of one type (float32 / float16 /
    bfloat16) with unit stride inside a head and any other strides (slices of a
    packed projection); q_gamma, k_gamma: [D], or None to leave that norm out;
    cos_sin: [positions, rot_dim] float32, rot_dim / 2 cosines then sines, or
    None for no rotation; positions: [T] int64; style: "half" rotates elements
    (i, i + rot_dim / 2), "interleaved" (2i, 2i + 1).  q_out may be q, k_out k.
    A token whose position is outside the table keeps its output rows and sets
    watchdog bit 4.

    Positions of several axes (time, height, width): positions [axes, T] (unit
    stride along the tokens) and ``sections``, the rotation's pairs of each of up
    to four axes (a tuple; rot_dim / 2 in all).  section_order "blocks": the
    first axis's pairs, then the second's and so on; "cyclic": the axes in turn,
    one that has used its pairs up left out.  Pair i turns by column i of the
    table at its axis's position."""
    import torch
    dev, dt = q.device, q.dtype
    if q.dim() != 3:
        raise ValueError("q must be [T, heads, D]")
    T, Hq, D = q.shape
    hq = _heads("q", q, T, Hq, D, dt, dev)
    hk = _heads("k", k, T, None, D, dt, dev)
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=dt, device=dev)
    if k_out is None:
        k_out = torch.empty(k.shape, dtype=dt, device=dev)
    if sections is None:
        what, fn = "rarn_qk_norm_rope", library().rarn_qk_norm_rope
        rot = _rotation(cos_sin, positions, style, T, dev)
    else:
        what, fn = "rarn_qk_norm_rope_axes", library().rarn_qk_norm_rope_axes
        rot = _rotation_axes(cos_sin, positions, style, sections, section_order, T, dev)
    _on(dev, what, fn, _heads("q_out", q_out, T, Hq, D, dt, dev),
        _heads("k_out", k_out, T, hk.heads, D, dt, dev), hq, hk,
        _gamma("q_gamma", q_gamma, D, dt, dev), _gamma("k_gamma", k_gamma, D, dt, dev), rot, T, D,
        eps)
    return q_out, k_out


class KVCache:
    """A paged cache of keys and values held as e4m3 / e5m2 codes with binary32
    scales.  The tensors are the caller's; this object only describes them.

    k, v: [pages, heads, page_size, head_dim] uint8 (or float8 of the format)
    with unit stride along head_dim and the same strides (views of any layout:
    a pool that keeps tokens before heads is passed permuted); k_scale, v_scale:
    float32 [pages, heads, page_size] with equal strides (scale_mode "row": a
    scale per token and head, written with the codes) or one value each
    ("tensor": read)."""

    def __init__(self, k, v, k_scale, v_scale, fmt: str = "e4m3", scale_mode: str = "row"):
        import torch
        if fmt not in FP8_FORMATS or scale_mode not in SCALE_MODES:
            raise ValueError(f"fmt must be one of {sorted(FP8_FORMATS)}, scale_mode one of "
                             f"{sorted(SCALE_MODES)}")
        codes = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
        if k.dim() != 4:
            raise ValueError("k must be [pages, heads, page_size, head_dim]")
        for n, t in (("k", k), ("v", v)):
            if t.dtype not in (torch.uint8, codes[fmt]):
                raise TypeError(f"{n} must be uint8 or {codes[fmt]}")
            if not t.is_cuda or t.device != k.device:
                raise ValueError(f"{n} must be a CUDA tensor on {k.device}")
            if t.shape != k.shape or t.stride() != k.stride() or t.stride(3) != 1:
                raise ValueError("k and v must have one shape and layout, unit stride along "
                                 "head_dim")
        for n, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t.dtype != torch.float32 or not t.is_cuda or t.device != k.device:
                raise TypeError(f"{n} must be a float32 CUDA tensor on {k.device}")
            if scale_mode == "row":
                if t.shape != k.shape[:3] or t.stride() != k_scale.stride():
                    raise ValueError(f"{n} must be {list(k.shape[:3])}, k_scale and v_scale of "
                                     f"one layout")
            elif t.numel() != 1:
                raise ValueError(f"{n} must hold one value")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.fmt, self.scale_mode = fmt, scale_mode
        self.device = k.device
        self.num_pages, self.heads, self.page_size, self.head_dim = k.shape
        ps, hs, ss = k.stride()[:3]
        sp, sh, s1 = k_scale.stride() if scale_mode == "row" else (0, 0, 0)
        self._desc = KvCacheDesc(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(),
                                 v_scale.data_ptr(), ps, hs, ss, sp, sh, s1, self.num_pages,
                                 self.page_size, self.heads, self.head_dim, FP8_FORMATS[fmt],
                                 SCALE_MODES[scale_mode])
        self._ref = ctypes.byref(self._desc)

    @classmethod
    def empty(cls, pages: int, page_size: int, heads: int, head_dim: int, fmt: str = "e4m3",
              scale_mode: str = "row", device="cuda", k_scale: float = 1.0, v_scale: float = 1.0):
        """A cache of zero codes with tensors of its own (``k_scale``,
        ``v_scale``: the two scales of mode "tensor")."""
        import torch
        shape = (pages, heads, page_size, head_dim)
        k, v = (torch.zeros(shape, dtype=torch.uint8, device=device) for _ in range(2))
        if scale_mode == "row":
            ks, vs = (torch.ones(shape[:3], dtype=torch.float32, device=device) for _ in range(2))
        else:
            ks, vs = (torch.full((1,), float(x), dtype=torch.float32, device=device)
                      for x in (k_scale, v_scale))
        return cls(k, v, ks, vs, fmt, scale_mode)


def kv_cache_write(k, v, cache: KVCache, slots) -> None:
    """Keys and values k, v [T, heads, D] (one type, any strides) quantised into
    the cache: token t into slot slots[t] (int64; page * page_size + slot of the
    page; negative: left out; the others distinct)."""
    import torch
    dev, dt = cache.device, k.dtype
    T = k.shape[0]
    _on(dev, "rarn_kv_cache_write", library().rarn_kv_cache_write, cache._ref,
        _heads("k", k, T, cache.heads, cache.head_dim, dt, dev),
        _heads("v", v, T, cache.heads, cache.head_dim, dt, dev),
        _indices("slots", slots, torch.int64, T, dev), T)


def qk_norm_rope_kv_write(q, k, v, q_gamma, k_gamma, eps: float, cos_sin, positions,
                          cache: KVCache, slots, style: str = "half", q_out=None, sections=None,
                          section_order: str = "blocks"):
    """qk_norm_rope and kv_cache_write in one pass: returns the normalised,
    rotated queries; the keys (quantised from their binary32 values) and values
    go to the cache.  ``sections``, ``section_order``: positions of several axes,
    as in qk_norm_rope."""
    import torch
    dev, dt, H, D = cache.device, q.dtype, cache.heads, cache.head_dim
    T = q.shape[0]
    hq = _heads("q", q, T, None, D, dt, dev)
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=dt, device=dev)
    if sections is None:
        what, fn = "rarn_qk_norm_rope_kv_write", library().rarn_qk_norm_rope_kv_write
        rot = _rotation(cos_sin, positions, style, T, dev)
    else:
        what, fn = "rarn_qk_norm_rope_axes_kv_write", library().rarn_qk_norm_rope_axes_kv_write
        rot = _rotation_axes(cos_sin, positions, style, sections, section_order, T, dev)
    _on(dev, what, fn, _heads("q_out", q_out, T, hq.heads, D, dt, dev),
        cache._ref, hq, _heads("k", k, T, H, D, dt, dev), _heads("v", v, T, H, D, dt, dev),
        _gamma("q_gamma", q_gamma, D, dt, dev), _gamma("k_gamma", k_gamma, D, dt, dev), rot,
        _indices("slots", slots, torch.int64, T, dev), T, eps)
    return q_out


def _page_table(t, device):
    """Address, row stride, sequences and width of a page table."""
    import torch
    if t.dtype is not torch.int32 or t.get_device() != device.index:
        raise TypeError(f"page_table must be an int32 CUDA tensor on {device}")
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or (shape[1] > 1 and stride[1] != 1):
        raise ValueError("page_table must be [sequences, pages] with unit stride along a row")
    return t.data_ptr(), stride[0], shape[0], shape[1]


def kv_cache_read(cache: KVCache, page_table, starts, k_out, v_out):
    """The cached tokens of every sequence, dequantised: sequence b's go to rows
    starts[b] .. starts[b + 1] - 1 of k_out and v_out ([rows, heads, D], one
    type); page_table: [B, width] int32, starts: [B + 1] int32.  Rows past the
    last sequence stay as they were.  Returns (k_out, v_out)."""
    import torch
    dev, dt, H, D = cache.device, k_out.dtype, cache.heads, cache.head_dim
    rows = k_out.shape[0]
    hk = _heads("k_out", k_out, rows, H, D, dt, dev)
    hv = _heads("v_out", v_out, rows, H, D, dt, dev)
    table, stride, B, width = _page_table(page_table, dev)
    _on(dev, "rarn_kv_cache_read", library().rarn_kv_cache_read, hk, hv, cache._ref, table, stride,
        width, _indices("starts", starts, torch.int32, B + 1, dev), B, rows)
    return k_out, v_out


def tree_attention_workspace_bytes(tokens: int, sequences: int, q_heads: int, kv_heads: int,
                                   head_dim: int) -> int:
    """Workspace bytes tree_attention needs for these sizes (-1: unsupported)."""
    return int(library().rarn_tree_attention_workspace_bytes(tokens, sequences, q_heads, kv_heads,
                                                             head_dim))


def plan_tree_attention(tokens: int, sequences: int, q_heads: int, kv_heads: int, head_dim: int,
                        page_size: int) -> str:
    """Which kernel a tree_attention call of these sizes gets (host logic
    only)."""
    buf = ctypes.create_string_buffer(64)
    st = library().rarn_plan_tree_attention(tokens, sequences, q_heads, kv_heads, head_dim,
                                            page_size, buf, 64)
    if st not in (0, 2):
        _check(st, "rarn_plan_tree_attention")
    return buf.value.decode()


def tree_attention(q, cache: KVCache, page_table, context_lens, starts, mask=None,
                   scale: float | None = None, out=None, workspace=None):
    """Attention of drafted tokens over the cache: sequence b's drafted tokens
    are rows starts[b] .. starts[b + 1] - 1 of q [tokens, q_heads, D], their
    keys and values lie in the cache behind its context_lens[b] tokens.  Each
    sees the context and the drafted tokens whose bits are set in its row of
    ``mask`` ([tokens, words] int32, bit d % 32 of word d / 32 for drafted token
    d); without a mask itself and those before it (one token: the decode step).
    ``scale``: of the scores, 1 / sqrt(D) by default.  ``workspace``: a CUDA
    tensor of at least tree_attention_workspace_bytes bytes (allocated if None);
    calls that may overlap need one each.  Returns out (like q)."""
    import torch
    dev, dt, D = cache.device, q.dtype, cache.head_dim
    N = q.shape[0]
    hq = _heads("q", q, N, None, D, dt, dev)
    if out is None:
        out = torch.empty(q.shape, dtype=dt, device=dev)
    ho = _heads("out", out, N, hq.heads, D, dt, dev)
    table, stride, B, width = _page_table(page_table, dev)
    ctx = _indices("context_lens", context_lens, torch.int32, B, dev)
    st = _indices("starts", starts, torch.int32, B + 1, dev)
    pm, words = None, 0
    if mask is not None:
        if mask.dim() != 2 or mask.shape[0] != N:
            raise ValueError(f"mask must be [{N}, words]")
        if mask.shape[1] == 0:  # its address may be that of no mask at all
            raise ValueError("mask must have one word or more")
        words = mask.shape[1]
        pm = _indices("mask", mask, torch.int32, N * words, dev)
    if workspace is None:
        n = max(tree_attention_workspace_bytes(N, B, hq.heads, cache.heads, D), 16)
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous CUDA tensor on {dev}")
    _on(dev, "rarn_tree_attention", library().rarn_tree_attention, ho, hq, cache._ref, table,
        stride, width, ctx, st, pm, words, B, N, D ** -0.5 if scale is None else scale,
        workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out


class KVPages:
    """Which pages of a cache each sequence holds and which are free: the state that
    kv_step and kv_trim update in place.  Int32 CUDA tensors of the caller's:
    page_table [sequences, width] (unit stride along a row; what tree_attention and
    kv_cache_read take), held [sequences], free_pages [num_pages], free_count [1].
    A page belongs to one sequence at a time; calls on one object must be
    ordered.  One that is made while a graph is captured belongs to that graph's
    replays: its word of the calls' own is zeroed there."""

    def __init__(self, page_table, held, free_pages, free_count, page_size: int):
        import torch
        if not 1 <= page_size <= MAX_PAGE_SIZE:  # ctypes would cut it to 32 bits
            raise ValueError(f"page_size must be 1 .. {MAX_PAGE_SIZE}")
        dev = page_table.device
        table, stride, B, width = _page_table(page_table, dev)
        self.page_table, self.held = page_table, held
        self.free_pages, self.free_count = free_pages, free_count
        self.device, self.page_size = dev, page_size
        self.sequences, self.num_pages = B, free_pages.numel()
        # the calls' own word; its zero has to be there for a call on any stream
        self._ticket = torch.zeros(1, dtype=torch.int32, device=dev)
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(dev).synchronize()
        i32 = torch.int32
        self._desc = KvPagesDesc(table, stride, width, _indices("held", held, i32, B, dev),
                                 _indices("free_pages", free_pages, i32, self.num_pages, dev),
                                 _indices("free_count", free_count, i32, 1, dev),
                                 self._ticket.data_ptr(), B, self.num_pages, page_size)
        self._ref = ctypes.byref(self._desc)

    @classmethod
    def empty(cls, sequences: int, width: int, num_pages: int, page_size: int, device="cuda"):
        """Tensors of its own: no sequence holds a page, page 0 is the first taken."""
        import torch
        kw = dict(dtype=torch.int32, device=device)
        return cls(torch.full((sequences, width), -1, **kw), torch.zeros(sequences, **kw),
                   torch.arange(num_pages - 1, -1, -1, **kw), torch.full((1,), num_pages, **kw),
                   page_size)


def kv_step(pages: KVPages, context_lens, new_lens, tokens: int, starts=None, slots=None,
            positions=None, served=None):
    """Pages, slots and positions of a step: sequence b adds new_lens[b] tokens
    behind its context_lens[b] (int32 CUDA tensors of pages.sequences values), and
    gets the pages that they need.  Returns (starts [B + 1] int32, slots [tokens]
    int64, positions [tokens] int64, served [1] int32): row r of sequence b is r -
    starts[b] tokens behind its context, in slot and position; rows past the last
    sequence get slot -1 and position 0.  That is a chain's position; a tree's row
    lies as many tokens behind the context as it is deep, so for trees add each
    row's depth less its number in its sequence before the rows are turned (keys
    that kv_cache_compact moves stay turned as they were).  served < B: rows
    (``tokens``) or free pages ran out at that sequence, and it and those behind it
    got none.  Lengths that make no sense leave their sequence without rows and set
    watchdog bit 4."""
    import torch
    dev, B = pages.device, pages.sequences
    if starts is None:
        starts = torch.empty(B + 1, dtype=torch.int32, device=dev)
    if slots is None:
        slots = torch.empty(tokens, dtype=torch.int64, device=dev)
    if positions is None:
        positions = torch.empty(tokens, dtype=torch.int64, device=dev)
    if served is None:
        served = torch.empty(1, dtype=torch.int32, device=dev)
    i32, i64 = torch.int32, torch.int64
    _on(dev, "rarn_kv_step", library().rarn_kv_step, pages._ref,
        _indices("context_lens", context_lens, i32, B, dev),
        _indices("new_lens", new_lens, i32, B, dev), _indices("starts", starts, i32, B + 1, dev),
        _indices("slots", slots, i64, tokens, dev),
        _indices("positions", positions, i64, tokens, dev),
        _indices("served", served, i32, 1, dev), tokens)
    return starts, slots, positions, served


def kv_trim(pages: KVPages, lens) -> None:
    """Every sequence keeps the pages of its first lens[b] tokens (int32 CUDA
    tensor; 0: a finished sequence) and gives the others back.  A negative length
    keeps its pages; that, and a table entry that is no page (it goes back as it is,
    and the step that takes it gets no slots in it), set watchdog bit 4."""
    import torch
    _on(pages.device, "rarn_kv_trim", library().rarn_kv_trim, pages._ref,
        _indices("lens", lens, torch.int32, pages.sequences, pages.device))


def verify_drafts(probs, tokens, starts, uniforms, final_uniforms, most: int, draft_probs=None,
                  parents=None, new_tokens=None, path=None, lengths=None):
    """Drafted tokens verified against the target's probabilities, and the token
    behind the accepted ones drawn: what comes out is distributed as the target's
    own tokens.

    Sequence b's rows are starts[b] .. starts[b + 1] - 1 (int32, [B + 1]) of probs
    [rows, vocab] (float32 / float16 / bfloat16, unit stride along a row): row 0 its
    last known token, the others drafts; a row holds the target's distribution
    behind its token.  tokens: [rows] int64; parents: [rows] int32, each draft's
    parent row within its sequence (a tree), or None: the row before (a chain).
    uniforms: [rows] float32 in [0, 1), the number that decides among a row's drafts;
    final_uniforms: [B] float32, those of the drawn tokens.  draft_probs: like probs,
    row r the distribution that draft r was drawn from (chains only); None: drafts
    that were chosen without chance.  At most ``most`` drafts are accepted.

    Returns (new_tokens [B, most + 1] int64, path [B, most + 1] int32, lengths [B]
    int32): lengths[b] - 1 accepted drafts; path their rows behind row 0; new_tokens
    their tokens and the drawn one; -1 behind those.  A row without a distribution
    (a sum of 0, or of 2 and more) draws -1; that, and indices outside, set watchdog
    bit 4."""
    import torch
    dev, dt = probs.device, probs.dtype
    if probs.dim() != 2:
        raise ValueError("probs must be [rows, vocab]")
    shape, code = probs.shape, _code(probs)
    N, V = shape
    rp = _matrix("probs", probs, shape, dt, code, dev)
    rq = None
    if draft_probs is not None:
        if parents is not None:
            raise ValueError("draft_probs go with chains only: parents must be None")
        rq = ctypes.byref(_matrix("draft_probs", draft_probs, shape, dt, code, dev))
    B, W = starts.numel() - 1, most + 1
    i32, i64, f32 = torch.int32, torch.int64, torch.float32
    if B < 0 or most < 0:
        raise ValueError("starts must hold a value more than there are sequences, most be >= 0")
    if new_tokens is None:
        new_tokens = torch.empty(B, W, dtype=i64, device=dev)
    if path is None:
        path = torch.empty(B, W, dtype=i32, device=dev)
    if lengths is None:
        lengths = torch.empty(B, dtype=i32, device=dev)
    _on(dev, "rarn_verify_drafts", library().rarn_verify_drafts,
        _indices("new_tokens", new_tokens, i64, B * W, dev),
        _indices("path", path, i32, B * W, dev),
        _indices("lengths", lengths, i32, B, dev), rp, rq, _indices("tokens", tokens, i64, N, dev),
        None if parents is None else _indices("parents", parents, i32, N, dev),
        _indices("starts", starts, i32, B + 1, dev), _indices("uniforms", uniforms, f32, N, dev),
        _indices("final_uniforms", final_uniforms, f32, B, dev), B, N, V, most)
    return new_tokens, path, lengths


def kv_cache_compact(cache: KVCache, page_table, context_lens, path, lengths) -> None:
    """The tokens of an accepted path moved together: token context_lens[b] +
    path[b, j] goes to context_lens[b] + j, j = 1 .. lengths[b] - 1, with its scales.
    path: [B, width] int32, rising along a row; lengths: [B] int32 (as
    verify_drafts returns them)."""
    import torch
    dev = cache.device
    table, stride, B, width = _page_table(page_table, dev)
    if path.dim() != 2 or path.shape[0] != B:
        raise ValueError(f"path must be [{B}, width]")
    W = path.shape[1]
    _on(dev, "rarn_kv_cache_compact", library().rarn_kv_cache_compact, cache._ref, table, stride,
        width, _indices("context_lens", context_lens, torch.int32, B, dev),
        _indices("path", path, torch.int32, B * W, dev),
        _indices("lengths", lengths, torch.int32, B, dev), B, W)


def launch_floor(grid: int, block: int, rows=None, row_bytes: int = 0) -> None:
    """The row kernels' launch floor on the current stream of ``rows``'s
    device (else the current device): ``grid`` CTAs of ``block`` threads that
    only prefetch one row each (``row_bytes`` bytes of ``rows`` per CTA),
    wait for the previous kernel and let the next launch.  A measurement aid."""
    import torch
    dev = rows.device if rows is not None else torch.device("cuda", torch.cuda.current_device())
    if rows is not None and rows.numel() * rows.element_size() < grid * row_bytes:
        raise ValueError("rows must hold grid * row_bytes bytes")
    with torch.cuda.device(dev):
        _check(library().rarn_launch_floor(rows.data_ptr() if rows is not None else None,
                                           row_bytes, grid, block, _stream(dev)),
               "rarn_launch_floor")


def _addr(x) -> int:
    """A device address: a tensor's data pointer, or an int as given."""
    return x.data_ptr() if hasattr(x, "data_ptr") else int(x)


def tp_rows(T: int, world_size: int, rank: int):
    """Rows [r0, r1) that ``rank`` of ``world_size`` owns in the tensor-parallel
    form."""
    r0, r1 = ctypes.c_int64(0), ctypes.c_int64(0)
    _check(library().rarn_tp_rows(T, world_size, rank, ctypes.byref(r0), ctypes.byref(r1)),
           "rarn_tp_rows")
    return r0.value, r1.value


def _tp_group(buffers, rank, signals):
    g = TpGroup()
    g.world_size = len(buffers)
    g.rank = rank
    if len(buffers) > TP_MAX_RANKS:
        raise ValueError(f"at most {TP_MAX_RANKS} ranks")
    for q, b in enumerate(buffers):
        g.buffers[q] = _addr(b)
    if signals is not None:
        if len(signals) != len(buffers):
            raise ValueError("one signal pad per rank")
        for q, sg in enumerate(signals):
            g.signals[q] = _addr(sg)
    return g


def tp_reduce_add_rms_norm(buffers, rank: int, residual, gamma, eps: float, T: int,
                           signals=None):
    """This rank's part of the tensor-parallel form: ``buffers`` lists every
    rank's [T, H] buffer (tensors or device addresses as this process sees
    them; partial in, y for all T rows out), ``residual`` this rank's rows
    [r1 - r0, H] (updated in place), ``gamma`` [H]; ``signals`` every rank's
    pad (TP_SIGNAL_BYTES each) for the in-kernel barrier between ranks, or
    None when the caller orders the ranks.  Runs on the current stream of
    residual's device."""
    import torch
    H = gamma.numel()
    dev = residual.device
    _check_tensor("gamma", gamma, residual.dtype, dev)
    r0, r1 = tp_rows(T, len(buffers), rank)
    if tuple(residual.shape) != (r1 - r0, H) or not residual.is_contiguous():
        raise ValueError(f"residual must be this rank's rows, [{r1 - r0}, {H}], contiguous")
    g = _tp_group(buffers, rank, signals)
    with torch.cuda.device(dev):
        _check(library().rarn_tp_reduce_add_rms_norm(
            ctypes.byref(g), residual.data_ptr(), gamma.data_ptr(), T, H, float(eps),
            _dtype_code(residual), _stream(dev)), "rarn_tp_reduce_add_rms_norm")


def tp_reduce_add_rms_norm_world(buffers, residuals, gamma, eps: float, T: int, signals=None):
    """Every rank's part in one launch on this device (all buffers, residual
    rows and pads on it): ``residuals[q]`` is rank q's rows of the residual."""
    import torch
    H = gamma.numel()
    N = len(buffers)
    dev = gamma.device
    if len(residuals) != N:
        raise ValueError("one residual block per rank")
    for q, r in enumerate(residuals):
        r0, r1 = tp_rows(T, N, q)
        _check_tensor(f"residuals[{q}]", r, gamma.dtype, dev)
        if tuple(r.shape) != (r1 - r0, H):
            raise ValueError(f"residuals[{q}] must be [{r1 - r0}, {H}]")
    g = _tp_group(buffers, 0, signals)
    rp = (ctypes.c_void_p * N)(*[r.data_ptr() for r in residuals])
    with torch.cuda.device(dev):
        _check(library().rarn_tp_reduce_add_rms_norm_world(
            ctypes.byref(g), ctypes.cast(rp, ctypes.c_void_p), gamma.data_ptr(), T, H,
            float(eps), _dtype_code(gamma), _stream(dev)), "rarn_tp_reduce_add_rms_norm_world")


def ipc_export(x) -> bytes:
    """A handle (IPC_HANDLE_BYTES bytes) through which another process can
    address the device memory at ``x`` (a tensor or a device address)."""
    buf = ctypes.create_string_buffer(IPC_HANDLE_BYTES)
    _check(library().rarn_ipc_export(_addr(x), buf), "rarn_ipc_export")
    return buf.raw


def ipc_import(handle: bytes) -> int:
    """The address at which this process reaches the memory another process
    exported as ``handle``."""
    if len(handle) != IPC_HANDLE_BYTES:
        raise ValueError(f"an IPC handle has {IPC_HANDLE_BYTES} bytes")
    p = ctypes.c_void_p(0)
    _check(library().rarn_ipc_import(handle, ctypes.byref(p)), "rarn_ipc_import")
    return int(p.value)


def ipc_close(ptr: int) -> None:
    """Release a mapping ipc_import opened."""
    _check(library().rarn_ipc_close(ptr), "rarn_ipc_close")


def set_tuning(name: str, value: int) -> None:
    """Set one planner override (``TUNING`` names it; -1 restores the
    planner's choice).  Raises RarnError for a value outside the knob's list."""
    _check(library().rarn_set_tuning(TUNING[name], int(value)), f"rarn_set_tuning({name})")


def get_tuning(name: str) -> int:
    v = ctypes.c_int64(0)
    _check(library().rarn_get_tuning(TUNING[name], ctypes.byref(v)), "rarn_get_tuning")
    return v.value


def reset_tuning() -> None:
    """Every planner override back to the planner's choice."""
    _check(library().rarn_reset_tuning(), "rarn_reset_tuning")


class tuning:
    """Context manager: ``with tuning(gemm_pair=0): ...`` sets the named
    knobs and restores their previous values on exit."""

    def __init__(self, **knobs):
        self.knobs = knobs
        self.saved = {}

    def __enter__(self):
        for k, v in self.knobs.items():
            self.saved[k] = get_tuning(k)
            set_tuning(k, v)
        return self

    def __exit__(self, *exc):
        for k, v in self.saved.items():
            set_tuning(k, v)
        return False


def set_pdl(enable: bool) -> None:
    """Programmatic dependent launch for every later launch (process-wide)."""
    _check(library().rarn_set_pdl(int(bool(enable))), "rarn_set_pdl")


def get_pdl() -> bool:
    return bool(library().rarn_get_pdl())


def get_path() -> str:
    code = library().rarn_get_path()
    return {v: k for k, v in PATHS.items()}[code]


def plan(op: str, T: int, H: int, R: int, dtype: str, vec_ok: bool = True,
         num_sms: int = 0, rdtype: str | None = None) -> str:
    """The kernel the current path setting would launch for a problem
    (``rdtype``: the residual's storage type, default ``dtype``)."""
    buf = ctypes.create_string_buffer(256)
    st = library().rarn_plan_ex(OP_CODES[op], T, H, R, DTYPE_CODES[dtype],
                                DTYPE_CODES[rdtype or dtype], int(vec_ok), num_sms, buf, 256)
    if st not in (0, 2):
        _check(st, "rarn_plan")
    return buf.value.decode()


def watchdog(clear: bool = True) -> int:
    """Read (and by default clear) the current device's watchdog word."""
    v = ctypes.c_uint32(0)
    _check(library().rarn_watchdog(ctypes.byref(v), int(clear)), "rarn_watchdog")
    return v.value
