"""ctypes binding of libsmd.so (include/smd.h), with the same names.

Argument marshalling only: every step of the decode runs in the library's
CUDA kernels. There is no CPU path; if the library cannot be built or loaded
the import of a decode function raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

from . import build as _build

SMD_OK = 0
SMD_ERR_NULL = -1
SMD_ERR_SHAPE = -2
SMD_ERR_ALIGN = -3
SMD_ERR_LAUNCH = -4
SMD_ERR_TIMEOUT = -5
SMD_ERR_PLAN = -6
SMD_ERR_DEVICE = -7
SMD_ERR_WORKSPACE = -8
SMD_ERR_GROUP = -9
SMD_ERR_INDEX = -10
SMD_ERR_PAGES = -11

SMD_KERNEL_AUTO = 0
SMD_KERNEL_MMA = 1
SMD_KERNEL_TC = 2
SMD_KERNEL_GROUP = 3
SMD_KERNEL_TC_GROUP = 4
SMD_KERNEL_TC_SPREAD = 5

SMD_QUERY_E4M3 = 0
SMD_QUERY_BF16 = 1


class SmdPlan(ctypes.Structure):
    """smd_plan_t."""
    _fields_ = [(name, ctypes.c_int32) for name in (
        "kernel", "split", "tiles", "window", "wait_budget_us", "inject_stall", "key_cap",
        "grid_x", "grid_y", "cluster_x", "threads", "smem_bytes")]

    def as_dict(self) -> dict:
        return {name: int(getattr(self, name)) for name, _ in self._fields_}


class SmdHostOpts(ctypes.Structure):
    """smd_host_opts_t."""
    _fields_ = [(name, ctypes.c_int32) for name in ("row_group", "bf16_query", "chunks",
                                                     "copies")]


class SmdOptions(ctypes.Structure):
    """smd_options_t."""
    _fields_ = [("row_group", ctypes.c_int32), ("query_type", ctypes.c_int32),
                ("library_scratch", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64),
                ("status", ctypes.c_void_p), ("force", ctypes.POINTER(SmdPlan))]


class SmdPagedCache(ctypes.Structure):
    """smd_paged_cache_t."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("bounds", ctypes.c_void_p),
                ("k_stride", ctypes.c_int64 * 3), ("v_stride", ctypes.c_int64 * 3),
                ("pages", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("map", ctypes.c_uint64 * 36)]


class SmdPagedCache4(ctypes.Structure):
    """smd_paged4_cache_t."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("k_exp", ctypes.c_void_p),
                ("v_exp", ctypes.c_void_p), ("bounds", ctypes.c_void_p),
                ("k_stride", ctypes.c_int64 * 3), ("v_stride", ctypes.c_int64 * 3),
                ("pages", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("map", ctypes.c_uint64 * 68)]


class SmdError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = int(status)
        super().__init__(f"{what}: {smd_status_str(status)} ({status})" if what
                         else f"{smd_status_str(status)} ({status})")


_lock = threading.Lock()
_lib = None

_DECODE_ARGS = [
    ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,   # q, kv_pool, N
    ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,   # indices, W, counts
    ctypes.c_int32, ctypes.c_int32,                     # B, H
    ctypes.c_float, ctypes.c_float, ctypes.c_float,     # sm_scale, q_scale, k_scale
    ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,  # out, lse, status
    ctypes.c_void_p,                                    # stream
]


def lib() -> ctypes.CDLL:
    """The loaded library (built in-tree on first use if missing or stale):
    libsmd.so, or its tracing variant when SMD_TRACE_BUILD=1 (per-phase
    timestamps of the kernels; same results)."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.build(trace=os.environ.get("SMD_TRACE_BUILD") == "1")
            so = ctypes.CDLL(path)
            so.smd_sparse_mla_decode.restype = ctypes.c_int
            so.smd_sparse_mla_decode.argtypes = _DECODE_ARGS
            ws_args = _DECODE_ARGS[:-1] + [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]
            so.smd_sparse_mla_decode_ws.restype = ctypes.c_int
            so.smd_sparse_mla_decode_ws.argtypes = ws_args
            so.smd_sparse_mla_decode_ex.restype = ctypes.c_int
            so.smd_sparse_mla_decode_ex.argtypes = ws_args + [ctypes.POINTER(SmdPlan)]
            so.smd_sparse_mla_decode_noalloc.restype = ctypes.c_int
            so.smd_sparse_mla_decode_noalloc.argtypes = _DECODE_ARGS
            grp_args = _DECODE_ARGS[:8] + [ctypes.c_int32] + _DECODE_ARGS[8:]
            so.smd_sparse_mla_decode_grouped.restype = ctypes.c_int
            so.smd_sparse_mla_decode_grouped.argtypes = grp_args
            grp_ws = grp_args[:-1] + [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]
            so.smd_sparse_mla_decode_grouped_ws.restype = ctypes.c_int
            so.smd_sparse_mla_decode_grouped_ws.argtypes = grp_ws
            so.smd_sparse_mla_decode_grouped_ex.restype = ctypes.c_int
            so.smd_sparse_mla_decode_grouped_ex.argtypes = grp_ws + [ctypes.POINTER(SmdPlan)]
            so.smd_workspace_bytes_grouped.restype = ctypes.c_int64
            so.smd_workspace_bytes_grouped.argtypes = [ctypes.c_int32] * 4
            bq_args = ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                        ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32,
                        ctypes.c_float, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                        ctypes.c_void_p, ctypes.c_void_p])
            so.smd_sparse_mla_decode_bf16q.restype = ctypes.c_int
            so.smd_sparse_mla_decode_bf16q.argtypes = bq_args
            bq_ws = bq_args[:-1] + [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]
            so.smd_sparse_mla_decode_bf16q_ws.restype = ctypes.c_int
            so.smd_sparse_mla_decode_bf16q_ws.argtypes = bq_ws
            so.smd_sparse_mla_decode_bf16q_ex.restype = ctypes.c_int
            so.smd_sparse_mla_decode_bf16q_ex.argtypes = bq_ws + [ctypes.POINTER(SmdPlan)]
            so.smd_workspace_bytes_bf16q.restype = ctypes.c_int64
            so.smd_workspace_bytes_bf16q.argtypes = [ctypes.c_int32] * 3
            so.smd_plan_bf16q.restype = ctypes.c_int
            so.smd_plan_bf16q.argtypes = [ctypes.c_int32] * 3 + [ctypes.c_int64,
                                                                 ctypes.POINTER(SmdPlan)]
            so.smd_topk_select.restype = ctypes.c_int
            tk_args = [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int32,
                       ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                       ctypes.c_void_p, ctypes.c_void_p]
            so.smd_topk_select.argtypes = tk_args
            so.smd_topk_select_ex.restype = ctypes.c_int
            so.smd_topk_select_ex.argtypes = tk_args + [ctypes.c_int32]
            so.smd_plan_grouped.restype = ctypes.c_int
            so.smd_plan_grouped.argtypes = [ctypes.c_int32] * 4 + [ctypes.c_int64,
                                                                   ctypes.POINTER(SmdPlan)]
            so.smd_workspace_bytes.restype = ctypes.c_int64
            so.smd_workspace_bytes.argtypes = [ctypes.c_int32] * 3
            so.smd_workspace_bytes_ex.restype = ctypes.c_int64
            so.smd_workspace_bytes_ex.argtypes = [ctypes.c_int32] * 3 + [ctypes.POINTER(SmdPlan)]
            so.smd_plan.restype = ctypes.c_int
            so.smd_plan.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                    ctypes.POINTER(SmdPlan)]
            so.smd_plan_ws.restype = ctypes.c_int
            so.smd_plan_ws.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                       ctypes.POINTER(SmdPlan)]
            so.smd_plan_host.restype = ctypes.c_int
            so.smd_plan_host.argtypes = [ctypes.c_int32] * 3 + [ctypes.POINTER(SmdHostOpts),
                                                                ctypes.POINTER(ctypes.c_int32)]
            so.smd_workspace_bytes_host.restype = ctypes.c_int64
            so.smd_workspace_bytes_host.argtypes = [ctypes.c_int32] * 3 + [
                ctypes.POINTER(SmdHostOpts)]
            so.smd_sparse_mla_decode_host.restype = ctypes.c_int
            so.smd_sparse_mla_decode_host.argtypes = _DECODE_ARGS[:-1] + [
                ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(SmdHostOpts), ctypes.c_void_p]
            so.smd_workspace_bytes_topk_host.restype = ctypes.c_int64
            so.smd_workspace_bytes_topk_host.argtypes = [ctypes.c_int32] * 3
            so.smd_topk_select_host.restype = ctypes.c_int
            so.smd_topk_select_host.argtypes = tk_args[:-1] + [ctypes.c_void_p, ctypes.c_int64,
                                                               ctypes.c_int32, ctypes.c_void_p]
            so.smd_validate_indices.restype = ctypes.c_int
            so.smd_validate_indices.argtypes = [ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                                ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p,
                                                ctypes.c_void_p]
            so.smd_fp8_mma_probe.restype = ctypes.c_int
            so.smd_fp8_mma_probe.argtypes = [ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                                             ctypes.POINTER(ctypes.c_int32)]
            so.smd_scale_log2.restype = ctypes.c_float
            so.smd_scale_log2.argtypes = [ctypes.c_float] * 3
            so.smd_status_str.restype = ctypes.c_char_p
            so.smd_decode.argtypes = _DECODE_ARGS[:-2] + [ctypes.POINTER(SmdOptions),
                                                           ctypes.c_void_p]
            so.smd_decode.restype = ctypes.c_int
            so.smd_decode_plan.argtypes = [ctypes.c_int32] * 3 + [ctypes.POINTER(SmdOptions),
                                                                  ctypes.POINTER(SmdPlan)]
            so.smd_decode_plan.restype = ctypes.c_int
            so.smd_decode_workspace_bytes.argtypes = [ctypes.c_int32] * 3 + [
                ctypes.POINTER(SmdOptions)]
            so.smd_decode_workspace_bytes.restype = ctypes.c_int64
            so.smd_trace_enabled.argtypes = []
            so.smd_trace_enabled.restype = ctypes.c_int
            so.smd_trace_read.argtypes = [ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32]
            so.smd_trace_read.restype = ctypes.c_int
            so.smd_trace_clear.argtypes = [ctypes.c_int32]
            so.smd_trace_clear.restype = ctypes.c_int
            ptr, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
            cache = ctypes.POINTER(SmdPagedCache)
            so.smd_paged_cache_init.argtypes = [cache]
            so.smd_paged_cache_init.restype = ctypes.c_int
            so.smd_block_tables.argtypes = [ptr, ptr, i32, ptr, i64, i32, ptr, i32, ptr, i32, i32,
                                            ptr, ptr, ptr, ptr, ptr, ptr, ptr]
            so.smd_block_tables.restype = ctypes.c_int
            so.smd_paged_append.argtypes = [cache, ptr, i64, ptr, i64, ptr, i32, ptr]
            so.smd_paged_append.restype = ctypes.c_int
            rows = [ptr, i64, cache, ptr, i64, i32, ptr, i32, i32, i32]
            so.smd_block_scores.argtypes = rows + [i32, i32, ptr, i64, ptr]
            so.smd_block_scores.restype = ctypes.c_int
            so.smd_paged_workspace_bytes.argtypes = [cache]
            so.smd_paged_workspace_bytes.restype = i64
            so.smd_paged_decode.argtypes = rows + [ctypes.c_float, ptr, ptr, i32, ptr, ptr, ptr,
                                                   ptr, i64, ptr]
            so.smd_paged_decode.restype = ctypes.c_int
            so.smd_paged_decode_ex.argtypes = so.smd_paged_decode.argtypes + [ctypes.POINTER(SmdPlan)]
            so.smd_paged_decode_ex.restype = ctypes.c_int
            cache4 = ctypes.POINTER(SmdPagedCache4)
            so.smd_paged4_cache_init.argtypes = [cache4]
            so.smd_paged4_cache_init.restype = ctypes.c_int
            so.smd_paged4_append.argtypes = [cache4, ptr, i64, ptr, i64, ptr, i32, ptr]
            so.smd_paged4_append.restype = ctypes.c_int
            so.smd_paged4_read.argtypes = [cache4, ptr, i32, ptr, i64, ptr, i64, ptr]
            so.smd_paged4_read.restype = ctypes.c_int
            so.smd_paged4_workspace_bytes.argtypes = [cache4]
            so.smd_paged4_workspace_bytes.restype = i64
            so.smd_paged4_decode.argtypes = [cache4 if a is cache else a
                                             for a in so.smd_paged_decode.argtypes]
            so.smd_paged4_decode.restype = ctypes.c_int
            so.smd_paged4_decode_ex.argtypes = so.smd_paged4_decode.argtypes + [
                ctypes.POINTER(SmdPlan)]
            so.smd_paged4_decode_ex.restype = ctypes.c_int
            so.smd_qk_norm_rope.argtypes = [ptr, i64, ptr, i64, i32, i32, i32, i32, ptr, i64, i32, ptr,
                                            i32, i32, ptr, ptr, ctypes.c_float, ptr, i64, ptr, i64,
                                            ptr]
            so.smd_qk_norm_rope.restype = ctypes.c_int
            so.smd_verify_drafts.argtypes = [ptr, i64, ptr, i64, ptr, ptr, ptr, i32, i32, i32, ptr,
                                             ptr, ptr, ptr]
            so.smd_verify_drafts.restype = ctypes.c_int
            so.smd_block_trim.argtypes = [ptr, ptr, i32, ptr, i64, i32, ptr, i32, ptr, i32, ptr, ptr,
                                          ptr]
            so.smd_block_trim.restype = ctypes.c_int
            so.smd_status_str.argtypes = [ctypes.c_int]
            so.smd_version.restype = ctypes.c_int
            so.smd_version.argtypes = []
            _lib = so
    return _lib


def library_path() -> str:
    return _build.TRACE_LIB if os.environ.get("SMD_TRACE_BUILD") == "1" else _build.LIB


# ---- raw C-ABI calls (pointers as integers) -----------------------------------

def smd_sparse_mla_decode(q, kv_pool, N, indices, W, counts, B, H, sm_scale, q_scale, k_scale,
                          out, lse, status, stream) -> int:
    return lib().smd_sparse_mla_decode(q, kv_pool, N, indices, W, counts, B, H, sm_scale,
                                       q_scale, k_scale, out, lse, status, stream)


def smd_sparse_mla_decode_ws(q, kv_pool, N, indices, W, counts, B, H, sm_scale, q_scale, k_scale,
                             out, lse, status, workspace, workspace_bytes, stream) -> int:
    return lib().smd_sparse_mla_decode_ws(q, kv_pool, N, indices, W, counts, B, H, sm_scale,
                                          q_scale, k_scale, out, lse, status, workspace,
                                          workspace_bytes, stream)


def smd_sparse_mla_decode_ex(q, kv_pool, N, indices, W, counts, B, H, sm_scale, q_scale, k_scale,
                             out, lse, status, workspace, workspace_bytes, stream,
                             force: SmdPlan | None) -> int:
    ref = ctypes.byref(force) if force is not None else None
    return lib().smd_sparse_mla_decode_ex(q, kv_pool, N, indices, W, counts, B, H, sm_scale,
                                          q_scale, k_scale, out, lse, status, workspace,
                                          workspace_bytes, stream, ref)


def smd_sparse_mla_decode_noalloc(q, kv_pool, N, indices, W, counts, B, H, sm_scale, q_scale,
                                  k_scale, out, lse, status, stream) -> int:
    """The decode for callers that cannot allocate device memory: split
    partials go through the library's own static scratch (see smd.h)."""
    return lib().smd_sparse_mla_decode_noalloc(q, kv_pool, N, indices, W, counts, B, H, sm_scale,
                                               q_scale, k_scale, out, lse, status, stream)


def smd_sparse_mla_decode_grouped(q, kv_pool, N, indices, W, counts, B, H, row_group, sm_scale,
                                  q_scale, k_scale, out, lse, status, stream) -> int:
    return lib().smd_sparse_mla_decode_grouped(q, kv_pool, N, indices, W, counts, B, H,
                                               row_group, sm_scale, q_scale, k_scale, out, lse,
                                               status, stream)


def smd_sparse_mla_decode_grouped_ws(q, kv_pool, N, indices, W, counts, B, H, row_group,
                                     sm_scale, q_scale, k_scale, out, lse, status, workspace,
                                     workspace_bytes, stream) -> int:
    return lib().smd_sparse_mla_decode_grouped_ws(q, kv_pool, N, indices, W, counts, B, H,
                                                  row_group, sm_scale, q_scale, k_scale, out,
                                                  lse, status, workspace, workspace_bytes, stream)


def smd_sparse_mla_decode_grouped_ex(q, kv_pool, N, indices, W, counts, B, H, row_group,
                                     sm_scale, q_scale, k_scale, out, lse, status, workspace,
                                     workspace_bytes, stream, force: SmdPlan | None) -> int:
    ref = ctypes.byref(force) if force is not None else None
    return lib().smd_sparse_mla_decode_grouped_ex(q, kv_pool, N, indices, W, counts, B, H,
                                                  row_group, sm_scale, q_scale, k_scale, out,
                                                  lse, status, workspace, workspace_bytes,
                                                  stream, ref)


def smd_workspace_bytes_grouped(B: int, H: int, W: int, row_group: int) -> int:
    return int(lib().smd_workspace_bytes_grouped(B, H, W, row_group))


def smd_plan_grouped(B: int, H: int, W: int, row_group: int, workspace_bytes: int = 0) -> SmdPlan:
    p = SmdPlan()
    rc = lib().smd_plan_grouped(B, H, W, row_group, int(workspace_bytes), ctypes.byref(p))
    if rc != SMD_OK:
        raise SmdError(rc, "smd_plan_grouped")
    return p


def smd_sparse_mla_decode_bf16q(q, kv_pool, N, indices, W, counts, B, H, sm_scale, k_scale,
                                out, lse, status, stream) -> int:
    return lib().smd_sparse_mla_decode_bf16q(q, kv_pool, N, indices, W, counts, B, H, sm_scale,
                                             k_scale, out, lse, status, stream)


def smd_sparse_mla_decode_bf16q_ws(q, kv_pool, N, indices, W, counts, B, H, sm_scale, k_scale,
                                   out, lse, status, workspace, workspace_bytes, stream) -> int:
    return lib().smd_sparse_mla_decode_bf16q_ws(q, kv_pool, N, indices, W, counts, B, H, sm_scale,
                                                k_scale, out, lse, status, workspace,
                                                workspace_bytes, stream)


def smd_sparse_mla_decode_bf16q_ex(q, kv_pool, N, indices, W, counts, B, H, sm_scale, k_scale,
                                   out, lse, status, workspace, workspace_bytes, stream,
                                   force: SmdPlan | None) -> int:
    ref = ctypes.byref(force) if force is not None else None
    return lib().smd_sparse_mla_decode_bf16q_ex(q, kv_pool, N, indices, W, counts, B, H, sm_scale,
                                                k_scale, out, lse, status, workspace,
                                                workspace_bytes, stream, ref)


def smd_workspace_bytes_bf16q(B: int, H: int, W: int) -> int:
    return int(lib().smd_workspace_bytes_bf16q(B, H, W))


def smd_plan_bf16q(B: int, H: int, W: int, workspace_bytes: int = 0) -> SmdPlan:
    p = SmdPlan()
    rc = lib().smd_plan_bf16q(B, H, W, int(workspace_bytes), ctypes.byref(p))
    if rc != SMD_OK:
        raise SmdError(rc, "smd_plan_bf16q")
    return p


def smd_topk_select(logits, row_stride, row_ends, B, L, K, indices, counts, status,
                    stream) -> int:
    return lib().smd_topk_select(logits, row_stride, row_ends, B, L, K, indices, counts, status,
                                 stream)


def smd_topk_select_ex(logits, row_stride, row_ends, B, L, K, indices, counts, status, stream,
                       cluster) -> int:
    return lib().smd_topk_select_ex(logits, row_stride, row_ends, B, L, K, indices, counts,
                                    status, stream, cluster)


def smd_workspace_bytes(B: int, H: int, W: int) -> int:
    return int(lib().smd_workspace_bytes(B, H, W))


def smd_workspace_bytes_ex(B: int, H: int, W: int, force: SmdPlan | dict | None = None) -> int:
    if isinstance(force, dict):
        p = SmdPlan()
        for k, v in force.items():
            setattr(p, k, int(v))
        force = p
    ref = ctypes.byref(force) if force is not None else None
    return int(lib().smd_workspace_bytes_ex(B, H, W, ref))


def smd_plan(B: int, H: int, W: int) -> SmdPlan:
    p = SmdPlan()
    rc = lib().smd_plan(B, H, W, ctypes.byref(p))
    if rc != SMD_OK:
        raise SmdError(rc, "smd_plan")
    return p


def smd_plan_ws(B: int, H: int, W: int) -> SmdPlan:
    p = SmdPlan()
    rc = lib().smd_plan_ws(B, H, W, ctypes.byref(p))
    if rc != SMD_OK:
        raise SmdError(rc, "smd_plan_ws")
    return p


def _host_opts(row_group: int = 1, bf16_query: bool = False, chunks: int = 0,
               copies: int = 0) -> SmdHostOpts:
    return SmdHostOpts(int(row_group), 1 if bf16_query else 0, int(chunks), int(copies))


def smd_plan_host(B: int, H: int, W: int, row_group: int = 1, bf16_query: bool = False,
                  chunks: int = 0) -> int:
    """The number of row chunks smd_sparse_mla_decode_host pipelines."""
    n = ctypes.c_int32(0)
    o = _host_opts(row_group, bf16_query, chunks)
    rc = lib().smd_plan_host(B, H, W, ctypes.byref(o), ctypes.byref(n))
    if rc != SMD_OK:
        raise SmdError(rc, "smd_plan_host")
    return int(n.value)


def smd_workspace_bytes_host(B: int, H: int, W: int, row_group: int = 1,
                             bf16_query: bool = False, chunks: int = 0) -> int:
    o = _host_opts(row_group, bf16_query, chunks)
    return int(lib().smd_workspace_bytes_host(B, H, W, ctypes.byref(o)))


def smd_sparse_mla_decode_host(q, kv_pool, N, indices, W, counts, B, H, sm_scale, q_scale,
                               k_scale, out, lse, status, workspace, workspace_bytes,
                               opts: SmdHostOpts | None, stream) -> int:
    ref = ctypes.byref(opts) if opts is not None else None
    return lib().smd_sparse_mla_decode_host(q, kv_pool, N, indices, W, counts, B, H, sm_scale,
                                            q_scale, k_scale, out, lse, status, workspace,
                                            workspace_bytes, ref, stream)


def smd_workspace_bytes_topk_host(B: int, L: int, K: int) -> int:
    return int(lib().smd_workspace_bytes_topk_host(B, L, K))


def smd_topk_select_host(logits, row_stride, row_ends, B, L, K, indices, counts, status,
                         workspace, workspace_bytes, copies, stream) -> int:
    return lib().smd_topk_select_host(logits, row_stride, row_ends, B, L, K, indices, counts,
                                      status, workspace, workspace_bytes, copies, stream)


def smd_validate_indices(indices, W, counts, B, N, status, stream) -> int:
    return lib().smd_validate_indices(indices, W, counts, B, N, status, stream)


def smd_fp8_mma_probe(iters: int, status, stream) -> int:
    """Launches the FP8 tensor-pipe rate probe; returns the CTAs launched."""
    n = ctypes.c_int32(0)
    rc = lib().smd_fp8_mma_probe(iters, status, stream, ctypes.byref(n))
    if rc != SMD_OK:
        raise SmdError(rc, "smd_fp8_mma_probe")
    return n.value


def _as_plan(force):
    if isinstance(force, dict):
        p = SmdPlan()
        for k, v in force.items():
            setattr(p, k, int(v))
        return p
    return force


def smd_options(row_group: int = 1, query_type: int = SMD_QUERY_E4M3, library_scratch: bool = False,
                workspace: int = 0, workspace_bytes: int = 0, status: int = 0,
                force: SmdPlan | dict | None = None, reserved: int = 0) -> SmdOptions:
    """An smd_options_t (pointers as integers). The forced plan, if any, is
    kept alive by the returned struct."""
    o = SmdOptions()
    o.row_group, o.query_type, o.library_scratch, o.reserved = (int(row_group), int(query_type),
                                                                int(bool(library_scratch)),
                                                                int(reserved))
    o.workspace, o.workspace_bytes, o.status = int(workspace) or None, int(workspace_bytes), \
        int(status) or None
    force = _as_plan(force)
    if force is not None:
        o._force = force
        o.force = ctypes.pointer(force)
    return o


def smd_decode(q, kv_pool, N, indices, W, counts, B, H, sm_scale, q_scale, k_scale, out, lse,
               options: SmdOptions | None, stream) -> int:
    ref = ctypes.byref(options) if options is not None else None
    return int(lib().smd_decode(q, kv_pool, N, indices, W, counts, B, H, sm_scale, q_scale, k_scale,
                                out, lse, ref, stream))


def smd_decode_plan(B: int, H: int, W: int, options: SmdOptions | None = None) -> SmdPlan:
    p = SmdPlan()
    ref = ctypes.byref(options) if options is not None else None
    rc = lib().smd_decode_plan(B, H, W, ref, ctypes.byref(p))
    if rc != SMD_OK:
        raise SmdError(rc, "smd_decode_plan")
    return p


def smd_decode_workspace_bytes(B: int, H: int, W: int, options: SmdOptions | None = None) -> int:
    ref = ctypes.byref(options) if options is not None else None
    return int(lib().smd_decode_workspace_bytes(B, H, W, ref))


def smd_trace_enabled() -> int:
    return int(lib().smd_trace_enabled())


def smd_trace_read(kernel: int, host, n: int) -> int:
    return int(lib().smd_trace_read(kernel, host, n))


def smd_trace_clear(kernel: int) -> int:
    return int(lib().smd_trace_clear(kernel))


def smd_scale_log2(sm_scale: float, q_scale: float, k_scale: float) -> float:
    return float(lib().smd_scale_log2(sm_scale, q_scale, k_scale))


def smd_status_str(status: int) -> str:
    return lib().smd_status_str(int(status)).decode()


def smd_version() -> int:
    return int(lib().smd_version())


# ---- torch-level marshalling ----------------------------------------------------

def _ptr(t) -> int:
    return 0 if t is None else int(t.data_ptr())


def _bytes_view(t, name: str):
    import torch
    if t.dtype == torch.float8_e4m3fn:
        t = t.view(torch.uint8)
    if t.dtype != torch.uint8:
        raise TypeError(f"{name}: expected uint8 / float8_e4m3fn, got {t.dtype}")
    return t


def sparse_mla_decode(q, kv_pool, indices, counts, sm_scale: float, q_scale: float,
                      k_scale: float, out=None, lse=None, status=None, stream=None,
                      plan: SmdPlan | dict | None = None, workspace=None, row_group: int = 1):
    """Decode on the GPU. q [B,H,576] and kv_pool [N,576] E4M3 (uint8 or
    float8_e4m3fn), indices [B,W] int32, counts [B] int32, all CUDA tensors.
    Returns (out [B,H,512] bfloat16, lse [B,H] float32). ``plan`` forces
    plan fields (smd_sparse_mla_decode_ex); ``status`` is an optional int32
    CUDA tensor that receives device-side errors; ``workspace`` an optional
    CUDA tensor for smd_sparse_mla_decode_ws (at least
    smd_workspace_bytes(B, H, W) bytes: the spread kernel's or the L2
    exchange of split partials); ``row_group`` > 1 calls
    smd_sparse_mla_decode_grouped (rows in groups sharing one index list)."""
    import torch

    q = _bytes_view(q, "q")
    kv_pool = _bytes_view(kv_pool, "kv_pool")
    for name, t in (("q", q), ("kv_pool", kv_pool), ("indices", indices), ("counts", counts)):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (the decode has no CPU path)")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if indices.dtype != torch.int32 or counts.dtype != torch.int32:
        raise TypeError("indices and counts must be int32")
    if q.dim() != 3 or q.shape[2] != 576 or kv_pool.dim() != 2 or kv_pool.shape[1] != 576:
        raise ValueError("q must be [B,H,576] and kv_pool [N,576]")
    B, H = int(q.shape[0]), int(q.shape[1])
    W = int(indices.shape[1]) if indices.dim() == 2 else 0
    if indices.dim() != 2 or indices.shape[0] < B or counts.shape[0] < B:
        raise ValueError("indices must be [>=B, W] and counts [>=B]")
    if out is None:
        out = torch.empty((B, H, 512), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    args = (_ptr(q), _ptr(kv_pool), int(kv_pool.shape[0]), _ptr(indices), W, _ptr(counts), B, H,
            float(sm_scale), float(q_scale), float(k_scale), _ptr(out), _ptr(lse), _ptr(status))
    ws = (_ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size())
    if workspace is not None and not workspace.is_cuda:
        raise ValueError("workspace must be a CUDA tensor")
    if isinstance(plan, dict):
        p = SmdPlan()
        for k, v in plan.items():
            setattr(p, k, int(v))
        plan = p
    if row_group != 1:
        g_args = args[:8] + (int(row_group),) + args[8:]
        if plan is not None:
            rc = smd_sparse_mla_decode_grouped_ex(*g_args, *ws, int(stream), plan)
        elif workspace is not None:
            rc = smd_sparse_mla_decode_grouped_ws(*g_args, *ws, int(stream))
        else:
            rc = smd_sparse_mla_decode_grouped(*g_args, int(stream))
        if rc != SMD_OK:
            raise SmdError(rc, "smd_sparse_mla_decode_grouped")
        return out, lse
    if plan is None and workspace is None:
        rc = smd_sparse_mla_decode(*args, int(stream))
    elif plan is None:
        rc = smd_sparse_mla_decode_ws(*args, *ws, int(stream))
    else:
        rc = smd_sparse_mla_decode_ex(*args, *ws, int(stream), plan)
    if rc != SMD_OK:
        raise SmdError(rc, "smd_sparse_mla_decode")
    return out, lse


def decode(q, kv_pool, indices, counts, sm_scale: float, q_scale: float, k_scale: float,
           out=None, lse=None, status=None, stream=None, plan: SmdPlan | dict | None = None,
           workspace=None, row_group: int = 1, library_scratch: bool = False):
    """Decode on the GPU through smd_decode (one call for every variant).
    q [B,H,576]: E4M3 (uint8 or float8_e4m3fn, with q_scale) or bfloat16 (the
    split query; q_scale is not used); kv_pool [N,576] E4M3, indices [B,W]
    int32, counts [B] int32, all CUDA tensors. ``row_group`` 2 or 4: rows in
    groups sharing one index list; ``workspace``, ``plan``, ``status`` as in
    sparse_mla_decode; ``library_scratch``: the no-alloc exchange. Returns
    (out [B,H,512] bfloat16, lse [B,H] float32)."""
    import torch

    bf16 = q.dtype == torch.bfloat16
    if not bf16:
        q = _bytes_view(q, "q")
    kv_pool = _bytes_view(kv_pool, "kv_pool")
    for name, t in (("q", q), ("kv_pool", kv_pool), ("indices", indices), ("counts", counts)):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (the decode has no CPU path)")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if indices.dtype != torch.int32 or counts.dtype != torch.int32:
        raise TypeError("indices and counts must be int32")
    if q.dim() != 3 or q.shape[2] != 576 or kv_pool.dim() != 2 or kv_pool.shape[1] != 576:
        raise ValueError("q must be [B,H,576] and kv_pool [N,576]")
    B, H = int(q.shape[0]), int(q.shape[1])
    if indices.dim() != 2 or indices.shape[0] < B or counts.shape[0] < B:
        raise ValueError("indices must be [>=B, W] and counts [>=B]")
    W = int(indices.shape[1])
    if workspace is not None and not workspace.is_cuda:
        raise ValueError("workspace must be a CUDA tensor")
    if out is None:
        out = torch.empty((B, H, 512), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    opts = smd_options(row_group=row_group, query_type=SMD_QUERY_BF16 if bf16 else SMD_QUERY_E4M3,
                       library_scratch=library_scratch, workspace=_ptr(workspace),
                       workspace_bytes=0 if workspace is None
                       else workspace.numel() * workspace.element_size(),
                       status=_ptr(status), force=plan)
    rc = smd_decode(_ptr(q), _ptr(kv_pool), int(kv_pool.shape[0]), _ptr(indices), W, _ptr(counts),
                    B, H, float(sm_scale), float(q_scale), float(k_scale), _ptr(out), _ptr(lse),
                    opts, int(stream))
    if rc != SMD_OK:
        raise SmdError(rc, "smd_decode")
    return out, lse


def sparse_mla_decode_bf16q(q, kv_pool, indices, counts, sm_scale: float, k_scale: float,
                            out=None, lse=None, status=None, stream=None,
                            plan: SmdPlan | dict | None = None, workspace=None):
    """Decode with a bfloat16 query q [B,H,576] (split into E4M3 hi + lo per
    (row, head) on the GPU: smd_sparse_mla_decode_bf16q). kv_pool [N,576] E4M3,
    indices [B,W] int32, counts [B] int32, all CUDA tensors. Returns
    (out [B,H,512] bfloat16, lse [B,H] float32)."""
    import torch

    kv_pool = _bytes_view(kv_pool, "kv_pool")
    if q.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise TypeError(f"q: expected bfloat16, got {q.dtype}")
    for name, t in (("q", q), ("kv_pool", kv_pool), ("indices", indices), ("counts", counts)):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (the decode has no CPU path)")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if indices.dtype != torch.int32 or counts.dtype != torch.int32:
        raise TypeError("indices and counts must be int32")
    if q.dim() != 3 or q.shape[2] != 576 or kv_pool.dim() != 2 or kv_pool.shape[1] != 576:
        raise ValueError("q must be [B,H,576] and kv_pool [N,576]")
    B, H = int(q.shape[0]), int(q.shape[1])
    if indices.dim() != 2 or indices.shape[0] < B or counts.shape[0] < B:
        raise ValueError("indices must be [>=B, W] and counts [>=B]")
    W = int(indices.shape[1])
    if out is None:
        out = torch.empty((B, H, 512), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    args = (_ptr(q), _ptr(kv_pool), int(kv_pool.shape[0]), _ptr(indices), W, _ptr(counts), B, H,
            float(sm_scale), float(k_scale), _ptr(out), _ptr(lse), _ptr(status))
    ws = (_ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size())
    if isinstance(plan, dict):
        p = SmdPlan()
        for k, v in plan.items():
            setattr(p, k, int(v))
        plan = p
    if plan is not None:
        rc = smd_sparse_mla_decode_bf16q_ex(*args, *ws, int(stream), plan)
    elif workspace is not None:
        rc = smd_sparse_mla_decode_bf16q_ws(*args, *ws, int(stream))
    else:
        rc = smd_sparse_mla_decode_bf16q(*args, int(stream))
    if rc != SMD_OK:
        raise SmdError(rc, "smd_sparse_mla_decode_bf16q")
    return out, lse


def sparse_mla_decode_host(q, kv_pool, indices, counts, sm_scale: float, q_scale: float,
                           k_scale: float, out=None, lse=None, status=None, stream=None,
                           workspace=None, row_group: int = 1, bf16_query: bool = False,
                           chunks: int = 0, copies: int = 0):
    """Decode with q, indices and counts in HOST memory and out / lse returned
    to host memory (smd_sparse_mla_decode_host); kv_pool stays a CUDA tensor.
    q [B,H,576] E4M3 (uint8 or float8_e4m3fn), or bfloat16 with bf16_query;
    indices [B,W] int32; counts [B] int32: contiguous CPU tensors, page-locked
    (``pin_memory()``) for the copies to overlap. ``workspace``: a CUDA tensor
    of at least smd_workspace_bytes_host bytes (allocated here if None).
    Returns (out [B,H,512] bfloat16, lse [B,H] float32) CPU tensors, complete
    once ``stream`` has reached the end of the call (synchronize before
    reading them)."""
    import torch

    if bf16_query:
        if q.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
            raise TypeError(f"q: expected bfloat16, got {q.dtype}")
    else:
        q = _bytes_view(q, "q")
    kv_pool = _bytes_view(kv_pool, "kv_pool")
    if not kv_pool.is_cuda:
        raise ValueError("kv_pool must be a CUDA tensor")
    for name, t in (("q", q), ("indices", indices), ("counts", counts)):
        if t.is_cuda:
            raise ValueError(f"{name} must be a CPU tensor (this call copies it to the GPU)")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if indices.dtype != torch.int32 or counts.dtype != torch.int32:
        raise TypeError("indices and counts must be int32")
    if q.dim() != 3 or q.shape[2] != 576 or kv_pool.dim() != 2 or kv_pool.shape[1] != 576:
        raise ValueError("q must be [B,H,576] and kv_pool [N,576]")
    B, H = int(q.shape[0]), int(q.shape[1])
    if indices.dim() != 2 or indices.shape[0] != B or counts.shape[0] != B:
        raise ValueError("indices must be [B, W] and counts [B]")
    W = int(indices.shape[1])
    if out is None:
        out = torch.empty((B, H, 512), dtype=torch.bfloat16).pin_memory()
    if lse is None:
        lse = torch.empty((B, H), dtype=torch.float32).pin_memory()
    for name, t in (("out", out), ("lse", lse)):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CPU tensor")
    opts = _host_opts(row_group, bf16_query, chunks, copies)
    if workspace is None:
        nb = smd_workspace_bytes_host(B, H, W, row_group, bf16_query, chunks)
        if nb < 0:
            raise SmdError(nb, "smd_workspace_bytes_host")
        workspace = torch.empty(max(nb, 16), dtype=torch.uint8, device=kv_pool.device)
    if stream is None:
        stream = torch.cuda.current_stream(kv_pool.device).cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    rc = smd_sparse_mla_decode_host(
        _ptr(q), _ptr(kv_pool), int(kv_pool.shape[0]), _ptr(indices), W, _ptr(counts), B, H,
        float(sm_scale), float(q_scale), float(k_scale), _ptr(out), _ptr(lse), _ptr(status),
        _ptr(workspace), workspace.numel() * workspace.element_size(), opts, int(stream))
    if rc != SMD_OK:
        raise SmdError(rc, "smd_sparse_mla_decode_host")
    return out, lse


def topk_select(logits, K: int, row_ends=None, indices=None, counts=None, stream=None,
                status=None, cluster: int = 0):
    """Top-k select on the GPU (smd_topk_select). logits: bfloat16 CUDA tensor
    [B, L] with unit column stride (a column slice of a wider tensor is fine;
    16-byte aligned rows are read fastest); row_ends: optional
    int32 [B]. Returns (indices int32 [B, K], counts int32 [B]), ready to be
    the decode's index list and counts."""
    import torch

    if logits.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise TypeError(f"logits: expected bfloat16, got {logits.dtype}")
    if not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor (the select has no CPU path)")
    if logits.dim() != 2 or logits.stride(1) != 1:
        raise ValueError("logits must be [B, L] with unit column stride")
    B, L = int(logits.shape[0]), int(logits.shape[1])
    stride = int(logits.stride(0)) if B > 1 else L
    if row_ends is not None and (row_ends.dtype != torch.int32 or not row_ends.is_cuda):
        raise TypeError("row_ends must be an int32 CUDA tensor")
    if indices is None:
        indices = torch.empty((B, K), dtype=torch.int32, device=logits.device)
    if counts is None:
        counts = torch.empty((B,), dtype=torch.int32, device=logits.device)
    if stream is None:
        stream = torch.cuda.current_stream(logits.device).cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    rc = smd_topk_select_ex(_ptr(logits), stride, _ptr(row_ends), B, L, int(K), _ptr(indices),
                            _ptr(counts), _ptr(status), int(stream), int(cluster))
    if rc != SMD_OK:
        raise SmdError(rc, "smd_topk_select")
    return indices, counts


def validate_indices(indices, counts, N: int, status=None, stream=None):
    """Range check of an index list on the GPU (smd_validate_indices): every
    valid entry (i < clamp(counts[b], 0, W)) of the int32 CUDA tensor
    indices [B, W] must lie in [0, N). Returns the int32 status tensor (one
    element, zeroed here unless given), which holds SMD_ERR_INDEX after the
    stream reaches the check if an entry lies outside."""
    import torch
    if indices.dim() != 2 or indices.dtype != torch.int32 or counts.dtype != torch.int32:
        raise ValueError("indices [B, W] and counts [B] must be int32")
    if not (indices.is_cuda and counts.is_cuda) or not indices.is_contiguous():
        raise ValueError("indices and counts must be contiguous CUDA tensors")
    B, W = indices.shape
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=indices.device)
    stream = torch.cuda.current_stream(indices.device) if stream is None else stream
    rc = smd_validate_indices(_ptr(indices), W, _ptr(counts), B, int(N), _ptr(status),
                              int(stream.cuda_stream))
    if rc != SMD_OK:
        raise SmdError(rc, "smd_validate_indices")
    return status


def topk_select_host(logits, K: int, row_ends=None, indices=None, counts=None, stream=None,
                     status=None, workspace=None, copies: int = 0, device=None):
    """Top-k select with host buffers (smd_topk_select_host): logits a bfloat16
    CPU tensor [B, L] with unit column stride, row_ends an optional int32 CPU
    tensor [B]; page-locked (``pin_memory()``) for the select to read them in
    place. Returns (indices int32 [B, K], counts int32 [B]) CPU tensors,
    complete once ``stream`` has reached the end of the call."""
    import torch

    if logits.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise TypeError(f"logits: expected bfloat16, got {logits.dtype}")
    if logits.is_cuda or logits.dim() != 2 or logits.stride(1) != 1:
        raise ValueError("logits must be a CPU tensor [B, L] with unit column stride")
    B, L = int(logits.shape[0]), int(logits.shape[1])
    stride = int(logits.stride(0)) if B > 1 else L
    if row_ends is not None and (row_ends.dtype != torch.int32 or row_ends.is_cuda):
        raise TypeError("row_ends must be an int32 CPU tensor")
    if indices is None:
        indices = torch.empty((B, K), dtype=torch.int32).pin_memory()
    if counts is None:
        counts = torch.empty((B,), dtype=torch.int32).pin_memory()
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    if workspace is None and copies:
        workspace = torch.empty(max(smd_workspace_bytes_topk_host(B, L, int(K)), 16),
                                dtype=torch.uint8, device=dev)
    if stream is None:
        stream = torch.cuda.current_stream(dev).cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = smd_topk_select_host(_ptr(logits), stride, _ptr(row_ends), B, L, int(K), _ptr(indices),
                              _ptr(counts), _ptr(status), _ptr(workspace), nbytes, int(copies),
                              int(stream))
    if rc == SMD_ERR_WORKSPACE and workspace is None:
        # the buffers could not be read in place: copy through a workspace
        workspace = torch.empty(max(smd_workspace_bytes_topk_host(B, L, int(K)), 16),
                                dtype=torch.uint8, device=dev)
        rc = smd_topk_select_host(_ptr(logits), stride, _ptr(row_ends), B, L, int(K),
                                  _ptr(indices), _ptr(counts), _ptr(status), _ptr(workspace),
                                  workspace.numel(), int(copies), int(stream))
    if rc != SMD_OK:
        raise SmdError(rc, "smd_topk_select_host")
    return indices, counts


# ---- the paged cache ------------------------------------------------------------------

class PagedCache:
    """A paged key/value cache in E4M3 (smd_paged_cache_t), over the caller's
    tensors, which it keeps alive.

    k, v: [pages, heads, page_size, head_dim] E4M3 (uint8 or float8_e4m3fn), any
    strides in 16-byte steps with contiguous columns (a token-major pool is
    passed as ``pool.transpose(1, 2)``); k_scale, v_scale: [pages, heads]
    float32; bounds: [pages, heads, 2, head_dim] bfloat16 or None. All on one GPU,
    where the calls on the cache run and every other tensor of theirs must be. A cache
    that only block_scores reads may leave k, v and the scales out (then
    ``page_size`` says how many tokens a page holds)."""

    def __init__(self, k=None, v=None, k_scale=None, v_scale=None, bounds=None, page_size=None):
        import torch

        c = SmdPagedCache()
        shape = None
        for name, t in (("k", k), ("v", v)):
            if t is None:
                continue
            t = _bytes_view(t, name)
            if t.dim() != 4 or t.stride(3) != 1:
                raise ValueError(f"{name} must be [pages, heads, page_size, head_dim] with "
                                 "contiguous columns")
            if shape is not None and tuple(t.shape) != shape:
                raise ValueError("k and v must have one shape")
            shape = tuple(t.shape)
            setattr(c, name, _ptr(t))
            setattr(c, name + "_stride", (ctypes.c_int64 * 3)(*t.stride()[:3]))
        if shape is None:
            if bounds is None or page_size is None:
                raise ValueError("a cache without k and v needs bounds and page_size")
            shape = (bounds.shape[0], bounds.shape[1], int(page_size), bounds.shape[3])
        elif page_size is not None and int(page_size) != shape[2]:
            raise ValueError(f"page_size {page_size} is not that of k and v ({shape[2]})")
        for name, t, want, dtype in (
                ("k_scale", k_scale, shape[:2], torch.float32),
                ("v_scale", v_scale, shape[:2], torch.float32),
                ("bounds", bounds, (shape[0], shape[1], 2, shape[3]), torch.bfloat16)):
            if t is None:
                continue
            if tuple(t.shape) != tuple(want) or t.dtype != dtype or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {want}")
            setattr(c, name, _ptr(t))
        self.device = _gpu(k if k is not None else v if v is not None else bounds, "the cache")
        for name, t in (("k", k), ("v", v), ("k_scale", k_scale), ("v_scale", v_scale),
                        ("bounds", bounds)):
            if t is not None and t.get_device() != self.device:
                raise ValueError(f"{name} must be on cuda:{self.device}")
        c.pages, c.heads, c.page_size, c.head_dim = (int(x) for x in shape)
        rc = lib().smd_paged_cache_init(ctypes.byref(c))
        if rc != SMD_OK:
            raise SmdError(rc, "smd_paged_cache_init")
        self.k, self.v, self.k_scale, self.v_scale, self.bounds = k, v, k_scale, v_scale, bounds
        self.pages, self.heads, self.page_size, self.head_dim = (int(x) for x in shape)
        self.c, self.ref = c, ctypes.byref(c)

    @classmethod
    def empty(cls, pages: int, heads: int, page_size: int, head_dim: int, bounds: bool = True,
              device="cuda"):
        """A cache of newly allocated tensors (zero scales: nothing written yet)."""
        import torch

        def codes():
            return torch.zeros((pages, heads, page_size, head_dim), dtype=torch.uint8, device=device)

        def scale():
            return torch.zeros((pages, heads), dtype=torch.float32, device=device)

        b = torch.zeros((pages, heads, 2, head_dim), dtype=torch.bfloat16, device=device) \
            if bounds else None
        return cls(codes(), codes(), scale(), scale(), b)


def _so() -> ctypes.CDLL:
    return _lib if _lib is not None else lib()  # no lock once it is loaded


_raw_stream = _cuda_device = None  # torch's, looked up once: an import costs a call 0.2 us


def _stream(stream, dev: int) -> int:
    if stream is None:
        global _raw_stream
        if _raw_stream is None:
            import torch
            _raw_stream = torch._C._cuda_getCurrentRawStream
        return _raw_stream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _gpu(t, name: str) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def _current_device() -> int:
    global _cuda_device
    if _cuda_device is None:
        import torch
        _cuda_device = torch._C._cuda_getDevice
    return _cuda_device()


def _entry(name: str, dev: int):
    """The library's call ``name``, made on GPU ``dev``: it launches on the current one."""
    call = getattr(_so(), name)
    if _current_device() == dev:
        return call
    import torch

    def there(*args):
        with torch.cuda.device(dev):
            return call(*args)
    return there


def _vector(t, name: str, dtype, dev: int, n: int | None = None):
    if t.get_device() != dev or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor on cuda:{dev}")
    if n is not None and t.numel() < n:
        raise ValueError(f"{name} must have at least {n} elements")


def _new(make, stream, shape, dtype, device):
    """A tensor made (torch.empty, torch.zeros) on the stream of the call that
    uses it, so that the allocator reuses its memory in that stream's order."""
    import torch
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=device)


def _output(t, name: str, dtype, n: int, like, stream):
    if t is None:
        import torch
        return _new(torch.empty, stream, n, dtype, like.device)
    _vector(t, name, dtype, like.get_device(), n)
    return t


def _table(table, R: int, dev: int):
    """Entries of a row that may be used, and from one row to the next."""
    import torch
    if table.get_device() == dev and table.dtype == torch.int32:
        shape, steps = table.shape, table.stride()
        if len(shape) == 2 and shape[0] >= R and steps[1] == 1:
            return shape[1], steps[0] if shape[0] > 1 else shape[1]
    raise ValueError(f"table must be an int32 tensor [>= {R}, width] on cuda:{dev} with contiguous rows")


def block_tables(lengths, new_tokens, table, ring, state, page_size: int, max_tokens: int | None = None,
                 new_lengths=None, new_state=None, starts=None, slots=None, positions=None,
                 status=None, stream=None):
    """Pages and slots of a step (smd_block_tables). lengths, new_tokens [R],
    ring [pages] int32, table [R, width] int32 (written in place where pages
    are given), state [2] int64, all CUDA tensors; a new_tokens below 0 ends
    the request. ``max_tokens``: the slots to make room for, if ``slots`` is not
    given. Returns (new_lengths [R], new_state [2], starts [R + 1], slots [T],
    positions [T]); the outputs may be given, and may not be the inputs."""
    import torch

    R, dev = lengths.numel(), _gpu(lengths, "lengths")
    _vector(lengths, "lengths", torch.int32, dev)
    _vector(new_tokens, "new_tokens", torch.int32, dev, R)
    _vector(ring, "ring", torch.int32, dev)
    _vector(state, "state", torch.int64, dev, 2)
    width, step = _table(table, R, dev)
    if slots is None:
        if max_tokens is None:
            raise ValueError("block_tables needs slots or max_tokens")
        slots = _new(torch.empty, stream, int(max_tokens), torch.int32, lengths.device)
    T = slots.numel()

    new_lengths = _output(new_lengths, "new_lengths", torch.int32, R, lengths, stream)
    new_state = _output(new_state, "new_state", torch.int64, 2, lengths, stream)
    starts = _output(starts, "starts", torch.int32, R + 1, lengths, stream)
    _vector(slots, "slots", torch.int32, dev)
    positions = _output(positions, "positions", torch.int32, T, lengths, stream)
    if new_lengths.data_ptr() == lengths.data_ptr() and R or new_state.data_ptr() == state.data_ptr():
        raise ValueError("new_lengths and new_state may not be lengths and state")
    if status is not None:
        _vector(status, "status", torch.int32, dev, 1)
    rc = _entry("smd_block_tables", dev)(
        lengths.data_ptr(), new_tokens.data_ptr(), R, table.data_ptr(), step, width,
        ring.data_ptr(), ring.numel(), state.data_ptr(), page_size, T,
        new_lengths.data_ptr(), new_state.data_ptr(), starts.data_ptr(), slots.data_ptr(),
        positions.data_ptr(), _ptr(status), _stream(stream, dev))
    if rc != SMD_OK:
        raise SmdError(rc, "smd_block_tables")
    return new_lengths, new_state, starts, slots, positions


def paged_append(cache: PagedCache, k, v, slots, stream=None) -> None:
    """Writes new keys and values into the cache (smd_paged_append). k, v
    [T, heads, head_dim] bfloat16 CUDA tensors whose tokens may lie apart
    (slices of a fused projection); slots [T] int32."""
    import torch

    dev = cache.device
    _vector(slots, "slots", torch.int32, dev)
    T, args = slots.numel(), (cache.ref,)
    for name, t in (("k", k), ("v", v)):
        if t.get_device() != dev or t.dtype != torch.bfloat16 or t.shape != (
                T, cache.heads, cache.head_dim):
            raise ValueError(f"{name} must be a bfloat16 tensor [{T}, {cache.heads}, "
                             f"{cache.head_dim}] on cuda:{dev}")
        steps = t.stride()
        if steps[2] != 1 or (cache.heads > 1 and steps[1] != cache.head_dim):
            raise ValueError(f"{name}: a token's heads must be contiguous")
        args += (t.data_ptr(), steps[0] if T > 1 else cache.heads * cache.head_dim)
    rc = _entry("smd_paged_append", dev)(*args, slots.data_ptr(), T, _stream(stream, dev))
    if rc != SMD_OK:
        raise SmdError(rc, "smd_paged_append")


def _paged_rows(q, cache, table, lengths, row_group):
    import torch

    R, dev = lengths.numel(), cache.device
    _vector(lengths, "lengths", torch.int32, dev)
    shape = q.shape
    if q.get_device() != dev or q.dtype != torch.bfloat16 or len(shape) != 3 \
            or shape[0] != R * row_group or shape[2] != cache.head_dim:
        raise ValueError(f"q must be a bfloat16 tensor [{R} * {row_group}, Hq, {cache.head_dim}] on "
                         f"cuda:{dev}")
    B, Hq, D = shape
    steps = q.stride()
    if steps[2] != 1 or (Hq > 1 and steps[1] != D):
        raise ValueError("q: a row's heads must be contiguous")
    q_stride = steps[0] if B > 1 else Hq * D
    width, step = _table(table, R, dev)
    return (q.data_ptr(), q_stride, cache.ref, table.data_ptr(), step, width, lengths.data_ptr(), R,
            row_group, Hq)


def block_scores(q, cache: PagedCache | PagedCache4, table, lengths, row_group: int = 1, keep_first: int = 0,
                 keep_last: int = 0, out=None, stream=None):
    """The score of each page for each row and kv head (smd_block_scores): an
    upper bound of q . k over the page's keys as they were appended (rounding to the cache's
    bits can lift a stored one above its page's bounds), the largest over the kv head's
    query heads. q [R * row_group, Hq, head_dim] bfloat16, table [R, width] and
    lengths [R] int32. Returns bfloat16 [R * row_group, heads, width], NaN past
    the pages a row sees; ``scores.flatten(0, 1)`` goes to topk_select."""
    import torch

    if isinstance(cache, PagedCache4):
        if cache.of_bounds is None:
            raise ValueError("the cache has no bounds")
        cache = cache.of_bounds
    args, dev = _paged_rows(q, cache, table, lengths, row_group), cache.device
    B, heads, width = q.shape[0], cache.heads, table.shape[1]
    if out is None:  # rows of a multiple of 8 scores: topk_select reads them in 16-byte pieces
        stride = (width + 7) // 8 * 8
        out = _new(torch.empty, stream, (B, heads, stride), torch.bfloat16, q.device)[:, :, :width]
    else:
        if out.get_device() != dev or out.dtype != torch.bfloat16 or out.shape != (B, heads, width) \
                or out.stride(2) != 1 \
                or (B > 1 and heads > 1 and out.stride(0) != heads * out.stride(1)):
            raise ValueError(f"out must be a bfloat16 tensor [{B}, {heads}, {width}] on cuda:{dev} "
                             "with evenly spaced rows")
        stride = out.stride(1) if heads > 1 else out.stride(0) if B > 1 else width
    rc = _entry("smd_block_scores", dev)(*args, keep_first, keep_last, out.data_ptr(), stride,
                                         _stream(stream, dev))
    if rc != SMD_OK:
        raise SmdError(rc, "smd_block_scores")
    return out


def paged_workspace_bytes(cache: PagedCache) -> int:
    """Bytes of workspace paged_decode needs for this cache, whatever the batch."""
    n = int(_entry("smd_paged_workspace_bytes", cache.device)(cache.ref))
    if n < 0:
        raise SmdError(n, "smd_paged_workspace_bytes")
    return n


def paged_decode(q, cache: PagedCache, table, lengths, sm_scale: float, row_group: int = 1,
                 block_lists=None, block_counts=None, out=None, lse=None, status=None,
                 workspace=None, stream=None, plan: SmdPlan | dict | None = None):
    """Attention over the cache (smd_paged_decode). q [R * row_group, Hq,
    head_dim] bfloat16 (rows may lie apart), table [R, width] and lengths [R]
    int32; block_lists [R * row_group, heads, K] int32: the pages of its request
    that each row and kv head attends (topk_select's output on block_scores),
    the first block_counts [R * row_group, heads] of them; None: all of its
    tokens. ``workspace``: a CUDA tensor of paged_workspace_bytes(cache) bytes,
    zeroed once before its first use (allocated here if None). ``status`` is an optional int32
    CUDA tensor: without one, a wait that runs out shows in NaN rows only. ``plan`` sets the
    testing hooks (smd_paged_decode_ex). Returns (out [R * row_group, Hq, head_dim] bfloat16,
    lse [R * row_group, Hq] float32)."""
    return _decode_call("smd_paged_decode", paged_workspace_bytes, q, cache, table, lengths, sm_scale,
                        row_group, block_lists, block_counts, out, lse, status, workspace, stream, plan)


def _decode_call(name, workspace_bytes, q, cache, table, lengths, sm_scale, row_group, block_lists,
                 block_counts, out, lse, status, workspace, stream, plan):
    """The decode ``name`` of a paged cache, whatever its bits."""
    import torch

    args, dev = _paged_rows(q, cache, table, lengths, row_group), cache.device
    B, Hq = q.shape[0], q.shape[1]
    K = 0
    if block_lists is not None:
        _vector(block_lists, "block_lists", torch.int32, dev)
        if block_lists.dim() != 3 or tuple(block_lists.shape[:2]) != (B, cache.heads):
            raise ValueError(f"block_lists must be [{B}, {cache.heads}, K]")
        K = block_lists.shape[2]
        if block_counts is not None:
            _vector(block_counts, "block_counts", torch.int32, dev, B * cache.heads)
    elif block_counts is not None:
        raise ValueError("block_counts without block_lists")
    if out is None:
        out = _new(torch.empty, stream, (B, Hq, cache.head_dim), torch.bfloat16, q.device)
    else:
        if out.shape != (B, Hq, cache.head_dim):
            raise ValueError(f"out must be [{B}, {Hq}, {cache.head_dim}]")
        _vector(out, "out", torch.bfloat16, dev)
    if lse is None:
        lse = _new(torch.empty, stream, (B, Hq), torch.float32, q.device)
    else:
        _vector(lse, "lse", torch.float32, dev, B * Hq)
    if workspace is None:
        workspace = _new(torch.zeros, stream, workspace_bytes(cache), torch.uint8, q.device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    if status is not None:
        _vector(status, "status", torch.int32, dev, 1)
    args += (sm_scale, _ptr(block_lists) if K or block_lists is None else workspace.data_ptr(),
             _ptr(block_counts), K, out.data_ptr(), lse.data_ptr(),
             _ptr(status), workspace.data_ptr(),
             workspace.numel() * workspace.element_size(), _stream(stream, dev))
    if plan is None:
        rc = _entry(name, dev)(*args)
    else:
        rc = _entry(name + "_ex", dev)(*args, ctypes.byref(_as_plan(plan)))
    if rc != SMD_OK:
        raise SmdError(rc, name)
    return out, lse


# ---- the paged cache in 4 bits, and the step around it -------------------------------------

class PagedCache4:
    """A paged key/value cache in E2M1 with an E4M3 scale for each token, head and
    block of 16 columns (smd_paged4_cache_t), over the caller's tensors, which it keeps
    alive.

    k, v: [pages, heads, page_size, head_dim / 2] uint8 (two codes a byte, the even
    column in the low bits), any strides in 16-byte steps with contiguous bytes (a
    token-major pool is passed as ``pool.transpose(1, 2)``); k_scales, v_scales: [pages,
    heads, page_size, head_dim / 16] E4M3 (uint8 or float8_e4m3fn), contiguous; k_exp,
    v_exp: [heads] int32 exponents of the heads' powers of two, or None (zeros); bounds:
    [pages, heads, 2, head_dim] bfloat16 or None. All on one GPU. block_scores takes
    such a cache too, if it has bounds."""

    def __init__(self, k, v, k_scales, v_scales, k_exp=None, v_exp=None, bounds=None):
        import torch

        c = SmdPagedCache4()
        shape = None
        for name, t in (("k", k), ("v", v)):
            if t.dtype != torch.uint8 or t.dim() != 4 or t.stride(3) != 1:
                raise ValueError(f"{name} must be uint8 [pages, heads, page_size, head_dim / 2] with "
                                 "contiguous bytes")
            if shape is not None and tuple(t.shape) != shape:
                raise ValueError("k and v must have one shape")
            shape = tuple(t.shape)
            setattr(c, name, _ptr(t))
            setattr(c, name + "_stride", (ctypes.c_int64 * 3)(*t.stride()[:3]))
        pages, heads, page_size, D = *shape[:3], 2 * shape[3]
        codes8 = (torch.uint8, torch.float8_e4m3fn)
        for name, t, want, dtypes in (
                ("k_scales", k_scales, (pages, heads, page_size, D // 16), codes8),
                ("v_scales", v_scales, (pages, heads, page_size, D // 16), codes8),
                ("k_exp", k_exp, (heads,), (torch.int32,)),
                ("v_exp", v_exp, (heads,), (torch.int32,)),
                ("bounds", bounds, (pages, heads, 2, D), (torch.bfloat16,))):
            if t is None and name[1:] != "_scales":
                continue
            if t is None or tuple(t.shape) != want or t.dtype not in dtypes or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {dtypes[0]} tensor of shape {want}")
            setattr(c, name, _ptr(t))
        self.device = _gpu(k, "the cache")
        for name, t in (("v", v), ("k_scales", k_scales), ("v_scales", v_scales), ("k_exp", k_exp),
                        ("v_exp", v_exp), ("bounds", bounds)):
            if t is not None and t.get_device() != self.device:
                raise ValueError(f"{name} must be on cuda:{self.device}")
        c.pages, c.heads, c.page_size, c.head_dim = pages, heads, page_size, D
        rc = lib().smd_paged4_cache_init(ctypes.byref(c))
        if rc != SMD_OK:
            raise SmdError(rc, "smd_paged4_cache_init")
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.k_exp, self.v_exp, self.bounds = k_exp, v_exp, bounds
        self.pages, self.heads, self.page_size, self.head_dim = pages, heads, page_size, D
        self.c, self.ref = c, ctypes.byref(c)
        # What block_scores reads: the bounds.
        self.of_bounds = PagedCache(bounds=bounds, page_size=page_size) if bounds is not None else None

    @classmethod
    def empty(cls, pages: int, heads: int, page_size: int, head_dim: int, bounds: bool = True,
              k_exp=None, v_exp=None, device="cuda"):
        """A cache of newly allocated tensors (zeros: nothing written yet)."""
        import torch

        def zeros(*shape, dtype=torch.uint8):
            return torch.zeros(shape, dtype=dtype, device=device)

        codes, scales = (pages, heads, page_size, head_dim // 2), (pages, heads, page_size, head_dim // 16)
        b = zeros(pages, heads, 2, head_dim, dtype=torch.bfloat16) if bounds else None
        return cls(zeros(*codes), zeros(*codes), zeros(*scales), zeros(*scales), k_exp, v_exp, b)


def _token_rows(t, name: str, shape: tuple, bfloat16, dev: int):
    """Pointer and token stride of bfloat16 [T, heads, D] whose tokens may lie apart."""
    if t.get_device() != dev or t.dtype != bfloat16 or t.shape != shape:
        raise ValueError(f"{name} must be a bfloat16 tensor {list(shape)} on cuda:{dev}")
    token, head, column = t.stride()
    T, heads, D = shape
    if column != 1 or (heads > 1 and head != D):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    return t.data_ptr(), token if T > 1 else heads * D


def paged4_append(cache: PagedCache4, k, v, slots, stream=None) -> None:
    """Writes new keys and values into the cache (smd_paged4_append). k, v
    [T, heads, head_dim] bfloat16 CUDA tensors whose tokens may lie apart
    (slices of a fused projection); slots [T] int32."""
    import torch

    dev = cache.device
    _vector(slots, "slots", torch.int32, dev)
    T, bfloat16 = slots.numel(), torch.bfloat16
    shape = (T, cache.heads, cache.head_dim)
    rc = _entry("smd_paged4_append", dev)(
        cache.ref, *_token_rows(k, "k", shape, bfloat16, dev), *_token_rows(v, "v", shape, bfloat16, dev),
        slots.data_ptr(), T, _stream(stream, dev))
    if rc != SMD_OK:
        raise SmdError(rc, "smd_paged4_append")


def paged4_read(cache: PagedCache4, slots, k=None, v=None, stream=None):
    """The keys and values of slots [T] int32 as bfloat16 [T, heads, head_dim] each
    (smd_paged4_read), into ``k`` and ``v`` if given (whose tokens may lie apart). Rows of
    slots outside the pool are left as they are. Returns (k, v)."""
    import torch

    dev = cache.device
    _vector(slots, "slots", torch.int32, dev)
    T, bfloat16 = slots.numel(), torch.bfloat16
    shape = (T, cache.heads, cache.head_dim)
    if k is None:
        k = _new(torch.zeros, stream, shape, bfloat16, slots.device)
    if v is None:
        v = _new(torch.zeros, stream, shape, bfloat16, slots.device)
    rc = _entry("smd_paged4_read", dev)(
        cache.ref, slots.data_ptr(), T, *_token_rows(k, "k", shape, bfloat16, dev),
        *_token_rows(v, "v", shape, bfloat16, dev), _stream(stream, dev))
    if rc != SMD_OK:
        raise SmdError(rc, "smd_paged4_read")
    return k, v


def paged4_workspace_bytes(cache: PagedCache4) -> int:
    """Bytes of workspace paged4_decode needs for this cache, whatever the batch."""
    n = int(_entry("smd_paged4_workspace_bytes", cache.device)(cache.ref))
    if n < 0:
        raise SmdError(n, "smd_paged4_workspace_bytes")
    return n


def paged4_decode(q, cache: PagedCache4, table, lengths, sm_scale: float, row_group: int = 1,
                  block_lists=None, block_counts=None, out=None, lse=None, status=None,
                  workspace=None, stream=None, plan: SmdPlan | dict | None = None):
    """Attention over the cache (smd_paged4_decode); the arguments and results are
    paged_decode's, the workspace is of paged4_workspace_bytes(cache) bytes."""
    return _decode_call("smd_paged4_decode", paged4_workspace_bytes, q, cache, table, lengths, sm_scale,
                        row_group, block_lists, block_counts, out, lse, status, workspace, stream, plan)


def qk_norm_rope(q, k, positions, freqs, q_weight=None, k_weight=None, eps: float = 1e-6,
                 interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """The norm of each query and key head and the position rotation, in one pass
    (smd_qk_norm_rope). q [T, Hq, head_dim] and k [T, Hk, head_dim] (or None) bfloat16 CUDA
    tensors whose tokens may lie apart; positions [T] or [axes, T] int32; freqs [rot / 2] or
    [axes, rot / 2] float32, radians a position, 0 where a pair does not turn with an axis; both
    None: no rotation. q_weight, k_weight [head_dim] bfloat16 or None (no norm). q_out, k_out:
    outputs, which may be q and k themselves; new tensors if None. Returns (q_out, k_out);
    tokens whose position on the first axis is negative are left as they are (zeros in new
    tensors)."""
    import torch

    dev = _gpu(q, "q")
    if q.dim() != 3:
        raise ValueError("q must be [T, Hq, head_dim]")
    bfloat16 = torch.bfloat16
    q_shape = tuple(q.shape)
    T, Hq, D = q_shape
    if k is not None:
        Hk = k.shape[1]
        k_shape = (T, Hk, D)
        k_args = _token_rows(k, "k", k_shape, bfloat16, dev)
    elif k_out is None:
        Hk, k_args = 0, (0, 0)
    else:
        raise ValueError("k_out without k")
    if (positions is None) != (freqs is None):
        raise ValueError("positions and freqs go together")
    axes, rot, pos_ptr, pos_step, f_ptr = 1, 0, 0, 0, 0
    if positions is not None:
        steps, shape = positions.stride(), positions.shape
        if positions.get_device() != dev or positions.dtype != torch.int32 or len(shape) not in (1, 2) \
                or shape[-1] != T or (T > 1 and steps[-1] != 1):
            raise ValueError(f"positions must be an int32 tensor [{T}] or [axes, {T}] on cuda:{dev} with "
                             "contiguous rows")
        pos_ptr, pos_step = positions.data_ptr(), T
        if len(shape) == 2:
            axes = shape[0]
            if axes > 1:
                pos_step = steps[0]
        _vector(freqs, "freqs", torch.float32, dev)
        f_shape = freqs.shape
        if len(f_shape) != len(shape) or (len(f_shape) == 2 and f_shape[0] != axes):
            raise ValueError("freqs must be [rot / 2] or [axes, rot / 2], as positions")
        rot, f_ptr = 2 * f_shape[-1], freqs.data_ptr()
    for w in (q_weight, k_weight):
        if w is not None:
            _vector(w, "q_weight" if w is q_weight else "k_weight", bfloat16, dev)
            if w.numel() != D:
                raise ValueError(f"{'q_weight' if w is q_weight else 'k_weight'} must have {D} elements")
    if q_out is None:
        q_out = _new(torch.zeros, stream, q_shape, bfloat16, q.device)
    if k is not None and k_out is None:
        k_out = _new(torch.zeros, stream, k_shape, bfloat16, q.device)
    args = (*_token_rows(q, "q", q_shape, bfloat16, dev), *k_args)
    out = (*_token_rows(q_out, "q_out", q_shape, bfloat16, dev),
           *(_token_rows(k_out, "k_out", k_shape, bfloat16, dev) if k is not None else k_args))
    rc = _entry("smd_qk_norm_rope", dev)(*args, T, Hq, Hk, D, pos_ptr, pos_step, axes, f_ptr, rot,
                                         int(bool(interleaved)), _ptr(q_weight), _ptr(k_weight), eps,
                                         *out, _stream(stream, dev))
    if rc != SMD_OK:
        raise SmdError(rc, "smd_qk_norm_rope")
    return q_out, k_out


def _probability_rows(t, name: str, shape: tuple, float32, dev: int):
    """Pointer and row stride of float32 [R, n, V] whose rows are evenly spaced."""
    if t.get_device() != dev or t.dtype != float32 or t.shape != shape:
        raise ValueError(f"{name} must be a float32 tensor {list(shape)} on cuda:{dev}")
    (R, n, V), (request, row, column) = shape, t.stride()
    if V > 1 and column != 1 or (R > 1 and n > 1 and request != n * row):
        raise ValueError(f"{name}: rows must be contiguous and evenly spaced")
    return t.data_ptr(), row if n > 1 else request if R > 1 else V


def verify_drafts(target, tokens, accept, sample, draft=None, out_tokens=None, accepted=None,
                  rejected=None, stream=None):
    """Which drafted tokens stay, and the token after them (smd_verify_drafts). target
    [R, G, V] float32: the target's probabilities after each of 0 .. G - 1 drafted tokens; tokens
    [R, G - 1] int32: the drafted ones (one outside the vocabulary ends a request's drafts); accept
    [R, G - 1] and sample [R] float32: random numbers from [0, 1); draft [R, G - 1, V] float32: what the
    drafted tokens were drawn from, or None (each was the only choice). Returns (out_tokens [R, G]: the
    tokens that stay, the one drawn after them, then -1; accepted [R]; rejected [R]: G - 1 - accepted, which
    block_trim takes off requests that were granted G slots; of n < G granted ones it is n - 1 - accepted, and
    nothing of none, as after a refusal of block_tables), int32."""
    import torch

    dev = _gpu(target, "target")
    if target.dim() != 3:
        raise ValueError("target must be [R, G, V]")
    shape, float32 = tuple(target.shape), torch.float32
    R, G, V = shape
    args = _probability_rows(target, "target", shape, float32, dev)
    _vector(sample, "sample", float32, dev, R)
    _vector(tokens, "tokens", torch.int32, dev, R * (G - 1))
    _vector(accept, "accept", float32, dev, R * (G - 1))
    draft_args = (0, 0)
    if draft is not None:
        draft_args = _probability_rows(draft, "draft", (R, G - 1, V), float32, dev)
    if out_tokens is None:
        out_tokens = _new(torch.empty, stream, (R, G), torch.int32, target.device)
    else:
        _vector(out_tokens, "out_tokens", torch.int32, dev, R * G)
    accepted = _output(accepted, "accepted", torch.int32, R, target, stream)
    rejected = _output(rejected, "rejected", torch.int32, R, target, stream)
    rc = _entry("smd_verify_drafts", dev)(*args, *draft_args, tokens.data_ptr(), accept.data_ptr(),
                                          sample.data_ptr(), R, G, V, out_tokens.data_ptr(),
                                          accepted.data_ptr(), rejected.data_ptr(), _stream(stream, dev))
    if rc != SMD_OK:
        raise SmdError(rc, "smd_verify_drafts")
    return out_tokens, accepted, rejected


def block_trim(lengths, drop, table, ring, state, page_size: int, new_lengths=None, new_state=None,
               stream=None):
    """Takes drop [R] int32 tokens off the end of requests (smd_block_trim): their pages
    past the new lengths go back to the ring. lengths, table, ring and state as in block_tables. Returns
    (new_lengths [R], new_state [2]), which may be given and may not be the inputs."""
    import torch

    R, dev = lengths.numel(), _gpu(lengths, "lengths")
    _vector(lengths, "lengths", torch.int32, dev)
    _vector(drop, "drop", torch.int32, dev, R)
    _vector(ring, "ring", torch.int32, dev)
    _vector(state, "state", torch.int64, dev, 2)
    width, step = _table(table, R, dev)
    new_lengths = _output(new_lengths, "new_lengths", torch.int32, R, lengths, stream)
    new_state = _output(new_state, "new_state", torch.int64, 2, lengths, stream)
    if new_lengths.data_ptr() == lengths.data_ptr() and R or new_state.data_ptr() == state.data_ptr():
        raise ValueError("new_lengths and new_state may not be lengths and state")
    rc = _entry("smd_block_trim", dev)(
        lengths.data_ptr(), drop.data_ptr(), R, table.data_ptr(), step, width, ring.data_ptr(),
        ring.numel(), state.data_ptr(), page_size, new_lengths.data_ptr(), new_state.data_ptr(),
        _stream(stream, dev))
    if rc != SMD_OK:
        raise SmdError(rc, "smd_block_trim")
    return new_lengths, new_state
