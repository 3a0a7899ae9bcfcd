"""Sparse MLA decode over an FP8 (E4M3) latent KV cache, for GB300 (sm_103a).

Beside it, a paged grouped-query cache in FP8 with a scale for each page and
head: its tables, its writes, page scores and attention; the same in 4 bits (E2M1
with block scales), and what a step around it needs: norm and rotation of queries
and keys, the verification of drafted tokens, the pages of rejected ones.

The calls run in libsmd.so (hand-written CUDA, C ABI in include/smd.h);
``binding`` is its ctypes wrapper. ``inputs`` holds the seeded synthetic
workloads. Submodules load lazily so that importing ``inputs`` does not need
the CUDA library.
"""
import importlib

__all__ = ["binding", "inputs", "build", "sparse_mla_decode", "smd_plan", "PagedCache",
           "block_tables", "paged_append", "block_scores", "paged_decode", "PagedCache4",
           "qk_norm_rope", "paged4_append", "paged4_read", "paged4_decode", "verify_drafts",
           "block_trim"]


def __getattr__(name):
    if name in ("binding", "inputs", "build"):
        return importlib.import_module(f".{name}", __name__)
    if name in ("sparse_mla_decode", "smd_plan", "smd_sparse_mla_decode",
                "smd_sparse_mla_decode_ex", "smd_scale_log2", "smd_status_str", "SmdPlan",
                "SmdError", "PagedCache", "block_tables", "paged_append", "block_scores",
                "paged_decode", "paged_workspace_bytes", "PagedCache4", "qk_norm_rope",
                "paged4_append", "paged4_read", "paged4_decode", "paged4_workspace_bytes",
                "verify_drafts", "block_trim"):
        return getattr(importlib.import_module(".binding", __name__), name)
    raise AttributeError(name)
