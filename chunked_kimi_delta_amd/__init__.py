"""Chunked Kimi Delta Attention (KDA) forward (and its backward) on AMD Instinct MI355X (gfx950).

The compute lives in libkda_fwd.so (hand-written HIP kernels behind the C ABI of
include/kda_fwd.h). This package is a thin ctypes binding: it marshals torch tensors' device
pointers and the current HIP stream into that ABI and nothing else. There is no fallback: if
the shared library is missing or cannot be loaded, every entry point raises.
"""
from .api import KdaBwdPlan, KdaFwdPlan, kda_bwd, kda_fwd, workspace_bytes  # noqa: F401
from .act8 import Packed8, pack8, unpack8  # noqa: F401
from .gdn import GdnBwdPlan, GdnFwdPlan, GdnStepPlan, gdn_bwd, gdn_fwd, gdn_step  # noqa: F401
from .glr import GlrBwdPlan, GlrFwdPlan, GlrStepPlan, glr_bwd, glr_fwd, glr_step  # noqa: F401
from .pool import pool_alloc, pool_compact, pool_copy, pool_fork, pool_free  # noqa: F401
from .autograd import ChunkGDNFunction, ChunkGLRFunction, ChunkKDAFunction, chunk_gdn, chunk_glr, chunk_kda  # noqa: F401
from ._lib import KDA_BF16, KDA_FP32, library_path, load  # noqa: F401

__all__ = ["kda_fwd", "KdaFwdPlan", "kda_bwd", "KdaBwdPlan", "chunk_kda", "ChunkKDAFunction",
           "gdn_fwd", "GdnFwdPlan", "gdn_bwd", "GdnBwdPlan", "chunk_gdn", "ChunkGDNFunction", "gdn_step", "GdnStepPlan", "Packed8", "pack8", "unpack8",
           "glr_fwd", "GlrFwdPlan", "glr_bwd", "GlrBwdPlan", "chunk_glr", "ChunkGLRFunction", "glr_step", "GlrStepPlan",
           "pool_copy", "pool_fork", "pool_alloc", "pool_free", "pool_compact",
           "workspace_bytes", "load", "library_path", "KDA_BF16", "KDA_FP32"]
