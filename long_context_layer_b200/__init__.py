"""DELTA decode attention stack for NVIDIA B200 (sm_100a).

The compute path is libdelta_attn.so (include/delta_attn.h); this package is a thin
binding over it plus the per-step stack schedule.  There is no CPU fallback: importing
the binding fails when the library is missing.
"""
from . import _native  # noqa: F401  (fails loudly if the library is not built)
from ._native import (  # noqa: F401
    DELTA_BF16, DELTA_E4M3, DELTA_F32, DELTA_HEAD_MAX, DELTA_HEAD_SUM, DELTA_INT8, DELTA_ROPE_BANDS,
    DELTA_ROPE_HALF, DELTA_ROPE_INTERLEAVED, DELTA_ROPE_LINEAR, DELTA_ROPE_PLAIN, DeltaDesc, DeltaError,
    DeltaPageTable, DeltaQ8Cache, DeltaRope, DeltaRopeParams, DeltaSelectParams, choose_layers, full_attn,
    full_attn_noalloc, full_attn_q8, kv_append, kv_append_layers, kv_append_layers_q8, kv_append_q8, kv_read_q8,
    kv_write_q8, layer_shift, read_device_error, rope, rope_table, sel_capacity, select_attn, select_attn_q8,
    sparse_attn, sparse_attn_q8, sparse_attn_settled, sparse_attn_settled_q8, status_string, window_attn,
    window_attn_q8, workspace_init, workspace_size, workspace_size_q8, workspace_size_reduce,
)
