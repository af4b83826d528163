"""Exact, IO-aware softmax attention for NVIDIA GB300 (sm_103a).

The compute lives in ``libfa_gb300.so`` (hand-written CUDA, C-ABI in
``include/fa.h``); this package is its Python binding. Importing it does not
load the library; the first call does, and raises if it has not been built.
"""
from ._build import build  # noqa: F401
from .api import (FAError, FlashAttention, Session, alloc_workspace, fa_backward,  # noqa: F401
                  fa_backward_dkdv, fa_backward_dq, fa_backward_grads, fa_backward_noalloc,
                  fa_backward_preprocess,
                  fa_backward_workspace_size, fa_forward, fa_get_device_status,
                  fa_online_softmax_stats, fa_standard_forward, fa_standard_matrix_bytes,
                  fa_selftest_mma, fa_selftest_wait_timeout, flash_attention, lib, status_string, version)
from .cache4 import (alloc_cache4, alloc_cache4_workspace, fa_cache4_append,  # noqa: F401
                     fa_cache4_decode, fa_cache4_read)
from .decode import alloc_prefix_workspace, fa_cache_append, fa_prefix_decode  # noqa: F401
from .packed import (FlashAttentionPacked, PackedPlan, alloc_packed_workspace,  # noqa: F401
                     fa_packed_backward, fa_packed_forward, fa_packed_plan,
                     flash_attention_packed)
from .rope import (QKNormRope, alloc_qk_norm_rope_workspace, fa_qk_norm_rope,  # noqa: F401
                   fa_qk_norm_rope_backward, fa_rope_append, qk_norm_rope, rope_table)
