"""GB300-native dynamic block-sparse attention (BSA) forward.

``plan`` maps a logical u8 block mask onto 128-row physical tiles (retain,
combine or subdivide) and emits a per-(head, q-tile) CSR list of K/V tiles, a
longest-row-first schedule and an optional GQA union table; ``forward`` runs a
persistent tcgen05/TMA kernel over exactly those tiles.  Both run in libbsa.so
(include/bsa.h); this package is its ctypes binding plus the seeded workload
generators.  ``Cache`` / ``cache_*``: a paged K/V cache in 8 bits, with its
writers, attention for decoding, the forward over it, its page operations, and
eviction by the attention weight that its tokens gather.
``rope``: rotary positions of queries and keys; ``prompt_attention``: packed prompts
without a plan.
"""
from ._cache import (  # noqa: F401
    Cache, cache_append, cache_attention, cache_compact, cache_copy_pages, cache_create, cache_evict, cache_fork,
    cache_forward, cache_free, cache_resize, cache_status, cache_weigh,
)
from ._lib import (  # noqa: F401
    BsaError, Layout, Plan, PLAN_NO_UNION, PLAN_Q64, PLAN_REMAP, STAGE_ALL, STAGE_BOUNDED, STAGE_EXACT, STAGE_KNORM, STAGE_PREPARE,
    STAGE_ROWBOUND, attention, attention_static, attention_static_status, forward, library, plan, plan_affine,
    plan_check, plan_layout, plan_workspace_bytes, select_flags, sync_status, watchdog_selftest,
)
from ._prompt import Rope, prompt_attention, prompt_status, prompt_workspace_bytes, rope, rope_create  # noqa: F401

__all__ = ["BsaError", "Cache", "cache_append", "cache_attention", "cache_compact", "cache_copy_pages", "cache_create",
           "cache_evict", "cache_fork", "cache_forward", "cache_free", "cache_resize", "cache_status", "cache_weigh", "Layout", "Plan", "PLAN_NO_UNION", "PLAN_Q64", "PLAN_REMAP", "STAGE_ALL", "STAGE_BOUNDED",
           "STAGE_EXACT", "STAGE_KNORM", "STAGE_PREPARE", "STAGE_ROWBOUND", "attention", "attention_static", "attention_static_status", "forward", "library",
           "plan", "plan_affine", "plan_check", "plan_layout", "plan_workspace_bytes", "prompt_attention", "prompt_status", "prompt_workspace_bytes", "Rope", "rope", "rope_create", "select_flags", "sync_status",
           "watchdog_selftest"]
