"""GB300-native batched draft-token verification for speculative decoding.

The compute path is libspecverify.so (hand-written sm_103a CUDA behind the C
ABI in include/); this package holds its sources (csrc/), the in-tree build
(_build.py) and a thin ctypes binding (binding.py; cache.py for the 4-bit paged
cache, prompt.py for the attention of prompts, tree.py for trees of drafts).
"""
from ._build import build  # noqa: F401
from .binding import (  # noqa: F401
    EXPORTS, SpecError, StepController, draft_confidence, load_library, new_workspace,
    prefix_stats, restore_rows, step_cost_additive, step_cost_sps,
    verify_greedy, verify_greedy_active, verify_greedy_margin, verify_greedy_noalloc, verify_relaxed_topk,
    verify_sample, workspace_bytes,
)
from .cache import (  # noqa: F401
    CacheCall, PagedCache, cache_append, cache_attend, cache_attend_tree, cache_evict, cache_read,
    cache_weights, cache_workspace_bytes, new_cache, new_cache_workspace,
)
from .prompt import new_prompt_workspace, prompt_attend, prompt_workspace_bytes  # noqa: F401
from .tree import adjust_logits, tree_accept  # noqa: F401

__all__ = ["build", "load_library", "new_workspace", "workspace_bytes", "verify_greedy",
           "verify_greedy_noalloc", "verify_greedy_margin", "verify_greedy_active",
           "verify_relaxed_topk", "verify_sample", "draft_confidence", "prefix_stats",
           "restore_rows", "StepController", "step_cost_sps", "step_cost_additive", "SpecError", "EXPORTS",
           "PagedCache", "CacheCall", "new_cache", "new_cache_workspace", "cache_workspace_bytes",
           "cache_append", "cache_read", "cache_attend", "cache_attend_tree", "cache_weights", "cache_evict",
           "prompt_attend", "new_prompt_workspace", "prompt_workspace_bytes", "tree_accept", "adjust_logits"]
