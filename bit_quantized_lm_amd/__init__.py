"""2-bit speculative-draft LM head for MI355X (gfx950).

The head computes x[M, K] @ W[K, N] for one tensor-parallel rank's vocabulary
shard with int2 weights, keeps the top KCAND columns of every 64-column block,
reranks the best R candidates exactly against the bf16 weight and returns the
argmax token.  All per-call steps run in hand-written HIP kernels behind a
C ABI (include/drafthead.h); `_binding` is a thin ctypes layer over it.  The
draft layer's attention before the head (include/draftlayer.h: rotary append to
an 8-bit paged cache, its reading back, attention over it) is in the same
library, bound by `_layer`, and so is what several branches of one context need
(include/draftbranch.h: pages forked and drawn together, attention over shared
prefixes, log probabilities), bound by `_branch`.

Importing the package loads nothing native: the binding's names are resolved
on first attribute access, and the native library is loaded on first call
(raising if it has not been built).
"""
_BINDING_NAMES = (
    "DraftHeadError", "draft_head_sizes", "draft_head_quantize_pack", "draft_head_tile",
    "draft_head_coarse", "draft_head_rerank", "draft_head_argmax", "draft_head_last_error",
    "DraftHead", "library_path", "load_library",
)

_LAYER_NAMES = (
    "draft_layer_rope_table", "draft_layer_append", "draft_layer_read", "draft_layer_attend",
    "draft_layer_workspace_bytes", "draft_layer_workspace", "DraftCache",
)

_BRANCH_NAMES = (
    "draft_branch_fork", "draft_branch_compact", "draft_branch_pages_workspace_bytes", "draft_branch_pages_workspace",
    "draft_branch_attend", "draft_branch_attend_workspace_bytes", "draft_branch_attend_workspace",
    "draft_branch_logprobs", "draft_branch_logprobs_workspace_bytes", "draft_branch_logprobs_workspace",
)

__all__ = list(_BINDING_NAMES + _LAYER_NAMES + _BRANCH_NAMES)


def __getattr__(name):
    if name in _BINDING_NAMES:
        from . import _binding as home
    elif name in _LAYER_NAMES:
        from . import _layer as home
    elif name in _BRANCH_NAMES:
        from . import _branch as home
    else:
        raise AttributeError(name)
    value = globals()[name] = getattr(home, name)   # found here from now on
    return value
