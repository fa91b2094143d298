"""GB300-native (sm_103a) LiLiCorr draft-time rerank.

The CUDA library (liblilicorr.so, built in-tree by build.build()) holds the whole path;
this package marshals arguments to its C ABI.
"""
from .decode import (  # noqa: F401
    KV8Cache,
    beam_reorder,
    beam_select,
    beam_select_workspace,
    kv8_append,
    kv8_attention,
    kv8_attention_workspace,
)
from .cross import cross_attention, cross_attention_workspace  # noqa: F401
from .logits import adjust_logits  # noqa: F401
from .pages import (  # noqa: F401
    kv8_compact,
    kv8_copy,
    kv8_fork,
    kv8_free,
    kv8_grow,
    kv8_pages_workspace,
)
from .api import (  # noqa: F401
    LilicorrError,
    Weights,
    device_error,
    diag_wait_timeout,
    greedy_walk,
    viterbi,
    launch_count,
    lm_head_topk_lse,
    lm_head_workspace_bytes,
    rerank,
    rerank_host,
    rerank_host_workspace,
    sample_walk,
    stage_timing,
    stage_times,
    topk_lse,
    topk_lse_merge,
    topk_lse_shard,
    topk_lse_workspace,
)
from ._lib import BF16, F32, LIB_PATH  # noqa: F401
