"""Routed mixture-of-experts verify layer for AMD Instinct MI355X (gfx950).

One routed-MoE FFN block (F32 softmax top-k router, Q8_0 / Q4_K / Q2_K / Q3_K / Q6_K experts,
SwiGLU, a shared expert and a weighted combine) applied to the verify batch
of MTP speculative decoding, implemented as hand-written HIP kernels behind
the C ABI of ``include/moe_layer.h``, plus greedy MTP verify/accept
(``include/moe_accept.h``), log probabilities of the tokens it accepts
(``include/moe_logprobs.h``), and the attention half of the verify step on a
paged 4-bit key/value cache (``include/moe_kv.h``), and the step on a tree of
drafts: plan, attention and commit (``include/moe_tree.h``), sampled
verification of chains and trees (``include/moe_sample.h``).  This package is the thin
Python binding of that ABI (``_binding``) and the build helper (``build``).
"""

from ._binding import (  # noqa: F401
    ACCEPT_MAX_ROWS,
    C_SYMBOLS,
    DraftTree,
    KvBatch,
    KvDesc,
    LIB_PATH,
    LOGPROBS_MAX_TOP,
    LayerDesc,
    LayerWeights,
    NOALLOC_MAX_WORKSPACE,
    MoeError,
    PreparedForward,
    TREE_MAX_ROWS,
    accept_workspace,
    kv_cache,
    kv_workspace,
    lib,
    logprobs_workspace,
    moe_accept_workspace_bytes,
    moe_dequant_rows,
    moe_kv_append,
    moe_kv_attention,
    moe_kv_attention_workspace_bytes,
    moe_kv_cache_bytes,
    moe_kv_commit,
    moe_kv_read,
    moe_kv_tree_attention,
    moe_layer_forward,
    moe_layer_forward_noalloc,
    moe_layer_forward_timed,
    moe_logprobs,
    moe_logprobs_workspace_bytes,
    moe_route,
    moe_sample_workspace_bytes,
    moe_stage_count,
    moe_stage_name,
    moe_strerror,
    moe_tensor_bytes,
    moe_tree_plan,
    moe_verify_accept,
    moe_verify_sample,
    moe_version,
    moe_workspace_bytes,
    sample_workspace,
    workspace,
)
