"""GB300 (sm_103a) kernels for the target-side verification step of speculative decoding.

The compute path is the C-ABI library built from csrc/ (declared in include/spec_verify.h);
`binding` exposes its entry points under the same names for torch CUDA tensors.
"""

from .binding import (  # noqa: F401
    SpecVerifyError,
    attention_workspace_bytes,
    library,
    make_attention_workspace,
    make_workspace,
    workspace_reset,
    spec_attention,
    spec_kv_compact,
    spec_kv_read,
    spec_kv_write,
    spec_logits_process,
    spec_ngram_draft,
    spec_verify_chain,
    spec_verify_ngram,
    spec_verify_tree_greedy,
    spec_verify_tree_walk,
    workspace_bytes,
)
