"""B200-native fused linear cross-entropy (FLCE).

The hot path is a C-ABI CUDA library (`include/flce.h`, sources in `csrc/`)
with hand-written sm_100a kernels: tcgen05/TMEM bf16 GEMM tiles fed by TMA
with the softcap, an online fp32 logsumexp and the label gather fused into the
forward epilogue, and a backward that recomputes logit tiles, forms dZ in
registers and feeds two more tensor-core GEMMs (dHidden, split-K dWeight).
Beside the loss the library scores with the same head: log probabilities of given
tokens, entropies and top alternatives, with gradients; and it looks up rows of the
weight where it is tied to the embedding, with its gradient.
This package is its thin PyTorch binding.
"""
from .flce import (  # noqa: F401
    FlceForward, FusedLinearCrossEntropy, alloc_workspace, backward, forward,
    fused_linear_cross_entropy, status, workspace_bytes,
)
from .embedding import (  # noqa: F401
    embedding_backward, embedding_forward, embedding_workspace_bytes, fused_embedding,
)
from .logprobs import (  # noqa: F401
    Logprobs, fused_linear_logprobs, logprobs_backward, logprobs_forward,
    logprobs_workspace_bytes,
)
from ._native import FlceError, get_option, load, options, set_option  # noqa: F401

__all__ = [
    "FlceForward", "FusedLinearCrossEntropy", "FlceError", "Logprobs", "alloc_workspace",
    "backward", "embedding_backward", "embedding_forward", "embedding_workspace_bytes",
    "forward", "fused_embedding", "fused_linear_cross_entropy", "fused_linear_logprobs",
    "get_option", "load", "logprobs_backward", "logprobs_forward", "logprobs_workspace_bytes", "options",
    "set_option", "status", "workspace_bytes",
]
