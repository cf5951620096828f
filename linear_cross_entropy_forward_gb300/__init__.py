"""Fused linear cross-entropy + entropy for NVIDIA GB300 (sm_103a).

loss, entropy = linear_cross_entropy(hidden, weight, labels, reduction="mean")

The [N, V] logits are never materialised: tcgen05 tensor-core GEMM tiles feed
fused online-softmax (forward) and dlogits (backward) epilogues inside
libflce.so, reached through a C ABI (include/flce.h).  The gradient-in-forward
mode (flce_forward_backward, linear_cross_entropy(..., grad_in_forward=True))
keeps one token chunk's logits instead and skips the backward's recompute.

Around the head: policy_loss and preference_loss read its log-probabilities,
linear_policy_loss is the first on top of the head in one call, and embedding is the
lookup in a (tied) table, each with its gradient.  linear is the dense layer below the head (or
its logits), flce_process_logits and logits_logprob the distribution that a sampler sees of them, and
AdamW the step that the gradients go into.
"""
from .adamw import AdamW, flce_grad_norm  # noqa: F401
from ._binding import (FlceError, FlceParams, flce_backward, flce_combine_shards,  # noqa: F401
                       flce_forward, flce_forward_backward, flce_scale_bf16,
                       flce_shard_stats, flce_status, kernel_launches,
                       linear_cross_entropy, load_library, make_params, plan_tiles,
                       selftest_wait_timeout, workspace_size,
                       LIB_PATH, EXPORTED)
from .embedding import (embedding, embedding_params, embedding_workspace_size,  # noqa: F401
                        flce_embedding, flce_embedding_backward)
from .linear import (flce_linear, flce_linear_backward, linear, linear_params,  # noqa: F401
                     linear_workspace_size)
from .logits import (flce_logits_logprob, flce_logits_logprob_backward,  # noqa: F401
                     flce_process_logits, logits_logprob)
from .losses import (flce_policy_forward_backward, flce_policy_loss,  # noqa: F401
                     flce_preference_loss, linear_policy_loss, policy_loss, policy_params,
                     policy_workspace_size, preference_loss, preference_params,
                     preference_workspace_size)
from .pipeline import HostPipeline  # noqa: F401
from .vocab_parallel import (exchange_stats, reduce_dhidden,  # noqa: F401
                             vocab_parallel_linear_cross_entropy)
from .workloads import IGNORE_INDEX, WORKLOADS  # noqa: F401

__version__ = "0.2.0"
