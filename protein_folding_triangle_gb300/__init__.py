"""libtriattn: triangular (pair-biased, slice-batched) attention forward and
backward on NVIDIA GB300 (sm_103a), behind a C ABI (include/triattn.h), with
the triangle-attention module around it, the triangle multiplicative update,
the transition (gated feed-forward block), norms of queries and keys with the
position rotation, the learned relative position bias, the global gradient norm
with clipping, and the orthogonalisation of a list of updates.

``triattn`` is the ctypes binding, ``build`` compiles the CUDA library
in-tree, ``synthetic`` draws seeded inputs, ``sharding`` splits the outer axis
across GPUs or into memory-bounded chunks on one GPU, ``layers`` wraps the
module, the multiplicative update, the transition, the norms and the position
bias as autograd functions and torch modules, and clips and orthogonalises the
gradients of their parameters.
"""
from . import build, synthetic, triattn  # noqa: F401
from .triattn import (TriAttnError, bwd_workspace_bytes, device_status, set_wait_limit_ns,  # noqa: F401
                      tri_attn_bwd, tri_attn_fwd, tri_attn_module_bwd, tri_attn_module_fwd, triangle_attention,
                      triattn_clip_grad_norm, triattn_grad_norm, triattn_orthogonalize, triattn_qk_norm_bwd,
                      triattn_qk_norm_fwd, triattn_relpos_bwd, triattn_relpos_fwd, triattn_transition_bwd,
                      triattn_transition_fwd, triattn_trimul_bwd, triattn_trimul_fwd)
