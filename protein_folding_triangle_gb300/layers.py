"""Autograd functions and torch modules over the library's entry points.

Every computation runs in libtriattn's kernels; these classes only hold
parameters, keep the forward's context buffer
for the backward, and hand the library's gradients to autograd.  The
library's parameter gradients are FP32; autograd casts them to each
parameter's dtype (BF16 projection matrices, FP32 LayerNorm parameters).

- ``TriangleAttention``: the triangle-attention module around the core
  (LayerNorm, projections into q, k, v and the pair bias, core, output
  projection; "TurboPairFormer", Figure 6).  Returns the update; the caller
  adds it to z.
- ``TriangleMultiplication``: the triangle multiplicative update, outgoing or
  incoming ("TurboPairFormer", Figure 12).  Returns the update.
- ``Transition``: the gated feed-forward block over the pair rows.  Returns
  the update; its forward keeps only its inputs for the backward.
- ``QKNorm``: norms of queries and keys for each head with the position
  rotation, in front of the core (``triattn.triangle_attention``).
- ``RelativePosition``: a learned relative position bias by buckets, added to
  the core's bias planes or to the pair features.
- ``clip_grad_norm_``: clips the gradients of a model's parameters by their
  global norm, in place.
- ``orthogonalize_grads_``: orthogonalises the gradients of its matrices, in
  place; ``matrix_parameters``: which of a model's parameters those are.

Forward and backward may be captured into a CUDA graph.  Before a backward is
captured, drop what holds an eager autograd graph of the same parameters (a
loss that is still referenced, say): torch ties the accumulation of a leaf to
the stream of the graph that used it first, and a capture that reaches another
stream fails.
"""
from __future__ import annotations

import math
import warnings
from typing import Optional

import torch

from . import triattn as T


class TriangleAttentionFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, z, ln_w, ln_b, w_in, w_o, mask, H: int, D: int):
        z = z.contiguous()
        out, buf = T.tri_attn_module_fwd(z, mask, ln_w, ln_b, w_in, w_o, H, D)
        ctx.save_for_backward(z, ln_w, w_in, w_o, buf)
        ctx.mask, ctx.H, ctx.D = mask, H, D
        return out

    @staticmethod
    def backward(ctx, d_out):
        z, ln_w, w_in, w_o, buf = ctx.saved_tensors
        dz, dlw, dlb, dwi, dwo = T.tri_attn_module_bwd(z, ctx.mask, ln_w, w_in, w_o, buf, d_out.contiguous(), ctx.H,
                                                       ctx.D)
        return dz, dlw, dlb, dwi, dwo, None, None, None


class TriangleMultiplicationFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, z, ln_in_w, ln_in_b, w_p, ln_out_w, ln_out_b, w_o, mask, direction: str):
        z = z.contiguous()
        out, buf = T.triattn_trimul_fwd(z, mask, ln_in_w, ln_in_b, w_p, ln_out_w, ln_out_b, w_o, direction)
        ctx.save_for_backward(z, ln_in_w, w_p, ln_out_w, w_o, buf)
        ctx.mask, ctx.direction = mask, direction
        return out

    @staticmethod
    def backward(ctx, d_out):
        z, ln_in_w, w_p, ln_out_w, w_o, buf = ctx.saved_tensors
        dz, dliw, dlib, dwp, dlow, dlob, dwo = T.triattn_trimul_bwd(z, ctx.mask, ln_in_w, w_p, ln_out_w, w_o, buf,
                                                                    d_out.contiguous(), ctx.direction)
        return dz, dliw, dlib, dwp, dlow, dlob, dwo, None, None


class TransitionFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, z, ln_w, ln_b, w_in, w_o, mask, activation: str):
        z = z.contiguous()
        out = T.triattn_transition_fwd(z, mask, ln_w, ln_b, w_in, w_o, activation)
        ctx.save_for_backward(z, ln_w, ln_b, w_in, w_o, mask)
        ctx.activation = activation
        return out

    @staticmethod
    def backward(ctx, d_out):
        z, ln_w, ln_b, w_in, w_o, mask = ctx.saved_tensors
        dz, dlw, dlb, dwi, dwo = T.triattn_transition_bwd(z, mask, ln_w, ln_b, w_in, w_o, d_out.contiguous(),
                                                          ctx.activation)
        return dz, dlw, dlb, dwi, dwo, None, None


def _rows(t: torch.Tensor) -> bool:
    """Whether a [B, N_o, H, N, D] view is one of rows that the kernels take as it is:
    the rules of tri_attn_fwd_strided."""
    if t.dim() != 5 or t.stride(4) != 1 or t.data_ptr() % 16:
        return False
    B, No, H, N, D = t.shape
    example, piece, head, row = t.stride()[:4]
    if (B > 1 and example != No * piece) or not all(s > 0 and s % 8 == 0 for s in (piece, head, row)):
        return False
    if head < row or (head == row and H == 1):  # heads inside a row
        inner, n_inner, outer, n_outer = head, H, row, N
    elif piece == H * head and (head != row or N == 1):
        inner, n_inner, outer, n_outer = row, N, head, H
    else:
        return False
    width = (n_inner - 1) * inner + D
    return inner >= D and width <= outer and (n_outer - 1) * outer + width <= piece < 1 << 36


def _aligned(t: torch.Tensor) -> torch.Tensor:
    """``t``, or a copy that is contiguous and starts on 16 bytes: a part of a batch of
    planes of an odd number of tokens does not."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class QKNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, w_q, w_k, positions, rotary: str, theta: float, eps: float):
        if q.stride() != k.stride() or not (_rows(q) and _rows(k)):
            q, k = _aligned(q), _aligned(k)
        out = T.triattn_qk_norm_fwd(q, k, w_q, w_k, positions, rotary, theta=theta, eps=eps)
        ctx.save_for_backward(q, k, w_q, w_k, positions)
        ctx.rotary, ctx.theta, ctx.eps = rotary, theta, eps
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_q, d_k):
        q, k, w_q, w_k, positions = ctx.saved_tensors
        return (*T.triattn_qk_norm_bwd(q, k, w_q, w_k, _aligned(d_q), _aligned(d_k), positions, ctx.rotary,
                                       theta=ctx.theta, eps=ctx.eps), None, None, None, None)


class RelativePositionFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, base, positions, chains, layout: str, kind: str, max_distance: int):
        if base is not None:
            base = _aligned(base)
        out = T.triattn_relpos_fwd(_aligned(table), base, positions, chains, layout=layout, kind=kind,
                                   max_distance=max_distance)
        ctx.save_for_backward(positions, chains)
        ctx.buckets, ctx.how = table.shape[0], dict(layout=layout, kind=kind, max_distance=max_distance)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_out):
        positions, chains = ctx.saved_tensors
        d_table = None
        if ctx.needs_input_grad[0]:
            d_table = T.triattn_relpos_bwd(_aligned(d_out), ctx.buckets, positions, chains, **ctx.how)
        return d_table, d_out if ctx.needs_input_grad[1] else None, None, None, None, None, None


class TriangleAttention(torch.nn.Module):
    """Triangle attention over the pair tensor z [B, N, N, C] (BF16).  ``mask``
    (optional) is the core's additive key mask [B, N, N] (BF16, 0 or -inf):
    key k of slice i is masked where mask[b, i, k] = -inf."""

    def __init__(self, c_z: int, n_heads: int, head_dim: int, device=None):
        super().__init__()
        self.H, self.D = n_heads, head_dim
        f = 3 * n_heads * head_dim + n_heads
        self.ln_w = torch.nn.Parameter(torch.ones(c_z, dtype=torch.float32, device=device))
        self.ln_b = torch.nn.Parameter(torch.zeros(c_z, dtype=torch.float32, device=device))
        self.w_in = torch.nn.Parameter(
            (torch.randn(c_z, f, device=device) / math.sqrt(c_z)).to(torch.bfloat16))
        self.w_o = torch.nn.Parameter(
            (torch.randn(n_heads * head_dim, c_z, device=device) / math.sqrt(n_heads * head_dim)).to(torch.bfloat16))

    def forward(self, z: torch.Tensor, mask: Optional[torch.Tensor] = None) -> torch.Tensor:
        return TriangleAttentionFunction.apply(z, self.ln_w, self.ln_b, self.w_in, self.w_o, mask, self.H, self.D)


class TriangleMultiplication(torch.nn.Module):
    """Triangle multiplicative update of z [B, N, N, C_z] (BF16), ``direction``
    "outgoing" or "incoming".  ``mask`` (optional) is the multiplicative pair
    mask [B, N, N] (BF16, 1 keeps a pair)."""

    def __init__(self, c_z: int, c_hidden: int, direction: str = "outgoing", device=None):
        super().__init__()
        if direction not in T.TRIMUL_DIRECTIONS:
            raise ValueError(f"direction must be one of {tuple(T.TRIMUL_DIRECTIONS)}")
        self.direction = direction
        f = 4 * c_hidden + c_z
        self.ln_in_w = torch.nn.Parameter(torch.ones(c_z, dtype=torch.float32, device=device))
        self.ln_in_b = torch.nn.Parameter(torch.zeros(c_z, dtype=torch.float32, device=device))
        self.w_p = torch.nn.Parameter((torch.randn(c_z, f, device=device) / math.sqrt(c_z)).to(torch.bfloat16))
        self.ln_out_w = torch.nn.Parameter(torch.ones(c_hidden, dtype=torch.float32, device=device))
        self.ln_out_b = torch.nn.Parameter(torch.zeros(c_hidden, dtype=torch.float32, device=device))
        self.w_o = torch.nn.Parameter(
            (torch.randn(c_hidden, c_z, device=device) / math.sqrt(c_hidden)).to(torch.bfloat16))

    def forward(self, z: torch.Tensor, mask: Optional[torch.Tensor] = None) -> torch.Tensor:
        return TriangleMultiplicationFunction.apply(z, self.ln_in_w, self.ln_in_b, self.w_p, self.ln_out_w,
                                                    self.ln_out_b, self.w_o, mask, self.direction)


class Transition(torch.nn.Module):
    """Gated feed-forward block over the rows of z [..., C] (BF16):
    out = mask * ((act(a) * b) w_o), [a | b] = LayerNorm(z) w_in, with
    ``c_hidden`` hidden features (4 c_z by default) and ``activation`` "silu",
    "sigmoid" or "gelu" (tanh form).  ``mask`` (optional) is [...] (BF16, 1
    keeps a row); a row whose mask is 0 gives 0 and takes no part in any
    gradient, whatever z holds there."""

    def __init__(self, c_z: int, c_hidden: Optional[int] = None, activation: str = "silu", device=None):
        super().__init__()
        if activation not in T.ACTIVATIONS:
            raise ValueError(f"activation must be one of {tuple(T.ACTIVATIONS)}")
        self.activation = activation
        h = 4 * c_z if c_hidden is None else c_hidden
        self.ln_w = torch.nn.Parameter(torch.ones(c_z, dtype=torch.float32, device=device))
        self.ln_b = torch.nn.Parameter(torch.zeros(c_z, dtype=torch.float32, device=device))
        self.w_in = torch.nn.Parameter((torch.randn(c_z, 2 * h, device=device) / math.sqrt(c_z)).to(torch.bfloat16))
        self.w_o = torch.nn.Parameter((torch.randn(h, c_z, device=device) / math.sqrt(h)).to(torch.bfloat16))

    def forward(self, z: torch.Tensor, mask: Optional[torch.Tensor] = None) -> torch.Tensor:
        return TransitionFunction.apply(z, self.ln_w, self.ln_b, self.w_in, self.w_o, mask, self.activation)


class QKNorm(torch.nn.Module):
    """Norms of queries and keys [B, N_o, H, N, D] (BF16; contiguous, or views of
    one layout with contiguous features, as in a projection's rows) for each head,
    y = w[h] * x rsqrt(mean x^2 + eps), turned by the position's angles: pairs
    (i, i + D/2) with ``rotary`` "half", (2 i, 2 i + 1) with "interleaved", none
    with "none".  ``shared``: one weight [D] for all heads.  ``positions``
    (optional) [B, N] int32, the token's index if None.  Returns (q, k)."""

    NOT_MATRICES = ("w_q", "w_k")  # a vector for each head

    def __init__(self, n_heads: int, head_dim: int, rotary: str = "half", theta: float = 10000.0, eps: float = 1e-6,
                 shared: bool = False, device=None):
        super().__init__()
        if rotary not in T.ROTARY:
            raise ValueError(f"rotary must be one of {tuple(T.ROTARY)}")
        self.rotary, self.theta, self.eps = rotary, theta, eps
        shape = (head_dim,) if shared else (n_heads, head_dim)
        self.w_q = torch.nn.Parameter(torch.ones(shape, dtype=torch.float32, device=device))
        self.w_k = torch.nn.Parameter(torch.ones(shape, dtype=torch.float32, device=device))
        self.w_q.not_matrix = self.w_k.not_matrix = True

    def forward(self, q: torch.Tensor, k: torch.Tensor, positions: Optional[torch.Tensor] = None):
        return QKNormFunction.apply(q, k, self.w_q, self.w_k, positions, self.rotary, self.theta, self.eps)


class RelativePosition(torch.nn.Module):
    """Learned relative position bias: adds a row of the table (FP32, zeros at
    first) by the bucket of pos[i] - pos[j] to ``base`` (BF16), the bias planes
    [B, features, N, N] of the core (``layout`` "heads": features are heads) or
    pair features [B, N, N, features] ("pairs").  ``kind`` "clip" has
    2 max_distance + 1 buckets; "log" ``buckets``, an even number, half of them
    for each sign, logarithmic up to max_distance.  ``chains``: one row more, for
    pairs of different chains, whose indices [B, N] int32 each call then takes.
    ``positions`` (optional) [B, N] int32, the token's index if None.  Without
    ``base`` the bias alone, for the B and N of ``positions``."""

    NOT_MATRICES = ("table",)  # a vector for each bucket

    def __init__(self, features: int, layout: str = "heads", kind: str = "clip", max_distance: int = 32,
                 buckets: Optional[int] = None, chains: bool = False, device=None):
        super().__init__()
        if layout not in T.RELPOS_LAYOUTS:
            raise ValueError(f"layout must be one of {tuple(T.RELPOS_LAYOUTS)}")
        if kind not in T.BUCKETS:
            raise ValueError(f"kind must be one of {tuple(T.BUCKETS)}")
        if buckets is None:
            if kind != "clip":
                raise ValueError("buckets must be given")
            buckets = 2 * max_distance + 1
        self.layout, self.kind, self.max_distance, self.chains = layout, kind, max_distance, chains
        self.table = torch.nn.Parameter(
            torch.zeros(buckets + (1 if chains else 0), features, dtype=torch.float32, device=device))
        self.table.not_matrix = True

    def forward(self, base: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                chains: Optional[torch.Tensor] = None) -> torch.Tensor:
        if (chains is not None) != self.chains:
            raise ValueError("chains must be given" if self.chains else "this bias has no row for other chains")
        return RelativePositionFunction.apply(self.table, base, positions, chains, self.layout, self.kind,
                                              self.max_distance)


def clip_grad_norm_(parameters, max_norm: float, norm_type: float = 2.0) -> torch.Tensor:
    """Scale the gradients of ``parameters`` (BF16 and FP32) in place so that
    their global norm (2 or inf) is at most ``max_norm``.  Parameters without a
    gradient are skipped.  Returns the norm before clipping (0-dim FP32 on the
    gradients' device; nothing waits for it).  Captured into a graph, it keeps
    the gradients' addresses: zero them between replays, do not free them."""
    parameters = [parameters] if isinstance(parameters, torch.Tensor) else parameters
    return T.triattn_clip_grad_norm([p.grad for p in parameters if p.grad is not None], max_norm, norm_type)


def matrix_parameters(module: torch.nn.Module) -> list:
    """The parameters of ``module`` that are matrices of a product: 2-D, but not the
    weights of ``QKNorm`` (a vector for each head), the table of
    ``RelativePosition`` and those of embeddings (a vector for each row), and not
    what another module names in its ``NOT_MATRICES``."""
    skip = set()
    for m in module.modules():
        rows = ("weight",) if isinstance(m, (torch.nn.Embedding, torch.nn.EmbeddingBag)) else ()
        names = getattr(m, "NOT_MATRICES", rows)
        skip.update(id(p) for n, p in m.named_parameters(recurse=False) if n in names)
    return [p for p in module.parameters() if p.dim() == 2 and id(p) not in skip]


def orthogonalize_grads_(parameters, steps: int = 5, *, coefficients=T.ORTHOGONALIZE, eps: float = 1e-7) -> None:
    """Replace gradients of matrices (BF16 and FP32) by their orthogonalised ones
    (Newton-Schulz products, rounded to BF16), in place.  ``parameters`` is a model,
    of which the ``matrix_parameters`` are taken, or parameters, of which every 2-D
    one is, whatever it stands for: the heads' weights of a ``QKNorm``, a bias table
    and an embedding are 2-D as well, so hand over the model, or the matrices alone
    (a weight or table as a module above made it is warned of).
    Parameters of other dimensions or without a gradient stay as they are.  Captured
    into a graph, it keeps the gradients' addresses, as clip_grad_norm_ does.  To
    orthogonalise running means of gradients, hand those to
    ``triattn.triattn_orthogonalize``."""
    if isinstance(parameters, torch.nn.Module):
        parameters = matrix_parameters(parameters)
    parameters = [parameters] if isinstance(parameters, torch.Tensor) else parameters
    parameters = [p for p in parameters if p.grad is not None and p.dim() == 2]
    if any(getattr(p, "not_matrix", False) for p in parameters):
        warnings.warn("lists of vectors (norm weights, a bias table) are orthogonalised as matrices: hand over the "
                      "model, or matrix_parameters(model)", stacklevel=2)
    grads = [p.grad for p in parameters]
    if not grads:
        return
    wide = [g for g in grads if g.dtype != torch.bfloat16]
    narrow = [torch.empty(g.shape, dtype=torch.bfloat16, device=g.device) for g in wide]
    it = iter(narrow)
    T.triattn_orthogonalize(grads, steps, coefficients=coefficients, eps=eps,
                            out=[g if g.dtype == torch.bfloat16 else next(it) for g in grads])
    for g, o in zip(wide, narrow):
        g.copy_(o)
