"""FP64 oracle of the transition (gated feed-forward block over rows) and of
the global gradient norm with clipping (test infrastructure only).

  x = LayerNorm(z), eps 1e-5;  [a | b] = x W_in;  h = act(a) b;
  out = m (h W_o), rows with m = 0 left out (0 output, no gradient, whatever
  they hold)

Every step in float64 numpy; the rows whose mask is 0 are taken out of the
arrays before anything is computed.
"""
from __future__ import annotations

import numpy as np

from .trimul import _f64, layernorm, layernorm_bwd, sigmoid

ACTIVATIONS = ("silu", "sigmoid", "gelu")


def act(a, kind):
    """(act(a), act'(a))."""
    if kind == "silu":
        s = sigmoid(a)
        return a * s, s + a * s * (1.0 - s)
    if kind == "sigmoid":
        s = sigmoid(a)
        return s, s * (1.0 - s)
    if kind == "gelu":
        k, c = np.sqrt(2.0 / np.pi), 0.044715
        t = np.tanh(k * (a + c * a ** 3))
        return 0.5 * a * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * a * (1.0 - t ** 2) * k * (1.0 + 3.0 * c * a ** 2)
    raise ValueError(kind)


def run(z, mask, ln_w, ln_b, w_in, w_o, d_out=None, kind="silu"):
    """{"out"} and, with d_out, the gradients of <out, d_out>: dz, dln_w,
    dln_b, dw_in, dw_o."""
    z, mask, ln_w, ln_b, w_in, w_o, d_out = (_f64(t) for t in (z, mask, ln_w, ln_b, w_in, w_o, d_out))
    H, C = w_o.shape
    rows = z.reshape(-1, C)
    m = np.ones(rows.shape[0]) if mask is None else mask.reshape(-1)
    keep = m != 0.0
    m = m[keep][:, None]
    x, xhat, rstd = layernorm(rows[keep], ln_w, ln_b)
    p = x @ w_in
    a, b = p[:, :H], p[:, H:]
    f, df = act(a, kind)
    h = f * b
    out = np.zeros_like(rows)
    out[keep] = m * (h @ w_o)
    res = {"out": out.reshape(z.shape)}
    if d_out is None:
        return res
    g = m * d_out.reshape(-1, C)[keep]
    dh = g @ w_o.T
    dp = np.concatenate([dh * b * df, dh * f], axis=1)
    dz = np.zeros_like(rows)
    dz[keep], dgamma, dbeta = layernorm_bwd(dp @ w_in.T, xhat, rstd, ln_w)
    res.update(dz=dz.reshape(z.shape), dln_w=dgamma, dln_b=dbeta, dw_in=x.T @ dp, dw_o=h.T @ g)
    return res


def clip(tensors, max_norm, kind="l2"):
    """(norm, clipped tensors) of a list of arrays."""
    ts = [_f64(t) for t in tensors]
    if kind == "l2":
        norm = np.sqrt(sum(float((t * t).sum()) for t in ts))
    else:
        norm = max([float(np.abs(t).max()) for t in ts if t.size], default=0.0)
    coef = min(1.0, max_norm / (norm + 1e-6))
    return norm, [t * coef for t in ts]
