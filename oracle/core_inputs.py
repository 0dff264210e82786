"""FP64 oracle of what prepares the attention core's inputs (test infrastructure
only): the norms of queries and keys for each head with the position rotation,
and the learned relative position bias by buckets, with their gradients.

Plain float64 numpy.  The rotation is a product of complex numbers, the angles
are reduced to a turn in whole numbers, the logarithmic buckets' borders are
found by comparing whole numbers.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np

from .trimul import _f64


def turns(positions, D: int, theta: float = 10000.0):
    """exp(i pos theta^(-2 i / D)) [B, N, D / 2]: the angle's fraction of a turn
    from exact products (a position times a frequency in 2^-80 turns)."""
    pos = np.asarray(positions, dtype=np.int64)
    out = np.empty(pos.shape + (D // 2,), dtype=np.complex128)
    for i in range(D // 2):
        f = int(Fraction(float(theta) ** (-2.0 * i / D) / (2.0 * np.pi)) * (1 << 80))
        frac = np.array([((int(p) * f) % (1 << 80)) / float(1 << 80) for p in pos.ravel()])
        out[..., i] = np.exp(2j * np.pi * frac).reshape(pos.shape)
    return out


def _pairs(u, kind):
    D = u.shape[-1]
    return u[..., : D // 2] + 1j * u[..., D // 2:] if kind == "half" else u[..., 0::2] + 1j * u[..., 1::2]


def _unpair(z, kind):
    out = np.empty(z.shape[:-1] + (2 * z.shape[-1],))
    if kind == "half":
        out[..., : z.shape[-1]], out[..., z.shape[-1]:] = z.real, z.imag
    else:
        out[..., 0::2], out[..., 1::2] = z.real, z.imag
    return out


def qk_norm(x, w, positions=None, kind="half", theta=10000.0, eps=1e-6, dy=None):
    """One of q, k [B, N_o, H, N, D] with its weight [H, D] or [D].  {"y"} and,
    with dy, "dx", "dw" and "dw_abs", the sum of dw's terms' sizes (of the turned
    pair of dy, whose length the turn keeps, times n)."""
    x, w, dy = (_f64(t) for t in (x, w, dy))
    B, _, _, N, D = x.shape
    pos = np.tile(np.arange(N), (B, 1)) if positions is None else np.asarray(positions)
    rot = None if kind == "none" else turns(pos, D, theta)[:, None, None]
    wf = w if w.ndim == 1 else w[:, None, :]
    eps = float(np.float32(eps))
    r = 1.0 / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    n = x * r
    u = n * wf
    out = {"y": u if rot is None else _unpair(_pairs(u, kind) * rot, kind)}
    if dy is None:
        return out
    g = dy if rot is None else _unpair(_pairs(dy, kind) * np.conj(rot), kind)
    out["dw"] = (g * n).sum(axis=(0, 1, 2, 3) if w.ndim == 1 else (0, 1, 3))
    z = None if rot is None else np.abs(_pairs(dy, kind))
    size = np.abs(g) if rot is None else _unpair(z + 1j * z, kind)
    out["dw_abs"] = (size * np.abs(n)).sum(axis=(0, 1, 2, 3) if w.ndim == 1 else (0, 1, 3))
    a = g * wf
    out["dx"] = r * (a - n * (a * n).mean(axis=-1, keepdims=True))
    return out


def bucket_of(d: int, kind: str, n: int, R: int) -> int:
    """The table's row of a difference of positions; n rows without that of other chains."""
    if kind == "clip":
        return min(max(d, -R), R) + R
    half = n // 2
    e = half // 2
    m = min(abs(d), R)
    k = m
    if m >= e:  # the largest t with (m / e)^(half - e) >= (R / e)^t, in whole numbers
        s = half - e
        k = e + max(t for t in range(s + 1) if m ** s * e ** t >= R ** t * e ** s)
        k = min(k, half - 1)
    return k + (half if d < 0 else 0)


def buckets(B, N, K, positions=None, chains=None, kind="clip", R=32):
    """The table's row of every pair [B, N, N]."""
    pos = np.tile(np.arange(N), (B, 1)) if positions is None else np.asarray(positions).astype(np.int64)
    n = K - (0 if chains is None else 1)
    rows = np.array([bucket_of(d, kind, n, R) for d in range(-R, R + 1)])
    k = rows[np.clip(pos[:, :, None] - pos[:, None, :], -R, R) + R]
    if chains is not None:
        c = np.asarray(chains)
        k = np.where(c[:, :, None] == c[:, None, :], k, K - 1)
    return k


def relpos(table, base, k, layout):
    table, base = _f64(table), _f64(base)
    e = table[k]
    e = e.transpose(0, 3, 1, 2) if layout == "heads" else e
    return e if base is None else base + e


def relpos_bwd(d_out, k, K, layout):
    d = _f64(d_out)
    d = d.transpose(0, 2, 3, 1) if layout == "heads" else d
    out = np.zeros((K, d.shape[-1]))
    np.add.at(out, k.ravel(), d.reshape(-1, d.shape[-1]))
    return out
