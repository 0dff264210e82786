"""Transition layers whose gates are all far out: closed (act(a) a tiny fraction
of a) or wide open (act'(a) of a sigmoid nearly 0).  There a gate has to be
right relative to itself, not to 1: nothing larger stands beside it in h.

Every a lies around `center`: x_0 is 4 in every row (ln_w_0 = 0, ln_b_0 = 4,
exact in BF16), w_in's first row is center / 4 in the a half, and the other
features spread a by `spread`.

Tolerances (relative RMSE).  A BF16 rounding spread evenly over its step has an
RMS of at most u = 2^-8 / sqrt(3) of the value.  x's reaches a as u spread and
act(a) or act'(a) as `amp` u spread (amp: the largest |d log act / da| and
|d log act' / da| within three spreads of the center; d log act' of an open SiLU
or GELU is far below 1); x reaches b as u; then h and out: sqrt((amp spread)^2 + 3) u
forward.  Backward x in a and in b again, then dh (rounded at C > 128), da or db,
and the result: sqrt((amp spread)^2 + 4) u.  d_ln_w and d_ln_b have few elements and
one far larger than the others, feature 0's, a sum over the rows of terms of either
sign: the terms' errors add like the terms' squares, whatever is left of the sum, so
they are held against the root of the sum of those squares.  The bound above is the
standard deviation of that one number's error, which is a sum over hundreds of rows
and so close to normal: 4 of them, passed by 6e-5 of draws, for the 72 that are
taken here.  FP32 sums of a add 2^-20 |a| at the
very most to a, amp of that to the gate: 2^-20 20 at
amp 1, 2^-20 6 12 at GELU's -6, below 1e-4; 2e-4 is added.
Up to 192 rows the forward rounds out alone, 2^-8, as in test_gpu_transition.py."""
import math

import numpy as np
import pytest
import torch

from parity_utils import cpu64, rel_rmse
from oracle import transition as TR
from oracle.trimul import layernorm
from protein_folding_triangle_gb300 import synthetic as S
from protein_folding_triangle_gb300 import triattn as T

pytestmark = pytest.mark.gpu

U = 2.0 ** -8 / math.sqrt(3.0)

# (activation, center, spread, amp)
GATES = [("sigmoid", -4.0, 0.3, 1.0), ("sigmoid", -6.0, 0.7, 1.0), ("sigmoid", -20.0, 0.7, 1.0),
         ("sigmoid", 10.0, 0.7, 1.0),
         ("silu", -4.0, 0.3, 1.1), ("silu", -6.0, 0.7, 1.1), ("silu", -20.0, 0.7, 1.1), ("silu", 9.0, 0.7, 1.0),
         ("gelu", -3.0, 0.2, 5.0), ("gelu", -4.0, 0.25, 7.0), ("gelu", -6.0, 0.2, 12.0), ("gelu", 4.0, 0.2, 1.0)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from protein_folding_triangle_gb300 import build
    build.build()
    T.load()


def params(d):
    return d["z"], d["mask"], d["ln_w"], d["ln_b"], d["w_in"], d["w_o"]


def make(M, C, H, center, spread):
    x = S.make_transition_inputs((M,), C, H, seed=M + C + H)
    x["ln_w"][0], x["ln_b"][0] = 0.0, 4.0
    w = x["w_in"].float()
    w[:, :H] *= spread
    w[0, :H], w[0, H:] = center / 4.0, 0.0
    x["w_in"] = w.to(torch.bfloat16)
    return x


def row_terms(x, kind):
    """dx and xhat of every row in FP64: d_ln_b and d_ln_w are the sums of dx and dx xhat."""
    z, lw, lb, wi, wo, g = (cpu64(x[k]) for k in ("z", "ln_w", "ln_b", "w_in", "w_o", "d_out"))
    H = wo.shape[0]
    xn, xhat, _ = layernorm(z, lw, lb)
    p = xn @ wi
    f, df = TR.act(p[:, :H], kind)
    dh = g @ wo.T
    return np.concatenate([dh * p[:, H:] * df, dh * f], axis=1) @ wi.T, xhat


def to_dev(x):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}


@pytest.mark.parametrize("gate", GATES, ids=lambda g: f"{g[0]}{g[1]:+.0f}")
@pytest.mark.parametrize("M,C,H", [(193, 128, 512), (900, 64, 96), (500, 256, 288)])
def test_far_gates(M, C, H, gate):
    kind, center, spread, amp = gate
    x = make(M, C, H, center, spread)
    ref = TR.run(*params(x), x["d_out"], kind)
    d = to_dev(x)
    out = T.triattn_transition_fwd(*params(d), kind)
    dz, dlw, dlb, dwi, dwo = T.triattn_transition_bwd(*params(d), d["d_out"], kind)
    torch.cuda.synchronize()
    assert T.device_status() == T.OK
    a2 = (amp * spread) ** 2
    errs = {"out": rel_rmse(cpu64(out), ref["out"])}
    for n, g in (("dz", dz), ("dw_o", dwo)):
        errs[n] = rel_rmse(cpu64(g), ref[n])
    dx, xhat = row_terms(x, kind)
    for n, g, terms in (("dln_w", dlw, dx * xhat), ("dln_b", dlb, dx)):
        errs[n] = float(np.sqrt(((cpu64(g) - ref[n]) ** 2).sum() / (terms ** 2).sum()))
    errs["dw_a"] = rel_rmse(cpu64(dwi[:, :H]), ref["dw_in"][:, :H])  # through act'
    errs["dw_b"] = rel_rmse(cpu64(dwi[:, H:]), ref["dw_in"][:, H:])  # through act
    print(gate, {k: f"{v:.2e}" for k, v in errs.items()})
    assert errs.pop("out") <= U * math.sqrt(a2 + 3) + 2e-4, errs
    for n, e in errs.items():
        assert e <= U * math.sqrt(a2 + 4) * (4 if n in ("dln_w", "dln_b") else 1) + 2e-4, (n, errs)


@pytest.mark.parametrize("gate", GATES, ids=lambda g: f"{g[0]}{g[1]:+.0f}")
@pytest.mark.parametrize("C,H", [(128, 512), (256, 96)])
def test_far_gates_of_a_few_rows(C, H, gate):
    """192 rows, and the same rows as part of 193: apart by both calls' errors."""
    kind, center, spread, amp = gate
    x = make(193, C, H, center, spread)
    ref = TR.run(*params(x), x["d_out"], kind)["out"][:192]
    d = to_dev(x)
    many = cpu64(T.triattn_transition_fwd(*params(d), kind))[:192]
    d["z"] = d["z"][:192].contiguous()
    few = cpu64(T.triattn_transition_fwd(*params(d), kind))
    tol_few, tol_many = 2.0 ** -8 + 5e-4, U * math.sqrt((amp * spread) ** 2 + 3) + 2e-4
    assert rel_rmse(few, ref) <= tol_few
    assert rel_rmse(many, few) <= tol_few + tol_many


@pytest.mark.parametrize("kind", TR.ACTIVATIONS)
@pytest.mark.parametrize("M", [5, 300])
def test_gates_past_the_exponent_range(M, kind):
    """Gates of +-200 and +-3e4, whose exponentials over- and underflow: closed
    ones give 0 (SiLU and GELU: -0 counts), open ones a or 1, nothing is NaN."""
    C, H = 64, 64
    x = make(M, C, H, 0.0, 0.0)
    w = x["w_in"].float()
    w[0, :H] = torch.tensor([-7500.0, -50.0, 50.0, 7500.0]).repeat(16)
    x["w_in"] = w.to(torch.bfloat16)
    ref = TR.run(*params(x), x["d_out"], kind)
    d = to_dev(x)
    out = T.triattn_transition_fwd(*params(d), kind)
    grads = T.triattn_transition_bwd(*params(d), d["d_out"], kind)
    torch.cuda.synchronize()
    assert rel_rmse(cpu64(out), ref["out"]) <= 8e-3
    for n, g in zip(("dz", "dln_w", "dln_b", "dw_in", "dw_o"), grads):
        assert bool(torch.isfinite(g).all()), n
        assert rel_rmse(cpu64(g), ref[n]) <= 1e-2, n
