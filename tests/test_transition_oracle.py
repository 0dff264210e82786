"""The FP64 oracle of the transition and of clipping against other routes:
torch's FP64 autograd, central differences, and torch's clip_grad_norm_."""
import numpy as np
import pytest
import torch

from oracle import transition as TR
from protein_folding_triangle_gb300 import synthetic as S

NAMES = ("z", "ln_w", "ln_b", "w_in", "w_o")


def torch_run(x, kind):
    p = {k: x[k].double().requires_grad_(True) for k in NAMES}
    H = x["w_o"].shape[0]
    h = torch.nn.functional.layer_norm(p["z"], (x["z"].shape[-1],), p["ln_w"], p["ln_b"], 1e-5) @ p["w_in"]
    f = {"silu": torch.nn.functional.silu, "sigmoid": torch.sigmoid,
         "gelu": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[kind](h[..., :H])
    out = (f * h[..., H:]) @ p["w_o"]
    if x["mask"] is not None:
        out = out * x["mask"].double()[..., None]
    out.backward(x["d_out"].double())
    return out.detach(), {k: p[k].grad for k in NAMES}


@pytest.mark.parametrize("kind", TR.ACTIVATIONS)
@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_matches_autograd(kind, drop):
    x = S.make_transition_inputs((2, 5, 7), 32, 64, seed=3, drop=drop)
    r = TR.run(x["z"], x["mask"], x["ln_w"], x["ln_b"], x["w_in"], x["w_o"], x["d_out"], kind)
    out, grads = torch_run(x, kind)
    # FP64 both: sums of at most 70 * 128 terms
    np.testing.assert_allclose(r["out"], out.numpy(), rtol=0, atol=1e-11)
    for name, key in zip(NAMES, ("dz", "dln_w", "dln_b", "dw_in", "dw_o")):
        np.testing.assert_allclose(r[key], grads[name].numpy(), rtol=0, atol=1e-10)


@pytest.mark.parametrize("kind", TR.ACTIVATIONS)
def test_central_differences(kind):
    rng = np.random.default_rng(0)
    C, H, M = 4, 3, 5
    p = {"z": rng.normal(size=(M, C)), "ln_w": rng.normal(size=C), "ln_b": rng.normal(size=C),
         "w_in": rng.normal(size=(C, 2 * H)), "w_o": rng.normal(size=(H, C))}
    mask = np.array([1.0, 0.5, 0.0, 1.0, 1.0])
    d = rng.normal(size=(M, C))
    r = TR.run(p["z"], mask, p["ln_w"], p["ln_b"], p["w_in"], p["w_o"], d, kind)
    eps = 1e-6
    for name, key in zip(NAMES, ("dz", "dln_w", "dln_b", "dw_in", "dw_o")):
        num = np.zeros_like(p[name])
        for i in np.ndindex(p[name].shape):
            f = []
            for sgn in (1, -1):
                q = {k: v.copy() for k, v in p.items()}
                q[name][i] += sgn * eps
                f.append((TR.run(q["z"], mask, q["ln_w"], q["ln_b"], q["w_in"], q["w_o"], None, kind)["out"] * d).sum())
            num[i] = (f[0] - f[1]) / (2 * eps)
        np.testing.assert_allclose(r[key], num, rtol=0, atol=1e-6 * max(1.0, np.abs(num).max()))


def test_masked_rows_may_hold_anything():
    x = S.make_transition_inputs((40,), 32, 32, seed=5, drop=0.4)
    args = lambda y: (y["z"], y["mask"], y["ln_w"], y["ln_b"], y["w_in"], y["w_o"], y["d_out"])  # noqa: E731
    a = TR.run(*args(x))
    bad = x["mask"] == 0
    x["z"][bad], x["d_out"][bad] = float("nan"), float("inf")
    b = TR.run(*args(x))
    for k in a:
        assert np.array_equal(a[k], b[k]) and np.isfinite(a[k]).all(), k


@pytest.mark.parametrize("kind,p", [("l2", 2.0), ("max", float("inf"))])
@pytest.mark.parametrize("limit", [0.5, 1e6])
def test_clip_matches_torch(kind, p, limit):
    g = torch.Generator().manual_seed(0)
    ts = [torch.randn(n, generator=g, dtype=torch.float64).float() for n in (1, 0, 17, 300)]
    params = [torch.nn.Parameter(torch.zeros_like(t, dtype=torch.float64)) for t in ts]
    for q, t in zip(params, ts):
        q.grad = t.double().clone()
    want = torch.nn.utils.clip_grad_norm_([q for q in params if q.numel()], limit, p)
    norm, out = TR.clip(ts, limit, kind)
    assert abs(norm - float(want)) <= 1e-12 * float(want)
    for q, o in zip(params, out):
        np.testing.assert_allclose(o, q.grad.numpy(), rtol=1e-12, atol=0)
