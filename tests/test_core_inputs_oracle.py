"""The oracle of the core's inputs (norms with rotation, relative position bias)
against independent statements of the same: central differences, torch's
automatic differentiation in 64 bits, and hand-written small cases."""
import math

import numpy as np
import pytest
import torch

from oracle import core_inputs as CI


@pytest.mark.parametrize("kind", ["none", "half", "interleaved"])
@pytest.mark.parametrize("shared", [False, True])
def test_qk_norm_gradients_against_differences(kind, shared):
    """Step 1e-5: the difference's own error is about 1e-10, so 1e-7 of the gradient's size."""
    g = np.random.default_rng(3)
    B, No, H, N, D = 2, 2, 2, 3, 8
    x, dy = g.normal(size=(2, B, No, H, N, D))
    w = 1.0 + 0.2 * g.normal(size=(D,) if shared else (H, D))
    pos = g.integers(-50, 1000, size=(B, N))
    r = CI.qk_norm(x, w, pos, kind, dy=dy, eps=1e-3)

    def loss(x, w):
        return float((CI.qk_norm(x, w, pos, kind, eps=1e-3)["y"] * dy).sum())

    for name, t in (("dx", x), ("dw", w)):
        num = np.zeros_like(t)
        for i in np.ndindex(t.shape):
            for s in (1, -1):
                v = t.copy()
                v[i] += s * 1e-5
                num[i] += s * (loss(v, w) if name == "dx" else loss(x, v)) / 2e-5
        assert np.abs(num - r[name]).max() <= 1e-7 * np.abs(r[name]).max(), name


@pytest.mark.parametrize("kind", ["half", "interleaved"])
def test_rotation_is_the_matrix_of_the_formula(kind):
    D, N = 16, 5
    x = np.random.default_rng(1).normal(size=(1, 1, 1, N, D))
    pos = np.array([[0, 1, 17, -3, 2_000_000]])
    y = CI.qk_norm(x, np.ones(D), pos, kind)["y"][0, 0, 0]
    for n in range(N):
        u = x[0, 0, 0, n] / math.sqrt((x[0, 0, 0, n] ** 2).mean() + float(np.float32(1e-6)))
        for i in range(D // 2):
            a, b = (i, i + D // 2) if kind == "half" else (2 * i, 2 * i + 1)
            t = float(pos[0, n]) * 10000.0 ** (-2.0 * i / D)
            want = (u[a] * math.cos(t) - u[b] * math.sin(t), u[a] * math.sin(t) + u[b] * math.cos(t))
            # the angle of 2e6 as a double is off by 2e6 2^-53
            assert np.abs(np.array(want) - (y[n, a], y[n, b])).max() <= 1e-9


def test_rotated_scores_depend_on_the_difference_only():
    g = np.random.default_rng(2)
    q, k = g.normal(size=(2, 1, 1, 1, 1, 32))
    w = np.ones(32)

    def score(a, b):
        return float((CI.qk_norm(q, w, [[a]], "half")["y"] * CI.qk_norm(k, w, [[b]], "half")["y"]).sum())

    assert abs(score(5, 2) - score(1_000_005, 1_000_002)) <= 1e-8


def test_clipped_buckets():
    assert [CI.bucket_of(d, "clip", 5, 2) for d in (-9, -2, -1, 0, 1, 2, 9)] == [0, 0, 1, 2, 3, 4, 4]
    k = CI.buckets(1, 4, 6, [[10, 11, 10, 14]], [[7, 7, 3, 7]], "clip", 2)[0]
    assert k.tolist() == [[2, 1, 5, 0], [3, 2, 5, 0], [5, 5, 2, 5], [4, 4, 5, 2]]


def test_logarithmic_buckets():
    """32 rows to 128: the first 8 distances of each sign exact, then a row per
    factor 2^(1/2) (borders 8, 11.3, 16, 22.6, 32, 45.3, 64, 90.5), the last from 90.5 on."""
    row = [CI.bucket_of(d, "log", 32, 128) for d in range(200)]
    first = {r: row.index(r) for r in sorted(set(row))}
    assert first == {**{i: i for i in range(8)}, 8: 8, 9: 12, 10: 16, 11: 23, 12: 32, 13: 46, 14: 64, 15: 91}
    assert [CI.bucket_of(-d, "log", 32, 128) for d in range(1, 200)] == [r + 16 for r in row[1:]]


@pytest.mark.parametrize("layout", ["heads", "pairs"])
def test_relpos_against_autograd(layout):
    g = torch.Generator().manual_seed(4)
    B, N, F, R = 2, 7, 3, 2
    table = torch.randn(6, F, generator=g, dtype=torch.float64, requires_grad=True)
    shape = (B, F, N, N) if layout == "heads" else (B, N, N, F)
    base, d = torch.randn((2,) + shape, generator=g, dtype=torch.float64)
    pos = torch.randint(-4, 5, (B, N), generator=g)
    chain = torch.randint(0, 2, (B, N), generator=g)
    rel = (pos[:, :, None] - pos[:, None, :]).clamp(-R, R) + R
    rel[chain[:, :, None] != chain[:, None, :]] = 5
    e = table[rel]
    out = base + (e.permute(0, 3, 1, 2) if layout == "heads" else e)
    out.backward(d)
    k = CI.buckets(B, N, 6, pos.numpy(), chain.numpy(), "clip", R)
    got = CI.relpos(table.detach().numpy(), base.numpy(), k, layout)
    assert np.allclose(got, out.detach().numpy(), rtol=0, atol=1e-14)
    assert np.allclose(CI.relpos_bwd(d.numpy(), k, 6, layout), table.grad.numpy(), rtol=0, atol=1e-12)
