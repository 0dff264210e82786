"""Gradients that are not finite, as a step that overflows has them: in sums over
rows every such value is part of its own sum and of no other.  The reference adds in
FP64, where an infinity stays one, and one of each sign or a NaN make a NaN; what is
finite lies within the bounds of the table's gradient: (N + 64) 2^-24 of the sum of
absolute values for planes (chains of FP32 additions), 528 * 2^-23 for pair features
(products that are cut off)."""
import numpy as np
import pytest
import torch

from oracle import core_inputs as CI
from parity_utils import cpu64
from protein_folding_triangle_gb300 import triattn as T

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from protein_folding_triangle_gb300 import build
    build.build()
    T.load()


def table_sums(d, k, K, layout):
    """Sums over the pairs of every bucket [K, F], and those of the sizes."""
    d = cpu64(d)
    d = d.transpose(0, 2, 3, 1) if layout == "heads" else d
    out = np.zeros((2, K, d.shape[-1]))
    with np.errstate(invalid="ignore"):
        for o, v in zip(out, (d, np.abs(d))):
            np.add.at(o, k.ravel(), v.reshape(-1, d.shape[-1]))
    return out


def check_table(layout, d, positions, chains, K, R):
    B, N = positions.shape
    got = cpu64(T.triattn_relpos_bwd(d, K, positions, chains, layout=layout, max_distance=R))
    assert T.device_status() == T.OK
    k = CI.buckets(B, N, K, positions.cpu().numpy(), chains.cpu().numpy(), "clip", R)
    want, size = table_sums(d, k, K, layout)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf])
    fin = np.isfinite(want)
    tol = (N + 64) * 2.0 ** -24 if layout == "heads" else 528 * 2.0 ** -23
    assert np.all(np.abs(got[fin] - want[fin]) <= tol * size[fin])
    assert fin.any() and inf.any() and np.isnan(want).any()


def ids(B, N):
    t = torch.arange(N)
    chain = (t * 2) // N
    pos = t - torch.searchsorted(chain, chain) + 5 * (t % 7 == 6)
    return pos.expand(B, N).int().contiguous().cuda(), chain.expand(B, N).int().contiguous().cuda()


def scatter(d, layout, seed):
    """Some values of d that are not finite, those of one head or feature all of one kind or missing."""
    g = torch.Generator().manual_seed(seed)
    F, N = (d.shape[1], d.shape[2]) if layout == "heads" else (d.shape[3], d.shape[1])
    for f, values in ((0, (INF,)), (1, (-INF,)), (2, (INF, -INF)), (3, (NAN,)), (F - 1, (INF, NAN))):
        for v in values:
            b, i, j = (int(torch.randint(0, n, (1,), generator=g)) for n in (d.shape[0], N, N))
            d[(b, f, i, j) if layout == "heads" else (b, i, j, f)] = v
    return d


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("B,N,F", [(1, 64, 6), (2, 131, 8), (1, 601, 5)])
def test_planes(B, N, F, fp32):
    d = torch.randn(B, F, N, N, generator=torch.Generator().manual_seed(N))
    d = scatter(d if fp32 else d.bfloat16(), "heads", N).cuda()
    check_table("heads", d, *ids(B, N), 66, 32)


@pytest.mark.parametrize("B,N,F,K", [(1, 9, 8, 18), (2, 40, 64, 66), (1, 131, 136, 66), (1, 75, 256, 202),
                                     (1, 400, 128, 66)])
def test_pair_features(B, N, F, K):
    d = torch.randn(B, N, N, F, generator=torch.Generator().manual_seed(N)).bfloat16()
    check_table("pairs", scatter(d, "pairs", N).cuda(), *ids(B, N), K, (K - 2) // 2)


def test_pair_features_that_are_all_broken():
    d = torch.full((1, 90, 90, 16), INF, dtype=torch.bfloat16, device="cuda")
    d[..., 8:] = NAN
    pos, chain = ids(1, 90)
    got = T.triattn_relpos_bwd(d, 18, pos, chain, layout="pairs", max_distance=8)
    assert T.device_status() == T.OK
    assert bool((got[:, :8] == INF).all()) and bool(torch.isnan(got[:, 8:]).all())


def test_pair_features_whose_sum_overflows():
    """Finite values whose sum FP32 does not hold: an infinity in their bucket, the others as they are."""
    g = torch.Generator().manual_seed(6)
    d = torch.randn(1, 70, 70, 24, generator=g).bfloat16()
    pos, chain = ids(1, 70)
    k = CI.buckets(1, 70, 18, pos.cpu().numpy(), chain.cpu().numpy(), "clip", 8)[0]
    i, j = np.argwhere(k == 3)[:2].T
    d[0, i, j, 5] = 3e38
    got = cpu64(T.triattn_relpos_bwd(d.cuda(), 18, pos, chain, layout="pairs", max_distance=8))
    want, size = table_sums(d, k[None], 18, "pairs")
    assert got[3, 5] == INF
    got[3, 5] = want[3, 5]
    assert np.all(np.abs(got - want) <= 528 * 2.0 ** -23 * size)


@pytest.mark.parametrize("shared", [False, True])
def test_norm_weights(shared):
    """An infinite gradient of one element: its feature's sum is not finite, the others are as without it."""
    g = torch.Generator().manual_seed(4)
    q, k, dq, dk = (torch.randn(1, 7, 3, 40, 32, generator=g).bfloat16().cuda() for _ in range(4))
    w = torch.ones(32, device="cuda") if shared else torch.ones(3, 32, device="cuda")
    want = T.triattn_qk_norm_bwd(q, k, w, w, dq, dk, None, "none")
    dq[0, 2, 1, 11, 5] = INF
    got = T.triattn_qk_norm_bwd(q, k, w, w, dq, dk, None, "none")
    a, b = (t[2].reshape(-1, 32).cpu() for t in (got, want))
    row = 0 if shared else 1
    assert not torch.isfinite(a[row, 5])
    a[row, 5] = b[row, 5]
    assert torch.equal(a, b) and torch.equal(got[3], want[3])
