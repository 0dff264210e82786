"""GPU tests of the orthogonalisation of matrices whose squares FP32 does not hold, above and
below its range, against the FP64 oracle: the norm is that of the values all the same.
Tolerance as for other sizes (operands of 22 bits, one rounding)."""
import numpy as np
import pytest
import torch

from oracle import orthogonalize as OR
from protein_folding_triangle_gb300 import triattn as T
from test_gpu_orthogonalize import TOL, far, update

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from protein_folding_triangle_gb300 import build
    build.build()
    T.load()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("size,eps", [(1e18, 1e-7), (1e19, 1e-7), (1e25, 1e-7), (1e37, 1e-7), (1e-18, 1e-24),
                                      (1e-21, 1e-30), (1e-25, 1e-32), (1e-36, 1e-38)])
def test_beyond_the_range_of_squares(size, eps, dtype):
    for shape in ((60, 200), (200, 130), (300, 60)):
        g = update(*shape, seed=1, dtype=dtype, size=size)
        assert bool(torch.isfinite(g).all())
        out, = T.triattn_orthogonalize([g], eps=eps)
        assert T.device_status() == T.OK
        assert far(out, OR.orthogonalize(g, eps=eps)) <= TOL


def test_one_large_value_among_small_ones():
    """Runs of 4096 elements of both kinds in one matrix."""
    g = torch.zeros(100, 300)
    g[3, 7], g[90, 250] = 2e38, 1e-20
    out, = T.triattn_orthogonalize([g.cuda()])
    ref = OR.orthogonalize(g.numpy())
    assert np.abs(out.float().cpu().numpy() - ref).max() <= TOL * ref.max()


def test_values_far_below_eps():
    """The result is G / eps times the polynomial's slope; zeros stay zeros."""
    g = update(64, 90, seed=2, dtype=torch.float32, size=1e-24)
    out, zero = T.triattn_orthogonalize([g, torch.zeros_like(g)], eps=1e-20)
    assert far(out, OR.orthogonalize(g, eps=1e-20)) <= TOL
    assert torch.count_nonzero(zero) == 0
