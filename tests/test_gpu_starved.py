"""A load that is left out (test hook): the products that wait for it give up after the
limit, every CTA ends by itself, peers of its team among them, the status word says
so, and the next call, with the hook off, gives the right bits."""
import pytest
import torch

from protein_folding_triangle_gb300 import triattn as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from protein_folding_triangle_gb300 import build
    build.build()
    T.load()


def starved(f):
    """f's outputs where nothing is left out, after a call where something is."""
    want = f()
    assert T.device_status() == T.OK
    T.set_wait_limit_ns(20_000_000)
    T.test_set_starve(True)
    try:
        f()
        status = T.device_status()
    finally:
        T.test_set_starve(False)
        T.set_wait_limit_ns(0)
    assert status == T.ERR_TIMEOUT
    again = f()
    assert T.device_status() == T.OK
    assert len(again) == len(want) and all(torch.equal(a, b) for a, b in zip(again, want))


def matrices(count, m, n):
    g = torch.Generator().manual_seed(m + n)
    return [torch.randn(m, n, generator=g).bfloat16().cuda() for _ in range(count)]


# teams of eight, one CTA for each matrix, columns that stay in shared memory and columns that do not
@pytest.mark.parametrize("count,m,n", [(1, 128, 512), (3, 90, 5000), (160, 100, 256), (160, 64, 700)])
def test_small_matrices(count, m, n):
    ms = matrices(count, m, n)
    starved(lambda: T.triattn_orthogonalize(ms))


@pytest.mark.parametrize("N,F", [(9, 8), (131, 128), (160, 256)])
def test_pair_features(N, F):
    d = torch.randn(1, N, N, F, generator=torch.Generator().manual_seed(N)).bfloat16().cuda()
    starved(lambda: [T.triattn_relpos_bwd(d, 65, layout="pairs")])
