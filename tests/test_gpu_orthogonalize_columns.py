"""GPU test of the orthogonalisation of blocks of columns of one matrix, in place: the bits
that each block has alone, and nothing beside them touched."""
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


@pytest.mark.parametrize("rows,widths", [(128, (128, 128, 128)), (60, (33, 7, 64, 1)), (300, (130, 200)),
                                         (200, (64, 96, 300))])
def test_blocks_of_a_fused_matrix(rows, widths):
    g = torch.Generator().manual_seed(rows)
    fused = torch.randn(rows, sum(widths) + 5, generator=g).bfloat16().cuda()
    blocks = list(torch.split(fused, list(widths) + [5], dim=1))[:-1]
    want = T.triattn_orthogonalize([b.contiguous() for b in blocks])
    rest = fused[:, -5:].clone()
    T.triattn_orthogonalize(blocks, out=blocks)
    assert T.device_status() == T.OK
    assert all(torch.equal(a, b) for a, b in zip(blocks, want)) and torch.equal(fused[:, -5:], rest)
