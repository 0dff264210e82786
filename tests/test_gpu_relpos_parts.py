"""GPU test of the position bias on parts of larger tensors, which need not start on 16
bytes: planes of one example of a batch, the gradient of a joined batch, a table that is
a part of one buffer of parameters."""
import pytest
import torch

from protein_folding_triangle_gb300 import layers
from protein_folding_triangle_gb300 import triattn as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from protein_folding_triangle_gb300 import build
    build.build()
    T.load()


@pytest.mark.parametrize("fp32_table_at", [0, 3])
@pytest.mark.parametrize("N,H", [(5, 1), (33, 3)])
def test_parts_of_a_batch(N, H, fp32_table_at):
    torch.manual_seed(N)
    rel = layers.RelativePosition(H, max_distance=4, device="cuda")
    flat = torch.randn(9 * H + 8, device="cuda")
    rel.table = torch.nn.Parameter(flat[fp32_table_at:fp32_table_at + 9 * H].view(9, H))
    base = torch.randn(3, H, N, N, device="cuda").bfloat16()
    assert base[1].data_ptr() % 16 != 0
    parts = [rel(base[b:b + 1]) for b in range(3)]
    d = torch.randn(3, H, N, N, device="cuda").bfloat16()
    torch.cat(parts).backward(d)
    got = rel.table.grad.clone()
    rel.zero_grad()
    whole = rel(base)
    assert torch.equal(torch.cat(parts), whole)
    for b in range(3):  # the same three sums, added in the same order
        rel(base[b:b + 1].clone()).backward(d[b:b + 1].clone())
    # autograd adds the parts' gradients in its own order: of three FP32 sums, 2 x 2^-24 of their sizes
    size = sum(T.triattn_relpos_bwd(d[b:b + 1].abs().clone(), 9, max_distance=4) for b in range(3))
    assert bool(((got - rel.table.grad).abs() <= 2.0 ** -22 * size).all())
