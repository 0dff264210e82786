"""GPU test of the norms' module on views that the kernels do not take as they are: copied,
with the results and gradients of contiguous tensors."""
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


def fused_heads(x):  # q's and k's heads side by side, as planes
    return x.view(2, 3, 4, 9, 16).chunk(2, dim=2)


def overlapping(x):  # rows that share elements
    return tuple(t.as_strided((2, 3, 2, 9, 16), (3 * 320, 320, 160, 8, 1), t.storage_offset()) for t in x)


def shifted(x):  # from 8 bytes on
    n = 2 * 3 * 2 * 9 * 16
    return tuple(x.flatten()[4 + i * n:4 + (i + 1) * n].view(2, 3, 2, 9, 16) for i in range(2))


@pytest.mark.parametrize("views", [fused_heads, overlapping, shifted])
def test_views(views):
    torch.manual_seed(0)
    norm = layers.QKNorm(2, 16, device="cuda")
    x = torch.randn(2, 4096, device="cuda").bfloat16()
    x = x[:, :3 * 4 * 9 * 16].contiguous() if views is fused_heads else x
    q, k = (t.detach().requires_grad_() for t in views(x))
    assert not (layers._rows(q) and layers._rows(k) and q.stride() == k.stride())
    a, b = norm(q, k)
    assert T.device_status() == T.OK
    da, db = torch.randn_like(a), torch.randn_like(b)
    (ga, gb) = torch.autograd.grad((a, b), (q, k), (da, db))
    want = T.triattn_qk_norm_fwd(q.detach().clone(memory_format=torch.contiguous_format),
                                 k.detach().clone(memory_format=torch.contiguous_format), norm.w_q, norm.w_k)
    grads = T.triattn_qk_norm_bwd(q.detach().clone(memory_format=torch.contiguous_format),
                                  k.detach().clone(memory_format=torch.contiguous_format), norm.w_q, norm.w_k, da, db)
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    assert torch.equal(ga, grads[0]) and torch.equal(gb, grads[1])
