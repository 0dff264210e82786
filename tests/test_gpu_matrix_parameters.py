"""GPU test of the orthogonalised gradients of a model: its matrices, and nothing else."""
import warnings

import numpy as np
import pytest
import torch

from oracle import orthogonalize as OR
from parity_utils import cpu64
from protein_folding_triangle_gb300 import layers
from protein_folding_triangle_gb300 import triattn as T
from test_gpu_core_inputs_together import Attention, draw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from protein_folding_triangle_gb300 import build
    build.build()
    T.load()


def test_a_model_keeps_the_gradients_of_its_vectors():
    """After a step the heads' weights and the table keep their clipped gradients, the
    projection has the orthogonalised one: its rounding, 2^-8, and its products, 1e-3
    as for the operator alone."""
    torch.manual_seed(1)
    m = Attention(96, 2, 16, "half", False, "clip")
    x, base, mask, positions, chains, d = draw(1, 9, 33, 96, 2, 16, seed=2)
    m(x, base, mask, positions, chains).backward(d)
    layers.clip_grad_norm_(m.parameters(), 1e-2)
    before = {n: p.grad.clone() for n, p in m.named_parameters()}
    layers.orthogonalize_grads_(m)
    assert T.device_status() == T.OK
    for n, p in m.named_parameters():
        if n == "w":
            want = OR.orthogonalize(before[n])
            assert np.linalg.norm(cpu64(p.grad) - want) <= (2.0 ** -8 + 1e-3) * np.linalg.norm(want)
        else:
            assert torch.equal(p.grad, before[n]), n


def test_a_list_with_vectors_is_warned_of():
    """A list is taken as it is, and the caller is told of the vectors in it."""
    norm, rel = layers.QKNorm(2, 16, device="cuda"), layers.RelativePosition(4, max_distance=4, device="cuda")
    w = torch.nn.Parameter(torch.randn(8, 9, device="cuda").bfloat16())
    for p in (norm.w_q, rel.table, w):
        p.grad = torch.randn_like(p)
    for ps in ([norm.w_q, w], [rel.table], list(norm.parameters())):
        with pytest.warns(UserWarning, match="vectors"):
            layers.orthogonalize_grads_(ps)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        layers.orthogonalize_grads_([w])
        layers.orthogonalize_grads_(torch.nn.ModuleList([norm, rel]))
        layers.orthogonalize_grads_([norm.w_k])  # no gradient
    assert T.device_status() == T.OK
