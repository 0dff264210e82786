"""GPU test of the binding without its native part: the same bits."""
import pytest
import torch

from protein_folding_triangle_gb300 import triattn as T
from test_gpu_host import calls, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from protein_folding_triangle_gb300 import build
    build.build()
    T.load()


@pytest.mark.parametrize("rows,shared,chains", [(0, 0, 1), (1, 1, 0)])
def test_the_bits_without_it(monkeypatch, rows, shared, chains):
    fs = calls(rows, shared, chains)
    want = [f() for f in fs]
    monkeypatch.setattr(T, "_HOST", T._General)
    for f, w in zip(fs, want):
        assert same(f(), w)
    assert T.device_status() == T.OK
