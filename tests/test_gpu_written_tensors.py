"""Tensors that a call writes through their addresses are known to autograd as
written: a graph that saved one of them refuses its backward instead of computing
it from other values, as after any in-place operation of torch."""
import pytest
import torch

from protein_folding_triangle_gb300 import layers
from protein_folding_triangle_gb300 import synthetic as S
from protein_folding_triangle_gb300 import triattn as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from protein_folding_triangle_gb300 import build
    build.build()
    T.load()


def saved_by(t):
    """A result whose backward needs t."""
    w = torch.ones(t.shape, device="cuda", requires_grad=True)
    return (w * t).sum()


def refuses(y):
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_clipped_in_place(dt):
    ts = [torch.ones(100, device="cuda", dtype=dt), torch.ones(7, device="cuda"), torch.empty(0, device="cuda")]
    y, z = saved_by(ts[0]), saved_by(ts[1])
    T.triattn_grad_norm(ts)
    y.backward(retain_graph=True)  # a norm alone writes nothing
    T.triattn_clip_grad_norm(ts, 1.0)
    refuses(y)
    refuses(z)


def test_clipped_into_others():
    ts, outs = [torch.ones(100, device="cuda")], [torch.ones(100, device="cuda")]
    y, z = saved_by(ts[0]), saved_by(outs[0])
    T.triattn_clip_grad_norm(ts, 1.0, out=outs)
    y.backward()
    refuses(z)


def test_gradients_of_parameters():
    p = torch.nn.Parameter(torch.ones(50, device="cuda"))
    p.grad = torch.ones(50, device="cuda")
    y = saved_by(p.grad)
    layers.clip_grad_norm_([p], 1.0)
    refuses(y)
    with torch.inference_mode():  # tensors without a version counter
        t = torch.ones(10, device="cuda")
        assert float(T.triattn_clip_grad_norm([t], 1.0)) == pytest.approx(10.0 ** 0.5, rel=1e-6)


@pytest.mark.parametrize("rows", [5, 300])
def test_transition_outputs(rows):
    x = S.make_transition_inputs((rows,), 64, 64, seed=1)
    d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}
    args = [d[k] for k in ("z", "mask", "ln_w", "ln_b", "w_in", "w_o")]
    out = T.triattn_transition_fwd(*args)
    grads = T.triattn_transition_bwd(*args, d["d_out"])
    ys = [saved_by(t) for t in (out,) + tuple(grads)]
    ys[0].backward(retain_graph=True)
    again = T.triattn_transition_fwd(*args, out=out)
    assert again is out
    T.triattn_transition_bwd(*args, d["d_out"], out=grads)
    for y in ys:
        refuses(y)
    keep = saved_by(d["z"])
    T.triattn_transition_fwd(*args)
    keep.backward()  # what is only read stays as it was
