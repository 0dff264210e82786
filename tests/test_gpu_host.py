"""GPU tests of the binding's native part: a usual call, which it takes, gives the bits
of the same call through the general path, follows the current stream and refuses
what the general path refuses."""
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


def randn(*shape, dtype=torch.bfloat16):
    return torch.randn(*shape, device="cuda").to(dtype)


def same(a, b):
    a, b = (x if isinstance(x, (tuple, list)) else (x,) for x in (a, b))
    return len(a) == len(b) and all(x.shape == y.shape and x.stride() == y.stride() and x.dtype == y.dtype
                                    and torch.equal(x, y) for x, y in zip(a, b))


def calls(rows, shared, chains):
    torch.manual_seed(7)
    if rows:  # a projection's rows
        q, k, dq, dk = (randn(2, 3, 21, 4 * 4 * 16)[..., c:c + 64].unflatten(-1, (4, 16)).permute(0, 1, 3, 2, 4)
                        for c in (0, 0, 8, 8))
    else:
        q, k, dq, dk = (randn(2, 3, 4, 21, 16) for _ in range(4))
    w = torch.rand(16, device="cuda") if shared else torch.rand(4, 16, device="cuda")
    pos = torch.randint(-90, 90, (2, 21), dtype=torch.int32, device="cuda")
    ch = torch.randint(0, 2, (2, 21), dtype=torch.int32, device="cuda") if chains else None
    K = 17 + chains
    table, planes, pairs = torch.randn(K, 8, device="cuda"), randn(2, 8, 21, 21), randn(2, 21, 21, 8)
    ms = [randn(30, 41), randn(150, 140, dtype=torch.float32), randn(9, 5)]
    how = dict(max_distance=8)
    return [lambda **kw: T.triattn_qk_norm_fwd(q, k, w, w, pos, "interleaved", theta=500, eps=1e-5, **kw),
            lambda **kw: T.triattn_qk_norm_bwd(q, k, w, w, dq, dk, None, "half", **kw),
            lambda **kw: T.triattn_relpos_fwd(table, planes, pos, ch, **how, **kw),
            lambda **kw: T.triattn_relpos_fwd(table, None, pos, ch, layout="pairs", **how, **kw),
            lambda **kw: T.triattn_relpos_bwd(planes, K, pos, ch, **how, **kw),
            lambda **kw: T.triattn_relpos_bwd(planes.float(), K, None, ch, **how, **kw),
            lambda **kw: T.triattn_relpos_bwd(pairs, K, pos, ch, layout="pairs", **how, **kw),
            lambda **kw: T.triattn_orthogonalize(ms, **kw)]


@pytest.mark.parametrize("rows", [0, 1])
@pytest.mark.parametrize("shared", [0, 1])
@pytest.mark.parametrize("chains", [0, 1])
def test_the_bits_of_the_general_path(rows, shared, chains):
    for f in calls(rows, shared, chains):
        assert same(f(), f(stream=torch.cuda.current_stream()))  # a stream by name goes the general way
    assert T.device_status() == T.OK


def test_the_native_part_takes_usual_calls(monkeypatch):
    """... and nothing but them: the general path's first check is not reached."""
    def reached(*a, **k):
        raise AssertionError("general path")
    fs = calls(1, 0, 1)
    monkeypatch.setattr(T, "_qk_norm_plan", reached)
    monkeypatch.setattr(T, "_relpos_plan", reached)
    monkeypatch.setattr(T, "_matrix_table", reached)
    for f in fs[:-1]:
        f()
    g = [randn(30, 41), randn(9, 5)]
    T.triattn_orthogonalize(g, out=g)
    for f in fs[:-1]:
        with pytest.raises(AssertionError):
            f(stream=torch.cuda.current_stream())


def test_on_the_current_stream():
    for f in calls(0, 0, 1):
        want = f()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        big = torch.randn(4096, 4096, device="cuda")
        with torch.cuda.stream(side):
            got = f()
        big = big @ big  # on another stream than the call
        side.synchronize()
        assert same(got, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = f()
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, want)


def test_refusals():
    q, w = randn(1, 3, 2, 9, 16), torch.rand(2, 16, device="cuda")
    table, planes = torch.randn(65, 4, device="cuda"), randn(1, 4, 9, 9)
    for f in (lambda: T.triattn_qk_norm_fwd(q.float(), q.float(), w, w),
              lambda: T.triattn_qk_norm_fwd(q, q[:, :2], w, w),
              lambda: T.triattn_qk_norm_fwd(q, q, w.bfloat16(), w),
              lambda: T.triattn_qk_norm_fwd(q, q.cpu(), w, w),
              lambda: T.triattn_qk_norm_fwd(q, q, w, w, None, "quarter"),
              lambda: T.triattn_qk_norm_fwd(q.transpose(2, 4), q.transpose(2, 4), w, w),
              lambda: T.triattn_relpos_fwd(table, planes.float()),
              lambda: T.triattn_relpos_fwd(table, planes, layout="rows"),
              lambda: T.triattn_relpos_fwd(table.t(), planes),
              lambda: T.triattn_relpos_bwd(planes[..., :8], 65),
              lambda: T.triattn_orthogonalize([q]),
              lambda: T.triattn_orthogonalize([w.double()]),
              lambda: T.triattn_orthogonalize([w], out=[w]),
              lambda: T.triattn_orthogonalize([w], out=[w.bfloat16().t()])):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: T.triattn_qk_norm_fwd(q, q, w, w, eps=-1.0),
              lambda: T.triattn_relpos_fwd(table, planes, max_distance=31),
              lambda: T.triattn_relpos_bwd(planes, 66),
              lambda: T.triattn_relpos_bwd(planes, 1 << 20, max_distance=1 << 19)):
        with pytest.raises(T.TriAttnError):
            f()
