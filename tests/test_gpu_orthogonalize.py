"""GPU tests of the orthogonalisation by Newton-Schulz products, against the FP64
oracle on the same inputs.

Tolerance, relative in the Frobenius norm.  The result is rounded once to BF16:
2^-8.  A step's products have operands of 22 bits and FP32 sums: off by at most
some 2^-19 |X|_F; the polynomial multiplies what a step has added by at most its
slope, a = 3.4445 at zero, in every later step, together 3.4445^5 / 2.4445 = 200
times 2^-19 = 3.8e-4 of |X|_F, which the steps leave between 0.6 and 1.3 of the
root of the rank (a few directions) or let grow (many).  1e-3 covers it.
"""
import numpy as np
import pytest
import torch

from oracle import orthogonalize as OR
from parity_utils import cpu64
from protein_folding_triangle_gb300 import triattn as T

pytestmark = pytest.mark.gpu

TOL = 2.0 ** -8 + 1e-3


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from protein_folding_triangle_gb300 import build
    build.build()
    T.load()


def update(m, n, seed, dtype=torch.bfloat16, rank=None, noise=0.3, size=1e-3):
    """A few strong directions and noise."""
    g = torch.Generator().manual_seed(seed)
    r = min(m, n, 16) if rank is None else rank
    x = torch.randn(m, r, generator=g) * torch.linspace(1.0, 0.1, r) @ torch.randn(r, n, generator=g)
    return ((x + noise * torch.randn(m, n, generator=g)) * size).to(dtype).cuda()


def far(got, ref):
    return float(np.linalg.norm(cpu64(got) - ref) / np.linalg.norm(ref))


SHAPES = [(1, 1), (1, 100), (100, 1), (5, 7), (16, 2), (64, 64), (63, 65), (128, 128), (127, 129), (128, 388),
          (388, 128), (128, 1024), (512, 128), (129, 130), (130, 129), (200, 700), (256, 1037), (300, 300),
          (1100, 512), (8, 1100), (640, 641)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}")
def test_one_matrix(shape, dtype):
    g = update(*shape, seed=sum(shape), dtype=dtype)
    out, = T.triattn_orthogonalize([g])
    assert T.device_status() == T.OK
    assert out.dtype is torch.bfloat16 and out.shape == g.shape
    assert far(out, OR.orthogonalize(g)) <= TOL


def test_a_list_is_its_matrices():
    """Mixed sizes and types, longer than one upload of the table: every result
    right, and near what the matrix gives alone (where more CTAs may share it, whose
    parts are added in another order), the list again bit for bit the same."""
    g = np.random.default_rng(0)
    ts = [update(*map(int, g.integers(1, 200, 2)), seed=i, dtype=(torch.bfloat16, torch.float32)[i % 2])
          for i in range(300)]
    ts[7] = torch.empty(0, 5, device="cuda")
    outs = T.triattn_orthogonalize(ts)
    assert outs[7].shape == (0, 5)
    for i in (0, 1, 2, 130, 255, 256, 257, 299):
        alone, = T.triattn_orthogonalize([ts[i]])
        assert far(alone, cpu64(outs[i])) <= TOL
    for i, (t, o) in enumerate(zip(ts, outs)):
        if t.numel():
            assert far(o, OR.orthogonalize(t)) <= TOL, i
    again = T.triattn_orthogonalize(ts)
    assert all(torch.equal(a, b) for a, b in zip(outs, again))


@pytest.mark.parametrize("count,m,n", [(1, 100, 5000), (1, 128, 2560), (1, 128, 2561), (1, 30, 20000), (20, 128, 640),
                                       (40, 100, 333), (160, 64, 700), (160, 700, 64), (310, 128, 321)])
def test_many_and_wide(count, m, n):
    """One CTA per matrix and teams of them, chunks that stay in shared memory and chunks that do not."""
    ts = [update(m, n, seed=i) for i in range(4)]
    outs = T.triattn_orthogonalize([ts[i % 4] for i in range(count)])
    assert T.device_status() == T.OK
    for i in range(min(4, count)):
        assert far(outs[i], OR.orthogonalize(ts[i])) <= TOL
        assert all(torch.equal(outs[k], outs[i]) for k in range(i, count, 4))


def test_few_directions():
    """A matrix of low rank: what rounding adds beside its directions grows by a in every step."""
    for m, n, r in ((128, 388, 4), (256, 300, 1), (90, 40, 2)):
        g = update(m, n, seed=r, dtype=torch.float32, rank=r, noise=0.0)
        assert far(T.triattn_orthogonalize([g])[0], OR.orthogonalize(g)) <= TOL


@pytest.mark.parametrize("size", [1e-30, 1e-9, 1e-4, 1.0, 1e6, 1e15])
def test_sizes_of_values(size):
    """Far below eps (the result is small, not orthogonal) to far above."""
    for shape in ((60, 200), (200, 130)):
        g = update(*shape, seed=1, dtype=torch.float32, size=size)
        out, = T.triattn_orthogonalize([g])
        ref = OR.orthogonalize(g)
        # values are held down to 2^-33, and an error grows by at most a in each of five steps
        least = 3.4445 ** 5 * 2.0 ** -33 * np.sqrt(ref.size)
        assert np.linalg.norm(cpu64(out) - ref) <= TOL * np.linalg.norm(ref) + least


def test_zero_and_broken_matrices_stay_by_themselves():
    ts = [update(100, 60, 1), torch.zeros(70, 90, device="cuda"), update(90, 150, 2), update(129, 129, 3)]
    want = T.triattn_orthogonalize(ts)
    assert torch.count_nonzero(want[1]) == 0
    ts[2] = ts[2].clone()
    ts[2][3, 4] = float("nan")
    got = T.triattn_orthogonalize(ts)
    assert not torch.isfinite(got[2]).any()
    for i in (0, 1, 3):
        assert torch.equal(got[i], want[i])


@pytest.mark.parametrize("steps,coef", [(1, (1.5, -0.5, 0.0)), (12, (1.5, -0.5, 0.0)), (6, (2.0, -1.5, 0.5)),
                                        (2, OR.COEFFICIENTS)])
def test_steps_and_coefficients(steps, coef):
    for shape in ((96, 200), (260, 140)):
        g = update(*shape, seed=4)
        out, = T.triattn_orthogonalize([g], steps, coefficients=coef)
        assert far(out, OR.orthogonalize(g, steps, coef)) <= TOL


def test_rows_apart_in_place_and_unaligned():
    """Rows with a stride, results over the inputs, at odd addresses; nothing beside them is touched."""
    buf = torch.full((70, 300), 5.0, dtype=torch.bfloat16, device="cuda")
    view = buf[3:63, 11:208]
    g = update(60, 197, seed=5)
    view.copy_(g)
    want, = T.triattn_orthogonalize([g])
    back = T.triattn_orthogonalize([view], out=[view])
    assert back[0] is view and torch.equal(view, want)
    view.fill_(5.0)
    assert (buf == 5.0).all()
    flat = torch.full((1 + 60 * 197 + 197 * 60 + 2,), 5.0, dtype=torch.bfloat16, device="cuda")
    a, b = flat[1:1 + 60 * 197].view(60, 197), flat[1 + 60 * 197:-2].view(197, 60)
    T.triattn_orthogonalize([g, g.t().contiguous()], out=[a, b])
    assert torch.equal(a, want) and far(b, OR.orthogonalize(g).T) <= TOL
    assert flat[0] == 5.0 and (flat[-2:] == 5.0).all()
    # an output over another matrix's input: all inputs are read first
    x, y = update(80, 90, 6), update(80, 90, 7)
    ref = T.triattn_orthogonalize([x, y])
    swapped = T.triattn_orthogonalize([x, y], out=[y, x])
    assert torch.equal(swapped[0], ref[0]) and torch.equal(swapped[1], ref[1])


def test_streams_graphs_and_two_at_once():
    ts = [update(128, 388, 1), update(512, 128, 2), update(200, 150, 3, torch.float32)]
    want = T.triattn_orthogonalize(ts)
    torch.cuda.synchronize()
    got = [T.triattn_orthogonalize(ts, stream=s) for s in (torch.cuda.Stream(), torch.cuda.Stream())]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for k in range(2):  # two graphs, replayed in turn
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[k]):
            outs.append(T.triattn_orthogonalize(ts[k:]))
    for k in (0, 1, 0, 1):
        for t in outs[k]:
            t.zero_()
        graphs[k].replay()
        eager = T.triattn_orthogonalize(ts[:1])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs[k], want[k:])) and torch.equal(eager[0], want[0])
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


def test_a_wait_that_gives_up_is_reported():
    """With a limit of a nanosecond the first wait for another CTA's tiles gives up: the
    call's kernels end by themselves, the status word says so, and the next call, with
    the limit as it was, is right."""
    gs = [update(200, 300, 1), update(300, 260, 2, torch.float32)]
    want = T.triattn_orthogonalize(gs)
    assert T.device_status() == T.OK
    T.set_wait_limit_ns(1)
    try:
        T.triattn_orthogonalize(gs)
        status = T.device_status()
    finally:
        T.set_wait_limit_ns(0)
    assert status == T.ERR_TIMEOUT
    again = T.triattn_orthogonalize(gs)
    assert T.device_status() == T.OK and all(torch.equal(a, b) for a, b in zip(again, want))
