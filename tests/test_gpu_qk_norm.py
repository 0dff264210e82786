"""GPU tests of the norms of queries and keys with the position rotation, against
the FP64 oracle on the same inputs.

Tolerances.  An output is rounded once to BF16: at most 2^-8 of its value.  Before
that everything is FP32: the norm, the weight, the turn by an angle that is right
to 5e-7 and whose cos and sin are right to 3e-7, some 30 roundings in all, each
2^-24 of terms no larger than a few times the row's largest value: 2^-18 of it
for the outputs.  The gradient's two terms can exceed their difference by the
square of the largest normed value, at most D = 32 times: 2^-15 of the row's
largest gradient.  dw adds T terms in FP32, in chains of at most `per` slices of a
thread, then rows / 8 of a block, then in FP64: with the terms' own errors
(per + rows / 8 + 32) 2^-24 of the sum of the terms' sizes; per <= N_o, rows <= 256.
A term's size is the length of its pair of dy times |n|: the turn back,
g_a = dy_a cos + dy_b sin, is off by its angle's and its products' errors times that
length, which is sqrt(g_a^2 + g_b^2), however small g_a itself is.
"""
import numpy as np
import pytest
import torch

from oracle import core_inputs as CI
from parity_utils import cpu64
from protein_folding_triangle_gb300 import triattn as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from protein_folding_triangle_gb300 import build
    build.build()
    T.load()


def heads_in_rows(rows, c, H, D):
    return rows[..., c:c + H * D].unflatten(-1, (H, D)).permute(0, 1, 3, 2, 4)


def make(B, No, N, H, D, seed, rows="heads", shared=False, scale=1.5):
    """q, k, dq_out, dk_out (bf16, in the given row layout), w_q, w_k."""
    g = torch.Generator().manual_seed(seed)

    def pair(scale):
        if rows == "heads":
            return [(torch.randn(B, No, H, N, D, generator=g) * scale).to(torch.bfloat16).cuda() for _ in range(2)]
        ld = (3 * H * D + H + 7) // 8 * 8
        t = (torch.randn(B, No, N, ld, generator=g) * scale).to(torch.bfloat16).cuda()
        return [heads_in_rows(t, c, H, D) for c in (0, H * D)]

    w = (D,) if shared else (H, D)
    ws = [(1.0 + 0.3 * torch.randn(w, generator=g)).cuda() for _ in range(2)]
    return pair(scale) + pair(1.0) + ws


def near(got, ref, rel, of_row):
    got, ref = cpu64(got), np.asarray(ref)
    tol = rel * np.abs(ref) + of_row * np.abs(ref).max(axis=-1, keepdims=True)
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (int(bad.sum()), bad.size, float((np.abs(got - ref) / np.maximum(tol, 1e-300)).max()))


def check(x, pos, kind, **kw):
    q, k, dqo, dko, wq, wk = x
    No, N = q.shape[1], q.shape[3]
    p = None if pos is None else pos.cuda()
    out = T.triattn_qk_norm_fwd(q, k, wq, wk, p, kind, **kw)
    grads = T.triattn_qk_norm_bwd(q, k, wq, wk, dqo, dko, p, kind, **kw)
    for m, (t, w, d) in enumerate(((q, wq, dqo), (k, wk, dko))):
        r = CI.qk_norm(t, w, None if pos is None else pos.numpy(), kind, dy=d, **kw)
        near(out[m], r["y"], 2.0 ** -8, 2.0 ** -18)
        near(grads[m], r["dx"], 2.0 ** -8, 2.0 ** -15)
        err = np.abs(cpu64(grads[2 + m]) - r["dw"])
        assert (err <= (No + 64) * 2.0 ** -24 * r["dw_abs"]).all(), (err / r["dw_abs"]).max()
    return tuple(out) + tuple(grads)


SHAPES = [  # B, N_o, N, H, D: one row; rows around a tile of 128 (D 32) or 256 (D 16) rows; every kind of remainder
    (1, 1, 1, 1, 16), (1, 1, 1, 1, 32), (1, 3, 5, 2, 32), (2, 7, 9, 3, 16), (1, 48, 48, 2, 16), (1, 5, 127, 1, 32),
    (1, 5, 128, 1, 32), (1, 5, 129, 2, 32), (3, 4, 85, 3, 16), (1, 33, 257, 1, 16), (2, 17, 31, 8, 32),
    (1, 2, 3, 150, 32), (1, 2, 2, 300, 16), (2, 131, 131, 6, 16)]


@pytest.mark.parametrize("rows", ["heads", "pairs"])
@pytest.mark.parametrize("kind", ["half", "interleaved", "none"])
@pytest.mark.parametrize("shape", SHAPES, ids=["x".join(map(str, s)) for s in SHAPES])
def test_matches_oracle(shape, kind, rows):
    B, No, N, H, D = shape
    pos = None
    if N % 2:
        pos = torch.randint(-300, 5000, (B, N), generator=torch.Generator().manual_seed(N), dtype=torch.int32)
    check(make(B, No, N, H, D, seed=N + H, rows=rows, shared=H % 2 == 0), pos, kind)


@pytest.mark.parametrize("theta", [10000.0, 100.0, 1e6, 0.5])
@pytest.mark.parametrize("kind", ["half", "interleaved"])
def test_far_positions(kind, theta):
    """The ends of 32 bits and everything between: the angle's fraction of a turn is what counts."""
    e = 2 ** 31
    pos = torch.tensor([[0, 1, -1, e - 1, -e, 1_000_003, -77_777_777, 2_000_000_011, 123, 65536, 900_000_000]],
                       dtype=torch.int32)
    check(make(1, 4, pos.shape[1], 2, 32, seed=5), pos, kind, theta=theta)


def test_rows_of_any_size():
    """Zero rows (1 / sqrt(eps) instead of a norm), rows far smaller and far larger than 1, a large eps."""
    x = make(1, 6, 40, 2, 32, seed=9)
    for t in x[:2]:
        t[0, 0] = 0.0
        t[0, 1] *= 1e-4
        t[0, 2] *= 1e4
        t[0, 3, :, ::2] = 0.0
    check(x, None, "half")
    check(x, None, "half", eps=0.5)


@pytest.mark.parametrize("D", [16, 32])
def test_views_give_the_same_bits(D):
    """Any valid layout on either side: bitwise what contiguous copies give; a
    gradient written over the incoming one; nothing else of the rows is touched."""
    B, No, N, H = 2, 5, 37, 3
    q, k, dqo, dko, wq, wk = make(B, No, N, H, D, seed=2, rows="pairs")
    pos = torch.arange(B * N, dtype=torch.int32, device="cuda").view(B, N) * 3
    want = T.triattn_qk_norm_fwd(q.contiguous(), k.contiguous(), wq, wk, pos)
    grads = T.triattn_qk_norm_bwd(q.contiguous(), k.contiguous(), wq, wk, dqo.contiguous(), dko.contiguous(), pos)
    ld = 2 * H * D + 24
    rows = torch.full((B, No, N, ld), 7.0, dtype=torch.bfloat16, device="cuda")
    out = tuple(heads_in_rows(rows, c, H, D) for c in (8, 16 + H * D))
    got = T.triattn_qk_norm_fwd(q, k, wq, wk, pos, out=out)
    assert got[0] is out[0] and all(torch.equal(a, b) for a, b in zip(got, want))
    for c0, c1 in ((0, 8), (8 + H * D, 16 + H * D), (16 + 2 * H * D, ld)):
        assert (rows[..., c0:c1] == 7.0).all()
    mixed = T.triattn_qk_norm_fwd(q, k, wq, wk, pos)
    assert mixed[0].is_contiguous() and all(torch.equal(a, b) for a, b in zip(mixed, want))
    got = T.triattn_qk_norm_bwd(q, k, wq, wk, dqo, dko, pos)
    # another order of the rows in memory: the same dq, dk; dw is added in another order
    assert all(torch.equal(a, b) for a, b in zip(got[:2], grads[:2]))
    again = T.triattn_qk_norm_bwd(q, k, wq, wk, dqo, dko, pos)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    over = T.triattn_qk_norm_bwd(q, k, wq, wk, dqo, dko, pos, out=(dqo, dko) + tuple(map(torch.empty_like, (wq, wk))))
    assert all(torch.equal(a, b) for a, b in zip(over, got))


def test_slices_past_32_bits():
    """Slices whose offsets pass 2^31 elements: a layout with a wide slice stride over one large buffer."""
    B, No, N, H, D = 1, 3, 4, 2, 32
    stride = (1 << 30) + 64
    buf = torch.empty(2 * stride + 2 * H * N * D, dtype=torch.bfloat16, device="cuda")
    q = buf.as_strided((B, No, H, N, D), (No * stride, stride, D, 2 * H * D, 1))
    k = buf.as_strided((B, No, H, N, D), (No * stride, stride, D, 2 * H * D, 1), H * D)
    x = make(B, No, N, H, D, seed=1)
    q.copy_(x[0])
    k.copy_(x[1])
    want = T.triattn_qk_norm_fwd(x[0], x[1], x[4], x[5])
    assert all(torch.equal(a, b) for a, b in zip(T.triattn_qk_norm_fwd(q, k, x[4], x[5]), want))


def test_many_slices_and_a_long_row():
    """More slices than tokens, and a slice longer than a wave of blocks."""
    check(make(1, 700, 3, 2, 32, seed=1), None, "half")
    check(make(1, 2, 9000, 3, 16, seed=2), None, "interleaved")


def test_streams_graphs_and_two_at_once():
    x = make(1, 64, 64, 4, 32, seed=3)
    q, k, dqo, dko, wq, wk = x
    want = T.triattn_qk_norm_fwd(q, k, wq, wk) + T.triattn_qk_norm_bwd(q, k, wq, wk, dqo, dko)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [T.triattn_qk_norm_fwd(q, k, wq, wk, stream=s) + T.triattn_qk_norm_bwd(q, k, wq, wk, dqo, dko, stream=s)
           for s in streams]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = T.triattn_qk_norm_fwd(q, k, wq, wk) + T.triattn_qk_norm_bwd(q, k, wq, wk, dqo, dko)
    for t in out:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
