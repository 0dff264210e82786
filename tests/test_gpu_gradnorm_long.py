"""The gradient norm and clipping of lists whose blocks walk many whole chunks
(32 KB each, 608 blocks): dense values, against FP64 on the device.

Tolerances: a block of n chunks adds at most 8 min(n, 64) squares per chain, one
rounding each, joins the chains (3), adds n / 64 such sums to its total, and the
block's threads pairwise (8); the FP64 sums above add nothing, the root halves it
and rounds once.  All terms are positive, so the roundings add up at worst:
norm_tol(n) = (8 min(n, 64) + n / 64 + 13) 2^-25.  A scaled element carries that,
the coefficient's roundings (2^-22) and its own, half a step."""
import math

import pytest
import torch

from protein_folding_triangle_gb300 import triattn as T

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
CHUNK, BLOCKS = 32768, 608


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from protein_folding_triangle_gb300 import build
    build.build()
    T.load()


def norm_tol(nbytes):
    n = nbytes / CHUNK / BLOCKS + 2
    return (8 * min(n, 64) + n / 64 + 13) * 2.0 ** -25


def dense(sizes, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.empty(n, device="cuda").normal_(0.0, 0.01, generator=g).to(dt) for n, dt in sizes]


def exact(ts, p):
    if p == math.inf:
        return max(float(t.abs().max()) for t in ts)
    return math.sqrt(math.fsum(float(t.double().square().sum()) for t in ts))


LISTS = {
    "60 M bf16": [(60_000_001, torch.bfloat16)],
    "40 M fp32": [(40_000_003, torch.float32)],
    "mixed": [(30_000_001, torch.bfloat16), (20_000_003, torch.float32), (11, torch.float32),
              (25_000_007, torch.bfloat16)],
    "1.4 GB bf16": [(700_000_001, torch.bfloat16)],  # 70 chunks per block: past the first 64
    "120 tensors": [(500_000 + 1009 * i, torch.bfloat16 if i % 3 else torch.float32) for i in range(120)],
}


@pytest.mark.parametrize("p", [2.0, math.inf])
@pytest.mark.parametrize("name", LISTS)
def test_dense_lists(name, p):
    ts = dense(LISTS[name], len(name))
    want = exact(ts, p)
    nt = norm_tol(sum(t.numel() * t.element_size() for t in ts)) if p == 2.0 else 0.0
    limit = 0.3 * want
    coef = limit / (want + 1e-6)
    outs = [torch.full_like(t, 9.0) for t in ts]
    alone = T.triattn_grad_norm(ts, p)
    norm = T.triattn_clip_grad_norm(ts, limit, p, out=outs)
    kept = [t.clone() for t in ts]
    inplace = T.triattn_clip_grad_norm(ts, limit, p)
    torch.cuda.synchronize()
    assert torch.equal(alone, norm) and torch.equal(norm, inplace)
    assert abs(float(norm) - want) <= nt * want + 2.0 ** -24 * want
    for t, o, k in zip(ts, outs, kept):
        assert torch.equal(t, o)
        bound = HALF[t.dtype] * (1 + 2.0 ** -10) + nt + 2.0 ** -22
        for i in range(0, t.numel(), 1 << 27):
            ref = k[i:i + (1 << 27)].double() * coef
            assert bool(((o[i:i + (1 << 27)].double() - ref).abs() <= ref.abs() * bound + 2.0 ** -133).all())


def test_sums_do_not_lose_what_is_small():
    """34 GB of FP32 elements whose square is 1 + 2^-12: where a single FP32 sum of
    13,800 squares per chain stands above 4096 it would drop the 2^-12 of every term."""
    n = (1 << 33) + 5
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 34 GB")
    v = torch.tensor(math.sqrt(1.0 + 2.0 ** -12 - 2.0 ** -20), dtype=torch.float32)
    t = torch.full((n,), float(v), device="cuda")
    want = float(v.double()) * math.sqrt(n)
    got = float(T.triattn_grad_norm([t]))
    del t
    assert abs(got - want) <= (norm_tol(4 * n) + 2.0 ** -24) * want, got / want - 1
