"""GPU tests of the learned relative position bias, against the FP64 oracle.

Tolerances.  Forward: one FP32 addition (2^-24 of the sum of absolute values) and
one rounding to BF16 (2^-8 of the value); without a base only the rounding.  The
table's gradient adds the values of a bucket.  Planes: a thread's chain of FP32
additions is at most the rows that it walks, each the sum of eight, then 8 warps
and 32 lanes, then FP64; with at most 16384 rows (here 2100): (N + 64) 2^-24 of
the sum of absolute values.  Pairs: the tensor cores add products of 16 to an FP32
accumulator, cut off instead of rounded (2^-23 each), at most 4 x 128 times before
the accumulators are joined in FP32 and then FP64: (512 + 16) 2^-23 of the sum of
absolute values."""
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


def ids(B, N, seed, how):
    """positions, chains [B, N] int32 (CPU)."""
    g = torch.Generator().manual_seed(seed)
    if how == "none":
        return None, None
    if how == "residues":  # chains one after the other, numbered anew, with a gap
        t = torch.arange(N)
        chain = (t * 3) // N
        pos = t - torch.searchsorted(chain, chain) + 5 * (t % 7 == 6)
        return pos.expand(B, N).to(torch.int32).contiguous(), chain.expand(B, N).to(torch.int32).contiguous()
    if how == "atoms":  # many tokens of one residue, no chains
        return torch.randint(0, 1 + N // 6, (B, N), generator=g, dtype=torch.int32), None
    assert how == "wild"  # no order at all, the ends of 32 bits among them
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (B, N), generator=g, dtype=torch.int64)
    pos = torch.where(torch.rand(B, N, generator=g) < 0.5, pos % 40, pos).to(torch.int32)
    return pos, torch.randint(-2, 2, (B, N), generator=g, dtype=torch.int32)


def make(layout, B, N, F, K, seed):
    g = torch.Generator().manual_seed(seed)
    shape = (B, F, N, N) if layout == "heads" else (B, N, N, F)
    return (torch.randn(K, F, generator=g).cuda(), torch.randn(shape, generator=g).to(torch.bfloat16).cuda(),
            torch.randn(shape, generator=g).cuda())


def check(layout, B, N, F, K, how, kind, R, seed=0, fp32=False, with_base=True):
    pos, chain = ids(B, N, seed, how)
    K += 0 if chain is None else 1
    table, base, d = make(layout, B, N, F, K, seed)
    d = d if fp32 else d.to(torch.bfloat16)
    dev = [None if t is None else t.cuda() for t in (pos, chain)]
    rule = dict(layout=layout, kind=kind, max_distance=R)
    out = T.triattn_relpos_fwd(table, base if with_base else None, *dev, **rule,
                               **({} if with_base else {"out": torch.empty_like(base)}))
    dt = T.triattn_relpos_bwd(d, K, *dev, **rule)
    assert T.device_status() == T.OK
    k = CI.buckets(B, N, K, *(None if t is None else t.numpy() for t in (pos, chain)), kind, R)
    ref = CI.relpos(table, base if with_base else None, k, layout)
    size = np.abs(CI.relpos(np.abs(cpu64(table)), np.abs(cpu64(base)) if with_base else None, k, layout))
    err = np.abs(cpu64(out) - ref)
    assert (err <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -24 * size if with_base else 0.0)).all(), err.max()
    want, total = CI.relpos_bwd(d, k, K, layout), CI.relpos_bwd(d.abs(), k, K, layout)
    tol = (N + 64) * 2.0 ** -24 if layout == "heads" else 528 * 2.0 ** -23
    err = np.abs(cpu64(dt) - want)
    assert (err <= tol * total).all(), float((err / np.maximum(total, 1e-300)).max())
    again = T.triattn_relpos_bwd(d, K, *dev, **rule)
    assert torch.equal(dt, again)
    return out, dt


RULES = [("clip", 65, 32), ("clip", 3, 1), ("clip", 255, 127), ("log", 32, 128), ("log", 4, 2), ("log", 254, 1024),
         ("log", 6, 1000)]
HOW = ["none", "residues", "atoms", "wild"]


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("B,N,F", [(1, 1, 1), (1, 7, 2), (2, 8, 5), (1, 9, 1), (3, 61, 3), (1, 64, 4), (2, 131, 8),
                                   (1, 200, 16), (1, 257, 2)])
def test_planes(B, N, F, how, fp32):
    for i, (kind, K, R) in enumerate(RULES[:4]):
        check("heads", B, N, F, K, how, kind, R, seed=N + i, fp32=fp32, with_base=i != 1)


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("B,N,F", [(1, 1, 8), (1, 7, 32), (2, 8, 64), (1, 9, 96), (3, 33, 128), (1, 64, 136),
                                   (2, 40, 256), (1, 75, 200), (1, 131, 128)])
def test_pairs(B, N, F, how):
    for i, (kind, K, R) in enumerate(RULES[:4]):
        check("pairs", B, N, F, K, how, kind, R, seed=N + i, with_base=i != 1)


@pytest.mark.parametrize("layout,F", [("heads", 3), ("pairs", 40)])
@pytest.mark.parametrize("rule", RULES, ids=lambda r: f"{r[0]}{r[1]}to{r[2]}")
def test_rules(rule, layout, F):
    for how in ("atoms", "wild"):
        check(layout, 1, 150, F, *rule[1:2], how, rule[0], rule[2], seed=1)
    # every distance of the rule and beyond, next to every border
    N = 1100
    pos = torch.arange(N, dtype=torch.int32)[None].cuda()
    table = torch.arange(rule[1], dtype=torch.float32, device="cuda")[:, None].expand(-1, 8).contiguous()
    out = T.triattn_relpos_fwd(table, None, pos, layout=layout, kind=rule[0], max_distance=rule[2])
    got = (out[0, 0] if layout == "heads" else out[0, :, :, 0]).float().cpu()
    want = torch.tensor([CI.bucket_of(d, rule[0], rule[1], rule[2]) for d in range(-N + 1, N)]).float()
    i = torch.arange(N)
    assert torch.equal(got, want[(i[:, None] - i[None, :]) + N - 1])  # up to 255: exact in BF16


@pytest.mark.parametrize("N,F,fp32", [(2056, 2, False), (2057, 1, True), (2100, 1, False)])
def test_rows_longer_than_a_block(N, F, fp32):
    check("heads", 1, N, F, 65, "residues", "clip", 32, fp32=fp32)


def test_many_pairs():
    """Runs of pairs at their longest: more than one wave of blocks."""
    N, F, K = 1200, 32, 65
    pos, chain = (t.cuda() for t in ids(1, N, 0, "residues"))
    d = torch.ones(1, N, N, F, dtype=torch.bfloat16, device="cuda")
    dt = T.triattn_relpos_bwd(d, K + 1, pos, chain, layout="pairs")
    k = CI.buckets(1, N, K + 1, pos.cpu().numpy(), chain.cpu().numpy())
    want = np.bincount(k.ravel(), minlength=K + 1)  # whole numbers below 2^24: every sum is exact
    assert (cpu64(dt) == want[:, None]).all()


def test_in_place_and_neighbours():
    """out may be base; what lies before and behind it stays."""
    for layout, N, F in (("heads", 33, 3), ("heads", 40, 3), ("pairs", 33, 16)):
        table, base, _ = make(layout, 2, N, F, 65, 1)
        n = base.numel()
        buf = torch.full((n + 64,), 3.0, dtype=torch.bfloat16, device="cuda")
        view = buf[32:32 + n].view(base.shape)
        view.copy_(base)
        want = T.triattn_relpos_fwd(table, base, layout=layout)
        got = T.triattn_relpos_fwd(table, view, layout=layout, out=view)
        assert got is view and torch.equal(got, want)
        assert (buf[:32] == 3.0).all() and (buf[32 + n:] == 3.0).all()


def test_the_core_takes_it():
    """The bias that the core is given and the gradient that it gives back, BF16 and FP32."""
    from protein_folding_triangle_gb300 import synthetic as S
    w = S.custom(1, 72, 2, 16)
    x = {k: (None if v is None else v.cuda()) for k, v in S.make_inputs(w, 3).items()}
    table = torch.randn(65, 2, device="cuda")
    bias = T.triattn_relpos_fwd(table, x["bias"])
    o, lse, resid = T.tri_attn_fwd(x["q"], x["k"], x["v"], bias, x["mask"])
    args = (x["q"], x["k"], x["v"], bias, x["mask"], o, resid, lse, x["do"])
    d16 = T.triattn_relpos_bwd(T.tri_attn_bwd(*args)[3], 65)
    d32 = T.triattn_relpos_bwd(T.tri_attn_bwd(*args, dbias_fp32=True)[3], 65)
    # the core's rows of dbias sum to zero, so the table's rows nearly do: the two differ by BF16's rounding of dbias
    total = T.triattn_relpos_bwd(T.tri_attn_bwd(*args)[3].abs(), 65)
    assert ((d16 - d32).abs() <= 2.0 ** -8 * total * (1 + 2.0 ** -7)).all()


def test_streams_graphs_and_two_at_once():
    for layout, F, N in (("heads", 4, 96), ("heads", 3, 77), ("pairs", 64, 96)):
        pos, chain = (t.cuda() for t in ids(1, N, 0, "residues"))
        table, base, d = make(layout, 1, N, F, 66, 0)
        d = d.to(torch.bfloat16)

        def run(**kw):
            return (T.triattn_relpos_fwd(table, base, pos, chain, layout=layout, **kw),
                    T.triattn_relpos_bwd(d, 66, pos, chain, layout=layout, **kw))

        want = run()
        torch.cuda.synchronize()
        got = [run(stream=s) for s in (torch.cuda.Stream(), torch.cuda.Stream())]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(run())
        for t in got[-1]:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for g in got:
            assert all(torch.equal(a, b) for a, b in zip(g, want))
