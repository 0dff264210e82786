"""The global gradient norm and clipping against FP64.

Tolerances: a thread's FP32 chain of k squares is off by at most k + 1
roundings of 2^-24 relative (all terms positive); at these sizes k <= 64, the
FP64 sums above it add nothing, and the root halves it: NORM_TOL = 2^-18.  A
scaled element carries the coefficient's error and its own rounding:
NORM_TOL + 2^-22 and half a step (2^-8 BF16, 2^-24 FP32)."""
import math

import pytest
import torch

from oracle import transition as TR
from protein_folding_triangle_gb300 import layers
from protein_folding_triangle_gb300 import synthetic as S
from protein_folding_triangle_gb300 import triattn as T

pytestmark = pytest.mark.gpu

NORM_TOL = 2.0 ** -18
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
KIND = {2.0: "l2", math.inf: "max"}
B, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from protein_folding_triangle_gb300 import build
    build.build()
    T.load()


def make(sizes, seed=0, scale=0.1):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * scale).to(dt).cuda() for n, dt in sizes]


def check(ts, limit, p, out=None):
    want, clipped = TR.clip([t.double().cpu().numpy() for t in ts], limit, KIND[p])
    alone = T.triattn_grad_norm(ts, p)
    before = [t.clone() for t in ts]
    norm = T.triattn_clip_grad_norm(ts, limit, p, out=out)
    torch.cuda.synchronize()
    assert norm.dtype == F and norm.dim() == 0 and torch.equal(norm, alone)
    assert abs(float(norm) - want) <= NORM_TOL * want
    for t, b, o, c in zip(ts, before, out or ts, clipped):
        ref = torch.from_numpy(c).cuda().reshape(b.shape)
        bound = ref.abs() * (HALF[b.dtype] * (1 + 2.0 ** -10) + NORM_TOL + 2.0 ** -22) + 2.0 ** -133
        assert bool(((o.double() - ref).abs() <= bound).all())
        if out is not None:
            assert torch.equal(t, b)
        elif limit > 2 * want:
            assert torch.equal(t, b)
    return norm


LISTS = {
    "one element": [(1, F)],
    "one bf16": [(1, B)],
    "ragged": [(n, B if n % 2 else F) for n in (1, 2, 3, 5, 7, 8, 9, 15, 16, 17, 31, 33, 1000, 8191, 8192, 8193, 0, 16385)],
    "two chunks and a bit": [(16384 * 2 + 5, B), (8192 * 2 + 3, F)],
    "block": [(128, F), (128, F), (128 * 1024, B), (512 * 128, B)],
    "large": [(3_000_001, B), (1_500_007, F)],
    "over the small table": [(37 + i, B if i % 3 else F) for i in range(97)],
    "over the large table": [(1 + i % 70, B if i % 2 else F) for i in range(2500)],
}


@pytest.mark.parametrize("p", [2.0, math.inf])
@pytest.mark.parametrize("name", LISTS)
def test_matches_oracle(name, p):
    ts = make(LISTS[name], seed=len(name))
    want, _ = TR.clip([t.double().cpu().numpy() for t in ts], 1.0, KIND[p])
    check([t.clone() for t in ts], 0.37 * want, p)
    check([t.clone() for t in ts], 100.0 * want, p)
    check(ts, 0.37 * want, p, out=[torch.full_like(t, 9.0) for t in ts])
    check(ts, 100.0 * want, p, out=[torch.full_like(t, 9.0) for t in ts])


@pytest.mark.parametrize("dt", [B, F])
def test_views_of_a_bucket_at_every_alignment(dt):
    """Neighbouring views of one buffer at odd offsets: each is scaled alone,
    what lies between them stays, also into a destination aligned otherwise."""
    flat = make([(200_000, dt)])[0]
    cuts = [1, 2, 4, 9, 40, 77, 1000, 16401, 17000, 50_001, 120_000, 199_999]
    ts = [flat[a:b - 1] for a, b in zip(cuts, cuts[1:]) if b - 1 > a]
    gaps = torch.ones(200_000, dtype=torch.bool)
    for a, b in zip(cuts, cuts[1:]):
        gaps[a:b - 1] = False
    keep = flat[gaps.cuda()].clone()
    into = torch.full((200_100,), 5.0, dtype=dt, device="cuda")
    for shift in (0, 1, 3, 8):
        into.fill_(5.0)
        outs = [into[shift + a:shift + b - 1] for a, b in zip(cuts, cuts[1:]) if b - 1 > a]
        check(ts, 0.1, 2.0, out=outs)
        mask = torch.ones(200_100, dtype=torch.bool)
        for o, (a, b) in zip(range(99), zip(cuts, cuts[1:])):
            mask[shift + a:shift + b - 1] = False
        assert bool((into[mask.cuda()] == 5.0).all())
    check(ts, 0.1, 2.0)
    assert torch.equal(flat[gaps.cuda()], keep)


def test_strides():
    base = make([(60 * 70, F)])[0].view(60, 70)
    check([base.t()], 0.3, 2.0)                                # dense in another order
    check([base[:1, :50]], 0.01, 2.0)
    with pytest.raises(ValueError):
        T.triattn_grad_norm([base[:, ::2]])
    with pytest.raises(ValueError):
        T.triattn_clip_grad_norm([base], 1.0, out=[base.t().clone().t()[:, :69]])


def test_nothing_to_clip():
    assert float(T.triattn_grad_norm([])) == 0.0 and float(T.triattn_clip_grad_norm([], 1.0)) == 0.0
    empty = torch.empty(0, device="cuda")
    assert float(T.triattn_clip_grad_norm([empty], 1.0)) == 0.0
    zero = torch.zeros(100, device="cuda")
    assert float(T.triattn_clip_grad_norm([zero], 1.0)) == 0.0 and bool((zero == 0).all())
    t = torch.ones(100, device="cuda")
    T.triattn_clip_grad_norm([t], 0.0)
    assert bool((t == 0).all())


@pytest.mark.parametrize("p", [2.0, math.inf])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_values_that_are_not_finite(p, bad):
    """As torch.nn.utils.clip_grad_norm_: NaN makes everything NaN; an
    infinite norm makes the coefficient 0."""
    for dt in (B, F):
        ts = make([(1000, dt), (50_000, dt)])
        ts[1][777] = bad
        norm = T.triattn_clip_grad_norm(ts, 1.0, p)
        if math.isnan(bad):
            assert math.isnan(float(norm)) and all(bool(t.isnan().all()) for t in ts)
        else:
            assert float(norm) == math.inf and bool((ts[0] == 0).all()) and bool(ts[1][777].isnan())


def test_shared_memory_is_refused():
    t = torch.ones(100, device="cuda")
    for bad in ([t, t], [t, t[99:]], [t[:60], t[59:]]):
        with pytest.raises(T.TriAttnError):
            T.triattn_clip_grad_norm(bad, 1.0)
    with pytest.raises(T.TriAttnError):
        T.triattn_clip_grad_norm([t], 1.0, out=[t])
    assert float(T.triattn_grad_norm([t, t])) == pytest.approx(math.sqrt(200.0), rel=1e-6)  # a norm may read twice
    assert bool((t == 1).all())
    for bad in ([t.half()], [t.double()], [t, t.cpu()], [t.to_sparse()]):
        with pytest.raises(ValueError):
            T.triattn_clip_grad_norm(bad, 1.0)
    with pytest.raises(ValueError):
        T.triattn_clip_grad_norm([t], 1.0, out=[])
    with pytest.raises(T.TriAttnError):
        T.triattn_clip_grad_norm([t], -1.0)


def test_past_32_bits():
    """2^31 + 77 BF16 elements: the last ones count and are scaled."""
    n = (1 << 31) + 77
    t = torch.zeros(n, dtype=B, device="cuda")
    t[-1] = 3.0
    t[-70] = -4.0
    t[12345] = 12.0
    norm = T.triattn_clip_grad_norm([t], 6.5)
    assert float(norm) == 13.0
    assert [float(t[i]) for i in (-1, -70, 12345)] == [1.5, -2.0, 6.0]
    assert int(torch.count_nonzero(t)) == 3


def test_repeatable_graph_and_side_stream():
    ts = make(LISTS["large"] + LISTS["ragged"])
    first = T.triattn_grad_norm(ts)
    for _ in range(3):
        assert torch.equal(T.triattn_grad_norm(ts), first)
    outs = [torch.empty_like(t) for t in ts]
    ref = [torch.empty_like(t) for t in ts]
    T.triattn_clip_grad_norm(ts, 1.0, out=ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    norm = T.triattn_clip_grad_norm(ts, 1.0, out=outs, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(norm, first) and all(torch.equal(a, b) for a, b in zip(outs, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = T.triattn_clip_grad_norm(ts, 1.0, out=outs)
    for t in ts:
        t.mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert float(norm) == pytest.approx(2 * float(first), rel=NORM_TOL)
    for o, r in zip(outs, ref):
        torch.testing.assert_close(o, r, rtol=2.0 ** -7 if o.dtype == B else 2.0 ** -18, atol=1e-30)


def test_a_pair_block_and_its_clipping():
    """The pair block as it is trained: multiplicative update, attention and
    transition with their residual sums, backward, then the gradients clipped
    by their norm.  Against the FP64 oracles in the same order.  Each stage's
    gradients are within 2e-2 of its oracle for the same inputs; the three
    stages' errors and the BF16 residual sums (2^-8 each) add in quadrature
    along the block: sqrt(3) 2e-2 + 2^-8 < 4e-2."""
    import numpy as np
    from oracle import module as MO
    from oracle import trimul as TMO
    N, C, H, D = 40, 64, 2, 16
    xm = S.make_trimul_inputs(1, N, C, 32, seed=2, pad_frac=0.1)
    xa = S.make_module_inputs(1, N, C, H, D, seed=3)
    xt = S.make_transition_inputs((1, N, N), C, 256, seed=4)
    mask = xm["mask"]
    key_mask = torch.where(mask[:, :1].expand(1, N, N) > 0, 0.0, -math.inf).to(B).contiguous()
    mul = layers.TriangleMultiplication(C, 32, "outgoing", device="cuda")
    att = layers.TriangleAttention(C, H, D, device="cuda")
    ffn = layers.Transition(C, 256, device="cuda")
    with torch.no_grad():
        for mod, x in ((mul, xm), (att, xa), (ffn, xt)):
            for n, p in mod.named_parameters():
                p.copy_(x[n])
    z0 = xm["z"].cuda().requires_grad_(True)
    z1 = z0 + mul(z0, mask.cuda())
    z2 = z1 + att(z1, key_mask.cuda())
    z3 = z2 + ffn(z2, mask.cuda())
    d = xm["d_out"]
    z3.backward(d.cuda())
    # the same in FP64
    f = lambda t: t.float().double().numpy()  # noqa: E731
    ma = (xm["ln_in_w"], xm["ln_in_b"], xm["w_p"], xm["ln_out_w"], xm["ln_out_b"], xm["w_o"])
    aa = (xa["ln_w"], xa["ln_b"], xa["w_in"], xa["w_o"])
    ta = (xt["ln_w"], xt["ln_b"], xt["w_in"], xt["w_o"])
    r0 = f(xm["z"])
    r1 = r0 + TMO.fwd(r0, mask, *ma, "outgoing")["out"]
    r2 = r1 + MO.fwd(r1, key_mask, *aa, H, D)["out"]
    gt = TR.run(r2, mask, *ta, d)
    g2 = f(d) + gt["dz"]
    ga = MO.bwd(r1, key_mask, *aa, g2, H, D)
    g1 = g2 + ga["dz"]
    gm = TMO.bwd(r0, mask, *ma, g1, "outgoing")
    want = {"ffn.w_in": gt["dw_in"], "ffn.w_o": gt["dw_o"], "ffn.ln_w": gt["dln_w"], "att.w_in": ga["dw_in"],
            "att.w_o": ga["dw_o"], "mul.w_p": gm["dw_p"], "mul.w_o": gm["dw_o"], "mul.ln_in_w": gm["dln_in_w"]}
    named = {f"{k}.{n}": p for k, m in (("ffn", ffn), ("att", att), ("mul", mul)) for n, p in m.named_parameters()}
    for n, r in want.items():
        e = named[n].grad.double().cpu().numpy() - r
        assert np.sqrt((e * e).mean() / (r * r).mean()) <= 4e-2, n
    before = {n: p.grad.clone() for n, p in named.items()}
    total, clipped = TR.clip([g.double().cpu().numpy() for g in before.values()], 1.0)
    norm = layers.clip_grad_norm_(named.values(), 1.0)
    assert total > 1.0 and abs(float(norm) - total) <= NORM_TOL * total
    for p, c in zip(named.values(), clipped):
        ref = torch.from_numpy(c).cuda()
        assert bool(((p.grad.double() - ref).abs() <= ref.abs() * (HALF[p.dtype] * (1 + 2.0 ** -10) + 2 * NORM_TOL)).all())
    again = T.triattn_grad_norm([p.grad for p in named.values()])
    # every element was rounded once more: at most 2^-8 of each, half of it on the root of the sum of squares
    assert abs(float(again) - 1.0) <= 2.0 ** -8
    layers.clip_grad_norm_([p for p in named.values()] + [torch.nn.Parameter(torch.zeros(3, device="cuda"))], 1.0)
