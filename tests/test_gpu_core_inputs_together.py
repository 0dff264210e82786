"""GPU tests of the norms, the position bias and the orthogonalisation as a model
uses them: a projection's rows -> norms with rotation -> bias planes with the
position bias -> the core -> gradients through autograd -> clipping ->
orthogonalised updates, against the same in FP64.

Tolerances, relative RMS.  The reference takes the rounded projection.  q and k are
rounded to BF16 once, 2^-8 at most and 1.6e-3 RMS of a value, and so is the bias: a
logit of two rows of norm about sqrt(D), scaled by 1/sqrt(D), is off by 1.6e-3
sqrt(2) + 1.6e-3 of bias values of about one, 2.8e-3 RMS, and the probabilities by as
much of themselves.  The core's own bars are 4e-3 for the output and 1e-2 for its
gradients; 2.8e-3 + 4e-3 is within 1e-2 for the output.  A gradient takes the
probabilities' error twice (P and dP - D), the core's, and BF16 roundings of dq, dk,
dbias, of the norms' gradients and of the projection's, 1.6e-3 each: root of the sum
of squares 1.2e-2, within 2e-2.
"""
import numpy as np
import pytest
import torch

from oracle import core_inputs as CI
from oracle import orthogonalize as OR
from parity_utils import cpu64
from protein_folding_triangle_gb300 import layers
from protein_folding_triangle_gb300 import triattn as T

pytestmark = pytest.mark.gpu

OUT, GRAD = 1e-2, 2e-2


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from protein_folding_triangle_gb300 import build
    build.build()
    T.load()


class Attention(torch.nn.Module):
    def __init__(self, C, H, D, rotary, shared, kind):
        super().__init__()
        self.H, self.D = H, D
        self.w = torch.nn.Parameter((torch.randn(C, 3 * H * D, device="cuda") / C ** 0.5).bfloat16())
        self.norm = layers.QKNorm(H, D, rotary, shared=shared, device="cuda")
        self.rel = layers.RelativePosition(H, kind=kind, max_distance=16, buckets=None if kind == "clip" else 16,
                                           chains=True, device="cuda")
        with torch.no_grad():
            for p in (self.norm.w_q, self.norm.w_k):
                p.copy_(1.0 + 0.2 * torch.randn_like(p))
            self.rel.table.copy_(0.5 * torch.randn_like(self.rel.table))

    def heads(self, y):
        return y.unflatten(-1, (3, self.H, self.D)).permute(3, 0, 1, 4, 2, 5)

    def forward(self, x, base, mask, positions, chains):
        q, k, v = self.heads(x @ self.w)
        q, k = self.norm(q, k, positions)
        return T.triangle_attention(q, k, v.contiguous(), self.rel(base, positions, chains), mask)


def draw(B, No, N, C, H, D, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, No, N, C, generator=g).bfloat16().cuda()
    base = torch.randn(B, H, N, N, generator=g).bfloat16().cuda().requires_grad_()
    mask = torch.where(torch.rand(B, No, N, generator=g) < 0.1, float("-inf"), 0.0).bfloat16()
    mask[..., 0] = 0.0
    chains = (torch.arange(N) >= N // 2 + 3).int().repeat(B, 1)
    positions = (torch.arange(N).repeat(B, 1) - chains * (N // 2 + 3)).int()
    d = torch.randn(B, No, H, N, D, generator=g).bfloat16().cuda()
    return x, base, mask.cuda(), positions.cuda(), chains.cuda(), d


def rel(got, ref):
    return float(np.linalg.norm(cpu64(got) - ref) / np.linalg.norm(ref))


def reference(m, x, base, mask, positions, chains, d):
    """Output and gradients, FP64, by the formulas and from the rounded projection."""
    q, k, v = (cpu64(t) for t in m.heads((x @ m.w).detach()))
    args = dict(positions=positions.cpu().numpy(), kind=m.norm.rotary)
    wq, wk = (cpu64(p) for p in (m.norm.w_q, m.norm.w_k))
    qn, kn = CI.qk_norm(q, wq, **args)["y"], CI.qk_norm(k, wk, **args)["y"]
    K = m.rel.table.shape[0]
    bk = CI.buckets(x.shape[0], x.shape[2], K, args["positions"], chains.cpu().numpy(), m.rel.kind, m.rel.max_distance)
    bias = CI.relpos(cpu64(m.rel.table), cpu64(base), bk, "heads")
    s = qn @ kn.swapaxes(-1, -2) / np.sqrt(m.D) + bias[:, None] + cpu64(mask)[:, :, None, None]
    p = np.exp(s - s.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    o, do = p @ v, cpu64(d)
    dp = do @ v.swapaxes(-1, -2)
    ds = p * (dp - (p * dp).sum(-1, keepdims=True))
    gq = CI.qk_norm(q, wq, dy=ds @ kn / np.sqrt(m.D), **args)
    gk = CI.qk_norm(k, wk, dy=ds.swapaxes(-1, -2) @ qn / np.sqrt(m.D), **args)
    dy = np.stack([gq["dx"], gk["dx"], p.swapaxes(-1, -2) @ do])  # [3, B, N_o, H, N, D]
    dy = dy.transpose(1, 2, 4, 0, 3, 5).reshape(x.shape[:3] + (-1,))
    db = ds.sum(1)
    return {"o": o, "w": np.einsum("bonc,bonf->cf", cpu64(x), dy), "base": db, "w_q": gq["dw"], "w_k": gk["dw"],
            "table": CI.relpos_bwd(db, bk, K, "heads")}


@pytest.mark.parametrize("B,No,N,H,D,rotary,shared,kind",
                         [(1, 40, 40, 2, 16, "half", False, "clip"), (2, 5, 131, 4, 32, "interleaved", True, "log"),
                          (1, 3, 200, 2, 32, "none", False, "clip")], ids=["40", "131", "200"])
def test_a_training_step(B, No, N, H, D, rotary, shared, kind):
    torch.manual_seed(N)
    m = Attention(96, H, D, rotary, shared, kind)
    x, base, mask, positions, chains, d = draw(B, No, N, 96, H, D, seed=N)
    o = m(x, base, mask, positions, chains)
    o.backward(d)
    ref = reference(m, x, base, mask, positions, chains, d)
    assert T.device_status() == T.OK
    assert rel(o, ref["o"]) <= OUT
    got = {"w": m.w.grad, "base": base.grad, "w_q": m.norm.w_q.grad, "w_k": m.norm.w_k.grad, "table": m.rel.table.grad}
    for name, g in got.items():
        assert rel(g, ref[name]) <= GRAD, name
    # the update: clipped, then the matrices (the BF16 projection, FP32 weights and table) orthogonalised
    layers.clip_grad_norm_(m.parameters(), 1e-2)
    clipped = {n: p.grad.clone() for n, p in m.named_parameters()}
    norm = np.sqrt(sum((cpu64(g) ** 2).sum() for g in clipped.values()))
    assert abs(norm / 1e-2 - 1.0) <= 2.0 ** -8
    layers.orthogonalize_grads_(m.parameters())
    for n, p in m.named_parameters():
        if p.dim() == 2:
            want = OR.orthogonalize(clipped[n])
            # the result's rounding and its products, as for the operator alone
            assert rel(p.grad, want) <= 2.0 ** -8 + 1e-3, n
        else:
            assert torch.equal(p.grad, clipped[n])


def test_a_captured_step_replays():
    """Forward, backward, clipping and orthogonalisation in one graph: on each
    replay's inputs the bits of the eager step."""
    torch.manual_seed(3)
    m = Attention(64, 2, 32, "half", False, "clip")
    inputs = [draw(1, 16, 70, 64, 2, 32, seed=s) for s in (5, 6)]

    def step(x, base, mask, positions, chains, d):
        m.zero_grad(set_to_none=False)
        o = m(x, base, mask, positions, chains)
        o.backward(d)
        norm = layers.clip_grad_norm_(m.parameters(), 1e-2)
        layers.orthogonalize_grads_(m.parameters())
        return o.detach(), norm

    want = []
    for i in inputs:
        o, norm = step(*i)
        want.append([o.clone(), norm.clone()] + [p.grad.clone() for p in m.parameters()])
        del o
    static = [t.clone().detach().requires_grad_(t.requires_grad) for t in inputs[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.zero_grad()
        step(*static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, norm = step(*static)
    for i in (1, 0, 1):
        with torch.no_grad():
            for a, b in zip(static, inputs[i]):
                a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert T.device_status() == T.OK
        for a, b in zip([o, norm] + [p.grad for p in m.parameters()], want[i]):
            assert torch.equal(a, b)


def test_bias_alone_and_pairs():
    """Without a base; as pair features in front of an autograd path of torch's;
    gradients that arrive expanded or transposed; an output that nothing uses."""
    torch.manual_seed(4)
    pos = torch.randint(-50, 50, (2, 37), dtype=torch.int32, device="cuda")
    alone = layers.RelativePosition(8, "pairs", max_distance=8, device="cuda")
    z = torch.randn(2, 37, 37, 8, device="cuda").bfloat16().requires_grad_()
    with torch.no_grad():
        alone.table.copy_(torch.randn_like(alone.table))
    a, b = alone(positions=pos), alone(z, pos)
    assert torch.equal(a, alone.table.bfloat16()[(pos[:, :, None] - pos[:, None, :]).clamp(-8, 8).long() + 8])
    g = torch.randn(2, 37, 37, 8, device="cuda").bfloat16()
    b.transpose(1, 2).backward(g)
    assert torch.equal(z.grad, g.transpose(1, 2))
    k = CI.buckets(2, 37, 17, pos.cpu().numpy(), None, "clip", 8)
    want = CI.relpos_bwd(cpu64(g).swapaxes(1, 2), k, 17, "pairs")
    # FP32 sums of BF16 values, 2^-20 of the sum of their sizes at most here
    assert np.all(np.abs(cpu64(alone.table.grad) - want)
                  <= 2.0 ** -20 * CI.relpos_bwd(np.abs(cpu64(g)).swapaxes(1, 2), k, 17, "pairs") + 1e-30)
    alone.zero_grad()
    a.sum().backward()  # an expanded gradient: the buckets' counts
    count = np.bincount(k.ravel(), minlength=17).astype(np.float64)
    assert np.array_equal(cpu64(alone.table.grad), np.repeat(count[:, None], 8, 1))

    norm = layers.QKNorm(2, 16, device="cuda")
    q = torch.randn(1, 3, 2, 9, 16, device="cuda").bfloat16().requires_grad_()
    k = torch.randn(1, 3, 9, 2, 16, device="cuda").bfloat16().requires_grad_()
    qn, kn = norm(q, k.transpose(2, 3))  # of two layouts
    ref = T.triattn_qk_norm_fwd(q.detach(), k.detach().transpose(2, 3).contiguous(), norm.w_q, norm.w_k)
    assert torch.equal(qn, ref[0]) and torch.equal(kn, ref[1])
    views = torch.randn(2, 1, 9, 3, 2, 17, device="cuda").bfloat16()[..., :16]  # not rows that a call takes: copied
    a, b = norm(*views.transpose(2, 4).transpose(2, 3))
    ref = T.triattn_qk_norm_fwd(*(t.contiguous() for t in views.transpose(2, 4).transpose(2, 3)), norm.w_q, norm.w_k)
    assert torch.equal(a, ref[0]) and torch.equal(b, ref[1])
    one = torch.randn(1, 1, 2, 9, 16, device="cuda").bfloat16().requires_grad_()
    a, b = norm(one.expand(1, 3, 2, 9, 16), one.expand(1, 3, 2, 9, 16))  # broadcast over slices
    (a.float().sum() + b.float().sum()).backward()
    g = T.triattn_qk_norm_bwd(*(one.detach().expand(1, 3, 2, 9, 16).contiguous() for _ in range(2)), norm.w_q, norm.w_k,
                              torch.ones_like(a), torch.ones_like(b))
    # the slices' and q's and k's gradients, alike: 6 values added in BF16, 2^-8 of the running sum each
    want = cpu64(g[0]).sum(1, keepdims=True) + cpu64(g[1]).sum(1, keepdims=True)
    assert np.all(np.abs(cpu64(one.grad) - want) <= 6 * 2.0 ** -8 * np.abs(want) + 1e-30)
    qn.backward(torch.randn_like(qn))
    assert not bool(k.grad.any()) and bool(q.grad.any())


def test_refusals_of_the_modules():
    with pytest.raises(ValueError):
        layers.QKNorm(2, 16, "quarter")
    for bad in (dict(layout="rows"), dict(kind="linear"), dict(kind="log")):
        with pytest.raises(ValueError):
            layers.RelativePosition(4, **bad)
    base = torch.zeros(1, 4, 9, 9, dtype=torch.bfloat16, device="cuda")
    chains = torch.zeros(1, 9, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        layers.RelativePosition(4, device="cuda")(base, chains=chains)
    with pytest.raises(ValueError):
        layers.RelativePosition(4, chains=True, device="cuda")(base)
    with pytest.raises(ValueError):
        layers.RelativePosition(4, device="cuda")()
    with pytest.raises(T.TriAttnError):  # heads of 64 features, which the core has not either
        layers.QKNorm(2, 64, device="cuda")(*torch.zeros(2, 1, 3, 2, 9, 64, dtype=torch.bfloat16, device="cuda"))
    p = torch.nn.Parameter(torch.zeros(4, device="cuda"))
    layers.orthogonalize_grads_([p])  # nothing to do
    p.grad = torch.ones(4, device="cuda")
    layers.orthogonalize_grads_(p)
    assert bool((p.grad == 1).all())
