"""GPU parity of the transition (gated feed-forward block), forward and
backward, through the C ABI, against the FP64 oracle on the same seeded BF16
inputs.

Tolerances (relative RMSE against FP64).  A BF16 rounding is off by at most
2^-8 = 3.9e-3 of the value, so it adds at most that to the relative RMSE of
what is linear in it, and independent ones add in quadrature.  Forward: x
(which enters out through a and through b: at most 2, and at most
max |a act'(a) / act(a)| in place of 1 for a, which for normal a averages below
1.3), a, b, h, out: sqrt(1.3^2 + 1 + 1.3^2 + 1 + 1 + 1) 2^-8 = 1.06e-2 if each
were at its largest; rounding errors spread evenly over half a step have an RMS
of 1 / sqrt(3) of that at most: 6.1e-3.  The hardware tanh adds 2^-11.
TOL_OUT = 8e-3 covers both.  Backward: those of x, a, b again (through act,
act' and both products), then dh, [da | db], dx, and the result, at most twice
the forward's count: 6.1e-3 sqrt(2) < 1e-2 = TOL_GRADS.
"""
import json

import numpy as np
import pytest
import torch

from parity_utils import cpu64, rel_rmse
from oracle import transition as TR
from protein_folding_triangle_gb300 import layers
from protein_folding_triangle_gb300 import synthetic as S
from protein_folding_triangle_gb300 import triattn as T

pytestmark = pytest.mark.gpu

TOL_OUT = 8e-3
TOL_GRADS = 1e-2
NAMES = ("dz", "dln_w", "dln_b", "dw_in", "dw_o")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from protein_folding_triangle_gb300 import build
    build.build()
    T.load()


def to_dev(x):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}


def params(d):
    return d["z"], d["mask"], d["ln_w"], d["ln_b"], d["w_in"], d["w_o"]


def run_gpu(x, kind="silu", **kw):
    d = to_dev(x)
    out = T.triattn_transition_fwd(*params(d), kind)
    grads = T.triattn_transition_bwd(*params(d), d["d_out"], kind, **kw)
    torch.cuda.synchronize()
    assert T.device_status() == T.OK
    return (out,) + tuple(grads)


def run_oracle(x, kind="silu"):
    r = TR.run(*params(x), x["d_out"], kind)
    return [r[k] for k in ("out",) + NAMES]


def check(x, kind="silu", case=None):
    got, ref = run_gpu(x, kind), run_oracle(x, kind)
    errs = {n: rel_rmse(cpu64(g), r) for n, g, r in zip(("out",) + NAMES, got, ref)}
    print(json.dumps({"case": case, "kind": kind, **{k: round(v, 6) for k, v in errs.items()}}))
    assert errs["out"] <= TOL_OUT, errs
    for n in NAMES:
        assert errs[n] <= TOL_GRADS, (n, errs)
    return got


CASES = [
    # (lead, C, H, drop): one row; rows around a tile; every width class; hidden
    # widths that end inside a 64-column block; several examples
    ((1,), 128, 512, 0.0),
    ((1,), 32, 32, 0.0),
    ((3,), 64, 256, 0.0),
    ((127,), 128, 512, 0.3),
    ((128,), 128, 512, 0.0),
    ((129,), 128, 512, 0.0),
    ((257,), 64, 64, 0.3),
    ((1, 40, 40), 128, 512, 0.1),
    ((2, 33, 33), 64, 256, 0.2),
    ((700,), 96, 288, 0.0),
    ((700,), 32, 96, 0.1),
    ((515,), 160, 32, 0.0),
    ((515,), 192, 352, 0.2),
    ((300,), 224, 896, 0.0),
    ((1031,), 256, 1024, 0.1),
    ((193,), 128, 512, 0.2),
    ((255,), 64, 96, 0.0),
    ((256,), 256, 512, 0.2),
    ((5000,), 128, 160, 0.0),
    ((70, 257), 128, 480, 0.1),
]


@pytest.mark.parametrize("case", CASES, ids=["x".join(map(str, c[0])) + f"C{c[1]}H{c[2]}" for c in CASES])
def test_matches_oracle(case):
    lead, C, H, drop = case
    check(S.make_transition_inputs(lead, C, H, seed=C + H + lead[0], drop=drop), case=list(map(str, case)))


@pytest.mark.parametrize("kind", TR.ACTIVATIONS)
@pytest.mark.parametrize("C,H", [(128, 512), (64, 128), (256, 288)])
def test_activations(kind, C, H):
    x = S.make_transition_inputs((900,), C, H, seed=11, drop=0.1)
    x["w_in"] = (x["w_in"].float() * 3.0).to(torch.bfloat16)  # a out to about +-12: both ends of the gate
    x["d_out"][5] = 0.0
    check(x, kind, case=["activations", C, H])


@pytest.mark.parametrize("C,H", [(128, 512), (192, 64)])
def test_masked_rows_may_hold_anything(C, H):
    """A row whose mask is 0: out and dz are exactly 0 and every gradient is
    bitwise what it is with clean rows there, for NaN, infinities and the
    type's lowest value."""
    x = S.make_transition_inputs((513,), C, H, seed=8, drop=0.4)
    clean = run_gpu(x)
    bad = x["mask"] == 0
    rows = bad.nonzero()[:, 0]
    for k, v in enumerate((float("nan"), float("inf"), -float("inf"), torch.finfo(torch.bfloat16).min)):
        x["z"][rows[k::4]] = v
        x["d_out"][rows[(k + 1) % 4::4]] = v
    x["mask"][rows[0]] = -0.0
    got = run_gpu(x)
    assert torch.count_nonzero(got[0][bad.cuda()]) == 0 and torch.count_nonzero(got[1][bad.cuda()]) == 0
    for a, b in zip(clean, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("C,H", [(128, 512), (64, 96)])
def test_every_row_masked(C, H):
    x = S.make_transition_inputs((200,), C, H, seed=8, drop=1.0)
    x["z"].fill_(float("nan"))
    x["d_out"].fill_(float("nan"))
    for t in run_gpu(x):
        assert torch.count_nonzero(t) == 0


def test_mask_values_other_than_one():
    x = S.make_transition_inputs((300,), 128, 256, seed=9, drop=0.2)
    x["mask"] = x["mask"] * torch.tensor([0.5, 1.0, -2.0, 0.25, 3.0]).repeat(60).to(torch.bfloat16)
    check(x, case=["mask values"])


def test_rows_without_spread():
    """Constant rows (variance 0: x = ln_b), tiny and large rows."""
    x = S.make_transition_inputs((64,), 128, 256, seed=10)
    x["z"][0] = 3.0
    x["z"][1] = 0.0
    x["z"][2] = (x["z"][2].float() * 1e-4).to(torch.bfloat16)
    x["z"][3] = (x["z"][3].float() * 1e4).to(torch.bfloat16)
    d = to_dev(x)
    out = T.triattn_transition_fwd(*params(d))
    assert rel_rmse(cpu64(out), TR.run(*params(x))["out"]) <= TOL_OUT
    for r in range(4):  # row by row: a large row does not hide a small one
        assert rel_rmse(cpu64(out[r]), TR.run(*params(x))["out"][r]) <= 4 * TOL_OUT, r


@pytest.mark.parametrize("C,H", [(128, 512), (96, 64), (256, 64)])
def test_rows_far_from_zero(C, H):
    """Rows with a common offset of many standard deviations, and rows whose
    first features lie far from the others.  z is what the oracle has too, so
    only the FP32 statistics differ: the mean of C values within 2^12 standard
    deviations is off by at most log2(C) + 2 half steps of 2^12, 10 * 2^-12 =
    2.5e-3 standard deviations, that of the other rows by far less; both add
    in quadrature to the tolerance of an ordinary row."""
    x = S.make_transition_inputs((640,), C, H, seed=16)
    z = x["z"].float()
    z[0:128] += 8.0
    z[128:256] -= 40.0
    z[256:384, :8] += 300.0  # the features that the one-pass statistics start from
    z[384:512, -8:] -= 300.0
    z[512:576] = 4096.0 + 32.0 * (z[512:576] > 0)  # two values, a step of BF16 apart
    z[576:640] *= 1e-3
    x["z"] = z.to(torch.bfloat16)
    ref = run_oracle(x)
    got = run_gpu(x)
    for i in range(0, 640, 64):
        r = slice(i, i + 64)
        assert rel_rmse(cpu64(got[0][r]), ref[0][r]) <= (TOL_OUT**2 + 2.5e-3**2) ** 0.5, i
        assert rel_rmse(cpu64(got[1][r]), ref[1][r]) <= (TOL_GRADS**2 + 2.5e-3**2) ** 0.5, i


@pytest.mark.parametrize("kind", TR.ACTIVATIONS)
@pytest.mark.parametrize("C,H", [(32, 32), (64, 4096), (96, 288), (128, 512), (160, 64), (192, 352), (224, 96), (256, 1024)])
@pytest.mark.parametrize("M", [1, 2, 5, 48, 191, 192])
def test_forward_of_a_few_rows(C, H, M, kind):
    """Few rows are computed in FP32 and rounded once: an element is off by at
    most half a step of BF16, 2^-8 of its value, and by the FP32 sums' errors, at
    most about (C + H) 2^-24 = 2.6e-4 of the root sum of squares of the terms,
    which is the size of the value itself for these inputs.  Masked rows hold
    NaN."""
    x = S.make_transition_inputs((M,), C, H, seed=C + H + M, drop=0.3 if M > 2 else 0.0)
    ref = TR.run(*params(x), x["d_out"], kind)["out"]
    if x["mask"] is not None:
        x["z"][x["mask"] == 0] = float("nan")
    d = to_dev(x)
    out = T.triattn_transition_fwd(*params(d), kind)
    assert rel_rmse(cpu64(out), ref) <= 2.0**-8 + 3e-4
    if x["mask"] is not None:
        assert torch.count_nonzero(out[d["mask"] == 0]) == 0
    again = torch.full((M + 2, C), 7.0, dtype=torch.bfloat16, device="cuda")
    T.triattn_transition_fwd(*params(d), kind, out=again[1:M + 1])
    assert torch.equal(again[1:M + 1], out) and bool((again[0] == 7.0).all()) and bool((again[M + 1] == 7.0).all())


def test_no_rows():
    x = S.make_transition_inputs((0,), 64, 128, seed=1)
    got = run_gpu(x)
    assert got[0].shape == (0, 64) and got[1].shape == (0, 64)
    for t in got[2:]:
        assert torch.count_nonzero(t) == 0
    for t in run_gpu(x, grads_bf16=True)[2:]:
        assert t.dtype == torch.bfloat16 and torch.count_nonzero(t) == 0


@pytest.mark.parametrize("C,H,M", [(128, 512, 3000), (256, 288, 700), (64, 64, 5)])
def test_bf16_gradients_are_the_rounded_fp32_ones(C, H, M):
    x = S.make_transition_inputs((M,), C, H, seed=12, drop=0.1)
    a, b = run_gpu(x), run_gpu(x, grads_bf16=True)
    assert torch.equal(a[1], b[1])
    for p, q in zip(a[2:], b[2:]):
        assert q.dtype == torch.bfloat16 and torch.equal(p.to(torch.bfloat16), q)


@pytest.mark.parametrize("C,H", [(128, 512), (160, 96)])
def test_bitwise_repeatable_and_outside_untouched(C, H):
    """Three calls give the same bits; outputs written into the middle of a
    larger buffer leave what is around them."""
    x = S.make_transition_inputs((777,), C, H, seed=13, drop=0.1)
    first = run_gpu(x)
    for _ in range(2):
        for a, b in zip(first, run_gpu(x)):
            assert torch.equal(a, b)
    d = to_dev(x)
    n = 777 * C
    pad = 512
    buf = torch.full((2, pad + n + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    out, dz = (buf[i, pad:pad + n].view(777, C) for i in range(2))
    T.triattn_transition_fwd(*params(d), out=out)
    T.triattn_transition_bwd(*params(d), d["d_out"], out=(dz,) + tuple(torch.empty_like(t) for t in first[2:]))
    assert torch.equal(out, first[0]) and torch.equal(dz, first[1])
    assert bool((buf[:, :pad] == 7.0).all()) and bool((buf[:, pad + n:] == 7.0).all())


def test_large_tensor_sampled():
    """crop768 at C = 128: sampled rows of out and dz against the oracle (a
    row depends on itself alone), and d_w_o, d_w_in by a random projection:
    u^T dW v in FP64 from the rows, both sides linear in dW."""
    M, C, H = 768 * 768, 128, 512
    x = S.make_transition_inputs((1, 768, 768), C, H, seed=14, drop=0.05)
    got = run_gpu(x)
    rows = np.random.default_rng(0).integers(0, M, 300)
    rows[:4] = (0, M - 1, M - 2, M // 2)
    pick = lambda t: t.reshape(M, -1)[torch.as_tensor(rows)]  # noqa: E731
    y = dict(x, z=pick(x["z"]), d_out=pick(x["d_out"]), mask=x["mask"].reshape(M)[torch.as_tensor(rows)])
    ref = TR.run(*params(y), y["d_out"])
    assert rel_rmse(cpu64(got[0].reshape(M, C)[rows]), ref["out"]) <= TOL_OUT
    assert rel_rmse(cpu64(got[1].reshape(M, C)[rows]), ref["dz"]) <= TOL_GRADS
    full = TR.run(*params(x), x["d_out"])
    for n, g in zip(NAMES[1:], got[2:]):
        assert rel_rmse(cpu64(g), full[n]) <= TOL_GRADS, n


def test_gradients_against_differences():
    """<out, d_out> along a random direction of each parameter, from two
    forwards a step apart, against the backward's gradient.  Step h moves the
    FP64 loss by h <grad, dir>; the loss's own error is that of out (TOL_OUT)
    on either side, in quadrature over the M C independent elements of out:
    2 TOL_OUT |out| |d_out| / sqrt(M C) / (2 h) on the quotient."""
    M, C, H = 4096, 128, 512
    x = S.make_transition_inputs((M,), C, H, seed=15)
    d = to_dev(x)
    got = run_gpu(x)
    g = torch.Generator().manual_seed(1)
    for name, grad in (("ln_w", got[2]), ("ln_b", got[3])):
        direction = torch.randn(C, generator=g).cuda()
        h = 0.125
        loss = []
        for sgn in (1.0, -1.0):
            q = dict(d)
            q[name] = d[name] + sgn * h * direction
            loss.append(float((T.triattn_transition_fwd(*params(q)).double() * d["d_out"].double()).sum()))
        quotient = (loss[0] - loss[1]) / (2 * h)
        want = float((grad.double() * direction.double()).sum())
        scale = float(got[0].double().norm() * d["d_out"].double().norm())
        noise = 2 * TOL_OUT * scale / np.sqrt(M * C) / (2 * h)
        # the quotient's own curvature error, from the FP64 oracle at the same step
        ref = []
        for sgn in (1.0, -1.0):
            q = dict(x)
            q[name] = x[name] + sgn * h * direction.cpu()
            ref.append(float((TR.run(*params(q))["out"] * cpu64(x["d_out"])).sum()))
        exact = run_oracle(x)[2 if name == "ln_w" else 3]
        curvature = (ref[0] - ref[1]) / (2 * h) - float((exact * direction.cpu().double().numpy()).sum())
        tol = 4 * noise + TOL_GRADS * float(grad.double().norm() * direction.double().norm()) / np.sqrt(C)
        assert abs(quotient - curvature - want) <= tol, (name, quotient, curvature, want, tol)


def test_autograd_module_matches_direct_calls():
    x = S.make_transition_inputs((1, 20, 20), 64, 256, seed=16, drop=0.1)
    d = to_dev(x)
    m = layers.Transition(64, device="cuda")
    with torch.no_grad():
        for n in ("ln_w", "ln_b", "w_in", "w_o"):
            getattr(m, n).copy_(d[n])
    z = d["z"].transpose(1, 2).contiguous().transpose(1, 2).detach().requires_grad_(True)  # a strided input
    assert not z.is_contiguous()
    out = m(z, d["mask"])
    out.backward(d["d_out"].transpose(1, 2).contiguous().transpose(1, 2))
    ref = run_gpu(x)
    assert torch.equal(out, ref[0]) and torch.equal(z.grad, ref[1])
    for n, g in zip(("ln_w", "ln_b", "w_in", "w_o"), ref[2:]):
        assert torch.equal(getattr(m, n).grad, g.to(getattr(m, n).dtype))
    m.zero_grad()
    m(d["z"]).sum().backward()  # an expanded gradient, no mask
    assert m.w_o.grad is not None


def test_graph_replay_and_side_stream():
    """Captured forward and backward replay on new inputs; a call on a side
    stream gives the same bits while another stream is busy."""
    x = S.make_transition_inputs((600,), 128, 512, seed=17, drop=0.1)
    y = S.make_transition_inputs((600,), 128, 512, seed=18, drop=0.1)
    ref_x, ref_y = run_gpu(x), run_gpu(y)
    d = to_dev(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    big = torch.randn(4096, 4096, device="cuda")
    for _ in range(4):
        big = big @ big * 1e-3
    out = T.triattn_transition_fwd(*params(d), stream=side)
    grads = T.triattn_transition_bwd(*params(d), d["d_out"], stream=side)
    torch.cuda.synchronize()
    for a, b in zip(ref_x, (out,) + grads):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = T.triattn_transition_fwd(*params(d))
        grads = T.triattn_transition_bwd(*params(d), d["d_out"])
    for src, ref in ((x, ref_x), (y, ref_y), (x, ref_x)):
        for k in ("z", "d_out", "mask", "ln_w", "ln_b", "w_in", "w_o"):
            d[k].copy_(src[k])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(ref, (out,) + grads):
            assert torch.equal(a, b)


def test_two_calls_at_once():
    """Two streams at the same time, each with its own workspace."""
    xs = [S.make_transition_inputs((20000,), 128, 512, seed=20 + i, drop=0.1) for i in range(2)]
    refs = [run_gpu(x) for x in xs]
    ds = [to_dev(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for _ in range(3):
        for d, s in zip(ds, streams):
            out = T.triattn_transition_fwd(*params(d), stream=s)
            got.append((out,) + tuple(T.triattn_transition_bwd(*params(d), d["d_out"], stream=s)))
    torch.cuda.synchronize()
    assert T.device_status() == T.OK
    for k, g in enumerate(got):
        for a, b in zip(refs[k % 2], g):
            assert torch.equal(a, b)


def test_refusals_on_device():
    x = to_dev(S.make_transition_inputs((8,), 64, 64, seed=1))
    z, mask, lw, lb, wi, wo = params(x)
    for bad in [(z[:, :32], None, lw, lb, wi, wo), (z.float(), None, lw, lb, wi, wo),
                (z, torch.ones(9, dtype=torch.bfloat16, device="cuda"), lw, lb, wi, wo),
                (z, torch.ones(8, device="cuda"), lw, lb, wi, wo), (z, None, lw.bfloat16(), lb, wi, wo),
                (z, None, lw, lb, wi[:, :64], wo), (z, None, lw, lb, wi, wo.t()),
                (z.t().contiguous().t(), None, lw, lb, wi, wo), (z, None, lw.cpu(), lb, wi, wo)]:
        with pytest.raises(ValueError):
            T.triattn_transition_fwd(*bad)
        with pytest.raises(ValueError):
            T.triattn_transition_bwd(*bad, x["d_out"])
    with pytest.raises(ValueError):
        T.triattn_transition_bwd(z, None, lw, lb, wi, wo, x["d_out"][:4])
    with pytest.raises(T.TriAttnError):
        T.triattn_transition_bwd(z, None, lw, lb, wi, wo, x["d_out"],
                                 workspace=torch.empty(128, dtype=torch.uint8, device="cuda"))
    odd = torch.empty(8 * 64 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(8, 64)  # 8-byte aligned
    with pytest.raises(T.TriAttnError):
        T.triattn_transition_fwd(odd, None, lw, lb, wi, wo)


@pytest.mark.parametrize("C,H", [(128, 512), (96, 64), (256, 64)])
def test_tensors_on_16_byte_boundaries(C, H):
    """Row tensors and the mask that start at odd multiples of 16 (2) bytes give
    the same bits, written into views aligned the same way."""
    M = 333
    x = S.make_transition_inputs((M,), C, H, seed=30, drop=0.2)
    ref = run_gpu(x)
    d = to_dev(x)

    def shifted(t, by):
        buf = torch.empty(t.numel() + 64, dtype=t.dtype, device="cuda")
        v = buf[by:by + t.numel()].view(t.shape)
        return v.copy_(t)

    for k in ("z", "d_out", "w_in", "w_o"):
        d[k] = shifted(d[k], 8)
    d["ln_w"], d["ln_b"], d["mask"] = shifted(d["ln_w"], 4), shifted(d["ln_b"], 4), shifted(d["mask"], 1)
    out = T.triattn_transition_fwd(*params(d), out=shifted(ref[0], 8))
    grads = T.triattn_transition_bwd(*params(d), d["d_out"], out=tuple(
        shifted(t, 8 if t.dtype == torch.bfloat16 else 4) for t in ref[1:]))
    torch.cuda.synchronize()
    for a, b in zip(ref, (out,) + tuple(grads)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("C,H", [(32, 2112), (64, 1504), (128, 1024), (128, 4096), (160, 2048), (224, 96), (256, 1536)])
@pytest.mark.parametrize("M", [1, 300, 2600])
def test_hidden_widths_past_shared_memory(C, H, M):
    """Hidden widths whose weights do not stay in shared memory, with fewer and
    more row tiles than a cluster pair takes at once."""
    check(S.make_transition_inputs((M,), C, H, seed=C + H + M, drop=0.1 if M > 1 else 0.0), case=[C, H, M])
