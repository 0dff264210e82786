"""The transition (gated feed-forward block over pair rows, forward and
backward) and the global gradient norm with clipping: the cases they are
measured on, their plain forms and their definition in 64 bits.

A case is a dict: ``op`` is "fwd" (the transition's forward), "train" (forward
and backward), "clip" (norm and clipped gradients) or "norm".  ``run`` makes
the library's calls when ``own`` is true and computes the same with elementary
torch operations otherwise.
"""
import math

import torch

own = False

if own:
    from protein_folding_triangle_gb300 import triattn  # noqa: F401

EPS = 1e-5


def listed():
    t = {"act": "silu", "pad": 0.0}
    return [
        # one row at the pair stack's width: latency only
        dict(t, name="fwd one row", op="fwd", rows=1, side=0, C=128, H=512),
        # a short chain (97 tokens) in a narrow pair tensor, last tokens padding
        dict(t, name="fwd 97 tokens C64", op="fwd", rows=97 * 97, side=97, C=64, H=256, pad=0.1),
        # the crop the library quotes its core on, 4-fold expansion
        dict(t, name="fwd crop768 C128", op="fwd", rows=768 * 768, side=768, C=128, H=512),
        # the widest pair tensor the layers take, with padding tokens
        dict(t, name="fwd crop384 C256", op="fwd", rows=384 * 384, side=384, C=256, H=1024, act="gelu", pad=0.1),
        # training steps at the usual crops
        dict(t, name="train crop384 C128", op="train", rows=384 * 384, side=384, C=128, H=512, pad=0.1),
        dict(t, name="train crop768 C128", op="train", rows=768 * 768, side=768, C=128, H=512),
        # an odd token count and a hidden width that is no power of two
        dict(t, name="train 131 tokens C96", op="train", rows=131 * 131, side=131, C=96, H=288, act="sigmoid", pad=0.08),
        # a narrow tensor, where the bytes weigh more than the products
        dict(t, name="train crop640 C64", op="train", rows=640 * 640, side=640, C=64, H=256, pad=0.05),
        # the gradients of one pair block (24 tensors): launch latency
        dict(name="clip one block", op="clip", blocks=1, tensors=0, total=0, dtype="mixed", kind=2, due=True),
        # a stack of 48 pair blocks (1152 tensors in two buckets)
        dict(name="clip 48 blocks", op="clip", blocks=48, tensors=0, total=0, dtype="mixed", kind=2, due=True),
        # FP32 main gradients, in place, a step whose largest gradient is under the limit
        dict(name="clip max 120M not due", op="clip", blocks=0, tensors=300, total=120_000_007, dtype="fp32", kind=0,
             due=False),
        # the norm alone (for a log), BF16, ragged tensors
        dict(name="norm 200M bf16", op="norm", blocks=0, tensors=77, total=200_000_003, dtype="bf16", kind=2,
             due=False),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["fwd", "fwd", "train", "train", "clip", "norm"])
    if op in ("fwd", "train"):
        C = 32 * rng.randint(1, 8)
        H = min(1024, C * rng.choice([1, 2, 4]) + 32 * rng.choice([0, 0, 1, 3]))
        most = 768 * 768 * 128 * 512 // (C * H)
        return {"op": op, "rows": log_int(1, min(most, 768 * 768)), "side": 0, "C": C, "H": H,
                "act": rng.choice(["silu", "silu", "sigmoid", "gelu"]), "pad": rng.choice([0.0, 0.05, 0.3])}
    dtype = rng.choice(["bf16", "fp32", "mixed"])
    total = log_int(1000, 120_000_000)
    return {"op": op, "blocks": 0, "tensors": log_int(1, min(1200, total // 8)), "total": total, "dtype": dtype,
            "kind": 2 if op == "norm" else rng.choice([2, 2, 0]), "due": op == "clip" and rng.random() < 0.7}


# ------------------------------------------------------------------- inputs
def _ffn_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    C, H, rows = case["C"], case["H"], case["rows"]
    lead = (1, case["side"], case["side"]) if case["side"] else (rows,)

    def normal(shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    s = {"case": case, "z": normal(lead + (C,)), "ln_w": normal((C,), 0.1, torch.float32) + 1.0,
         "ln_b": normal((C,), 0.1, torch.float32), "w_in": normal((C, 2 * H), C ** -0.5),
         "w_o": normal((H, C), H ** -0.5), "mask": None, "d_out": None}
    if case["pad"] > 0:
        if case["side"]:  # the last tokens are padding: every pair that touches one is masked
            keep = torch.ones(case["side"], device="cuda")
            keep[case["side"] - int(case["pad"] * case["side"]):] = 0.0
            s["mask"] = (keep[:, None] * keep[None, :]).expand(lead).contiguous().to(torch.bfloat16)
        else:
            s["mask"] = (torch.rand(lead, generator=g, device="cuda") >= case["pad"]).to(torch.bfloat16)
    if case["op"] == "train":
        s["d_out"] = normal(lead + (C,))
    return s


def _sizes(case, seed):
    """(elements, is_fp32) of every gradient tensor."""
    if case["blocks"]:  # per block: two attention modules, two multiplicative updates, a transition, at 128 features
        C, F = 128, 3 * 128 + 4
        att = [(C, True), (C, True), (C * F, False), (C * C, False)]
        mul = [(C, True), (C, True), (C * 5 * C, False), (C, True), (C, True), (C * C, False)]
        ffn = [(C, True), (C, True), (C * 8 * C, False), (4 * C * C, False)]
        return (2 * att + 2 * mul + ffn) * case["blocks"]
    n, total = case["tensors"], case["total"]
    g = torch.Generator().manual_seed(n * 1000003 + total)  # the sizes belong to the case, the values to the seed
    cuts = torch.sort(torch.randint(0, total + 1, (n - 1,), generator=g)).values.tolist()
    sizes = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    fp32 = {"bf16": lambda i: False, "fp32": lambda i: True, "mixed": lambda i: i % 3 == 0}[case["dtype"]]
    return [(m, fp32(i)) for i, m in enumerate(sizes)]


def _views(flat, sizes):
    """The tensors as consecutive views of one bucket, as a data-parallel run holds them."""
    return list(torch.split(flat, sizes)) if sizes else []


def _clip_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    sizes = _sizes(case, seed)
    s = {"case": case, "flats": [], "outs": [], "grads": [], "into": []}
    for want, dtype in ((False, torch.bfloat16), (True, torch.float32)):
        part = [m for m, f in sizes if f == want]
        if part:
            flat = torch.empty(sum(part), device="cuda").normal_(0.0, 1e-2, generator=g).to(dtype)
            s["flats"].append(flat)
            s["grads"] += _views(flat, part)
            if case["op"] == "clip" and case["due"]:
                s["outs"].append(torch.empty_like(flat))
                s["into"] += _views(s["outs"][-1], part)
    expect = 1e-2 * math.sqrt(sum(m for m, _ in sizes)) if case["kind"] == 2 else 4e-2
    s["max_norm"] = expect * (0.3 if case["due"] else 8.0)  # due: the norm is over the limit
    s["norm_type"] = 2.0 if case["kind"] == 2 else math.inf
    return s


def prepare(case, seed):
    return _ffn_inputs(case, seed) if case["op"] in ("fwd", "train") else _clip_inputs(case, seed)


# --------------------------------------------------------------- plain forms
def _act(a, kind):
    """act(a) and its derivative."""
    if kind == "gelu":
        k = math.sqrt(2.0 / math.pi)
        t = torch.tanh(k * (a + 0.044715 * a * a * a))
        return 0.5 * a * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * a * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * a * a)
    s = 1.0 / (1.0 + torch.exp(-a))
    return (s, s * (1.0 - s)) if kind == "sigmoid" else (a * s, s * (1.0 + a * (1.0 - s)))


def _plain_ffn(s):
    C, H = s["case"]["C"], s["case"]["H"]
    z = s["z"].float().reshape(-1, C)
    zc = z - z.mean(dim=1, keepdim=True)
    rstd = torch.rsqrt((zc * zc).mean(dim=1, keepdim=True) + EPS)
    xhat = zc * rstd
    x = xhat * s["ln_w"] + s["ln_b"]
    w_in, w_o = s["w_in"].float(), s["w_o"].float()
    p = x @ w_in
    a, b = p[:, :H], p[:, H:]
    f, df = _act(a, s["case"]["act"])
    h = f * b
    m = None if s["mask"] is None else s["mask"].float().reshape(-1, 1)
    out = h @ w_o
    out = out if m is None else torch.where(m == 0, 0.0, out * m)
    out = out.to(torch.bfloat16).reshape(s["z"].shape)
    if s["d_out"] is None:
        return out
    g = s["d_out"].float().reshape(-1, C)
    g = g if m is None else torch.where(m == 0, 0.0, g * m)
    dw_o = h.t() @ g
    dh = g @ w_o.t()
    dp = torch.cat([dh * b * df, dh * f], dim=1)
    dw_in = x.t() @ dp
    dx = dp @ w_in.t()
    dg = dx * s["ln_w"]
    dz = rstd * (dg - dg.mean(dim=1, keepdim=True) - xhat * (dg * xhat).mean(dim=1, keepdim=True))
    grads = (dz.reshape(s["z"].shape), (dx * xhat).sum(dim=0), dx.sum(dim=0), dw_in, dw_o)
    return (out,) + tuple(t.to(torch.bfloat16) for t in grads)


def _plain_clip(s):
    if s["norm_type"] == math.inf:
        norm = torch.stack([t.float().abs().max() for t in s["grads"] if t.numel()]).max()
    else:
        norm = torch.stack([t.float().square().sum() for t in s["grads"]]).sum().sqrt()
    if s["case"]["op"] == "norm":
        return (norm,)
    coef = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    if not s["into"]:  # in place; the limit is over the norm, so the values stay
        [t.copy_(t.float() * coef) for t in s["grads"]]
        return (norm, *s["flats"])
    [o.copy_(t.float() * coef) for o, t in zip(s["into"], s["grads"])]
    return (norm, *s["outs"])


# -------------------------------------------------------- the library's calls
def _own_ffn(s):
    from protein_folding_triangle_gb300 import triattn as T
    act = s["case"]["act"]
    out = T.triattn_transition_fwd(s["z"], s["mask"], s["ln_w"], s["ln_b"], s["w_in"], s["w_o"], act)
    if s["d_out"] is None:
        return out
    return (out,) + tuple(T.triattn_transition_bwd(s["z"], s["mask"], s["ln_w"], s["ln_b"], s["w_in"], s["w_o"],
                                                   s["d_out"], act, grads_bf16=True))


def _own_clip(s):
    from protein_folding_triangle_gb300 import triattn as T
    if s["case"]["op"] == "norm":
        return (T.triattn_grad_norm(s["grads"], s["norm_type"]),)
    norm = T.triattn_clip_grad_norm(s["grads"], s["max_norm"], s["norm_type"], out=s["into"] or None)
    return (norm, *(s["outs"] or s["flats"]))


def run(state):
    if state["case"]["op"] in ("fwd", "train"):
        return _own_ffn(state) if own else _plain_ffn(state)
    return _own_clip(state) if own else _plain_clip(state)


# ---------------------------------------------------------------------- work
def work(case):
    if case["op"] in ("fwd", "train"):
        M, C, H = case["rows"], case["C"], case["H"]
        mask = 2 * M if case["pad"] > 0 else 0
        by = 4 * M * C + mask + 6 * C * H + 8 * C  # z in, out out, the mask, the weights
        fl = 6 * M * C * H
        if case["op"] == "train":  # d_out in, dz out, the parameters' gradients out; the backward's five products
            by += 4 * M * C + 6 * C * H + 4 * C
            fl += 12 * M * C * H
        return {"bytes": by, "flops": fl}
    sizes = _sizes(case, 0)
    n = sum((4 if f else 2) * m for m, f in sizes)
    return {"bytes": n * (2 if case["due"] else 1), "flops": 2 * sum(m for m, _ in sizes)}


# --------------------------------------------------------------------- exact
def _exact_ffn(case, seed):
    """By automatic differentiation in 64 bits, some rows at a time."""
    s = _ffn_inputs(case, seed)
    C, H = case["C"], case["H"]
    par = [s[k].double().requires_grad_(True) for k in ("ln_w", "ln_b", "w_in", "w_o")]
    z_all = s["z"].reshape(-1, C)
    m_all = None if s["mask"] is None else s["mask"].reshape(-1)
    act = {"silu": torch.nn.functional.silu, "sigmoid": torch.sigmoid,
           "gelu": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[case["act"]]
    outs, dzs = [], []
    for lo in range(0, z_all.shape[0], 1 << 16):
        z = z_all[lo:lo + (1 << 16)].double().requires_grad_(True)
        x = torch.nn.functional.layer_norm(z, (C,), par[0], par[1], EPS)
        o = (act(x @ par[2][:, :H]) * (x @ par[2][:, H:])) @ par[3]
        if m_all is not None:
            o = o * m_all[lo:lo + (1 << 16), None].double()
        if s["d_out"] is not None:
            o.backward(s["d_out"].reshape(-1, C)[lo:lo + (1 << 16)].double())
            dzs.append(z.grad)
        outs.append(o.detach())
    out = torch.cat(outs).reshape(s["z"].shape)
    if s["d_out"] is None:
        return out
    return (out, torch.cat(dzs).reshape(s["z"].shape), *(p.grad for p in par))


def _exact_clip(case, seed):
    s = _clip_inputs(case, seed)
    parts = [f.double() for f in s["flats"]]
    if s["norm_type"] == math.inf:
        norm = max(float(p.abs().max()) for p in parts if p.numel())
    else:
        norm = math.sqrt(math.fsum(float((p * p).sum()) for p in parts))
    n = torch.tensor(norm, dtype=torch.float64)
    if case["op"] == "norm":
        return (n,)
    coef = min(1.0, s["max_norm"] / (norm + 1e-6))
    return (n, *(p * coef for p in parts))


def exact(case, seed):
    return _exact_ffn(case, seed) if case["op"] in ("fwd", "train") else _exact_clip(case, seed)
