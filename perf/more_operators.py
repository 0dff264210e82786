"""Operators around the attention core and at the end of a training step: the
norms of queries and keys for each head with the position rotation, the learned
relative position bias by buckets (as planes for the core and as pair features),
and the orthogonalisation of a list of updates: the cases they are measured on,
their plain forms and their definition in 64 bits.

A case is a dict: ``op`` is "qk" (norms and rotation), "rel" (relative position
bias) or "orth" (orthogonalisation); ``train`` adds the gradients.  ``run``
makes the library's calls when ``own`` is true and computes the same with
elementary torch operations otherwise.
"""
import functools
import math

import torch

own = False

if own:
    from protein_folding_triangle_gb300 import triattn  # noqa: F401

EPS = 1e-6
STEPS = 5
COEF = (3.4445, -4.7750, 2.0315)
BLOCK = [(128, 388), (128, 128), (128, 388), (128, 128), (128, 640), (128, 128), (128, 640), (128, 128),
         (128, 1024), (512, 128)]  # the matrices of a pair block at 128 features (two attention modules, two
#                                    multiplicative updates, a transition)


def listed():
    qk = {"op": "qk", "B": 1, "rotary": "half", "rows": "heads", "start": 0, "chains": 1, "shared": False}
    rel = {"op": "rel", "B": 1, "kind": "clip", "R": 32, "buckets": 65, "start": 1, "chains": 1, "base": True,
           "grad": "bf16"}
    return [
        # a short chain: latency only
        dict(qk, name="qk fwd 48 tokens", train=False, N=48, H=2, D=16),
        # inference on the crop the core is quoted on
        dict(qk, name="qk fwd crop768", train=False, N=768, H=4, D=32),
        # two complexes of an odd token count whose residue numbers start far out, heads in the projections' pair rows
        dict(qk, name="qk train 2x131 tokens", train=True, B=2, N=131, H=6, D=16, rotary="interleaved", rows="pairs",
             start=900_000_000, chains=3, shared=True),
        # a training step at the crop the core is quoted on, in the module's pair rows
        dict(qk, name="qk train crop768 pair rows", train=True, N=768, H=4, D=32, rows="pairs", chains=2),
        # the planes of a crop, a table of 32 logarithmic buckets
        dict(rel, name="bias fwd crop768", train=False, layout="heads", N=768, F=4, kind="log", R=128, buckets=32),
        # a long complex of four chains, forward and gradient
        dict(rel, name="bias train 2048 tokens", train=True, layout="heads", N=2048, F=16, chains=4, buckets=66),
        # an odd token count (rows off every alignment), the core's FP32 gradient
        dict(rel, name="bias train 3x301 tokens", train=True, layout="heads", B=3, N=301, F=8, chains=2, buckets=66,
             grad="fp32"),
        # the pair tensor of a crop, as the first thing that is added to it
        dict(rel, name="pair fwd crop768", train=False, layout="pairs", N=768, F=128, chains=2, buckets=66),
        # its training step
        dict(rel, name="pair train crop640", train=True, layout="pairs", N=640, F=128, chains=2, buckets=66),
        # the matrices of one pair block: launch latency
        dict(op="orth", name="orth one block", blocks=1, m=0, n=0, count=0, dtype="bf16", rank=16),
        # a stack of 48 pair blocks
        dict(op="orth", name="orth 48 blocks", blocks=48, m=0, n=0, count=0, dtype="bf16", rank=16),
        # the projections of the widest pair tensor, FP32 momentum, an odd width
        dict(op="orth", name="orth 256x1037", blocks=0, m=256, n=1037, count=12, dtype="fp32", rank=40),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["qk", "qk", "rel", "rel", "rel", "orth"])
    start = rng.choice([0, 1, 5000, 900_000_000])
    if op == "qk":
        B, H, D = rng.choice([1, 1, 2]), rng.choice([1, 2, 4, 6, 8]), rng.choice([16, 32])
        most = int(math.sqrt(768 * 768 * 128 / (B * H * D)))
        return {"op": op, "train": rng.random() < 0.5, "B": B, "N": log_int(5, min(most, 768)), "H": H, "D": D,
                "rotary": rng.choice(["half", "half", "interleaved", "none"]), "rows": rng.choice(["heads", "pairs"]),
                "start": start, "chains": rng.choice([1, 2, 5]), "shared": rng.random() < 0.3}
    if op == "rel":
        layout = rng.choice(["heads", "pairs"])
        B = rng.choice([1, 1, 2])
        F = rng.choice([1, 4, 5, 8, 16]) if layout == "heads" else 32 * rng.randint(1, 8)
        most = int(math.sqrt(640 * 640 * 128 / (B * F)))
        chains = rng.choice([1, 2, 5])
        kind = rng.choice(["clip", "clip", "log"])
        R = rng.choice([8, 32, 32, 50, 100] if kind == "clip" else [64, 128, 500])
        buckets = (2 * R + 1 if kind == "clip" else rng.choice([16, 32, 64])) + (1 if chains > 1 else 0)
        return {"op": op, "train": rng.random() < 0.6, "B": B, "layout": layout, "N": log_int(5, min(most, 2048)),
                "F": F, "kind": kind, "R": R, "buckets": buckets, "start": start, "chains": chains,
                "base": rng.random() < 0.8, "grad": rng.choice(["bf16", "fp32"]) if layout == "heads" else "bf16"}
    m, n = log_int(8, 512), log_int(8, 1100)
    most = 48 * 1_500_000_000 // (STEPS * (4 * min(m, n) ** 2 * max(m, n) + 2 * min(m, n) ** 3))
    return {"op": op, "blocks": 0, "m": m, "n": n, "count": log_int(1, max(1, min(200, most))),
            "dtype": rng.choice(["bf16", "fp32"]), "rank": log_int(4, 64)}


# ------------------------------------------------------------------- inputs
def _residues(case):
    """Residue numbers and chain ids [B, N]: chains one after the other, each numbered from the same start, a gap
    in every chain.  They belong to the case."""
    B, N, n = case["B"], case["N"], case["chains"]
    t = torch.arange(N)
    chain = (t * n) // N
    first = torch.searchsorted(chain, chain)
    pos = t - first
    pos = pos + torch.where(pos > N // (3 * n), 7, 0) + case["start"]
    return pos.expand(B, N).to(torch.int32).contiguous().cuda(), chain.expand(B, N).to(torch.int32).contiguous().cuda()


def _normal(g, shape, scale=1.0, dtype=torch.bfloat16):
    return torch.empty(shape, device="cuda").normal_(0.0, scale, generator=g).to(dtype)


def _qk_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    B, N, H, D = case["B"], case["N"], case["H"], case["D"]

    def pair(scale):
        if case["rows"] == "heads":
            return _normal(g, (B, N, H, N, D), scale), _normal(g, (B, N, H, N, D), scale)
        f = (3 * H * D + H + 7) // 8 * 8  # the module's projection [q | k | v | bias], row by row
        rows = _normal(g, (B, N, N, f), scale)
        return tuple(rows[..., c:c + H * D].unflatten(-1, (H, D)).permute(0, 1, 3, 2, 4) for c in (0, H * D))

    q, k = pair(1.7)
    w = (D,) if case["shared"] else (H, D)
    s = {"case": case, "q": q, "k": k, "w_q": _normal(g, w, 0.2, torch.float32) + 1.0,
         "w_k": _normal(g, w, 0.2, torch.float32) + 1.0, "pos": None, "d": None}
    if case["rotary"] != "none":
        s["pos"] = _residues(case)[0]
    if case["train"]:
        s["d"] = pair(1.0)
    return s


def _rel_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    B, N, F = case["B"], case["N"], case["F"]
    shape = (B, F, N, N) if case["layout"] == "heads" else (B, N, N, F)
    pos, chain = _residues(case)
    s = {"case": case, "table": _normal(g, (case["buckets"], F), 0.5, torch.float32), "pos": pos,
         "chain": chain if case["chains"] > 1 else None, "base": _normal(g, shape) if case["base"] else None, "d": None}
    if case["train"]:
        s["d"] = _normal(g, shape, 1.0, torch.float32 if case["grad"] == "fp32" else torch.bfloat16)
    return s


def _orth_inputs(case, seed):
    """Updates as training has them: a few strong directions and noise."""
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
    shapes = BLOCK * case["blocks"] or [(case["m"], case["n"])] * case["count"]
    ts = []
    for m, n in shapes:
        r = min(m, n, case["rank"])
        u, v = _normal(g, (m, r), 1.0, torch.float32), _normal(g, (r, n), 1.0, torch.float32)
        ts.append(((u * torch.linspace(1.0, 0.1, r, device="cuda") @ v + _normal(g, (m, n), 0.3, torch.float32))
                   * 1e-3).to(dt))
    flat = torch.empty(sum(t.numel() for t in ts), dtype=torch.bfloat16, device="cuda")  # the updates, in one bucket
    into = [v.view(t.shape) for v, t in zip(torch.split(flat, [t.numel() for t in ts]), ts)]
    return {"case": case, "grads": ts, "flat": flat, "into": into}


def prepare(case, seed):
    return {"qk": _qk_inputs, "rel": _rel_inputs, "orth": _orth_inputs}[case["op"]](case, seed)


# --------------------------------------------------------------- plain forms
def _angles(s, D):
    """cos and sin [B, 1, 1, N, D / 2] of position times frequency (the angle in 64 bits)."""
    f = 10000.0 ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
    a = s["pos"].double()[:, None, None, :, None] * f
    return torch.cos(a).float(), torch.sin(a).float()


def _turn(x, cos, sin, kind):
    if kind == "half":
        a, b = x.chunk(2, dim=-1)
        return torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)


def _plain_qk_one(s, x, w, d):
    kind, D = s["case"]["rotary"], s["case"]["D"]
    x, wf = x.float(), (w if w.dim() == 1 else w[:, None, :])
    r = torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS)
    n = x * r
    y = n * wf
    cos, sin = _angles(s, D) if kind != "none" else (None, None)
    y = _turn(y, cos, sin, kind) if kind != "none" else y
    y = y.to(torch.bfloat16)
    if d is None:
        return (y,)
    g = d.float()
    g = _turn(g, cos, -sin, kind) if kind != "none" else g
    p = (g * n).sum(dim=3)  # [B, N_o, H, D]: over the tokens of a slice
    dw = p.double().sum(dim=(0, 1, 2) if w.dim() == 1 else (0, 1)).float()
    a = g * wf
    dx = r * (a - n * (a * n).mean(dim=-1, keepdim=True))
    return y, dx.to(torch.bfloat16), dw


def _plain_qk(s):
    d = s["d"] or (None, None)
    a, b = _plain_qk_one(s, s["q"], s["w_q"], d[0]), _plain_qk_one(s, s["k"], s["w_k"], d[1])
    return tuple(t for both in zip(a, b) for t in both)


def _buckets(s):
    """The table's row of every pair [B, N, N]."""
    c = s["case"]
    d = s["pos"].long()[:, :, None] - s["pos"].long()[:, None, :]
    if c["kind"] == "clip":
        k = d.clamp(-c["R"], c["R"]) + c["R"]
    else:  # half of the rows for each sign, half of those exact, the others logarithmic up to R
        half = (c["buckets"] - (1 if s["chain"] is not None else 0)) // 2
        exact = half // 2
        far = (d.abs().clamp(min=exact).double() / exact).log() / math.log(c["R"] / exact) * (half - exact)
        k = torch.where(d.abs() < exact, d.abs(), (exact + (far + 1e-9).floor().long()).clamp(max=half - 1))
        k = k + torch.where(d < 0, half, 0)
    if s["chain"] is not None:
        k = torch.where(s["chain"][:, :, None] == s["chain"][:, None, :], k, c["buckets"] - 1)
    return k


def _plain_rel(s):
    c = s["case"]
    k = _buckets(s)
    heads = c["layout"] == "heads"
    e = s["table"][k]
    e = e.permute(0, 3, 1, 2) if heads else e
    out = (e if s["base"] is None else s["base"].float() + e).to(torch.bfloat16).contiguous()
    if s["d"] is None:
        return out
    hot = (k[..., None] == torch.arange(c["buckets"], device="cuda")).float().flatten(0, 1)  # [B N, N, buckets]
    d = s["d"].float()
    d = (d.permute(0, 2, 3, 1) if heads else d).flatten(0, 1)  # [B N, N, F]
    return out, torch.bmm(hot.transpose(1, 2), d).double().sum(dim=0).float()


def _step(x, _):
    a = torch.bmm(x, x.transpose(1, 2))
    return COEF[0] * x + torch.bmm(COEF[1] * a + COEF[2] * torch.bmm(a, a), x)


def _plain_orth_group(ts):
    """Matrices of one shape at once."""
    x = torch.stack(ts).float()
    tall = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2) if tall else x
    x = x / (x.square().sum(dim=(1, 2), keepdim=True).sqrt() + 1e-7)
    x = functools.reduce(_step, range(STEPS), x)
    return list((x.transpose(1, 2) if tall else x).to(torch.bfloat16).contiguous().unbind())


def _plain_orth(s):
    shapes = [tuple(t.shape) for t in s["grads"]]
    done = {sh: iter(_plain_orth_group([t for t in s["grads"] if tuple(t.shape) == sh])) for sh in set(shapes)}
    [o.copy_(next(done[sh])) for o, sh in zip(s["into"], shapes)]
    return s["flat"]


# -------------------------------------------------------- the library's calls
def _own_qk(s):
    from protein_folding_triangle_gb300 import triattn as T
    kind = s["case"]["rotary"]
    out = T.triattn_qk_norm_fwd(s["q"], s["k"], s["w_q"], s["w_k"], s["pos"], kind, eps=EPS)
    if s["d"] is None:
        return out
    dq, dk, dwq, dwk = T.triattn_qk_norm_bwd(s["q"], s["k"], s["w_q"], s["w_k"], s["d"][0], s["d"][1], s["pos"], kind,
                                             eps=EPS)
    return (*out, dq, dk, dwq, dwk)


def _own_rel(s):
    from protein_folding_triangle_gb300 import triattn as T
    c = s["case"]
    rule = dict(layout=c["layout"], kind=c["kind"], max_distance=c["R"])
    out = T.triattn_relpos_fwd(s["table"], s["base"], s["pos"], s["chain"], **rule)
    if s["d"] is None:
        return out
    return out, T.triattn_relpos_bwd(s["d"], c["buckets"], s["pos"], s["chain"], **rule)


def _own_orth(s):
    from protein_folding_triangle_gb300 import triattn as T
    T.triattn_orthogonalize(s["grads"], STEPS, coefficients=COEF, eps=1e-7, out=s["into"])
    return s["flat"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"qk": _own_qk, "rel": _own_rel, "orth": _own_orth}[op](state)
    return {"qk": _plain_qk, "rel": _plain_rel, "orth": _plain_orth}[op](state)


# ---------------------------------------------------------------------- work
def work(case):
    if case["op"] == "qk":
        e = case["B"] * case["N"] ** 2 * case["H"] * case["D"]
        # q, k in and out; for training also their gradients in and out
        return {"bytes": 2 * 2 * e * (4 if case["train"] else 2), "flops": 2 * e * (24 if case["train"] else 8)}
    if case["op"] == "rel":
        e = case["B"] * case["N"] ** 2 * case["F"]
        by = 2 * e * (2 if case["base"] else 1) + 4 * case["buckets"] * case["F"]
        if case["train"]:
            by += e * (4 if case["grad"] == "fp32" else 2) + 4 * case["buckets"] * case["F"]
        return {"bytes": by, "flops": e * (2 if case["train"] else 1)}
    shapes = BLOCK * case["blocks"] or [(case["m"], case["n"])] * case["count"]
    size = 4 if case["dtype"] == "fp32" else 2
    return {"bytes": sum(m * n for m, n in shapes) * (size + 2),
            "flops": STEPS * sum(4 * min(s) ** 2 * max(s) + 2 * min(s) ** 3 for s in shapes)}


# --------------------------------------------------------------------- exact
def _exact_qk(case, seed):
    """The rotation as a product of complex numbers, gradients by automatic differentiation, a slice of the outer
    axis at a time."""
    s = _qk_inputs(case, seed)
    N, D = case["N"], case["D"]
    unit = None
    if case["rotary"] != "none":
        f = torch.tensor([10000.0 ** (-2.0 * i / D) for i in range(D // 2)], dtype=torch.float64, device="cuda")
        ang = s["pos"].double()[..., None] * f
        unit = torch.polar(torch.ones_like(ang), ang)[:, None, None]  # [B, 1, 1, N, D / 2]
    got = []
    for x_all, w, d_all in ((s["q"], s["w_q"], (s["d"] or (None, None))[0]),
                            (s["k"], s["w_k"], (s["d"] or (None, None))[1])):
        w = w.double().requires_grad_(True)
        ys, dxs = [], []
        for o in range(0, N, 64):
            x = x_all[:, o:o + 64].double().requires_grad_(True)
            y = x / torch.linalg.vector_norm(torch.cat([x, torch.full_like(x[..., :1], math.sqrt(EPS * D))], -1),
                                             dim=-1, keepdim=True) * math.sqrt(D)
            y = y * (w if w.dim() == 1 else w.unsqueeze(1))
            if case["rotary"] == "half":
                z = torch.complex(y[..., :D // 2], y[..., D // 2:]) * unit
                y = torch.cat([z.real, z.imag], dim=-1)
            elif case["rotary"] == "interleaved":
                y = torch.view_as_real(torch.view_as_complex(y.unflatten(-1, (D // 2, 2)).contiguous())
                                       * unit).flatten(-2)
            if d_all is not None:
                y.backward(d_all[:, o:o + 64].double())
                dxs.append(x.grad)
            ys.append(y.detach())
        got.append((torch.cat(ys, 1),) if d_all is None else (torch.cat(ys, 1), torch.cat(dxs, 1), w.grad))
    return tuple(t for both in zip(*got) for t in both)


def _exact_rel(case, seed):
    """Buckets from a list of the smallest distance of each, found by trying every distance."""
    s = _rel_inputs(case, seed)
    R, F = case["R"], case["F"]
    other = s["chain"] is not None
    if case["kind"] == "clip":
        row = {d: d + R for d in range(-R, R + 1)}
    else:
        half = (case["buckets"] - (1 if other else 0)) // 2
        e = half // 2
        # bucket e + t from the first distance a with (a / e)^(half - e) >= (R / e)^t, in whole numbers
        up = [a if a < e else e + sum(a ** (half - e) * e ** t >= R ** t * e ** (half - e)
                                      for t in range(1, half - e)) for a in range(R + 1)]
        row = {d: up[abs(d)] + (half if d < 0 else 0) for d in range(-R, R + 1)}
    rows = torch.tensor([row[d] for d in range(-R, R + 1)], device="cuda")
    table = s["table"].double()
    outs, dt = [], torch.zeros(case["buckets"], F, dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        p = s["pos"][b].tolist()
        lo = min(p)
        p = torch.tensor([v - lo for v in p], device="cuda")
        k = rows[(p[:, None] - p[None, :]).clamp(-R, R) + R]
        if other:
            k[s["chain"][b][:, None] != s["chain"][b][None, :]] = case["buckets"] - 1
        for f in ([slice(h, h + 1) for h in range(F)] if case["layout"] == "heads" else [slice(0, F)]):
            v = table[:, f][k]  # [N, N, 1 or F]
            v = v[..., 0] if case["layout"] == "heads" else v
            outs.append(v if s["base"] is None else v + (s["base"][b, f.start] if case["layout"] == "heads"
                                                         else s["base"][b]).double())
            if s["d"] is not None:
                d = (s["d"][b, f.start][..., None] if case["layout"] == "heads" else s["d"][b]).double()
                order = torch.argsort(k.flatten(), stable=True)  # sums of the sorted pairs' prefixes
                run_ = torch.cat([torch.zeros_like(d[:1, 0]), d.flatten(0, 1)[order].cumsum(dim=0)])
                end = torch.bincount(k.flatten(), minlength=case["buckets"]).cumsum(0)
                dt[:, f] += run_[end] - run_[torch.cat([end.new_zeros(1), end[:-1]])]
    out = torch.stack(outs).reshape(s["base"].shape if s["base"] is not None else
                                    ((case["B"], F, case["N"], case["N"]) if case["layout"] == "heads" else
                                     (case["B"], case["N"], case["N"], F)))
    return out if s["d"] is None else (out, dt)


def _exact_orth(case, seed):
    """The polynomial of the singular values: the products leave the singular vectors as they are."""
    s = _orth_inputs(case, seed)
    outs = [None] * len(s["grads"])
    by_shape = {}
    for i, t in enumerate(s["grads"]):
        by_shape.setdefault(tuple(t.shape), []).append(i)
    for sh, idx in by_shape.items():
        for lo in range(0, len(idx), 16):
            part = idx[lo:lo + 16]
            x = torch.stack([s["grads"][i] for i in part]).double()
            wide = x.transpose(1, 2) if sh[0] > sh[1] else x
            # X = U S V^T: U and S^2 from X X^T, then X -> U diag(p(S) / S) U^T X, p(S) / S a polynomial in S^2
            val, u = torch.linalg.eigh(wide @ wide.transpose(1, 2))
            norm = torch.linalg.vector_norm(wide, dim=(1, 2)) + 1e-7
            t = val / norm[:, None] ** 2
            fac = torch.ones_like(t)
            for _ in range(STEPS):  # sigma <- sigma (a + b sigma^2 + c sigma^4)
                q = t * fac ** 2
                fac = fac * (COEF[0] + COEF[1] * q + COEF[2] * q * q)
            y = (u * fac[:, None, :]) @ (u.transpose(1, 2) @ wide) / norm[:, None, None]
            y = y.transpose(1, 2) if sh[0] > sh[1] else y
            for i, v in zip(part, y):
                outs[i] = v.flatten()
    return torch.cat(outs)


def exact(case, seed):
    return {"qk": _exact_qk, "rel": _exact_rel, "orth": _exact_orth}[case["op"]](case, seed)
