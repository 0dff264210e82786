"""Argument checks of the norms of queries and keys and of the relative position
bias, without a GPU: bad calls are answered before anything is launched."""
import ctypes

import pytest
import torch

from protein_folding_triangle_gb300 import build as B
from protein_folding_triangle_gb300 import triattn as T

FAKE = 1 << 20  # aligned, never dereferenced: validation fails first
V = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    B.build()
    return T.load()


def qk(lib, s, lays=(None, None, None), ws=FAKE, nbytes=1 << 40, bwd=False, **kw):
    names = ("q", "k", "w_q", "w_k", "positions", "d_q_out", "d_k_out", "q_out", "k_out", "d_w_q", "d_w_k")
    p = {n: V(FAKE) for n in names}
    p.update({n: V(v) for n, v in kw.items()})
    lay = [None if u is None else ctypes.byref(T.Layout(*u)) for u in lays]
    if not bwd:
        return lib.triattn_qk_norm_fwd(ctypes.byref(s), p["q"], p["k"], lay[0], p["w_q"], p["w_k"], p["positions"],
                                       p["q_out"], p["k_out"], lay[1], None)
    return lib.triattn_qk_norm_bwd(ctypes.byref(s), p["q"], p["k"], lay[0], p["w_q"], p["w_k"], p["positions"],
                                   p["d_q_out"], p["d_k_out"], lay[1], p["q_out"], p["k_out"], lay[2], p["d_w_q"],
                                   p["d_w_k"], V(ws), ctypes.c_size_t(nbytes), None)


OK_QK = dict(B=1, N_o=5, N=7, H=2, D=16, w_heads=2, rotary=1, eps=1e-6, theta=1e4, flags=0)


def shape(**kw):
    return T.QKNormShape(**{**OK_QK, **kw})


def test_qk_norm_shapes(lib):
    inf, nan = float("inf"), float("nan")
    for kw in [dict(), dict(w_heads=1), dict(D=32), dict(rotary=0), dict(rotary=2), dict(N_o=1 << 20, N=1)]:
        assert lib.triattn_qk_norm_workspace_bytes(ctypes.byref(shape(**kw))) > 0, kw
    for kw in [dict(B=0), dict(N_o=0), dict(N=0), dict(H=0), dict(D=0), dict(w_heads=0), dict(H=4, w_heads=2),
               dict(rotary=3), dict(rotary=-1), dict(eps=0.0), dict(eps=-1.0), dict(eps=nan), dict(eps=inf),
               dict(theta=0.0), dict(theta=nan), dict(theta=inf), dict(flags=1)]:
        assert lib.triattn_qk_norm_workspace_bytes(ctypes.byref(shape(**kw))) == 0, kw
        for bwd in (False, True):
            assert qk(lib, shape(**kw), bwd=bwd) == T.ERR_INVALID_ARG, kw
    for kw in [dict(D=8), dict(D=64), dict(D=24), dict(B=65536), dict(N=1 << 29, H=2), dict(B=1 << 12, N_o=1 << 20)]:
        assert lib.triattn_qk_norm_workspace_bytes(ctypes.byref(shape(**kw))) == 0, kw
        for bwd in (False, True):
            assert qk(lib, shape(**kw), bwd=bwd) == T.ERR_UNSUPPORTED, kw


def test_qk_norm_pointers(lib):
    s = shape()
    for n in ("q", "k", "q_out", "k_out", "w_q", "w_k"):
        for bwd in (False, True):
            assert qk(lib, s, bwd=bwd, **{n: None}) == T.ERR_INVALID_ARG, n
            assert qk(lib, s, bwd=bwd, **{n: FAKE + 2}) == T.ERR_INVALID_ARG, n
    for n in ("d_q_out", "d_k_out", "d_w_q", "d_w_k"):
        assert qk(lib, s, bwd=True, **{n: None}) == T.ERR_INVALID_ARG, n
        assert qk(lib, s, bwd=True, **{n: FAKE + 2}) == T.ERR_INVALID_ARG, n
    assert qk(lib, s, positions=FAKE + 2) == T.ERR_INVALID_ARG
    need = lib.triattn_qk_norm_workspace_bytes(ctypes.byref(s))
    assert qk(lib, s, bwd=True, nbytes=need - 1) == T.ERR_WORKSPACE
    assert qk(lib, s, bwd=True, ws=FAKE + 16) == T.ERR_WORKSPACE
    assert qk(lib, s, bwd=True, ws=None) == T.ERR_WORKSPACE
    good, bad = (7 * 48, 16, 48), (7 * 48, 16, 44)
    for at in range(3):
        lays = [good] * 3
        lays[at] = bad
        if at < 2:
            assert qk(lib, s, lays) == T.ERR_INVALID_ARG
        assert qk(lib, s, lays, bwd=True) == T.ERR_INVALID_ARG


def test_qk_norm_outputs_of_their_own(lib):
    """Outputs that are each other or an input; dq, dk over d_q_out, d_k_out want
    their layout."""
    s, at = shape(), [FAKE + (i << 24) for i in range(12)]
    names = ("q", "k", "w_q", "w_k", "positions", "d_q_out", "d_k_out", "q_out", "k_out", "d_w_q", "d_w_k")
    apart = dict(zip(names, at))
    for a, b in (("q_out", "k_out"), ("q_out", "q"), ("q_out", "k"), ("k_out", "q"), ("k_out", "k")):
        for bwd in (False, True):
            assert qk(lib, s, bwd=bwd, **{**apart, a: apart[b]}) == T.ERR_INVALID_ARG, (a, b)
    for a, b in (("d_w_q", "d_w_k"), ("q_out", "d_k_out"), ("k_out", "d_q_out")):
        assert qk(lib, s, bwd=True, **{**apart, a: apart[b]}) == T.ERR_INVALID_ARG, (a, b)
    rows = (7 * 96, 16, 96)
    for a, b in (("q_out", "d_q_out"), ("k_out", "d_k_out")):
        assert qk(lib, s, (None, rows, None), bwd=True, **{**apart, a: apart[b]}) == T.ERR_INVALID_ARG, (a, b)


def rel(lib, s, table=FAKE, base=FAKE, positions=FAKE, chains=None, out=FAKE):
    return lib.triattn_relpos_fwd(ctypes.byref(s), V(table), V(base), V(positions), V(chains), V(out), None)


def rel_bwd(lib, s, d_out=FAKE, positions=FAKE, chains=None, d_table=FAKE, ws=FAKE, nbytes=1 << 40):
    return lib.triattn_relpos_bwd(ctypes.byref(s), V(d_out), V(positions), V(chains), V(d_table), V(ws),
                                  ctypes.c_size_t(nbytes), None)


OK_REL = dict(B=1, N=9, F=8, layout=0, kind=0, buckets=65, max_distance=32, flags=0)


def rshape(**kw):
    return T.RelposShape(**{**OK_REL, **kw})


def test_relpos_shapes(lib):
    for kw in [dict(), dict(layout=1), dict(flags=4), dict(N=16384, F=1), dict(buckets=256, max_distance=127)]:
        assert lib.triattn_relpos_workspace_bytes(ctypes.byref(rshape(**kw))) > 0, kw
    for kw in [dict(B=0), dict(N=0), dict(F=0), dict(buckets=0), dict(max_distance=0), dict(layout=2), dict(kind=2),
               dict(kind=-1), dict(flags=1), dict(flags=8)]:
        assert lib.triattn_relpos_workspace_bytes(ctypes.byref(rshape(**kw))) == 0, kw
        assert rel(lib, rshape(**kw)) == T.ERR_INVALID_ARG and rel_bwd(lib, rshape(**kw)) == T.ERR_INVALID_ARG, kw
    for kw in [dict(N=16385), dict(buckets=257, max_distance=128), dict(max_distance=1025, kind=1, buckets=32),
               dict(B=8, N=16384), dict(F=65536), dict(layout=1, F=12), dict(layout=1, F=264), dict(layout=1, flags=4)]:
        assert lib.triattn_relpos_workspace_bytes(ctypes.byref(rshape(**kw))) == 0, kw
        assert rel(lib, rshape(**kw)) == T.ERR_UNSUPPORTED and rel_bwd(lib, rshape(**kw)) == T.ERR_UNSUPPORTED, kw
    # the number of rows against the rule, with and without the row of other chains
    for kw, chains in [(dict(buckets=66), None), (dict(buckets=65), FAKE), (dict(buckets=64), None),
                       (dict(kind=1, buckets=33), None), (dict(kind=1, buckets=32), FAKE), (dict(kind=1, buckets=2), None),
                       (dict(kind=1, buckets=32, max_distance=8), None), (dict(kind=1, buckets=4, max_distance=1), None)]:
        assert rel(lib, rshape(**kw), chains=chains) == T.ERR_INVALID_ARG, kw
        assert rel_bwd(lib, rshape(**kw), chains=chains) == T.ERR_INVALID_ARG, kw


def test_relpos_pointers(lib):
    s = rshape()
    for n, off in (("table", 8), ("base", 8), ("out", 8), ("positions", 2)):
        assert rel(lib, s, **{n: FAKE + off}) == T.ERR_INVALID_ARG, n
    assert rel(lib, s, table=None) == T.ERR_INVALID_ARG and rel(lib, s, out=None) == T.ERR_INVALID_ARG
    assert rel(lib, rshape(buckets=66), chains=FAKE + 2) == T.ERR_INVALID_ARG
    for n, off in (("d_out", 8), ("d_table", 2), ("positions", 2)):
        assert rel_bwd(lib, s, **{n: FAKE + off}) == T.ERR_INVALID_ARG, n
    assert rel_bwd(lib, s, d_out=None) == T.ERR_INVALID_ARG and rel_bwd(lib, s, d_table=None) == T.ERR_INVALID_ARG
    need = lib.triattn_relpos_workspace_bytes(ctypes.byref(s))
    assert rel_bwd(lib, s, nbytes=need - 1) == T.ERR_WORKSPACE
    assert rel_bwd(lib, s, ws=FAKE + 16) == T.ERR_WORKSPACE and rel_bwd(lib, s, ws=None) == T.ERR_WORKSPACE


def test_python_refusals(lib):
    q, w, t = torch.zeros(1, 2, 1, 3, 16, dtype=torch.bfloat16), torch.ones(16), torch.zeros(65, 4)
    for f in (lambda: T.triattn_qk_norm_fwd(q, q, w, w),                      # not on a GPU
              lambda: T.triattn_qk_norm_fwd(q[0], q[0], w, w),
              lambda: T.qk_norm_shape(q.shape, w, "quarter"),
              lambda: T.triattn_relpos_fwd(t, torch.zeros(1, 4, 9, 9, dtype=torch.bfloat16)),
              lambda: T.triattn_relpos_fwd(t),                                # neither base nor positions
              lambda: T.triattn_relpos_fwd(t[0]),
              lambda: T.triattn_relpos_bwd(torch.zeros(4, 9, 9), 65),
              lambda: T.relpos_shape(1, 9, 4, 65, "rows"),
              lambda: T.relpos_shape(1, 9, 4, 65, kind="linear")):
        with pytest.raises(ValueError):
            f()
