"""Argument checks of the transition and the gradient norm, without a GPU:
bad calls are answered before anything is launched."""
import ctypes

import pytest
import torch

from protein_folding_triangle_gb300 import build as B
from protein_folding_triangle_gb300 import layers
from protein_folding_triangle_gb300 import triattn as T

FAKE = 1 << 20  # aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    B.build()
    return T.load()


def fwd(lib, shape, **kw):
    names = ("z", "ln_w", "ln_b", "w_in", "w_o", "out")
    p = {n: ctypes.c_void_p(FAKE) for n in names}
    p["mask"] = None
    p.update(kw)
    return lib.triattn_transition_fwd(ctypes.byref(shape), p["z"], p["mask"], p["ln_w"], p["ln_b"], p["w_in"],
                                      p["w_o"], p["out"], None)


def bwd(lib, shape, nbytes, ws=FAKE, **kw):
    names = ("z", "ln_w", "ln_b", "w_in", "w_o", "d_out", "dz", "d_ln_w", "d_ln_b", "d_w_in", "d_w_o")
    p = {n: ctypes.c_void_p(FAKE) for n in names}
    p["mask"] = None
    p.update(kw)
    return lib.triattn_transition_bwd(ctypes.byref(shape), p["z"], p["mask"], p["ln_w"], p["ln_b"], p["w_in"],
                                      p["w_o"], p["d_out"], p["dz"], p["d_ln_w"], p["d_ln_b"], p["d_w_in"],
                                      p["d_w_o"], ctypes.c_void_p(ws), ctypes.c_size_t(nbytes), None)


UNSUPPORTED = [(10, 48, 64), (10, 288, 64), (10, 16, 64), (10, 64, 40), (10, 64, 4128), (1 << 31, 64, 64)]


def test_transition_shapes(lib):
    for M, C, H in [(1, 32, 32), (0, 128, 512), (589824, 128, 512), ((1 << 31) - 1, 256, 4096)]:
        assert T.transition_workspace_bytes(M, C, H) > 0
    for bad in UNSUPPORTED:
        s = T.TransitionShape(*bad, 0, 0)
        assert T.transition_workspace_bytes(*bad) == 0, bad
        assert fwd(lib, s) == T.ERR_UNSUPPORTED and bwd(lib, s, 1 << 40) == T.ERR_UNSUPPORTED, bad
    for bad in [(-1, 64, 64, 0, 0), (1, 0, 64, 0, 0), (1, 64, 0, 0, 0), (1, 64, 64, 3, 0), (1, 64, 64, -1, 0),
                (1, 64, 64, 0, 1)]:
        s = T.TransitionShape(*bad)
        assert lib.triattn_transition_workspace_bytes(ctypes.byref(s)) == 0
        assert fwd(lib, s) == T.ERR_INVALID_ARG and bwd(lib, s, 1 << 40) == T.ERR_INVALID_ARG, bad
    with pytest.raises(ValueError):
        T.transition_shape(1, 64, 64, "tanh")


def test_stream_of_another_device():
    class Stream:
        device = torch.device("cuda", 1)
        cuda_stream = 0

    with pytest.raises(ValueError, match="stream is on cuda:1"):
        T._on_stream(torch.device("cuda", 0), Stream())


def test_transition_pointers_and_workspace(lib):
    s = T.TransitionShape(10, 64, 64, 0, 0)
    nb = T.transition_workspace_bytes(10, 64, 64)
    for n in ("z", "ln_w", "ln_b", "w_in", "w_o", "out"):
        assert fwd(lib, s, **{n: None}) == T.ERR_INVALID_ARG, n
        assert fwd(lib, s, **{n: ctypes.c_void_p(FAKE + 8)}) == T.ERR_INVALID_ARG, n
    for n in ("z", "ln_w", "ln_b", "w_in", "w_o", "d_out", "dz", "d_ln_w", "d_ln_b", "d_w_in", "d_w_o"):
        assert bwd(lib, s, nb, **{n: None}) == T.ERR_INVALID_ARG, n
        assert bwd(lib, s, nb, **{n: ctypes.c_void_p(FAKE + 8)}) == T.ERR_INVALID_ARG, n
    assert fwd(lib, s, mask=ctypes.c_void_p(FAKE + 1)) == T.ERR_INVALID_ARG
    assert bwd(lib, s, nb, mask=ctypes.c_void_p(FAKE + 1)) == T.ERR_INVALID_ARG
    assert bwd(lib, s, nb - 1) == T.ERR_WORKSPACE
    assert bwd(lib, s, nb, ws=FAKE + 16) == T.ERR_WORKSPACE
    assert bwd(lib, s, nb, ws=0) == T.ERR_WORKSPACE
    # no rows: nothing to launch, and nothing to point at
    empty = T.TransitionShape(0, 64, 64, 0, 0)
    assert fwd(lib, empty, z=None, out=None) == T.OK


def table(*entries):
    return (T.Tensor * len(entries))(*entries)


def clip(lib, ts, n, out=None, kind=0, limit=1.0, norm=FAKE, ws=FAKE, nbytes=1 << 30):
    return lib.triattn_clip_grad_norm(ts, out, n, kind, limit, ctypes.c_void_p(norm), ctypes.c_void_p(ws),
                                      ctypes.c_size_t(nbytes), None)


def norm(lib, ts, n, kind=0, out=FAKE, ws=FAKE, nbytes=1 << 30):
    return lib.triattn_grad_norm(ts, n, kind, ctypes.c_void_p(out), ctypes.c_void_p(ws), ctypes.c_size_t(nbytes), None)


def test_grad_norm_refusals(lib):
    ok = table((FAKE, 100, 0), (FAKE + 4096, 100, 1))
    for f in (norm, clip):
        for bad in [table((None, 1, 0)), table((FAKE + 1, 4, 0)), table((FAKE + 2, 4, 1)), table((FAKE, -1, 0))]:
            assert f(lib, bad, 1) == T.ERR_INVALID_ARG
        assert f(lib, table((FAKE, 4, 2)), 1) == T.ERR_UNSUPPORTED
        assert f(lib, table((FAKE, 1 << 40, 0)), 1) == T.ERR_UNSUPPORTED
        assert f(lib, ok, -1) == T.ERR_INVALID_ARG
        assert f(lib, None, 2) == T.ERR_INVALID_ARG
        assert f(lib, ok, 2, kind=2) == T.ERR_INVALID_ARG
        assert f(lib, ok, 2, ws=0) == T.ERR_WORKSPACE
        assert f(lib, ok, 2, ws=FAKE + 16) == T.ERR_WORKSPACE
        assert f(lib, ok, 2, nbytes=lib.triattn_grad_norm_workspace_bytes(2) - 1) == T.ERR_WORKSPACE
    assert norm(lib, ok, 2, out=0) == T.ERR_INVALID_ARG and norm(lib, ok, 2, out=FAKE + 2) == T.ERR_INVALID_ARG
    assert clip(lib, ok, 2, norm=0) == T.ERR_INVALID_ARG
    for limit in (-1.0, float("nan")):
        assert clip(lib, ok, 2, limit=limit) == T.ERR_INVALID_ARG
    assert lib.triattn_grad_norm_workspace_bytes(-1) == 0


def test_clip_refuses_shared_memory(lib):
    a = FAKE
    assert clip(lib, table((a, 100, 0), (a, 100, 0)), 2) == T.ERR_INVALID_ARG        # the same tensor twice
    assert clip(lib, table((a + 4096, 8, 0), (a, 2049, 0)), 2) == T.ERR_INVALID_ARG  # the last element
    src, dst = table((a, 100, 0), (a + 4096, 100, 1)), (a + 8192, a + 16384)
    for o in [table((a, 100, 0), (dst[1], 100, 1)), table((dst[0], 100, 0), (a + 198, 100, 1)),
              table((dst[0], 100, 0), (dst[0] + 100, 100, 1)), table((a + 4096 + 396, 100, 0), (dst[1], 100, 1)),
              table((dst[0], 99, 0), (dst[1], 100, 1)), table((dst[0], 100, 1), (dst[1], 100, 1)),
              table((dst[0] + 1, 100, 0), (dst[1], 100, 1)), table((None, 100, 0), (dst[1], 100, 1))]:
        assert clip(lib, src, 2, out=o) == T.ERR_INVALID_ARG


def test_python_refusals(lib):
    m = layers.Transition(c_z=64)
    assert tuple(m.w_in.shape) == (64, 512) and tuple(m.w_o.shape) == (256, 64)
    assert m.w_in.dtype == torch.bfloat16 and m.ln_w.dtype == torch.float32
    assert tuple(layers.Transition(c_z=64, c_hidden=96).w_o.shape) == (96, 64)
    with pytest.raises(ValueError):
        layers.Transition(c_z=64, activation="relu6")
    with pytest.raises(ValueError):
        m(torch.zeros(3, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        T.triattn_grad_norm([torch.zeros(3)])
    with pytest.raises(ValueError):
        T.triattn_clip_grad_norm([torch.zeros(3)], 1.0, 1.0)


def test_dense_views():
    t = torch.zeros(4, 6, 5)
    assert T._dense(t.permute(2, 0, 1)) and T._dense(t[1:2].transpose(0, 1)) and T._dense(t[:, :1, :1][:1])
    assert not T._dense(t[:, ::2]) and not T._dense(t[:, :, 1:]) and not T._dense(torch.zeros(1).expand(3))
