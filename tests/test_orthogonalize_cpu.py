"""The oracle of the orthogonalisation against the singular value decomposition,
and the entry point's argument checks, without a GPU."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import orthogonalize as OR
from protein_folding_triangle_gb300 import build as B
from protein_folding_triangle_gb300 import triattn as T

FAKE = 1 << 20  # aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    B.build()
    return T.load()


@pytest.mark.parametrize("shape", [(5, 9), (9, 5), (6, 6), (1, 4)])
def test_oracle_is_the_polynomial_of_the_singular_values(shape):
    g = np.random.default_rng(0).normal(size=shape)
    u, s, vt = np.linalg.svd(g, full_matrices=False)
    a, b, c = (float(np.float32(v)) for v in OR.COEFFICIENTS)
    s = s / (np.sqrt((s * s).sum()) + float(np.float32(1e-7)))
    for _ in range(5):
        s = a * s + b * s ** 3 + c * s ** 5
    assert np.abs(OR.orthogonalize(g) - (u * s) @ vt).max() <= 1e-12
    assert (s > 0.6).all() and (s < 1.3).all()


class Matrix(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("rows", ctypes.c_longlong), ("cols", ctypes.c_longlong),
                ("stride", ctypes.c_longlong), ("dtype", ctypes.c_int)]


def table(*entries):
    return (Matrix * max(len(entries), 1))(*entries)


COEF = (ctypes.c_float * 3)(*OR.COEFFICIENTS)


def call(lib, ms, out, n, steps=5, coef=COEF, eps=1e-7, ws=FAKE, nbytes=1 << 50):
    return lib.triattn_orthogonalize(ms, out, n, steps, coef, eps, ctypes.c_void_p(ws), ctypes.c_size_t(nbytes), None)


def test_refusals(lib):
    at = FAKE * 16
    ok, dst = table((FAKE, 8, 9, 9, 0), (FAKE, 8, 9, 16, 1)), table((at, 8, 9, 9, 0), (at + 4096, 8, 9, 9, 0))
    need = lib.triattn_orthogonalize_workspace_bytes(ok, 2)
    assert need > 0 and lib.triattn_orthogonalize_workspace_bytes(None, 0) > 0
    for i, bad in enumerate([(None, 8, 9, 9, 0), (FAKE + 1, 8, 9, 9, 0), (FAKE + 2, 8, 9, 9, 1), (FAKE, -1, 9, 9, 0),
                             (FAKE, 8, -1, 9, 0), (FAKE, 8, 9, 8, 0), (FAKE, 8, 9, 1 << 40, 0)]):
        assert lib.triattn_orthogonalize_workspace_bytes(table(bad), 1) == 0
        assert call(lib, table(bad), dst, 1) == T.ERR_INVALID_ARG, i
        if i != 2:
            assert call(lib, table((FAKE, 8, 9, 9, 0)), table(bad), 1) == T.ERR_INVALID_ARG, i
    for bad in [(FAKE, 8, 9, 9, 2), (FAKE, 65537, 1, 1, 0), (FAKE, 1, 65537, 65537, 0)]:
        assert lib.triattn_orthogonalize_workspace_bytes(table(bad), 1) == 0
        assert call(lib, table(bad), table((at,) + bad[1:4] + (0,)), 1) == T.ERR_UNSUPPORTED
    assert call(lib, ok, table((at, 8, 9, 9, 1), (at + 4096, 8, 9, 9, 0)), 2) == T.ERR_UNSUPPORTED  # an FP32 out
    for bad in [table((at, 8, 9, 9, 0), (at + 142, 8, 9, 9, 0)), table((at, 8, 9, 9, 0), (at, 8, 9, 9, 0)),
                table((at, 8, 9, 40, 0), (at + 200, 8, 9, 9, 0)),                                   # overlapping outs
                table((at, 9, 8, 8, 0), (at + 4096, 8, 9, 9, 0)), None]:
        assert call(lib, ok, bad, 2) == T.ERR_INVALID_ARG
    inf, nan = float("inf"), float("nan")
    for kw in [dict(steps=0), dict(steps=-1), dict(eps=0.0), dict(eps=nan), dict(eps=inf), dict(coef=None),
               dict(coef=(ctypes.c_float * 3)(1.0, nan, 0.0)), dict(n=-1)]:
        assert call(lib, ok, dst, kw.pop("n", 2), **kw) == T.ERR_INVALID_ARG
    assert call(lib, ok, dst, 2, steps=65) == T.ERR_UNSUPPORTED
    assert call(lib, None, dst, 1) == T.ERR_INVALID_ARG
    for kw in [dict(ws=0), dict(ws=FAKE + 16), dict(nbytes=need - 1)]:
        assert call(lib, ok, dst, 2, **kw) == T.ERR_WORKSPACE
    assert call(lib, None, None, 0) == T.OK
    assert call(lib, table((None, 0, 5, 5, 0)), table((None, 0, 5, 5, 0)), 1) == T.OK  # nothing to do


def test_python_refusals(lib):
    t = torch.zeros(3, 4)
    dev = torch.device("cpu")
    for bad in (t[0], t.t(), t.double(), t[:, ::2], t[:1].expand(3, 4)):
        with pytest.raises(ValueError):
            T._matrix_table([bad], "tensors", dev)
    for good in (t, t[:, 1:3], t[:1], t[:, :1], t[::2]):
        assert len(T._matrix_table([good], "tensors", dev)[0]) == 40
    with pytest.raises(ValueError):
        T.triattn_orthogonalize([t])
    with pytest.raises(ValueError):
        T.triattn_orthogonalize([t], coefficients=(1.0, 2.0))
