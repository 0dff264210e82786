"""Which views of q and k the norms' module hands on as they are: those that the
library takes, and no others, without a GPU."""
import itertools

import pytest
import torch

from protein_folding_triangle_gb300 import layers
from protein_folding_triangle_gb300 import triattn as T
from test_core_inputs_abi_cpu import lib, qk, shape  # noqa: F401

BUF = torch.empty(1 << 16, dtype=torch.bfloat16)
NAMES = ("q", "k", "w_q", "w_k", "positions", "d_q_out", "d_k_out", "q_out", "k_out", "d_w_q", "d_w_k")
APART = {n: (1 << 20) + (i << 24) for i, n in enumerate(NAMES)}


def taken(lib, B, No, H, N, D, strides):  # noqa: F811
    s = shape(B=B, N_o=No, H=H, N=N, D=D, w_heads=1)
    code = qk(lib, s, (strides, None, None), bwd=True, nbytes=0, **APART)  # a valid call lacks its workspace
    assert code in (T.ERR_WORKSPACE, T.ERR_INVALID_ARG)
    return code == T.ERR_WORKSPACE


@pytest.mark.parametrize("H,N", [(1, 1), (1, 3), (2, 1), (2, 3)])
def test_as_the_library(lib, H, N):  # noqa: F811
    seen = set()
    for strides in itertools.product((0, 8, 12, 16, 24, 32, 48, 64, 96, 128), repeat=3):
        t = BUF.as_strided((1, 2, H, N, 16), (0, *strides, 1))
        want = taken(lib, 1, 2, H, N, 16, strides)
        assert layers._rows(t) == want, strides
        seen.add(want)
    assert seen == {False, True}


def test_others():
    t = BUF[:2 * 2 * 3 * 4 * 16].view(2, 2, 3, 4, 16)
    assert layers._rows(t) and layers._rows(t[:, :1][:1])
    assert not layers._rows(t[:, :1])                          # examples further apart than their slices
    assert not layers._rows(t[0]) and not layers._rows(t.transpose(3, 4))
    assert not layers._rows(BUF[4:4 + t.numel()].view(t.shape))  # from 8 bytes on
    assert layers._rows(t.transpose(2, 3)) and not layers._rows(t[:, :, :2])  # heads of more than are taken
