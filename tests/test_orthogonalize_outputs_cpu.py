"""Outputs that share elements are refused, outputs that lie beside one another are not,
without a GPU: a call that passes the check is answered for its workspace."""
import itertools

import pytest

from protein_folding_triangle_gb300 import triattn as T
from test_orthogonalize_cpu import call, lib, table  # noqa: F401

AT = 1 << 24


def answer(lib, *outs):  # (element, rows, columns, stride) of one buffer  # noqa: F811
    ms = table(*((AT << 8 | i << 20, r, c, c, 0) for i, (_, r, c, _) in enumerate(outs)))
    dst = table(*((AT + 2 * at, r, c, s, 0) for at, r, c, s in outs))
    return call(lib, ms, dst, len(outs), ws=1 << 20, nbytes=0)


@pytest.mark.parametrize("outs", [
    [(0, 8, 9, 9), (72, 8, 9, 9)],                                     # one behind the other
    [(0, 8, 16, 40), (16, 8, 24, 40)],                                 # two blocks of columns
    [(0, 64, 128, 388), (128, 64, 128, 388), (256, 64, 128, 388), (384, 64, 4, 388)],
    [(16, 8, 8, 40), (40 * 4, 4, 16, 40), (0, 3, 16, 40)],             # of other rows
    [(0, 8, 16, 40), (16, 1, 24, 24), (40 + 16, 1, 24, 24)],           # single rows beside a block
    [(0, 8, 1, 4), (1, 8, 1, 4), (2, 8, 2, 4)],                        # single columns
    [(0, 8, 9, 40), (8 * 40, 3, 5, 7)],                                # behind, of another stride
    [(0, 0, 9, 9), (0, 8, 9, 9)]])                                     # one without elements
def test_apart(lib, outs):  # noqa: F811
    for order in itertools.permutations(outs):
        assert answer(lib, *order) == T.ERR_WORKSPACE


@pytest.mark.parametrize("outs", [
    [(0, 8, 9, 9), (71, 8, 9, 9)],
    [(0, 8, 17, 40), (16, 8, 24, 40)],                                 # a column of both
    [(0, 8, 16, 40), (16, 8, 25, 40)],                                 # into the next row
    [(0, 8, 16, 40), (40 * 7 + 15, 1, 1, 1)],
    [(0, 8, 16, 40), (40 * 7 + 16, 4, 24, 40), (40 * 8, 1, 17, 17)],   # of three, two that are not neighbours
    [(0, 1, 50, 50), (40, 8, 5, 5)],
    [(0, 8, 16, 40), (20, 8, 4, 20)],                                  # other strides: taken to overlap
    [(0, 8, 9, 9), (0, 8, 9, 9)]])
def test_overlapping(lib, outs):  # noqa: F811
    for order in itertools.permutations(outs):
        assert answer(lib, *order) == T.ERR_INVALID_ARG


def test_against_the_elements(lib):  # noqa: F811
    """Every pair of small matrices: what shares an element is refused; what is apart is not
    refused where both are blocks of columns of the same rows."""
    shapes = [(r, c, s) for r in (1, 2, 3) for s in (4, 6) for c in (1, 2, 4)]

    def elements(at, r, c, s):
        return {at + i * s + j for i in range(r) for j in range(c)}
    refused = 0
    for (r, c, s), (r2, c2, s2), at in itertools.product(shapes, shapes, range(14)):
        got = answer(lib, (at, r, c, s), (5, r2, c2, s2))
        if elements(at, r, c, s) & elements(5, r2, c2, s2):
            assert got == T.ERR_INVALID_ARG
            refused += 1
        elif s == s2 and r == r2 and c + max(at - 5, 0) % s <= s and (at - 5) % s >= c2 and (5 - at) % s >= c:
            assert got == T.ERR_WORKSPACE, (at, r, c, s, r2, c2)
    assert refused > 1000
