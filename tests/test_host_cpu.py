"""The binding's native part without a GPU: it takes no call that is not plainly a
usual one, and the general path then says what is wrong."""
import pytest
import torch

from protein_folding_triangle_gb300 import build as B
from protein_folding_triangle_gb300 import triattn as T


@pytest.fixture(scope="module")
def host():
    B.build()
    T.load()
    return T._host()


def test_it_takes_no_other_calls(host):
    q, w = torch.zeros(1, 2, 1, 3, 16, dtype=torch.bfloat16), torch.ones(16)
    table, planes = torch.zeros(65, 4), torch.zeros(1, 4, 9, 9, dtype=torch.bfloat16)
    pos = torch.zeros(1, 3, dtype=torch.int32)
    for bad in (q, q.float(), q[0], None, 3, "q", [q]):  # none of them on a GPU
        assert host.qk_norm_fwd(bad, q, w, w, pos, 1, 1e4, 1e-6) is None
        assert host.qk_norm_bwd(q, q, w, w, bad, q, None, 1, 1e4, 1e-6) is None
        assert host.relpos_fwd(bad, planes, None, None, 0, 0, 32) is None
        assert host.relpos_fwd(table, bad, pos, None, 0, 0, 32) is None
        assert host.relpos_bwd(bad, 65, None, None, 0, 0, 32) is None
    for number in (1 << 40, -(1 << 80), 1.5, None, "half"):
        assert host.qk_norm_fwd(q, q, w, w, None, number, 1e4, 1e-6) is None
        assert host.relpos_bwd(planes, number, None, None, 0, 0, 32) is None
    assert host.qk_norm_fwd(q) is None and host.qk_norm_bwd() is None
    assert host.relpos_fwd() is None and host.relpos_bwd(planes) is None
    for lists in (([q],), ([table], [table], 0), ([table], None, -1), ([3], None, 0), (table, None, 0),
                  ([], [table], 0), ([table], table, 0), ([table], None, "0")):
        assert host.matrix_tables(*lists) is None
    assert host.matrix_tables([], None, 0) == (b"", None) and host.matrix_tables([], [], 0) == (b"", b"")


def test_addresses(host):
    with pytest.raises(TypeError):
        host.bind(1, 2)
    with pytest.raises((ValueError, TypeError)):
        host.bind(0, 0, 0, 0, 0, 0)
    with pytest.raises((ValueError, TypeError)):
        host.bind("a", 1, 1, 1, 1, 1)
