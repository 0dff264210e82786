"""The norms, the position bias and the orthogonalisation where the very first run of
the process is inside a graph capture (no warm-up), and in two graphs that are
replayed in turn."""
import os
import subprocess
import sys

import pytest
import torch

from protein_folding_triangle_gb300 import triattn as T

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import sys
import torch
from protein_folding_triangle_gb300 import triattn as T

T.load()
torch.manual_seed(1)
N, count = int(sys.argv[1]), int(sys.argv[2])
q, k, dq, dk = (torch.randn(1, 3, 2, N, 16, device="cuda").bfloat16() for _ in range(4))
w = torch.rand(2, 16, device="cuda")
table, planes = torch.randn(9, 8, device="cuda"), torch.randn(1, 8, N, N, device="cuda").bfloat16()
pairs = torch.randn(1, N, N, 8, device="cuda").bfloat16()
ms = [torch.randn(64 + i % 3, 90, device="cuda") for i in range(count)] + [torch.randn(200, 300, device="cuda")]


def calls():
    how = dict(max_distance=4)
    return [*T.triattn_qk_norm_fwd(q, k, w, w), *T.triattn_qk_norm_bwd(q, k, w, w, dq, dk),
            T.triattn_relpos_fwd(table, planes, **how), T.triattn_relpos_bwd(planes, 9, **how),
            T.triattn_relpos_fwd(table, pairs, layout="pairs", **how),
            T.triattn_relpos_bwd(pairs, 9, layout="pairs", **how), *T.triattn_orthogonalize(ms)]


torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = calls()
for _ in range(2):
    graph.replay()
torch.cuda.synchronize()
assert T.device_status() == T.OK
for a, b in zip(got, calls()):
    assert torch.equal(a, b)
"""


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from protein_folding_triangle_gb300 import build
    build.build()
    T.load()


@pytest.mark.parametrize("N,count", [(33, 3), (64, 300)])
def test_first_call_in_a_capture(N, count):
    r = subprocess.run([sys.executable, "-c", SCRIPT, str(N), str(count)], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]


def test_two_graphs_with_their_own_lists():
    """Each holds its own list of matrices (300, past what a launch's parameters
    hold, and a short one); replayed in turn, eager calls of a third between them."""
    g = torch.Generator(device="cuda").manual_seed(5)
    lists = [[torch.empty(3 + i % 40, 50 + i, device="cuda").normal_(generator=g) for i in range(n)]
             for n in (300, 9, 20)]
    outs = [[torch.empty(t.shape, dtype=torch.bfloat16, device="cuda") for t in ts] for ts in lists]
    want = [T.triattn_orthogonalize(ts) for ts in lists]
    torch.cuda.synchronize()
    graphs = []
    for k in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[k]):
            T.triattn_orthogonalize(lists[k], out=outs[k])
    for k in (0, 1, 1, 0, 1):
        for o in outs[k]:
            o.zero_()
        graphs[k].replay()
        T.triattn_orthogonalize(lists[2], out=outs[2])
        torch.cuda.synchronize()
        for j in (k, 2):
            assert all(torch.equal(a, b) for a, b in zip(outs[j], want[j]))
