"""Calls whose very first run of the process is inside a graph capture (no warm-up),
and graphs that hold lists of gradients too long for the kernels' parameters."""
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
from protein_folding_triangle_gb300 import synthetic as S, triattn as T

T.load()
names = ("z", "mask", "ln_w", "ln_b", "w_in", "w_o")
C, rows = int(sys.argv[1]), int(sys.argv[2])
x = S.make_transition_inputs((rows,), C, 96, seed=C, drop=0.2)
d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}
gs = [torch.ones(10 + i, device="cuda") for i in range(int(sys.argv[3]))]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = T.triattn_transition_fwd(*(d[n] for n in names))
    grads = T.triattn_transition_bwd(*(d[n] for n in names), d["d_out"])
    norm = T.triattn_clip_grad_norm(gs, 1e9)
for _ in range(2):
    graph.replay()
torch.cuda.synchronize()
assert T.device_status() == T.OK
assert torch.equal(out, T.triattn_transition_fwd(*(d[n] for n in names)))
for a, b in zip(grads, T.triattn_transition_bwd(*(d[n] for n in names), d["d_out"])):
    assert torch.equal(a, b)
assert torch.equal(norm, T.triattn_grad_norm(gs))
"""


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from protein_folding_triangle_gb300 import build
    build.build()
    T.load()


@pytest.mark.parametrize("C,rows,n", [(128, 700, 30), (64, 100, 200), (256, 700, 200), (160, 100, 30)])
def test_first_call_in_a_capture(C, rows, n):
    r = subprocess.run([sys.executable, "-c", SCRIPT, str(C), str(rows), str(n)], cwd=ROOT, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]


def test_two_graphs_with_long_lists():
    """Each holds its own list; replayed in turn, with eager calls of a third list
    between them."""
    g = torch.Generator(device="cuda").manual_seed(3)
    lists = [[torch.empty(50 + 13 * i, device="cuda").normal_(generator=g) for i in range(n)] for n in (150, 1100, 97)]
    outs = [[torch.empty_like(t) for t in ts] for ts in lists]
    refs = [[torch.empty_like(t) for t in ts] for ts in lists]
    want = [T.triattn_clip_grad_norm(ts, 1.0, out=r) for ts, r in zip(lists, refs)]
    torch.cuda.synchronize()
    graphs, norms = [], []
    for k in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[k]):
            norms.append(T.triattn_clip_grad_norm(lists[k], 1.0, out=outs[k]))
    for k in (0, 1, 1, 0, 1):
        for o in outs[k]:
            o.zero_()
        graphs[k].replay()
        third = T.triattn_clip_grad_norm(lists[2], 1.0, out=outs[2])
        torch.cuda.synchronize()
        assert torch.equal(norms[k], want[k]) and torch.equal(third, want[2])
        for j in (k, 2):
            assert all(torch.equal(a, b) for a, b in zip(outs[j], refs[j]))
