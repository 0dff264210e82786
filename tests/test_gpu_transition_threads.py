"""Host threads whose first calls of one width run at the same time: ctypes
releases the interpreter's lock, so both are inside the library at once.  Each
width and activation is a kernel of its own that is set up by its first call, so
the test runs in a process of its own."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import threading
import torch
from protein_folding_triangle_gb300 import synthetic as S, triattn as T

T.load()
names = ("z", "mask", "ln_w", "ln_b", "w_in", "w_o")
bad, got = [], {}
SIZES = (32, 160, 320, 2048)
for C in (32, 64, 96, 128, 160, 192, 224, 256):
    data = {}
    for H in SIZES:
        x = S.make_transition_inputs((300,), C, H, seed=H)
        data[H] = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}
    torch.cuda.synchronize()
    for kind in ("silu", "sigmoid", "gelu"):
        meet = threading.Barrier(4 * len(SIZES))

        def work(i, H):
            d = data[H]
            out = torch.empty_like(d["z"])
            meet.wait()
            try:
                for _ in range(20):
                    T.triattn_transition_fwd(*(d[n] for n in names), kind, out=out)
                T.triattn_transition_bwd(*(d[n] for n in names), d["d_out"], kind)
                got[C, kind, i] = out
            except Exception as e:
                bad.append((C, kind, H, str(e)))

        ts = [threading.Thread(target=work, args=(i, H)) for i, H in enumerate(SIZES * 4)]
        [t.start() for t in ts]
        [t.join() for t in ts]
        torch.cuda.synchronize()
        for i, H in enumerate(SIZES * 4):
            ref = T.triattn_transition_fwd(*(data[H][n] for n in names), kind)
            if (C, kind, i) in got and not torch.equal(got[C, kind, i], ref):
                bad.append((C, kind, H, "other output"))
assert T.device_status() == T.OK
print("BAD", bad)
raise SystemExit(1 if bad else 0)
"""


def test_first_calls_of_several_threads():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from protein_folding_triangle_gb300 import build
    build.build()
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
