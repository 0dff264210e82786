"""The transition on tensors of several row tiles per CTA pair: a wave is 76
pairs of 256 rows, 19456 rows, so that 45003 rows give every pair two or three
tiles and reach the loops over them (phases of the barriers that turn over, row
tiles and weights that are loaded again, one or two z tiles in shared memory).

Tolerances as in test_gpu_transition.py, here for every tile of 256 rows alone:
a tile's relative RMSE is over 256 C elements or more of the same distribution,
so a tile that is stale, or taken from another row, is off by about sqrt(2)."""
import numpy as np
import pytest
import torch

from parity_utils import cpu64, rel_rmse
from oracle import transition as TR
from protein_folding_triangle_gb300 import synthetic as S
from protein_folding_triangle_gb300 import triattn as T

pytestmark = pytest.mark.gpu

TOL_OUT = 8e-3
TOL_GRADS = 1e-2
NAMES = ("dz", "dln_w", "dln_b", "dw_in", "dw_o")
ROWS = 45003


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from protein_folding_triangle_gb300 import build
    build.build()
    T.load()


def params(d):
    return d["z"], d["mask"], d["ln_w"], d["ln_b"], d["w_in"], d["w_o"]


def worst_tile(got, ref):
    """Largest relative RMSE of a tile of 256 rows."""
    return max(rel_rmse(got[i:i + 256], ref[i:i + 256]) for i in range(0, len(ref), 256))


# (C, H, drop): hidden widths of one 64-wide chunk and of several, with W_in in
# shared memory throughout and through its ring
CASES = [(32, 64, 0.1), (64, 256, 0.0), (64, 1504, 0.1), (96, 96, 0.2), (128, 64, 0.0), (128, 512, 0.1),
         (160, 32, 0.1), (160, 320, 0.0), (192, 64, 0.0), (192, 768, 0.1), (224, 96, 0.1), (256, 64, 0.0),
         (256, 1024, 0.1)]


@pytest.mark.parametrize("C,H,drop", CASES)
def test_several_tiles_per_pair(C, H, drop):
    x = S.make_transition_inputs((ROWS,), C, H, seed=C + H, drop=drop)
    d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}
    ref = TR.run(*params(x), x["d_out"])
    out = T.triattn_transition_fwd(*params(d))
    grads = T.triattn_transition_bwd(*params(d), d["d_out"])
    torch.cuda.synchronize()
    assert T.device_status() == T.OK
    assert worst_tile(cpu64(out), ref["out"]) <= TOL_OUT
    assert worst_tile(cpu64(grads[0]), ref["dz"]) <= TOL_GRADS
    for n, g in zip(NAMES[1:], grads[1:]):
        assert rel_rmse(cpu64(g), ref[n]) <= TOL_GRADS, n
    for _ in range(3):  # the same bits whatever the order in which tiles came
        assert torch.equal(T.triattn_transition_fwd(*params(d)), out)
    again = T.triattn_transition_bwd(*params(d), d["d_out"])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, grads)) and T.device_status() == T.OK


@pytest.mark.parametrize("C", [32, 96, 160, 192, 224, 256])
@pytest.mark.parametrize("M", [19456, 19457, 38912, 38913])
def test_forward_at_the_edge_of_a_wave(C, M):
    """Whole waves, and one row more: a pair with a tile that the others do not
    have, of which one CTA has one row and the other none."""
    x = S.make_transition_inputs((M,), C, 64, seed=C)
    d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}
    buf = torch.full((M + 2, C), 7.0, dtype=torch.bfloat16, device="cuda")
    T.triattn_transition_fwd(*params(d), out=buf[1:M + 1])
    torch.cuda.synchronize()
    assert T.device_status() == T.OK
    got = cpu64(buf[1:M + 1])
    assert worst_tile(got[: M // 256 * 256], TR.run(*params(x))["out"][: M // 256 * 256]) <= TOL_OUT
    last = np.abs(got[-1] - TR.run(*params(dict(x, z=x["z"][-1:])))["out"][0])
    # one row is C elements, not 256 C: every rounding at its largest gives 1.06e-2
    assert np.sqrt((last ** 2).mean()) <= 2 * TOL_OUT * np.sqrt((got[-1] ** 2).mean())
    assert bool((buf[0] == 7.0).all()) and bool((buf[M + 1] == 7.0).all())


@pytest.mark.parametrize("C,H", [(160, 32), (192, 128), (224, 64), (256, 96)])
def test_wide_rows_under_load(C, H):
    """At C > 128 both CTAs of a pair write x to their shared memory and one of
    them starts the products on both: the same bits in every one of many calls,
    with a second stream's calls and memory traffic beside them."""
    x = S.make_transition_inputs((ROWS,), C, H, seed=C, drop=0.1)
    d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}
    ref = T.triattn_transition_fwd(*params(d))
    streams = [torch.cuda.Stream() for _ in range(2)]
    noise = torch.zeros(64 << 20, device="cuda")
    torch.cuda.synchronize()
    outs = [[torch.full_like(ref, 9.0) for _ in range(12)] for _ in streams]
    torch.cuda.synchronize()
    for k in range(12):
        for s, o in zip(streams, outs):
            T.triattn_transition_fwd(*params(d), out=o[k], stream=s)
        noise.add_(1.0)
    torch.cuda.synchronize()
    assert T.device_status() == T.OK
    assert all(torch.equal(o, ref) for os in outs for o in os)
