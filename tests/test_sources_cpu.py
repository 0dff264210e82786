"""What the library's sources must not hold."""
import glob
import os
import re

from protein_folding_triangle_gb300 import build as B


def test_no_copy_to_several_ctas_at_once():
    """The library is loaded by programs of several GPUs, and its kernels read memory of the
    caller's: no bulk copy goes to the shared memory of several CTAs at once."""
    copy = re.compile(r"cp\.async\.bulk[^;\"]*multi" + "cast")
    files = [p for d in (B.CSRC, B.INCLUDE) for p in glob.glob(os.path.join(d, "**", "*"), recursive=True)
             if os.path.isfile(p)]
    assert len(files) > 20
    for p in files:
        with open(p, errors="replace") as f:
            assert copy.search(f.read()) is None, p
