"""FP64 oracle of the orthogonalisation by Newton-Schulz products (test
infrastructure only): the formula as it stands, in float64 numpy."""
from __future__ import annotations

import numpy as np

from .trimul import _f64

COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def orthogonalize(g, steps=5, coefficients=COEFFICIENTS, eps=1e-7):
    x = _f64(g)
    a, b, c = (float(np.float32(v)) for v in coefficients)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    x = x / (np.sqrt((x * x).sum()) + float(np.float32(eps)))
    for _ in range(steps):
        s = x @ x.T
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.T if tall else x
