"""The dense product with its epilogue.

Oracle (test infrastructure only; see the package docstring). No counterpart in the pages: the router's product and a
layer's dense projections.
"""

import numpy as np
from scipy import special


def linear(x, w, bias=None, activation=None, residual=None):
    """(y, tol) float64: y = act(x w^T + bias) + residual, nothing rounded, and a bound of what FP32 sums, activation and
    addition may be off. u = 2^-24: the product's sum, taken 16 terms at a time by units that may truncate, is within
    (K/16 + 24) 2 u of its terms' magnitudes; no activation is steeper than 1.13; sigmoid, SiLU and GELU are within 16 u
    of their value, GELU's tail, whose logarithm's slope is z, within 4 z^2 u more."""
    u = 2.0 ** -24
    x, w = np.asarray(x, dtype=np.float64), np.asarray(w, dtype=np.float64)
    z = x @ w.T
    tol = (x.shape[1] / 16 + 24) * 2 * u * (np.abs(x) @ np.abs(w).T)
    if bias is not None:
        z = z + np.asarray(bias, dtype=np.float64)
        tol = tol + u * np.abs(z)
    slope, rel = {None: (1.0, 0.0), "relu": (1.0, 0.0), "silu": (1.1, 16.0), "gelu": (1.13, 16.0),
                  "sigmoid": (0.25, 16.0)}[activation]
    if activation == "gelu":
        rel = 16 + 4 * z * z
    y = {None: lambda v: v, "relu": lambda v: np.maximum(v, 0), "silu": lambda v: v * special.expit(v),
         "gelu": lambda v: v * special.ndtr(v), "sigmoid": special.expit}[activation](z)
    tol = slope * tol + rel * u * np.abs(y) + 2.0 ** -126
    if residual is not None:
        y = y + np.asarray(residual, dtype=np.float64)
        tol = tol + u * np.abs(y)
    return y, tol
