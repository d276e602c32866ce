"""Norm oracle in float64: h = x + residual, y = h / sqrt(mean(h^2) + eps) * w,
and its gradient.

Test infrastructure only (see ``oracle/__init__``).  The forward follows the
root-mean-square norm's definition (Zhang and Sennrich, "Root Mean Square
Layer Normalization", eq. 4, with eps under the root); the gradient is
checked against central differences of the forward in the tests.
"""

import numpy as np


def rms_norm(x, weight, eps, residual=None):
    """(h, y) of float64 rows x [T, H]."""
    h = np.asarray(x, dtype=np.float64)
    if residual is not None:
        h = h + np.asarray(residual, dtype=np.float64)
    size = np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    return h, h / size * np.asarray(weight, dtype=np.float64)


def rms_norm_grad(dy, h, weight, eps, dh=None):
    """{"dx", "dw"} and, for error bounds, "dx_mag" and "dw_mag": the sums of
    the magnitudes of the terms that dx and dw add up."""
    dy, h, w = (np.asarray(a, dtype=np.float64) for a in (dy, h, weight))
    r = 1.0 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    g = dy * w
    dx = r * g - h * r ** 3 * np.mean(g * h, axis=1, keepdims=True)
    mag = np.abs(r * g) + np.abs(h) * r ** 3 * np.mean(np.abs(g * h), axis=1, keepdims=True)
    if dh is not None:
        dx = dx + dh
        mag = mag + np.abs(dh)
    terms = dy * h * r
    return {"dx": dx, "dw": terms.sum(axis=0), "dx_mag": mag, "dw_mag": np.abs(terms).sum(axis=0)}
