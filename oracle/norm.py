"""RMS norm with the residual's addition, its 8-bit output and its gradient.

TEST INFRASTRUCTURE ONLY (see the package docstring): nothing in the product
path may import or call this module.

The statistic and the products are float64; y is rounded to float32 once and
from there to bf16, as the library documents.  The pages name no norm; the
formula is the usual one (no mean subtraction, eps inside the root).
"""
from __future__ import annotations

import numpy as np

from .numerics import bf16_rne

F64 = np.float64


def forward(x, gamma, eps, residual=None):
    """(s, y, r): the bf16 stream, the bf16 output and 1 / rms (float64), for bf16 values in float32 arrays."""
    x = np.asarray(x, np.float32)
    s = x if residual is None else bf16_rne(x + np.asarray(residual, np.float32))
    s64 = s.astype(F64)
    r = 1.0 / np.sqrt(np.mean(s64 * s64, axis=-1) + eps)
    with np.errstate(over="ignore"):
        y32 = (s64 * np.asarray(gamma, F64) * r[:, None]).astype(np.float32)
    return s, bf16_rne(y32), r


def backward(s, gamma, r, dy, dsum=None):
    """(dx, dgamma) in float64: gradients of sum(dy * y) + sum(dsum * s) on s and gamma, r the forward's 1 / rms."""
    s, gamma, dy, r = (np.asarray(v, F64) for v in (s, gamma, dy, r))
    r = r[:, None]
    a = dy * gamma
    dx = r * (a - s * r * r * np.mean(a * s, axis=-1, keepdims=True))
    if dsum is not None:
        dx = dx + np.asarray(dsum, F64)
    return dx, np.sum(dy * s * r, axis=0)
