"""Residual addition, RMS norm and its backward; the global gradient norm (oracle).

Test infrastructure only (see ``oracle/__init__.py``).

The norm divides a row by its root mean square and multiplies by a learned
weight; the layer's input is the normed residual stream.  Rounding steps of
the forward, in this order:
  h    = BF16(fl32(x + r))
  rstd = fl32(1 / sqrt(mean h^2 + eps))        evaluated in float64
  y    = BF16(fl32(fl32(h * rstd) * w))
and the 1x128 tiles of y by ``quant.quant_1x128``.
"""

import numpy as np

from .fp8 import bf16_round
from .quant import quant_1x128


def rmsnorm(x, residual, weight, eps, rule="fp32"):
    """x, residual [T, d] and weight [d] float32 arrays of BF16 values (residual may be None).
    Returns dict(sum, y, q, scale, rstd)."""
    x = np.asarray(x, np.float32)
    h = x if residual is None else bf16_round(x + np.asarray(residual, np.float32))
    ms = np.square(h.astype(np.float64)).sum(1) / h.shape[1]
    rstd = (1.0 / np.sqrt(ms + np.float64(np.float32(eps)))).astype(np.float32)
    y = bf16_round((h * rstd[:, None]).astype(np.float32) * np.asarray(weight, np.float32))
    q, scale = quant_1x128(y, rule)
    return dict(sum=h, y=y, q=q, scale=scale, rstd=rstd)


def rmsnorm_backward(dy, h, weight, rstd, dres=None):
    """(dh [T, d], dw [d]) in float64, unrounded."""
    dy, h, w = (np.asarray(a, np.float64) for a in (dy, h, weight))
    rs = np.asarray(rstd, np.float64)[:, None]
    xh, g = h * rs, dy * w
    dh = rs * (g - xh * (g * xh).mean(1, keepdims=True))
    if dres is not None:
        dh = dh + np.asarray(dres, np.float64)
    return dh, (dy * xh).sum(0)


def grad_norm(tensors, max_norm):
    """(norm, coef) in float64 over a list of arrays."""
    n = float(np.sqrt(sum(float(np.square(np.asarray(t, np.float64)).sum()) for t in tensors)))
    return n, 1.0 if n <= max_norm else max_norm / n
