"""fp64 CPU oracle for the group norm over heads -- TEST INFRASTRUCTURE ONLY.

Only ``tests/`` may import this module; it shares no code with the CUDA library.

Per token and head of ``x [T, H, d]``:

    m  = mean(x) ("mean") or 0 ("rms"),   xh = (x - m) / sqrt(mean((x - m)^2) + eps)
    n  = weight xh + bias
    y  = n act(z) with a gate z, act(n) without;   act = identity or silu

The pages print no formula for it; this is the norm's own definition.  The gradients
are the chain rule of these lines, written per element.
"""
from __future__ import annotations

import numpy as np

from . import _as_np, _widen


def _np(x):
    return None if x is None else _widen(_as_np(x)).astype(np.float64)


def _act(a, act):
    """act(a) and its derivative."""
    if act == "none":
        return a, np.ones_like(a)
    s = 0.5 * (1.0 + np.tanh(0.5 * a))
    return a * s, s + a * s * (1.0 - s)


def _xhat(x, norm, eps):
    c = x - x.mean(-1, keepdims=True) if norm == "mean" else x
    r = 1.0 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    return c * r, r


def group_norm(x, weight, bias=None, z=None, norm="rms", act="silu", eps=1e-6):
    x, weight, bias, z = map(_np, (x, weight, bias, z))
    n = _xhat(x, norm, eps)[0] * weight + (0.0 if bias is None else bias)
    return _act(n, act)[0] if z is None else n * _act(z, act)[0]


def group_norm_backward(dy, x, weight, bias=None, z=None, norm="rms", act="silu", eps=1e-6):
    """``(dx, dweight, dbias, dz)`` of ``<dy, y>`` (None where there is no such input)."""
    has_bias = bias is not None
    dy, x, weight, bias, z = map(_np, (dy, x, weight, bias, z))
    xh, r = _xhat(x, norm, eps)
    n = xh * weight + (0.0 if bias is None else bias)
    dz = None
    if z is None:
        dn = dy * _act(n, act)[1]
    else:
        value, slope = _act(z, act)
        dn, dz = dy * value, dy * n * slope
    axes = (0,) if weight.ndim == 2 else (0, 1)
    dw, db = (dn * xh).sum(axes), dn.sum(axes)
    # xh's Jacobian: r (I - xh xh^T / d), and I - 1 1^T / d in front of it when centred
    e = dn * weight
    dx = r * (e - xh * (e * xh).mean(-1, keepdims=True))
    if norm == "mean":
        dx = dx - dx.mean(-1, keepdims=True)
    return dx, dw, db if has_bias else None, dz
