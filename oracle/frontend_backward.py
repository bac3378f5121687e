"""fp64 CPU oracle for the front end's gradients -- TEST INFRASTRUCTURE ONLY.

Only ``tests/`` may import this module; it shares no code with the CUDA library.

The chain rule of ``oracle/frontend.py``'s lines, from the gradients of q, k, v,
log_alpha and beta to those of the raw inputs, the convolution weight and the gate
pre-activations, token by token within each sequence:

    du      = dv, or J dq with q = u / sqrt(u.u + eps):  r (dq - q <q, dq>), r = 1 / sqrt(u.u + eps)
    dy      = du act'(y)
    dx[t-j] += w[3 - j] dy[t],   dw[3 - j] += dy[t] x[t - j],   j = 0..3, t - j in the sequence
    da      = -sigmoid(a) dlog_alpha,   db = beta (1 - beta) dbeta
"""
from __future__ import annotations

import numpy as np

from . import _as_np, _widen
from .frontend import causal_conv, sigmoid


def frontend_backward(q_raw, k_raw, v_raw, conv_w, a, b, dq, dk, dv, dlog_alpha, dbeta,
                      cu_seqlens=None, act="none", eps=1e-6):
    """``(dq_raw, dk_raw, dv_raw, dconv_w, da, db)``; rows behind the last sequence are NaN."""
    T = q_raw.shape[0]
    cu = [0, T] if cu_seqlens is None else [int(c) for c in cu_seqlens]
    weights = _as_np(conv_w).astype(np.float64)
    outs, dws, at = [], [], 0
    for kind, (raw, grad) in enumerate(((q_raw, dq), (k_raw, dk), (v_raw, dv))):
        shape = tuple(raw.shape)
        C = shape[1] * shape[2]
        x, w = _widen(raw).reshape(T, C), weights[at:at + C]
        at += C
        y = causal_conv(x, w, cu)
        s = sigmoid(y)
        u, slope = (y * s, s + y * s * (1 - s)) if act == "silu" else (y, np.ones_like(y))
        du = _widen(grad)
        if kind < 2:
            u3 = u.reshape(shape)
            r = 1.0 / np.sqrt((u3 * u3).sum(-1, keepdims=True) + eps)
            q = u3 * r
            du = r * (du - q * (q * du).sum(-1, keepdims=True))
        dy = du.reshape(T, C) * slope
        dx, dw = np.full((T, C), np.nan), np.zeros((C, 4))
        for lo, hi in zip(cu[:-1], cu[1:]):
            dx[lo:hi] = 0.0
            for t in range(lo, hi):
                for j in range(min(3, t - lo) + 1):
                    dx[t - j] += w[:, 3 - j] * dy[t]
                    dw[:, 3 - j] += dy[t] * x[t - j]
        outs.append(dx.reshape(shape))
        dws.append(dw)
    ad, bd = _widen(a), _widen(b)
    be = sigmoid(bd)
    da, db = -sigmoid(ad) * _widen(dlog_alpha), be * (1 - be) * _widen(dbeta)
    da[cu[-1]:] = db[cu[-1]:] = np.nan
    return (*outs, np.concatenate(dws), da, db)
