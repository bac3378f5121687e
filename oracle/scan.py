"""fp64 CPU oracle for the per-channel gated recurrence -- TEST INFRASTRUCTURE ONLY.

Only ``tests/`` may import this module; it shares no code with the CUDA library.

    h_t = exp(log_alpha_t) h_{t-1} + x_t        within each packed sequence,

from ``h0`` (or zeros); ``h_final`` is the last state, ``h0`` for an empty sequence.
The gradients of ``<dh, h> + <dh_final, h_final>`` are the chain rule of that line,
token by token backwards; ``h`` may be given (the library reads the rounded forward
output) or is recomputed.
"""
from __future__ import annotations

import numpy as np

from . import _as_np, _widen


def _np(x):
    return None if x is None else _widen(_as_np(x)).astype(np.float64)


def _seqs(cu_seqlens, T):
    cu = [0, T] if cu_seqlens is None else [int(c) for c in cu_seqlens]
    return list(zip(cu[:-1], cu[1:]))


def scan(x, log_alpha, h0=None, cu_seqlens=None):
    x, a, h0 = _np(x), np.exp(_np(log_alpha)), _np(h0)
    seqs = _seqs(cu_seqlens, x.shape[0])
    h = np.full(x.shape, np.nan)
    final = np.zeros((len(seqs), *x.shape[1:])) if h0 is None else h0.copy()
    for n, (lo, hi) in enumerate(seqs):
        for t in range(lo, hi):
            final[n] = a[t] * final[n] + x[t]
            h[t] = final[n]
    return h, final


def scan_backward(log_alpha, h, dh, h0=None, dh_final=None, cu_seqlens=None):
    """``(dx, dlog_alpha, dh0)``; rows outside every sequence stay NaN."""
    a, h, dh, h0, dh_final = (np.exp(_np(log_alpha)), *map(_np, (h, dh, h0, dh_final)))
    seqs = _seqs(cu_seqlens, dh.shape[0])
    dx, dla = np.full(dh.shape, np.nan), np.full(dh.shape, np.nan)
    dh0 = np.zeros((len(seqs), *dh.shape[1:])) if dh_final is None else dh_final.copy()
    for n, (lo, hi) in enumerate(seqs):
        for t in range(hi - 1, lo - 1, -1):
            dx[t] = dh[t] + dh0[n]
            dh0[n] = a[t] * dx[t]
            before = h[t - 1] if t > lo else (0.0 if h0 is None else h0[n])
            dla[t] = dh0[n] * before
    return dx, dla, dh0
