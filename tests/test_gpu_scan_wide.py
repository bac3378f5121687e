"""The scan of many channels against the fp64 oracle: above 1,152 channels the tiles are smaller
and more blocks share an SM, and the gradients may run with one tile on its way.  The lengths are
several turns of a cluster; the oracle takes a slice of the channels."""
import numpy as np
import pytest
import torch

from linear_attention_12_b200 import gdn
from oracle import scan as oscan
from tests.test_gpu_scan import TYPES, U, _case, _cuda, _half_step, _limit, _np64

pytestmark = pytest.mark.gpu


def _check_channels(x, la, h0, dh, df, cu):
    """What test_gpu_scan's check does, with the same limits, at a few channels: the first tile's,
    those at a tile's border in the middle, and the last ones."""
    io, gate = x.dtype, la.dtype
    C = x.shape[1]
    mid = C // 2 // 64 * 64
    at = sorted({*range(8), *range(32, 36), *range(mid - 4, mid + 4), *range(C - 8, C)})
    cut = lambda t: None if t is None else t[:, at]
    sx, sla, sh0, sdh, sdf = map(cut, (x, la, h0, dh, df))
    end = x.shape[0] if cu is None else int(cu[-1])
    cx, cla, ch0, cdh, cdf, ccu = _cuda(x, la, h0, dh, df, cu)
    h, hf = gdn.scan(cx, cla, ch0, ccu, h=torch.full_like(cx, float("nan")))
    rh, rf = oscan.scan(sx, sla, sh0, cu)
    lim, flim, _ = _limit(sx, sla, sh0, cu)
    got = _np64(h)
    assert np.isnan(got[end:]).all() and np.isfinite(got[:end]).all()
    assert (np.abs(got[:, at] - rh) <= lim * (1 + _half_step(io)) +
            _half_step(io) * np.abs(rh))[:end].all()
    assert (np.abs(_np64(hf)[:, at] - rf) <= flim).all()

    hc = h.nan_to_num(0.0)
    dx, dla, dh0 = gdn.scan_backward(cla, hc, cdh, ch0, cdf, ccu,
                                     dx=torch.full_like(cx, float("nan")),
                                     dlog_alpha=torch.full_like(cla, float("nan")))
    sh = hc.cpu()[:, at]
    rx, rl, r0 = oscan.scan_backward(sla, sh, sdh, sh0, sdf, cu)
    mag = lambda t: None if t is None else t.abs()
    gabs, labs, uabs = oscan.scan_backward(sla, sh.abs(), sdh.abs(), mag(sh0), mag(sdf), cu)
    more, lmore, umore = oscan.scan_backward(sla, sh.abs(), 8 * np.nan_to_num(gabs), mag(sh0),
                                             None, cu)
    for out, ref, lim, step in ((dx, rx, U * (64 * gabs + more), _half_step(io)),
                                (dla, rl, U * (64 * labs + lmore), _half_step(gate))):
        got = _np64(out)
        assert np.isnan(got[end:]).all() and np.isfinite(got[:end]).all()
        assert (np.abs(got[:, at] - ref) <= lim * (1 + step) + step * np.abs(ref))[:end].all()
    assert (np.abs(_np64(dh0)[:, at] - r0) <= U * (64 * uabs + umore)).all()
    assert gdn.last_device_error() == gdn.GDN_OK


def _packed(T, N, seed):
    g = torch.Generator().manual_seed(seed)
    cuts = sorted(torch.randint(0, T + 1, (N - 2,), generator=g).tolist())
    return [0, *cuts, cuts[-1], T]  # (one empty sequence at least)


# 6,144 aligned channels of bf16 run the gradients with one tile on its way
@pytest.mark.parametrize("io,gate", TYPES)
@pytest.mark.parametrize("T,C", [(2500, 1280), (2049, 2048), (2500, 3001), (1500, 6144),
                                 (700, 1153), (130, 4099)])
@pytest.mark.parametrize("N", [1, 9])
def test_many_channels(T, C, N, io, gate):
    cu = None if N == 1 else _packed(T, N, T + C)
    _check_channels(*_case(T, C, cu, io, gate, T + C, h0=N > 1, mu=-2.0))


@pytest.mark.parametrize("io,gate", TYPES)
@pytest.mark.parametrize("C", [1280, 2051])
def test_many_channels_and_padding(C, io, gate):
    """Rows behind the last sequence are neither used nor written."""
    x, la, h0, dh, df, cu = _case(1300, C, [0, 300, 300, 1111], io, gate, C)
    for t in (x, la, dh):
        t[1111:] = float("nan")
    _check_channels(x, la, h0, dh, df, cu)


@pytest.mark.parametrize("C", [1280, 2051])
def test_many_channels_and_short_sequences(C):
    """Several boundaries within a warp's rows."""
    lens = torch.randint(0, 12, (200,), generator=torch.Generator().manual_seed(7)).tolist()
    cu = np.cumsum([0, *lens]).tolist()
    _check_channels(*_case(cu[-1], C, cu, torch.bfloat16, torch.float32, 9))
