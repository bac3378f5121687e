"""The per-channel recurrence's oracle against differences and closed forms, and the
refusals of gdn_scan, gdn_scan_backward and gdn_scan_step (CPU only)."""
import numpy as np
import pytest
import torch

from linear_attention_12_b200 import build as gdn_build
from linear_attention_12_b200 import gdn
from oracle import scan as oscan


@pytest.fixture(scope="module")
def L():
    gdn_build.build()
    return gdn.lib()


def test_oracle_closed_form():
    """h_t = sum_s exp(sum_{s < r <= t} log_alpha_r) x_s + exp(sum_{r <= t} log_alpha_r) h0."""
    rng = np.random.default_rng(1)
    T, C = 7, 3
    x, la, h0 = rng.normal(size=(T, C)), -rng.random((T, C)), rng.normal(size=(1, C))
    h, final = oscan.scan(x, la, h0)
    cum = np.cumsum(la, 0)
    for t in range(T):
        want = np.exp(cum[t]) * h0[0]
        for s in range(t + 1):
            want = want + np.exp(cum[t] - cum[s]) * x[s]
        assert np.allclose(h[t], want, rtol=1e-13, atol=1e-13)
    assert np.array_equal(final[0], h[-1])


def test_oracle_packing():
    rng = np.random.default_rng(2)
    cu = [0, 3, 3, 4, 9]
    x, la, h0 = rng.normal(size=(11, 2)), -rng.random((11, 2)), rng.normal(size=(4, 2))
    h, final = oscan.scan(x, la, h0, cu)
    for n, (lo, hi) in enumerate(zip(cu[:-1], cu[1:])):
        one, f = oscan.scan(x[lo:hi], la[lo:hi], h0[n:n + 1])
        assert np.array_equal(h[lo:hi], one) and np.array_equal(final[n], f[0])
    assert np.array_equal(final[1], h0[1]) and np.isnan(h[9:]).all()


def test_oracle_gradients_match_differences():
    rng = np.random.default_rng(3)
    cu, T, C = [0, 4, 4, 9], 9, 2
    v = dict(x=rng.normal(size=(T, C)), log_alpha=-rng.random((T, C)),
             h0=rng.normal(size=(3, C)))
    dh, df = rng.normal(size=(T, C)), rng.normal(size=(3, C))

    def loss(**a):
        h, f = oscan.scan(a["x"], a["log_alpha"], a["h0"], cu)
        return float((dh * h).sum() + (df * f).sum())

    h, _ = oscan.scan(v["x"], v["log_alpha"], v["h0"], cu)
    grads = dict(zip(("x", "log_alpha", "h0"),
                     oscan.scan_backward(v["log_alpha"], h, dh, v["h0"], df, cu)))
    step = 1e-6
    for name, g in grads.items():
        for i in np.ndindex(*g.shape):
            up, down = v[name].copy(), v[name].copy()
            up[i] += step
            down[i] -= step
            num = (loss(**{**v, name: up}) - loss(**{**v, name: down})) / (2 * step)
            # truncation step^2 and rounding 2^-53 |L| / step, ~1e-9
            assert abs(num - g[i]) <= 1e-7 * max(1.0, abs(g[i]))


P = 0x10000  # never dereferenced: the host checks fail, or there is no device here


def _scan(L, **kw):
    a = dict(x=P, xs=64, la=P, las=64, h0=None, cu=P, N=2, T=8, C=64, io=gdn.GDN_BF16,
             gate=gdn.GDN_F32, h=P, hs=64, hf=None, stream=None)
    a.update(kw)
    return L.gdn_scan(*a.values())


@pytest.mark.parametrize("kw,expect", [
    (dict(x=None), gdn.GDN_ERR_INVALID_ARG),
    (dict(la=None), gdn.GDN_ERR_INVALID_ARG),
    (dict(h=None), gdn.GDN_ERR_INVALID_ARG),
    (dict(x=P + 1), gdn.GDN_ERR_INVALID_ARG),
    (dict(la=P + 2), gdn.GDN_ERR_INVALID_ARG),
    (dict(cu=P + 2), gdn.GDN_ERR_INVALID_ARG),
    (dict(cu=None), gdn.GDN_ERR_INVALID_ARG),            # two sequences need their bounds
    (dict(h0=P + 2), gdn.GDN_ERR_INVALID_ARG),
    (dict(hf=P + 1), gdn.GDN_ERR_INVALID_ARG),
    (dict(xs=63), gdn.GDN_ERR_INVALID_ARG),
    (dict(las=0), gdn.GDN_ERR_INVALID_ARG),
    (dict(hs=-64), gdn.GDN_ERR_INVALID_ARG),
    (dict(N=0), gdn.GDN_ERR_INVALID_ARG),
    (dict(T=-1), gdn.GDN_ERR_INVALID_ARG),
    (dict(C=0), gdn.GDN_ERR_INVALID_ARG),
    (dict(C=1 << 23, xs=1 << 23, las=1 << 23, hs=1 << 23), gdn.GDN_ERR_INVALID_ARG),
    (dict(io=0), gdn.GDN_ERR_INVALID_ARG),
    (dict(gate=3), gdn.GDN_ERR_INVALID_ARG),
    (dict(), gdn.GDN_ERR_CUDA),                          # the host checks pass; no device here
])
def test_scan_rejects_bad_arguments_on_host(L, kw, expect):
    assert _scan(L, **kw) == expect


def _back(L, **kw):
    a = dict(la=P, las=64, h=P, hs=64, dh=P, dhs=64, h0=None, dhf=None, cu=P, N=2, T=8, C=64,
             io=gdn.GDN_BF16, gate=gdn.GDN_F32, dx=P, dxs=64, dla=P, dlas=64, dh0=None, stream=None)
    a.update(kw)
    return L.gdn_scan_backward(*a.values())


@pytest.mark.parametrize("kw,expect", [
    (dict(dh=None), gdn.GDN_ERR_INVALID_ARG),
    (dict(h=None), gdn.GDN_ERR_INVALID_ARG),
    (dict(dx=None), gdn.GDN_ERR_INVALID_ARG),
    (dict(dla=None), gdn.GDN_ERR_INVALID_ARG),
    (dict(dlas=10), gdn.GDN_ERR_INVALID_ARG),
    (dict(dhf=P + 1), gdn.GDN_ERR_INVALID_ARG),
    (dict(dh0=P + 2), gdn.GDN_ERR_INVALID_ARG),
    (dict(cu=None), gdn.GDN_ERR_INVALID_ARG),
    (dict(gate=0), gdn.GDN_ERR_INVALID_ARG),
    (dict(), gdn.GDN_ERR_CUDA),
])
def test_scan_backward_rejects_bad_arguments_on_host(L, kw, expect):
    assert _back(L, **kw) == expect


def _step(L, **kw):
    a = dict(x=P, xs=64, la=P, las=64, s=P, B=4, C=64, io=gdn.GDN_BF16, gate=gdn.GDN_BF16, h=P,
             hs=64, stream=None)
    a.update(kw)
    return L.gdn_scan_step(*a.values())


@pytest.mark.parametrize("kw,expect", [
    (dict(s=None), gdn.GDN_ERR_INVALID_ARG),
    (dict(s=P + 2), gdn.GDN_ERR_INVALID_ARG),
    (dict(x=None), gdn.GDN_ERR_INVALID_ARG),
    (dict(hs=32), gdn.GDN_ERR_INVALID_ARG),
    (dict(B=-1), gdn.GDN_ERR_INVALID_ARG),
    (dict(C=0), gdn.GDN_ERR_INVALID_ARG),
    (dict(B=0, x=None, s=None), gdn.GDN_OK),
    (dict(), gdn.GDN_ERR_CUDA),
])
def test_scan_step_rejects_bad_arguments_on_host(L, kw, expect):
    assert _step(L, **kw) == expect


def test_binding_refuses_what_is_not_on_a_gpu():
    x = torch.zeros(4, 8)
    for call in (lambda: gdn.scan(x, x), lambda: gdn.scan_backward(x, x, x),
                 lambda: gdn.scan_step(x, x, x)):
        with pytest.raises(TypeError):
            call()
