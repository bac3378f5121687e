"""The group norm's oracle against differences and known values, and the refusals of
gdn_group_norm and gdn_group_norm_backward (CPU only)."""
import itertools

import numpy as np
import pytest
import torch

from linear_attention_12_b200 import build as gdn_build
from linear_attention_12_b200 import gdn
from oracle import norm as onorm


@pytest.fixture(scope="module")
def L():
    gdn_build.build()
    return gdn.lib()


@pytest.mark.parametrize("norm,act,gated,per_head",
                         list(itertools.product(["rms", "mean"], ["none", "silu"], [False, True],
                                                [False, True])))
def test_oracle_gradients_match_differences(norm, act, gated, per_head):
    rng = np.random.default_rng(3)
    T, H, d = 2, 3, 5
    x, dy = rng.normal(size=(2, T, H, d))
    z = rng.normal(size=(T, H, d)) if gated else None
    w, b = rng.normal(size=(2, H, d)) if per_head else rng.normal(size=(2, d))
    args = dict(x=x, weight=w, bias=b, z=z)

    def loss(**a):
        return float((dy * onorm.group_norm(**a, norm=norm, act=act, eps=1e-3)).sum())

    dx, dw, db, dz = onorm.group_norm_backward(dy, **args, norm=norm, act=act, eps=1e-3)
    assert (dz is None) == (z is None)
    h = 1e-6
    for name, grad in (("x", dx), ("weight", dw), ("bias", db), ("z", dz)):
        if grad is None:
            continue
        assert grad.shape == args[name].shape
        for i in np.ndindex(*grad.shape):
            up, down = args[name].copy(), args[name].copy()
            up[i] += h
            down[i] -= h
            num = (loss(**{**args, name: up}) - loss(**{**args, name: down})) / (2 * h)
            # central differences: truncation h^2 (~1e-12) and rounding 2^-53 |L| / h (~1e-9)
            assert abs(num - grad[i]) <= 1e-7 * max(1.0, abs(grad[i]))


def test_oracle_known_values():
    x = np.array([[[3.0, -3.0]]])
    one = np.ones(2)
    assert np.allclose(onorm.group_norm(x, one, act="none", eps=0.0), [[[1.0, -1.0]]])
    assert np.allclose(onorm.group_norm(x + 7.0, one, norm="mean", act="none", eps=0.0),
                       [[[1.0, -1.0]]])
    z = np.array([[[0.0, 2.0]]])
    assert np.allclose(onorm.group_norm(x, one, z=z, act="none", eps=0.0), [[[0.0, -2.0]]])


P = 0x10000  # never dereferenced: the host checks fail, or there is no device here


def _fwd(L, **kw):
    a = dict(x=P, xs=256, z=None, zs=0, w=P, b=None, T=4, H=2, d=128, wh=1, norm=0, act=1,
             eps=1e-6, io=gdn.GDN_BF16, y=P, ys=256, stream=None)
    a.update(kw)
    return L.gdn_group_norm(*a.values())


@pytest.mark.parametrize("kw,expect", [
    (dict(x=None), gdn.GDN_ERR_INVALID_ARG),
    (dict(y=None), gdn.GDN_ERR_INVALID_ARG),
    (dict(w=None), gdn.GDN_ERR_INVALID_ARG),
    (dict(x=P + 1), gdn.GDN_ERR_INVALID_ARG),
    (dict(b=P + 2), gdn.GDN_ERR_INVALID_ARG),
    (dict(xs=255), gdn.GDN_ERR_INVALID_ARG),
    (dict(ys=0), gdn.GDN_ERR_INVALID_ARG),
    (dict(z=P, zs=-256), gdn.GDN_ERR_INVALID_ARG),
    (dict(T=-1), gdn.GDN_ERR_INVALID_ARG),
    (dict(H=0), gdn.GDN_ERR_INVALID_ARG),
    (dict(d=0), gdn.GDN_ERR_INVALID_ARG),
    (dict(wh=3), gdn.GDN_ERR_INVALID_ARG),
    (dict(norm=2), gdn.GDN_ERR_INVALID_ARG),
    (dict(act=2), gdn.GDN_ERR_INVALID_ARG),
    (dict(eps=-1.0), gdn.GDN_ERR_INVALID_ARG),
    (dict(eps=float("nan")), gdn.GDN_ERR_INVALID_ARG),
    (dict(io=0), gdn.GDN_ERR_INVALID_ARG),
    (dict(d=1025, xs=4096, ys=4096), gdn.GDN_ERR_UNSUPPORTED),
    (dict(T=0, x=None, y=None), gdn.GDN_OK),
])
def test_group_norm_rejects_bad_arguments_on_host(L, kw, expect):
    assert _fwd(L, **kw) == expect


def _bwd(L, **kw):
    a = dict(dy=P, dys=256, x=P, xs=256, z=None, zs=0, w=P, b=None, T=4, H=2, d=128, wh=1, norm=0,
             act=1, eps=1e-6, io=gdn.GDN_BF16, dx=P, dxs=256, dz=None, dzs=0, dw=P, db=None, ws=P,
             wsb=1 << 30, stream=None)
    a.update(kw)
    return L.gdn_group_norm_backward(*a.values())


@pytest.mark.parametrize("kw,expect", [
    (dict(dy=None), gdn.GDN_ERR_INVALID_ARG),
    (dict(dx=None), gdn.GDN_ERR_INVALID_ARG),
    (dict(dw=None), gdn.GDN_ERR_INVALID_ARG),
    (dict(z=P, zs=256), gdn.GDN_ERR_INVALID_ARG),      # a gate without its gradient
    (dict(dz=P, dzs=256), gdn.GDN_ERR_INVALID_ARG),    # and the other way round
    (dict(z=P, zs=256, dz=P, dzs=255), gdn.GDN_ERR_INVALID_ARG),
    (dict(dys=128), gdn.GDN_ERR_INVALID_ARG),
    (dict(wh=0), gdn.GDN_ERR_INVALID_ARG),
    (dict(ws=None), gdn.GDN_ERR_WORKSPACE),
    (dict(ws=P + 128), gdn.GDN_ERR_WORKSPACE),
    (dict(wsb=16), gdn.GDN_ERR_WORKSPACE),
    (dict(d=2048, dys=4096, xs=4096, dxs=4096), gdn.GDN_ERR_UNSUPPORTED),
])
def test_group_norm_backward_rejects_bad_arguments_on_host(L, kw, expect):
    assert _bwd(L, **kw) == expect


def test_group_norm_backward_workspace(L):
    size = L.gdn_group_norm_backward_workspace_size
    assert size(0, 48, 128, 1, gdn.GDN_BF16) == 0
    assert size(64, 48, 128, 2, gdn.GDN_BF16) == 0       # neither shared nor per head
    assert size(64, 48, 4096, 1, gdn.GDN_BF16) == 0
    # partial sums of dweight and dbias: at least one row each, bounded for any T
    assert size(1, 48, 128, 48, gdn.GDN_F32) >= 2 * 48 * 128 * 4
    assert size(1 << 20, 48, 128, 1, gdn.GDN_BF16) <= 2 * (148 * 8 * 128 * 4 + 256)


def test_binding_refuses_what_is_not_on_a_gpu():
    x = torch.zeros(4, 2, 8)
    with pytest.raises(TypeError):
        gdn.group_norm(x, torch.ones(8))
    with pytest.raises(TypeError):
        gdn.group_norm_backward(x, x, torch.ones(8))
