"""The oracle of the front end's gradients against differences of the front end's oracle,
and the refusals of gdn_frontend_backward (CPU only)."""
import numpy as np
import pytest
import torch

from linear_attention_12_b200 import build as gdn_build
from linear_attention_12_b200 import gdn
from oracle import frontend as fe
from oracle import frontend_backward as feb


@pytest.fixture(scope="module")
def L():
    gdn_build.build()
    return gdn.lib()


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("cu", [[0, 7], [0, 1, 1, 3, 7]])
def test_oracle_gradients_match_differences(act, cu):
    rng = np.random.default_rng(5)
    T, Hq, Hv, d = 7, 1, 2, 3
    v = dict(q_raw=rng.normal(size=(T, Hq, d)), k_raw=rng.normal(size=(T, Hq, d)),
             v_raw=rng.normal(size=(T, Hv, d)), conv_w=rng.normal(size=((2 * Hq + Hv) * d, 4)),
             a=rng.normal(size=(T, Hv)), b=rng.normal(size=(T, Hv)))
    g = [rng.normal(size=s) for s in [(T, Hq, d)] * 2 + [(T, Hv, d)] + [(T, Hv)] * 2]

    def loss(**kw):
        outs = fe.frontend(**kw, cu_seqlens=cu, act=act, eps=1e-2)
        return float(sum((p * q).sum() for p, q in zip(outs, g)))

    grads = feb.frontend_backward(**v, dq=g[0], dk=g[1], dv=g[2], dlog_alpha=g[3], dbeta=g[4],
                                  cu_seqlens=cu, act=act, eps=1e-2)
    h = 1e-6
    for (name, value), grad in zip(v.items(), grads):
        assert grad.shape == value.shape
        for i in np.ndindex(*value.shape):
            up, down = value.copy(), value.copy()
            up[i] += h
            down[i] -= h
            num = (loss(**{**v, name: up}) - loss(**{**v, name: down})) / (2 * h)
            # truncation ~h^2 times third derivatives (below 1e3 here), rounding 2^-53 |L| / h
            assert abs(num - grad[i]) <= 1e-7 * max(1.0, abs(grad[i]))


P = 0x10000  # never dereferenced: the host checks fail, or there is no device here


def _call(L, **kw):
    a = dict(q=P, k=P, v=P, w=P, a=P, b=P, cu=P, dq=P, dk=P, dv=P, dla=P, dbe=P, N=2, T=8, H_qk=2,
             H_v=6, hk=128, hv=128, io=gdn.GDN_BF16, act=1, eps=1e-6, dqr=P, dkr=P, dvr=P, dw=P,
             da=P, db=P, ws=P, wsb=1 << 30, stream=None)
    a.update(kw)
    return L.gdn_frontend_backward(*a.values())


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), gdn.GDN_ERR_INVALID_ARG),
    (dict(dv=P + 8), gdn.GDN_ERR_INVALID_ARG),
    (dict(dkr=None), gdn.GDN_ERR_INVALID_ARG),
    (dict(dw=None), gdn.GDN_ERR_INVALID_ARG),
    (dict(dw=P + 4), gdn.GDN_ERR_INVALID_ARG),
    (dict(dla=None), gdn.GDN_ERR_INVALID_ARG),
    (dict(da=P + 2), gdn.GDN_ERR_INVALID_ARG),
    (dict(cu=None), gdn.GDN_ERR_INVALID_ARG),
    (dict(cu=P + 1), gdn.GDN_ERR_INVALID_ARG),
    (dict(N=0), gdn.GDN_ERR_INVALID_ARG),
    (dict(T=-1), gdn.GDN_ERR_INVALID_ARG),
    (dict(H_qk=4), gdn.GDN_ERR_INVALID_ARG),
    (dict(act=5), gdn.GDN_ERR_INVALID_ARG),
    (dict(eps=-1.0), gdn.GDN_ERR_INVALID_ARG),
    (dict(io=9), gdn.GDN_ERR_INVALID_ARG),
    (dict(hk=64), gdn.GDN_ERR_UNSUPPORTED),
    (dict(ws=None), gdn.GDN_ERR_WORKSPACE),
    (dict(ws=P + 16), gdn.GDN_ERR_WORKSPACE),
    (dict(wsb=64), gdn.GDN_ERR_WORKSPACE),
    (dict(), gdn.GDN_ERR_CUDA),
])
def test_frontend_backward_rejects_bad_arguments_on_host(L, kw, expect):
    assert _call(L, **kw) == expect


def test_frontend_backward_workspace(L):
    size = lambda T, hq=16, hv=48: L.gdn_frontend_backward_workspace_size(T, hq, hv, 128, 128,
                                                                         gdn.GDN_BF16)
    assert size(0) == 0 and size(-1) == 0 and size(64, 5, 7) == 0
    row = 80 * 128 * 4 * 4
    assert size(1) == row and size(64) >= row
    assert size(1 << 20) <= 64 * row  # bounded by the SMs, not by the tokens


def test_binding_refuses_what_is_not_on_a_gpu():
    x = torch.zeros(4, 1, 128)
    g = torch.zeros(4, 1)
    with pytest.raises(TypeError):
        gdn.frontend_backward(x, x, x, torch.zeros(384, 4), g, g, x, x, x, g, g)
