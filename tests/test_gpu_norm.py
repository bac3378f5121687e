"""gdn_group_norm and gdn_group_norm_backward against the fp64 oracle."""
import itertools

import numpy as np
import pytest
import torch

from linear_attention_12_b200 import gdn
from oracle import norm as onorm

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32

# Errors of fp32 arithmetic, in units of 2^-24 of the largest intermediate: sums over
# a group of up to 1024 channels (each lane adds 32 terms at most, then 5 shuffles),
# the statistics' division and rsqrt (2 ulp), sigmoid by exp and division (2 + 1.16 |a|
# ulp for |a| <= 6, and 3 more, each ulp two units) and the products after them: below 128.
UNITS = 128 * 2.0 ** -24


def _half_step(dtype):
    return torch.finfo(dtype).eps / 2


def _close(got, ref, dtype, scale):
    got = got.float().cpu().double().numpy()
    assert np.isfinite(got).all()
    off = np.abs(got - ref)
    lim = _half_step(dtype) * (np.abs(ref) + UNITS * scale) + UNITS * scale
    assert (off <= lim).all(), (float((off / lim).max()), float(off.max()))


def _case(T, H, d, io, seed, gated=True, bias=True, per_head=True):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g)
    x, dy = rnd(T, H, d).to(io), rnd(T, H, d).to(io)
    z = rnd(T, H, d).to(io) if gated else None
    shape = (H, d) if per_head else (d,)
    w = 1.0 + 0.2 * rnd(*shape)
    b = 0.3 * rnd(*shape) if bias else None
    return x, dy, w, b, z


def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _scale(x, dy, w, b, z, norm, eps):
    """A bound on every intermediate of both directions."""
    r = onorm._xhat(onorm._np(x), norm, eps)[1].max() if x.numel() else 1.0
    n = float(w.abs().max()) * x.shape[-1] ** 0.5 + (0 if b is None else float(b.abs().max()))
    gate = max(1.1, 0 if z is None else float(z.float().abs().max()))
    return n * gate, max(1.0, r) * n * gate * float(dy.float().abs().max()) * 1.1


SIZES = [(1, 1, 1), (1, 1, 128), (3, 2, 8), (5, 3, 17), (7, 48, 128), (130, 5, 80), (33, 1, 1024),
         (9, 3, 1000), (2, 2, 1023), (64, 7, 96), (4099, 2, 16), (601, 33, 64), (2, 700, 4), (40, 3, 18), (21, 5, 130), (12, 2, 258),
         (6, 3, 1022), (9, 2, 190)]


@pytest.mark.parametrize("T,H,d", SIZES)
@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("norm", ["rms", "mean"])
def test_group_norm_and_gradients(T, H, d, io, norm):
    for i, (gated, bias, per_head, act) in enumerate(
            [(True, False, False, "silu"), (False, True, True, "silu"), (True, True, True, "none"),
             (False, False, False, "none")]):
        x, dy, w, b, z = _case(T, H, d, io, 100 * i + T, gated, bias, per_head)
        kw = dict(norm=norm, act=act, eps=1e-3)
        cx, cdy, cw, cb, cz = _cuda(x, dy, w, b, z)
        y = gdn.group_norm(cx, cw, cb, cz, **kw)
        dx, dw, db, dz = gdn.group_norm_backward(cdy, cx, cw, cb, cz, **kw)
        torch.cuda.synchronize()
        fs, bs = _scale(x, dy, w, b, z, norm, 1e-3)
        _close(y, onorm.group_norm(x, w, b, z, **kw), io, fs)
        rx, rw, rb, rz = onorm.group_norm_backward(dy, x, w, b, z, **kw)
        _close(dx, rx, io, bs)
        if gated:
            _close(dz, rz, io, bs)
        else:
            assert dz is None
        # sums of T (H) products, each within UNITS of the scale; the additions themselves run at
        # most 128 deep (a lane's own tokens, a block's groups, then the partial rows)
        terms = T * (1 if per_head else H)
        for got, ref in ((dw, rw), (db, rb)):
            if ref is None:
                assert got is None
                continue
            off = np.abs(got.cpu().double().numpy() - ref).max()
            assert off <= 2 * UNITS * terms * bs
    assert gdn.last_device_error() == gdn.GDN_OK


def test_large_sums_are_accurate():
    """dweight and dbias of many tokens: the error of a sum of random terms stays far below
    the worst case (here 1e-5 of the result's norm: 2^-24 x 128 additions deep is 8e-6)."""
    x, dy, w, b, z = _case(20000, 6, 128, BF16, 5, per_head=False)
    got = gdn.group_norm_backward(*_cuda(dy, x, w, b, z))
    ref = onorm.group_norm_backward(dy, x, w, b, z)
    for g, r in ((got[1], ref[1]), (got[2], ref[2])):
        assert np.linalg.norm(g.cpu().double().numpy() - r) <= 1e-5 * np.linalg.norm(r)


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("shift", [0, 1, 2])
def test_column_slices(io, shift):
    """Inputs and outputs that are column slices of wider tensors, on the wide path (shift 0),
    aligned to pairs of bf16 (2) and off both (1); what lies beside them stays as it was."""
    T, H, d = 37, 3, 64
    x, dy, w, b, z = _case(T, H, d, io, 9)
    n = H * d
    at = [8 * i + n * i + shift for i in range(3)]
    wide = torch.randn(T, 3 * n + 32).to(io).cuda()
    sl = [wide[:, a:a + n].view(T, H, d) for a in at]
    for s, v in zip(sl, (x, z, dy)):
        s.copy_(v.cuda())
    out = torch.full((T, 3 * n + 32), 7.0, dtype=io, device="cuda")
    so = [out[:, a:a + n].view(T, H, d) for a in at]
    cw, cb = w.cuda(), b.cuda()
    assert gdn.group_norm(sl[0], cw, cb, sl[1], y=so[0]) is so[0]
    dx, dw, db, dz = gdn.group_norm_backward(sl[2], sl[0], cw, cb, sl[1], dx=so[1], dz=so[2])
    ref = gdn.group_norm_backward(*_cuda(dy, x, w, b, z))
    torch.cuda.synchronize()
    fs, bs = _scale(x, dy, w, b, z, "rms", 1e-6)
    _close(so[0], onorm.group_norm(x, w, b, z), io, fs)
    rx, rw, rb, rz = onorm.group_norm_backward(dy, x, w, b, z)
    _close(so[1], rx, io, bs)
    _close(so[2], rz, io, bs)
    assert torch.allclose(dw, ref[1], rtol=1e-4, atol=1e-3)
    mask = torch.ones(3 * n + 32, dtype=torch.bool)
    for a in at:
        mask[a:a + n] = False
    assert (out[:, mask.cuda()] == 7.0).all()


def test_odd_rows():
    """Rows of zeros, huge and tiny rows, and a group that holds a NaN or an infinity: it
    stays within its group."""
    x, dy, w, b, z = _case(16, 4, 128, F32, 11, per_head=False)
    x[0] = 0.0
    x[1] *= 1e15
    x[2] *= 1e-12
    ref = onorm.group_norm(x, w, b, z, norm="mean")
    y = gdn.group_norm(*_cuda(x, w, b, z), norm="mean")
    _close(y, ref, F32, _scale(x[3:], dy, w, b, z, "mean", 1e-6)[0])
    bad = x.clone()
    bad[5, 1, 3] = float("nan")
    bad[6, 2, 0] = float("inf")
    got = gdn.group_norm(*_cuda(bad, w, b, z), norm="mean")
    dx = gdn.group_norm_backward(*_cuda(dy, bad, w, b, z), norm="mean")[0]
    dx0 = gdn.group_norm_backward(*_cuda(dy, x, w, b, z), norm="mean")[0]
    keep = torch.ones(16, 4, dtype=torch.bool)
    keep[5, 1] = keep[6, 2] = False
    assert torch.equal(got[keep.cuda()], y[keep.cuda()])
    assert torch.equal(dx[keep.cuda()], dx0[keep.cuda()])
    assert got[5, 1].isnan().all() and not got[6, 2].isfinite().all()


@pytest.mark.parametrize("T,H,d", [(5, 3, 17), (1, 1, 128), (40, 5, 128)])
def test_zero_eps_has_no_effect_on_idle_lanes(T, H, d):
    """With eps = 0 the lanes that hold no token add nothing to the weights' gradients."""
    x, dy, w, b, z = _case(T, H, d, F32, 13, per_head=False)
    got = gdn.group_norm_backward(*_cuda(dy, x, w, b, z), eps=0.0)
    ref = onorm.group_norm_backward(dy, x, w, b, z, eps=0.0)
    bs = _scale(x, dy, w, b, z, "rms", 0.0)[1]
    assert np.abs(got[1].cpu().double().numpy() - ref[1]).max() <= 2 * UNITS * T * H * bs


def test_no_tokens():
    x = torch.empty(0, 3, 64, dtype=BF16, device="cuda")
    w = torch.ones(3, 64, device="cuda")
    assert gdn.group_norm(x, w).shape == (0, 3, 64)
    dx, dw, db, dz = gdn.group_norm_backward(x, x, w, w)
    assert dx.shape == (0, 3, 64) and not dw.any() and not db.any() and dz is None


def test_same_bits_again_on_another_stream_and_in_a_graph():
    args = _cuda(*_case(300, 9, 128, BF16, 15))
    x, dy, w, b, z = args
    first = (gdn.group_norm(x, w, b, z), *gdn.group_norm_backward(dy, x, w, b, z))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    again = (gdn.group_norm(x, w, b, z, stream=side),
             *gdn.group_norm_backward(dy, x, w, b, z, stream=side))
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = (gdn.group_norm(x, w, b, z), *gdn.group_norm_backward(dy, x, w, b, z))
    for t in held:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, held))


def test_large_offsets():
    """Rows whose element offsets pass 2^31."""
    T, H, d, stride = 70000, 1, 64, 40000
    wide = torch.zeros(T * stride, dtype=BF16, device="cuda")
    cut = [torch.as_strided(wide, (T, H, d), (stride, d, 1), 64 * i) for i in range(5)]
    assert (T - 1) * stride > 2 ** 31
    x, dy, w, b, z = _cuda(*_case(T, H, d, BF16, 23))
    for s, v in zip(cut, (x, z, dy)):
        s.copy_(v)
    y = gdn.group_norm(cut[0], w, b, cut[1], y=cut[3])
    assert torch.equal(y, gdn.group_norm(x, w, b, z))
    got = gdn.group_norm_backward(cut[2], cut[0], w, b, cut[1], dx=cut[3], dz=cut[4])
    ref = gdn.group_norm_backward(dy, x, w, b, z)
    assert all(torch.equal(p, q) for p, q in zip(got, ref))


def test_bias_gradient_without_a_bias():
    """At the C level the gradient of a bias of zeros may be asked for."""
    T, H, d = 50, 3, 128
    x, dy, w, b, z = _case(T, H, d, BF16, 19, bias=False, per_head=False)
    cx, cdy, cw, _, cz = _cuda(x, dy, w, b, z)
    ref = gdn.group_norm_backward(cdy, cx, cw, torch.zeros_like(cw), cz)
    L = gdn.lib()
    ws = torch.empty(L.gdn_group_norm_backward_workspace_size(T, H, d, 1, gdn.GDN_BF16),
                     dtype=torch.uint8, device="cuda")
    dx, dz, dw, db = cx.clone(), cx.clone(), cw.clone(), cw.clone()
    n = H * d
    st = L.gdn_group_norm_backward(cdy.data_ptr(), n, cx.data_ptr(), n, cz.data_ptr(), n,
                                   cw.data_ptr(), None, T, H, d, 1, 0, 1, 1e-6, gdn.GDN_BF16,
                                   dx.data_ptr(), n, dz.data_ptr(), n, dw.data_ptr(), db.data_ptr(),
                                   ws.data_ptr(), ws.numel(),
                                   torch.cuda.current_stream().cuda_stream)
    assert st == gdn.GDN_OK
    torch.cuda.synchronize()
    for p, q in zip((dx, dw, db, dz), ref):
        assert torch.equal(p, q)


def test_keywords_and_given_workspaces():
    x, dy, w, b, z = _cuda(*_case(70, 5, 96, F32, 21))
    ref = gdn.group_norm_backward(dy, x, w, b, z)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda").fill_(255)
    got = gdn.group_norm_backward(dy=dy, x=x, weight=w, bias=b, z=z, workspace=ws)
    assert all(torch.equal(p, q) for p, q in zip(ref, got))
    assert torch.equal(gdn.group_norm(x=x, weight=w, bias=b, z=z), gdn.group_norm(x, w, b, z))


def test_refusals():
    x, dy, w, b, z = _cuda(*_case(6, 2, 64, BF16, 17))
    with pytest.raises(ValueError):
        gdn.group_norm(x, w[:, :32])
    with pytest.raises(ValueError):
        gdn.group_norm(x, w, norm="layer")
    with pytest.raises(ValueError):
        gdn.group_norm(x, w, act="gelu")
    with pytest.raises(ValueError):
        gdn.group_norm(x.transpose(1, 2), w)
    with pytest.raises(ValueError):
        gdn.group_norm(x[:1].expand(6, 2, 64), w)
    with pytest.raises(TypeError):
        gdn.group_norm(x, w, z=z.float())
    with pytest.raises(TypeError):
        gdn.group_norm(x.half(), w)
    with pytest.raises(ValueError):
        gdn.group_norm(x, w, b.t().contiguous().t())
    with pytest.raises(ValueError):
        gdn.group_norm_backward(dy, x, w, b, dz=z)
    with pytest.raises(gdn.GDNError):
        gdn.group_norm(x, w, eps=-1.0)
    with pytest.raises(gdn.GDNError):
        gdn.group_norm_backward(dy, x, w, b, workspace=torch.empty(64, dtype=torch.uint8,
                                                                    device="cuda"))
