"""gdn_frontend_backward against the fp64 oracle, and the layer's operators as they are used
together: front end, recurrence, norm, and back."""
import numpy as np
import pytest
import torch

import oracle
from linear_attention_12_b200 import gdn, inputs
from oracle import backward as oback
from oracle import frontend as fe
from oracle import frontend_backward as feb
from oracle import norm as onorm
from oracle import scan as oscan

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32

# fp32 arithmetic between the raw rows and dx, in units of 2^-24 of the largest intermediate:
# the convolution (4 products), sigmoid (2 + 1.16 |y| ulp of exp for |y| <= 8, division: 24
# units), two sums over 128 channels (4 + 5 additions each), rsqrt (2 ulp) used three times,
# and 8 products: below 128.  y's own error enters through slope and u, whose derivatives stay
# below 1.1, as 4 units of sum |w| |x| <= YMAX each.
UNITS = 128 * 2.0 ** -24
YMAX = 16.0


@pytest.fixture(autouse=True)
def _status_clean():
    yield
    assert gdn.last_device_error() == gdn.GDN_OK


def _half_step(dtype):
    return torch.finfo(dtype).eps / 2


def _case(lens, Hq, Hv, io, seed, extra=0):
    c = inputs.make_frontend("feb", lens, Hq, Hv, dtype=io, seed=seed)
    T = sum(lens) + extra
    g = torch.Generator().manual_seed(seed + 1)
    rnd = lambda *s: torch.randn(s, generator=g)
    pad = lambda t: torch.cat([t, torch.full((extra, *t.shape[1:]), float("nan"), dtype=t.dtype)])
    raw = [pad(t) for t in (c.q_raw, c.k_raw, c.v_raw)]
    gates = [pad(t) for t in (c.a, c.b)]
    grads = [rnd(*t.shape).to(io) for t in raw] + [rnd(T, Hv), rnd(T, Hv)]
    return [*raw, c.conv_w, *gates, *grads, c.cu_seqlens]


def _np64(t):
    return t.float().cpu().double().numpy()


def _check(args, act, eps=1e-6):
    io, end = args[0].dtype, int(args[-1][-1])
    got = gdn.frontend_backward(*[t.cuda() for t in args], act=act, eps=eps)
    ref = feb.frontend_backward(*args, act=act, eps=eps)
    # the largest |dy|: r (|dq| + |<q, dq>|) with 1 / r the smallest norm of a q or k head
    y = [fe._act(fe.causal_conv(np.nan_to_num(_np64(t)).reshape(t.shape[0], -1), w, args[-1]), act)[
        :end].reshape(-1, 128) for t, w in zip(args[:2], np.split(_np64(args[3]), [
            args[0].shape[1] * 128, 2 * args[0].shape[1] * 128])[:2])]
    r = max(1.0, float((1.0 / np.sqrt((np.concatenate(y) ** 2).sum(-1) + eps)).max()))
    big = r * 1.1 * (1 + 128 ** 0.5) * max(float(t.float().abs().max()) for t in args[6:9])
    w = float(args[3].abs().max())
    for p, q in zip(got[:3], ref[:3]):
        p = _np64(p)
        off, lim = np.abs(p - q)[:end], 4 * w * big * UNITS * (1 + YMAX / 8)
        assert (off <= lim + _half_step(io) * (np.abs(q[:end]) + lim)).all()
        if end and np.linalg.norm(q[:end]) > 1e-3:
            assert np.linalg.norm(off) <= (_half_step(io) + 2 * UNITS) * np.linalg.norm(q[:end])
    # sums over the tokens of products, each within the same bound times |x| <= 6
    off = np.abs(_np64(got[3]) - ref[3]).max()
    assert off <= 6 * end * big * UNITS * (1 + YMAX / 8)
    if end and np.linalg.norm(ref[3]) > 1e-3:
        assert np.linalg.norm(_np64(got[3]) - ref[3]) <= 4 * UNITS * np.linalg.norm(ref[3])
    for p, q in zip(got[4:], ref[4:]):
        assert (np.abs(_np64(p) - q)[:end] <= 16 * 2.0 ** -24 * 6).all()
    return got


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("lens,Hq,Hv", [
    ([1], 1, 1), ([2], 1, 1), ([3], 1, 2), ([4], 2, 2), ([31, 33], 1, 3), ([64], 16, 48),
    ([1, 1, 1, 1, 1, 2, 3, 4, 5], 1, 1), ([0, 5, 0, 0, 40, 0], 1, 2), ([300], 1, 1),
    ([97, 1, 0, 2, 130, 33], 2, 6), ([32, 32, 32, 32], 1, 1), ([35, 29, 34, 30, 33, 31], 1, 1)])
def test_gradients(lens, Hq, Hv, act, io):
    _check(_case(lens, Hq, Hv, io, sum(lens) + Hq), act)


@pytest.mark.parametrize("io", [BF16, F32])
def test_long_runs(io):
    """More tokens than runs: every run has tokens of its own and of its neighbours."""
    _check(_case([2500, 1, 2, 1300, 700], 8, 24, io, 31), "silu")


def test_rows_behind_the_last_sequence_are_not_used():
    """Padding behind cu[N] may hold anything (here NaN)."""
    args = _case([40, 30], 1, 2, F32, 33, extra=50)
    got = _check(args, "silu")
    cut = [t[:70] if i not in (3, 11) else t for i, t in enumerate(args)]
    ref = gdn.frontend_backward(*[t.cuda() for t in cut], act="silu")
    for i, (p, q) in enumerate(zip(got, ref)):
        if i != 3:
            assert torch.equal(p[:70], q)
        else:
            torch.testing.assert_close(p, q, rtol=1e-4, atol=1e-4)  # other runs, other sums


def test_rows_behind_the_last_sequence_are_not_written():
    """The same at the C level, where the outputs are the caller's."""
    args = [t.cuda() for t in _case([33, 20], 1, 2, BF16, 35, extra=40)]
    q, k, v, w, a, b, dq, dk, dv, dla, dbe, cu = args
    outs = [torch.full_like(t, 9.0) for t in (q, k, v, w, a, b)]
    L = gdn.lib()
    ws = torch.empty(L.gdn_frontend_backward_workspace_size(93, 1, 2, 128, 128, gdn.GDN_BF16),
                     dtype=torch.uint8, device="cuda")
    ptr = lambda t: t.data_ptr()
    st = L.gdn_frontend_backward(*map(ptr, (q, k, v, w, a, b, cu, dq, dk, dv, dla, dbe)), 2, 93, 1,
                                 2, 128, 128, gdn.GDN_BF16, 1, 1e-6, *map(ptr, outs), ptr(ws),
                                 ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == gdn.GDN_OK
    torch.cuda.synchronize()
    for i, t in enumerate(outs):
        if i != 3:
            assert (t[53:] == 9.0).all() and t[:53].isfinite().all()


def test_zero_rows():
    """Heads of zeros: the norm divides by sqrt(eps) alone."""
    args = _case([12], 1, 1, F32, 37)
    args[0].zero_()
    args[1][:9].zero_()
    _check(args, "none", eps=1e-2)


def test_nothing_crosses_a_boundary():
    args = _case([20, 30, 40], 1, 1, F32, 39)
    good = gdn.frontend_backward(*[t.cuda() for t in args], act="silu")
    args[0][25], args[7][49], args[2][20] = float("nan"), float("inf"), float("nan")
    bad = gdn.frontend_backward(*[t.cuda() for t in args], act="silu")
    for p, q in zip(bad[:3], good[:3]):
        assert torch.equal(p[:20], q[:20]) and torch.equal(p[50:], q[50:])


def test_large_offsets():
    """Values whose element offsets pass 2^31: the last sequence's gradients are those it has
    alone (each of its rows is the same arithmetic, whichever run takes it)."""
    T, Hq, Hv, at = 88000, 1, 192, 87400
    g = torch.Generator("cuda").manual_seed(3)
    rnd = lambda *s, **k: torch.randn(*s, generator=g, device="cuda", **k)
    assert at * Hv * 128 > 2 ** 31
    q, k, dq, dk = (rnd(T, Hq, 128, dtype=BF16) for _ in range(4))
    v, dv = (rnd(T, Hv, 128, dtype=BF16) for _ in range(2))
    a, b, dla, dbe = (rnd(T, Hv) for _ in range(4))
    w = rnd((2 * Hq + Hv) * 128, 4)
    cu = torch.tensor([0, at, T], dtype=torch.int32, device="cuda")
    got = gdn.frontend_backward(q, k, v, w, a, b, dq, dk, dv, dla, dbe, cu, act="silu")
    tail = [t[at:].contiguous() for t in (q, k, v, a, b, dq, dk, dv, dla, dbe)]
    ref = gdn.frontend_backward(*tail[:3], w, *tail[3:], act="silu")
    for i, (p, r) in enumerate(zip(got, ref)):
        if i != 3:
            assert torch.equal(p[at:], r)
    assert got[3].isfinite().all()


def test_no_tokens():
    e = lambda *s: torch.empty(*s, device="cuda")
    w = torch.randn(3 * 128, 4, device="cuda")
    x, g = e(0, 1, 128), e(0, 1)
    out = gdn.frontend_backward(x, x, x, w, g, g, x, x, x, g, g)
    assert out[0].shape == (0, 1, 128) and not out[3].any()


def test_same_bits_again_on_another_stream_and_in_a_graph():
    args = [t.cuda() for t in _case([100, 200], 2, 6, BF16, 41)]
    first = gdn.frontend_backward(*args, act="silu")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    again = gdn.frontend_backward(*args, act="silu", stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = gdn.frontend_backward(*args, act="silu")
    for t in held:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, held))


def test_refusals():
    args = [t.cuda() for t in _case([10], 1, 2, BF16, 43)]
    for i, bad in ((1, args[1].float()), (6, args[6].float()), (9, args[9].double())):
        with pytest.raises(TypeError):
            gdn.frontend_backward(*args[:i], bad, *args[i + 1:])
    for i, bad in ((8, args[8][:, :1]), (3, args[3][:128]), (2, args[2].transpose(0, 1)),
                   (0, args[0][:5])):
        with pytest.raises(ValueError):
            gdn.frontend_backward(*args[:i], bad, *args[i + 1:])
    with pytest.raises(ValueError):
        gdn.frontend_backward(*args, act="gelu")
    with pytest.raises(gdn.GDNError):
        gdn.frontend_backward(*args, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


# ---- the operators as a layer uses them ----
def _rel(p, q):
    return float(np.abs(_np64(p) - q).max() / np.abs(q).max())


def test_whole_layer_forward_and_gradients():
    """Raw projections -> front end -> delta rule -> gated norm, and the gradients back to the
    raw projections, against the oracles chained in fp64.  The chain carries the delta rule's
    bf16 products: its own bar of 1e-2 of the largest value for the recurrence's results, three
    times that behind the norm and the front end, which only scale them."""
    lens, Hq, Hv = [70, 33], 2, 6
    c = inputs.make_frontend("layer", lens, Hq, Hv, seed=51)
    T, N = sum(lens), len(lens)
    g = torch.Generator().manual_seed(52)
    z = torch.randn(T, Hv, 128, generator=g).to(BF16)
    dy = torch.randn(T, Hv, 128, generator=g).to(BF16)
    nw = 1 + 0.1 * torch.randn(128, generator=g)
    dev = lambda t: t.cuda()
    raw = [dev(t) for t in (c.q_raw, c.k_raw, c.v_raw, c.conv_w, c.a, c.b)]
    cu = dev(c.cu_seqlens)
    q, k, v, la, be = gdn.frontend(*raw, cu, act="silu")
    o, S, saved = gdn.prefill_train(q, k, v, la, be, cu_seqlens=cu)
    y = gdn.group_norm(o, dev(nw), None, dev(z), eps=1e-3)
    do, dnw, _, dz = gdn.group_norm_backward(dev(dy), o, dev(nw), None, dev(z), eps=1e-3)
    dq, dk, dv, dla, dbe, _ = gdn.prefill_backward(q, k, v, la, be, do, cu_seqlens=cu,
                                                   workspace=saved, saved=True)
    back = gdn.frontend_backward(*raw, dq, dk, dv, dla, dbe, cu, act="silu")

    args = (c.q_raw, c.k_raw, c.v_raw, c.conv_w, c.a, c.b)
    rq, rk, rv, rla, rbe = fe.frontend(*args, c.cu_seqlens, act="silu")
    f32 = [t.astype(np.float32) for t in (rq, rk, rv, rla, rbe)]
    ro, _ = oracle.prefill(*f32, cu_seqlens=c.cu_seqlens)
    ry = onorm.group_norm(ro, nw, None, z, eps=1e-3)
    rdo, rdnw, _, rdz = onorm.group_norm_backward(dy, ro, nw, None, z, eps=1e-3)
    rd = oback.prefill_backward(*f32, rdo, cu_seqlens=c.cu_seqlens.numpy())
    rback = feb.frontend_backward(*args, *rd[:5], c.cu_seqlens, act="silu")
    assert y.shape == (T, Hv, 128) and S.shape == (N, Hv, 128, 128)
    for p, r in ((y, ry), (dz, rdz), (dnw, rdnw), *zip(back, rback)):
        assert _rel(p, r) <= 3e-2


def test_scan_layer_forward_and_gradients():
    """The per-channel mixer in the same place: scan -> gated norm over heads, and back, against
    the oracles in fp64; h is rounded to bf16 once (2^-9 of it), which the norm passes on."""
    T, H, d, cu = 333, 4, 64, [0, 100, 333]
    g = torch.Generator().manual_seed(61)
    rnd = lambda *s: torch.randn(s, generator=g)
    x, z, dy = (rnd(T, H, d).to(BF16) for _ in range(3))
    la, h0, w = -torch.nn.functional.softplus(rnd(T, H, d)), rnd(2, H, d), 1 + 0.1 * rnd(H, d)
    cut = torch.tensor(cu, dtype=torch.int32).cuda()
    cx, cz, cdy, cla, ch0, cw = (t.cuda() for t in (x, z, dy, la, h0, w))
    h, hf = gdn.scan(cx, cla, ch0, cut)
    y = gdn.group_norm(h, cw, None, cz, norm="mean")
    dh, dw, _, dz = gdn.group_norm_backward(cdy, h, cw, None, cz, norm="mean")
    dx, dla, dh0 = gdn.scan_backward(cla, h, dh, ch0, None, cut)
    rh, rf = oscan.scan(x, la, h0, cu)
    ry = onorm.group_norm(rh, w, None, z, norm="mean")
    rdh, rdw, _, rdz = onorm.group_norm_backward(dy, rh, w, None, z, norm="mean")
    rdx, rdla, rdh0 = oscan.scan_backward(la, rh, rdh, h0, None, cu)
    for p, r in ((y, ry), (dw, rdw), (dz, rdz), (dx, rdx), (dla, rdla), (dh0, rdh0), (hf, rf)):
        assert _rel(p, r) <= 2e-2
