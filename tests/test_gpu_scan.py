"""gdn_scan, gdn_scan_backward and gdn_scan_step against the fp64 oracle."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from linear_attention_12_b200 import gdn
from oracle import scan as oscan

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(autouse=True)
def _status_clean():
    yield
    assert gdn.last_device_error() == gdn.GDN_OK


def _half_step(dtype):
    return torch.finfo(dtype).eps / 2


# A term of h_t that entered k tokens ago is a product of k gates and x: each gate carries
# exp's 2 ulp (4 U) and each product and sum one rounding (U each), and joining the pieces
# of a split scan adds a bounded number of products and sums, below 64.  With habs the
# recurrence of |x| and |h0|, that is at most U (64 habs_t + sum over s <= t of the gates
# between s and t times 8 habs_s), the second sum being the recurrence again.
def _limit(x, la, h0, cu):
    habs, fabs = oscan.scan(np.abs(oscan._np(x)), la, None if h0 is None else h0.abs(), cu)
    more, fmore = oscan.scan(8 * np.nan_to_num(habs), la, None, cu)
    return U * (64 * habs + more), U * (64 * fabs + fmore), habs


def _case(T, C, cu, io, gate, seed, h0=True, mu=0.0):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g)
    N = 1 if cu is None else len(cu) - 1
    x, dh = rnd(T, C).to(io), rnd(T, C).to(io)
    la = -torch.nn.functional.softplus(rnd(T, C) + mu).to(gate)
    s0, df = (rnd(N, C), rnd(N, C)) if h0 else (None, None)
    return x, la, s0, dh, df, None if cu is None else torch.tensor(cu, dtype=torch.int32)


def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _np64(t):
    return t.float().cpu().double().numpy()


def _check(x, la, h0, dh, df, cu):
    io, gate = x.dtype, la.dtype
    T = x.shape[0]
    end = T if cu is None else int(cu[-1])
    cx, cla, ch0, cdh, cdf, ccu = _cuda(x, la, h0, dh, df, cu)
    out = torch.full_like(cx, float("nan"))
    h, hf = gdn.scan(cx, cla, ch0, ccu, h=out)
    assert h is out
    rh, rf = oscan.scan(x, la, h0, cu)
    lim, flim, habs = _limit(x, la, h0, cu)
    got = _np64(h)
    assert np.isnan(got[end:]).all()
    assert (np.abs(got - rh) <= lim * (1 + _half_step(io)) + _half_step(io) * np.abs(rh))[:end].all()
    assert (np.abs(_np64(hf) - rf) <= flim).all()

    # the gradients read the rounded h
    hc = h.nan_to_num(0.0)
    dx, dla, dh0 = (torch.full_like(cx, float("nan")), torch.full_like(cla, float("nan")), None)
    dx, dla, dh0 = gdn.scan_backward(cla, hc, cdh, ch0, cdf, ccu, dx=dx, dlog_alpha=dla)
    rx, rl, r0 = oscan.scan_backward(la, hc.cpu(), dh, h0, df, cu)
    # the same argument for the reversed recurrence of |dh| and |dh_final|
    gabs, labs, uabs = oscan.scan_backward(la, hc.cpu().abs(), dh.abs(),
                                           None if h0 is None else h0.abs(),
                                           None if df is None else df.abs(), cu)
    more, lmore, umore = oscan.scan_backward(la, hc.cpu().abs(), 8 * np.nan_to_num(gabs),
                                             None if h0 is None else h0.abs(), None, cu)
    got = _np64(dx)
    assert np.isnan(got[end:]).all() and np.isnan(_np64(dla)[end:]).all()
    lim = U * (64 * gabs + more)
    assert (np.abs(got - rx) <= lim * (1 + _half_step(io)) + _half_step(io) * np.abs(rx))[:end].all()
    lim = U * (64 * labs + lmore)
    off = np.abs(_np64(dla) - rl)
    assert (off <= lim * (1 + _half_step(gate)) + _half_step(gate) * np.abs(rl))[:end].all()
    assert (np.abs(_np64(dh0) - r0) <= U * (64 * uabs + umore)).all()


TYPES = [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)]


@pytest.mark.parametrize("io,gate", TYPES)
@pytest.mark.parametrize("T,C", [(1, 1), (1, 6144), (2, 3), (7, 128), (63, 64), (64, 65),
                                 (65, 136), (257, 515), (1000, 8), (1031, 72), (2049, 256)])
def test_one_sequence(T, C, io, gate):
    _check(*_case(T, C, None, io, gate, T + C, h0=T % 2 == 1))


@pytest.mark.parametrize("io,gate", TYPES)
@pytest.mark.parametrize("C", [64, 100, 515, 1024])
@pytest.mark.parametrize("cu", [
    [0, 1], [0, 0, 5], [0, 5, 5], [0, 0, 0, 9, 9, 9], [0, 1, 2, 3, 4, 5, 6],
    [0, 63, 64, 128, 129, 300, 300, 555], list(range(0, 700, 7)), [0, 512, 1024, 1025],
    [0] * 40 + [33, 33, 90]])
def test_packed_sequences(C, cu, io, gate):
    _check(*_case(cu[-1], C, cu, io, gate, len(cu) + C, h0=C != 100))


@pytest.mark.parametrize("io,gate", TYPES)
@pytest.mark.parametrize("C", [64, 515])
@pytest.mark.parametrize("T,cu", [(10, [0, 0]), (200, [0, 70, 130]), (1030, [0, 1, 1000]),
                                  (640, [0, 100, 512])])
def test_rows_behind_the_last_sequence_stay(T, cu, C, io, gate):
    """Padding behind cu[N] may hold anything: it is neither used nor written."""
    x, la, h0, dh, df, cut = _case(T, C, cu, io, gate, T + C)
    for t in (x, la, dh):
        t[cu[-1]:] = float("nan")
    _check(x, la, h0, dh, df, cut)


@pytest.mark.parametrize("io,gate", [(BF16, BF16), (F32, F32)])
def test_long_memory(io, gate):
    """Gates near one over thousands of tokens."""
    _check(*_case(6000, 72, [0, 3000, 6000], io, gate, 3, mu=-6.0))


def test_many_short_sequences():
    lens = torch.randint(0, 4, (3000,), generator=torch.Generator().manual_seed(2)).tolist()
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    _check(*_case(cu[-1], 64, cu, BF16, F32, 4))


@pytest.mark.parametrize("C", [64, 515])
def test_closed_and_open_gates(C):
    """Gates of exactly 0 (log -inf) and 1 (log 0)."""
    x, la, h0, dh, df, cu = _case(400, C, [0, 150, 400], F32, F32, 6)
    la[::3] = 0.0
    la[5::7] = float("-inf")
    _check(x, la, h0, dh, df, cu)


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("C", [64, 515])
def test_nothing_crosses_a_boundary(io, C):
    """An infinity or a NaN in one sequence (input, state or gradient) stays in it."""
    cu = [0, 70, 71, 200, 333, 640]
    x, la, h0, dh, df, cut = _case(640, C, cu, io, io, 8)
    good = gdn.scan(*_cuda(x, la, h0, cut))
    hg = good[0]
    gback = gdn.scan_backward(*_cuda(la, hg, dh, h0, df, cut))
    x[69, 0], x[70], h0[3, 1], x[332, 2] = float("nan"), float("inf"), float("nan"), -float("inf")
    dh[71, 0], dh[199], df[3, 1] = float("nan"), float("inf"), float("nan")
    h, hf = gdn.scan(*_cuda(x, la, h0, cut))
    back = gdn.scan_backward(*_cuda(la, hg, dh, h0, df, cut))
    for n in (2, 4):
        assert torch.equal(h[cu[n]:cu[n + 1]], good[0][cu[n]:cu[n + 1]])
        assert torch.equal(hf[n], good[1][n])
    assert hf[0, 0].isnan() and hf[1].isinf().all() and hf[3, 1].isnan()
    for n in (0, 1, 4):
        for p, q in zip(back[:2], gback[:2]):
            assert torch.equal(p[cu[n]:cu[n + 1]], q[cu[n]:cu[n + 1]])
        assert torch.equal(back[2][n], gback[2][n])
    assert back[0][71, 0].isnan() and back[0][199].isinf().all()


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("io", [BF16, F32])
def test_column_slices_and_heads(io, shift):
    """x, log_alpha and the outputs as column slices of wider tensors, [T, H, d] layouts, on
    and off the wide path's alignment; what lies beside them stays."""
    T, H, d = 150, 3, 64
    n = H * d
    x, la, h0, dh, df, cu = _case(T, n, [0, 50, 150], io, io, 10)
    wide = torch.randn(T, 3 * n + 32).to(io).cuda()
    at = [n * i + 8 * i + shift for i in range(3)]
    cut = [wide[:, a:a + n].view(T, H, d) for a in at]
    for s, v in zip(cut, (x, la, dh)):
        s.copy_(v.cuda().view(T, H, d))
    out = torch.full((T, 3 * n + 32), 3.0, dtype=io, device="cuda")
    so = [out[:, a:a + n].view(T, H, d) for a in at]
    h0c, dfc = h0.cuda().view(2, H, d), df.cuda().view(2, H, d)
    h, hf = gdn.scan(cut[0], cut[1], h0c, cu.cuda(), h=so[0])
    dense = gdn.scan(*_cuda(x, la, h0, cu))
    assert hf.shape == (2, H, d)
    # the two paths may add in different orders: equal to a few steps of the type
    tol = dict(rtol=4 * torch.finfo(io).eps, atol=1e-5)
    torch.testing.assert_close(h.reshape(T, n), dense[0], **tol)
    torch.testing.assert_close(hf.reshape(2, n), dense[1], rtol=1e-5, atol=1e-5)
    back = gdn.scan_backward(cut[1], so[0], cut[2], h0c, dfc, cu.cuda(), dx=so[1], dlog_alpha=so[2])
    ref = gdn.scan_backward(*_cuda(la, h.reshape(T, n).contiguous(), dh, h0, df, cu))
    for p, q in zip(back[:2], ref[:2]):
        torch.testing.assert_close(p.reshape(T, n), q, **tol)
    torch.testing.assert_close(back[2].reshape(2, n), ref[2], rtol=1e-5, atol=1e-5)
    mask = torch.ones(3 * n + 32, dtype=torch.bool)
    for a in at:
        mask[a:a + n] = False
    assert (out[:, mask.cuda()] == 3.0).all()


@pytest.mark.parametrize("C", [64, 515])
def test_states_in_place(C):
    """h_final may be h0 itself."""
    x, la, h0, dh, df, cu = _case(300, C, [0, 0, 100, 300], F32, F32, 12)
    cx, cla, ch0, ccu = _cuda(x, la, h0, cu)
    h, hf = gdn.scan(cx, cla, ch0, ccu)
    s = ch0.clone()
    h2, s2 = gdn.scan(cx, cla, s, ccu, h_final=s)
    assert s2 is s and torch.equal(s, hf) and torch.equal(h, h2)


def test_no_tokens_and_no_state():
    x = torch.empty(0, 64, device="cuda")
    h0 = torch.randn(2, 64, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    h, hf = gdn.scan(x, x, h0, cu)
    assert h.shape == (0, 64) and torch.equal(hf, h0)
    assert not gdn.scan(x, x)[1].any()
    dx, dla, dh0 = gdn.scan_backward(x, x, x, h0, h0, cu)
    assert torch.equal(dh0, h0)
    y = torch.randn(9, 64, device="cuda")
    assert gdn.scan(y, -y.abs(), want_state=False)[1] is None
    assert gdn.scan_backward(-y.abs(), y, y, want_dh0=False)[2] is None


@pytest.mark.parametrize("io,gate", TYPES)
@pytest.mark.parametrize("B,C", [(1, 1), (1, 6144), (3, 515), (256, 1024), (17, 72)])
def test_step(B, C, io, gate):
    x, la, s0, _, _, _ = _case(B, C, list(range(B + 1)), io, gate, B + C)
    state = s0.cuda()
    h = gdn.scan_step(x.cuda(), la.cuda(), state)
    ref = np.exp(oscan._np(la)) * oscan._np(s0) + oscan._np(x)
    lim = 8 * U * (np.abs(oscan._np(s0)) + np.abs(oscan._np(x)))
    assert (np.abs(_np64(state) - ref) <= lim).all()
    assert (np.abs(_np64(h) - ref) <= lim * 1.01 + _half_step(io) * np.abs(ref)).all()
    # a step is a scan of one token per sequence
    h2, s2 = gdn.scan(*_cuda(x, la, s0, torch.arange(B + 1, dtype=torch.int32)))
    torch.testing.assert_close(state, s2, rtol=1e-6, atol=1e-6)
    wide = torch.randn(B, 2, C).to(io).cuda()
    wide[:, 1] = x.cuda()
    state3 = s0.cuda()
    assert torch.equal(gdn.scan_step(wide[:, 1], la.cuda(), state3, h=wide[:, 0]), h)
    assert torch.equal(state3, state) and torch.equal(wide[:, 1], x.cuda())


def test_step_of_nothing():
    x = torch.empty(0, 64, device="cuda")
    assert gdn.scan_step(x, x, x).shape == (0, 64)


@pytest.mark.parametrize("T,C", [(700, 256), (90, 515)])
def test_same_bits_again_on_another_stream_and_in_a_graph(T, C):
    x, la, h0, dh, df, cu = _cuda(*_case(T, C, [0, 33, T], BF16, F32, 14))
    state = h0.clone()

    def everything(**kw):
        h, hf = gdn.scan(x, la, h0, cu, **kw)
        return (h, hf, *gdn.scan_backward(la, h, dh, h0, df, cu, **kw))

    first = everything()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    again = everything(stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, again))
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = everything()
            gdn.scan_step(x[:2], la[:2], state)
        graphs.append((graph, held))
    for graph, held in graphs:
        for t in held:
            t.zero_()
    state.copy_(h0)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for (graph, _), s in zip(graphs, streams):
        with torch.cuda.stream(s):
            graph.replay()
        s.synchronize()
    for _, held in graphs:
        assert all(torch.equal(p, q) for p, q in zip(first, held))
    want = torch.exp(la[:2].float())
    ref = want * (want * h0 + x[:2].float()) + x[:2].float()
    torch.testing.assert_close(state, ref, rtol=1e-5, atol=1e-5)


def test_first_call_inside_a_capture():
    """A process whose first calls are captured (the kernels' attributes and the room for their
    clusters are asked for then)."""
    code = """
import torch
from linear_attention_12_b200 import gdn
g = torch.Generator("cuda").manual_seed(1)
x = torch.randn(3000, 320, generator=g, device="cuda")
la = -torch.rand(3000, 320, generator=g, device="cuda")
w = torch.ones(64, device="cuda")
gdn.lib()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    h, hf = gdn.scan(x=x, log_alpha=la)
    back = gdn.scan_backward(la, h, x)
    y = gdn.group_norm(h.view(3000, 5, 64), w)
    back += gdn.group_norm_backward(y, h.view(3000, 5, 64), w)[:2]
graph.replay()
torch.cuda.synchronize()
held = (h, hf, y, *back)
h, hf = gdn.scan(x, la)
back = gdn.scan_backward(la, h, x)
y = gdn.group_norm(h.view(3000, 5, 64), w)
back += gdn.group_norm_backward(y, h.view(3000, 5, 64), w)[:2]
assert all(torch.equal(p, q) for p, q in zip(held, (h, hf, y, *back)))
print("same")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                         timeout=300)
    assert out.stdout.strip().endswith("same"), out.stderr[-2000:]


@pytest.mark.parametrize("io,gate", TYPES)
def test_same_bits_from_a_cold_cache(io, gate):
    """The data and the code out of the caches before every call: the timing between the
    copies into a tile and the reads from it is another one then."""
    T, C, N = 4000, 2048, 20
    g = torch.Generator().manual_seed(31)
    cu = [0, *sorted(torch.randint(0, T + 1, (N - 1,), generator=g).tolist()), T]
    x, la, h0, dh, df, cu = _cuda(*_case(T, C, cu, io, gate, 31))
    ref = gdn.scan(x, la, h0, cu)
    back = gdn.scan_backward(la, ref[0], dh, h0, df, cu)
    flush = torch.empty(160 << 20, dtype=torch.uint8, device="cuda")
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for k in range(600):
        flush.fill_(k % 256)
        got = gdn.scan(x, la, h0, cu)
        flush.fill_(k % 255)
        got += gdn.scan_backward(la, ref[0], dh, h0, df, cu)
        for p, q in zip(got, ref + back):
            differ += (p != q).any()
    assert int(differ) == 0


def test_two_calls_at_once():
    """Calls on two streams that overlap do not disturb one another."""
    one = _cuda(*_case(5000, 256, [0, 1000, 5000], BF16, BF16, 16))
    two = _cuda(*_case(4000, 512, [0, 4000], F32, F32, 17))
    refs = [gdn.scan(a[0], a[1], a[2], a[5]) for a in (one, two)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for i, a in enumerate((one, two)):
            outs[i].append(gdn.scan(a[0], a[1], a[2], a[5], stream=streams[i]))
    torch.cuda.synchronize()
    for ref, got in zip(refs, outs):
        for h, hf in got:
            assert torch.equal(h, ref[0]) and torch.equal(hf, ref[1])


def test_large_offsets():
    """Rows whose element offsets pass 2^31."""
    T, C, stride = 70000, 64, 40000
    wide = torch.empty(T * stride, dtype=BF16, device="cuda")
    x = torch.as_strided(wide, (T, C), (stride, 1))
    h = torch.as_strided(wide, (T, C), (stride, 1), 64)
    assert (T - 1) * stride > 2 ** 31
    g = torch.Generator("cuda").manual_seed(1)
    xd = torch.randn(T, C, generator=g, device="cuda").to(BF16)
    la = -torch.rand(T, C, generator=g, device="cuda")
    x.copy_(xd)
    got, hf = gdn.scan(x, la, h=h)
    ref, rf = gdn.scan(xd, la)
    assert torch.equal(got, ref) and torch.equal(hf, rf)
    back = gdn.scan_backward(la, h, x)
    dense = gdn.scan_backward(la, ref, xd)
    assert all(torch.equal(p, q) for p, q in zip(back, dense))


def test_refusals():
    x, la, h0, dh, df, cu = _cuda(*_case(20, 64, [0, 8, 20], BF16, F32, 18))
    with pytest.raises(ValueError):
        gdn.scan(x, la[:10], h0, cu)
    with pytest.raises(ValueError):
        gdn.scan(x, la, h0[:1], cu)
    with pytest.raises(ValueError):
        gdn.scan(x, la, h0)                       # one sequence, two states
    with pytest.raises(TypeError):
        gdn.scan(x, la, h0.double(), cu)
    with pytest.raises(TypeError):
        gdn.scan(x, la.half(), h0, cu)
    with pytest.raises(TypeError):
        gdn.scan(x, la, h0, cu.long())
    with pytest.raises(ValueError):
        gdn.scan(x, la, h0, cu[:0])
    with pytest.raises(ValueError):
        gdn.scan(x[:, ::2], la[:, ::2])
    with pytest.raises(ValueError):
        gdn.scan(x[:1].expand(20, 64), la)
    with pytest.raises(TypeError):
        gdn.scan(x, la, h=torch.empty(20, 64, device="cuda"))
    with pytest.raises(TypeError):
        gdn.scan_backward(la, x, dh.float())
    with pytest.raises(ValueError):
        gdn.scan_step(x, la, h0)
    with pytest.raises(TypeError):
        gdn.scan(x, la.cpu())
