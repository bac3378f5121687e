"""Calls of the scan, norm and front-end gradients that their documentation allows and that stand
apart from the usual ones: states in place at the C level, the smallest and largest counts, calls
at once with workspaces, captures on a stream that is named."""
import numpy as np
import pytest
import torch

from linear_attention_12_b200 import gdn
from oracle import norm as onorm
from tests.test_gpu_norm import _case as norm_case
from tests.test_gpu_scan import _case as scan_case
from tests.test_gpu_scan import _cuda

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _status_clean():
    yield
    assert gdn.last_device_error() == gdn.GDN_OK


def _lens(kind, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, 5 if kind == "short" else 300, (400 if kind == "short" else 12,),
                         generator=g).tolist()


@pytest.mark.parametrize("kind", ["short", "long"])
@pytest.mark.parametrize("C", [64, 515, 1280, 2051])
def test_states_and_their_gradients_in_place(C, kind):
    """h_final may be h0, and dh0 may be dh_final."""
    cu = np.cumsum([0, *_lens(kind, C)]).tolist()
    x, la, h0, dh, df, cut = _cuda(*scan_case(cu[-1], C, cu, F32, F32, C))
    N, T = len(cu) - 1, cu[-1]
    h, hf = gdn.scan(x, la, h0, cut)
    dx, dla, dh0 = gdn.scan_backward(la, h, dh, h0, df, cut)
    s = h0.clone()
    h2, _ = gdn.scan(x, la, s, cut, h_final=s)
    assert torch.equal(h2, h) and torch.equal(s, hf)
    d, dx2, dla2 = df.clone(), torch.empty_like(dx), torch.empty_like(dla)
    p = lambda t: t.data_ptr()
    st = gdn.lib().gdn_scan_backward(p(la), C, p(h), C, p(dh), C, p(h0), p(d), p(cut), N, T, C,
                                     gdn.GDN_F32, gdn.GDN_F32, p(dx2), C, p(dla2), C, p(d),
                                     torch.cuda.current_stream().cuda_stream)
    assert st == gdn.GDN_OK
    assert torch.equal(dx2, dx) and torch.equal(dla2, dla) and torch.equal(d, dh0)


def test_many_empty_sequences():
    """A hundred thousand sequences, nearly all of them empty and most at one token."""
    N, T, C = 100000, 300, 72
    cu = torch.full((N + 1,), 150, dtype=torch.int32)
    cu[:40000], cu[-3:] = 0, T
    cu[40000:40010] = torch.arange(10)
    x, la, h0, dh, df, _ = _cuda(*scan_case(T, C, [0] * (N + 1), F32, F32, 5))
    cut = cu.cuda()
    h, hf = gdn.scan(x, la, h0, cut)
    back = gdn.scan_backward(la, h, dh, h0, df, cut)
    some = (cu[1:] > cu[:-1]).nonzero().flatten()
    keep = torch.unique(torch.cat([some, torch.tensor([0, N // 2, N - 1])]))
    few = [0]
    for n in keep.tolist():
        few.append(few[-1] + int(cu[n + 1] - cu[n]))
    few = torch.tensor(few, dtype=torch.int32).cuda()
    kc = keep.cuda()
    h2, hf2 = gdn.scan(x, la, h0[kc].contiguous(), few)
    back2 = gdn.scan_backward(la, h, dh, h0[kc].contiguous(), df[kc].contiguous(), few)
    assert torch.equal(h, h2) and torch.equal(hf[kc], hf2)
    assert torch.equal(back[0], back2[0]) and torch.equal(back[1], back2[1])
    assert torch.equal(back[2][kc], back2[2])
    rest = torch.ones(N, dtype=torch.bool, device="cuda")
    rest[kc] = False
    assert torch.equal(hf[rest], h0[rest]) and torch.equal(back[2][rest], df[rest])


@pytest.mark.parametrize("C", [1 << 22, (1 << 22) - 1])
def test_the_most_channels(C):
    T = 3
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(T, C, generator=g, device="cuda")
    la = -torch.rand(T, C, generator=g, device="cuda")
    h, hf = gdn.scan(x, la)
    a = la.double().exp()
    want = [x[0].double()]
    for t in range(1, T):
        want.append(a[t] * want[-1] + x[t].double())
    want = torch.stack(want)
    # (three terms below 6 each, a few units of 2^-24 of 18; h_{t-1} times that for dlog_alpha)
    assert (h - want).abs().max() < 1e-5 and torch.equal(hf[0], h[-1])
    dx, dla, dh0 = gdn.scan_backward(la, h, x)
    nxt = torch.zeros(C, dtype=torch.float64, device="cuda")
    for t in range(T - 1, -1, -1):
        dxt = x[t].double() + nxt
        nxt = a[t] * dxt
        assert (dx[t] - dxt).abs().max() < 1e-5
        before = h[t - 1].double() if t else torch.zeros_like(nxt)
        assert (dla[t] - nxt * before).abs().max() < 5e-5
    assert (dh0[0] - nxt).abs().max() < 1e-5


def test_steps_of_many_sequences_and_one_channel():
    B = 1 << 20
    x, la, s = (torch.randn(B, 1, device="cuda") for _ in range(3))
    la = -la.abs()
    want = la.double().exp() * s + x
    h = gdn.scan_step(x, la, s)
    assert (s - want).abs().max() < 2e-6 and torch.equal(h, s)


def test_rows_of_one_token_may_have_any_stride():
    base = torch.randn(64, device="cuda")
    x = base.as_strided((1, 64), (0, 1))
    assert torch.equal(gdn.scan(x, -x.abs())[0], x)
    y = gdn.group_norm(x.view(1, 1, 64), torch.ones(64, device="cuda"))
    assert torch.equal(y, gdn.group_norm(base.clone().view(1, 1, 64),
                                         torch.ones(64, device="cuda")))


@pytest.mark.parametrize("T,H,d", [(1, 1 << 18, 4), (200000, 1, 1), (1, 5000, 17), (3, 700, 1024)])
def test_norms_of_many_heads_or_tokens(T, H, d):
    x, dy, w, b, z = norm_case(T, H, d, F32, 3)
    args = _cuda(dy, x, w, b, z)
    y = gdn.group_norm(*args[1:], eps=1e-2)
    got = gdn.group_norm_backward(*args, eps=1e-2)
    ref = (onorm.group_norm(x, w, b, z, eps=1e-2),
           *onorm.group_norm_backward(dy, x, w, b, z, eps=1e-2))
    for p, r in zip((y, *got), ref):
        assert np.linalg.norm(p.cpu().double().numpy() - r) <= 1e-5 * np.linalg.norm(r)


def _layer(seed):
    g = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    T, Hq, Hv = 1500 + seed, 2, 6
    raw = [rnd(T, Hq, 128), rnd(T, Hq, 128), rnd(T, Hv, 128), rnd((2 * Hq + Hv) * 128, 4),
           rnd(T, Hv), rnd(T, Hv)]
    grads = [rnd(T, Hq, 128), rnd(T, Hq, 128), rnd(T, Hv, 128), rnd(T, Hv), rnd(T, Hv)]
    w, z, h0 = rnd(Hv, 128), rnd(T, Hv, 128), rnd(1, Hv, 128)
    la = -rnd(T, Hv, 128).abs()

    def call(**kw):
        h, hf = gdn.scan(raw[2], la, h0, **kw)
        y = gdn.group_norm(h, w, w, z, **kw)
        n = gdn.group_norm_backward(y, h, w, w, z, **kw)
        s = gdn.scan_backward(la, h, n[0], h0, **kw)
        return (h, hf, y, *n, *s, *gdn.frontend_backward(*raw, *grads, act="silu", **kw))

    return call


def test_calls_at_once_with_their_workspaces():
    calls = [_layer(1), _layer(2)]
    refs = [c() for c in calls]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for _ in range(6):
        for c, ref, s in zip(calls, refs, streams):
            with torch.cuda.stream(s):
                outs.append((c(), ref))
    torch.cuda.synchronize()
    for got, ref in outs:
        assert all(torch.equal(p, q) for p, q in zip(got, ref))


def test_graphs_replayed_at_once_and_captured_on_a_named_stream():
    calls = [_layer(3), _layer(4)]
    refs = [c() for c in calls]
    graphs = []
    for c in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = c(stream=torch.cuda.current_stream())
        graphs.append((graph, held))
    for _, held in graphs:
        for t in held:
            t.zero_()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        for (graph, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for (_, held), ref in zip(graphs, refs):
        assert all(torch.equal(p, q) for p, q in zip(held, ref))
