"""Cases and plain forms of the operators around the Gated DeltaNet mixer.

Six operators of a linear-attention layer, each with the calls a user makes
(``own`` true) and a plain form in elementary torch operations (``own`` false):

* ``scan``, ``scan_grad``, ``scan_step`` -- the gated linear recurrence
  ``h_t = exp(log_alpha_t) h_{t-1} + x_t`` per channel over packed sequences,
  its gradients, and one decode step;
* ``norm``, ``norm_grad`` -- the group norm over the heads of a mixer's output
  (one group per head and token, channels last) with its activation or its
  activated gate, and its gradients;
* ``front_grad`` -- the gradients of the front end (width-4 causal
  convolution, q/k L2 normalisation, gate activations).

A case is a dict: ``op``, sizes (``T`` tokens, ``N`` packed sequences, ``C``
channels, ``H`` / ``d`` heads and head size, ``Hq`` / ``Hv`` query/key and
value heads, ``B`` sequences of a decode step) and choices.
"""
import functools
import math

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}
_EPS = 1e-6


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a whole prompt through the recurrence, as wide as 48 value heads of 128; x and its
        # gate are the two halves of one fused projection
        {"name": "scan prompt", "op": "scan", "T": 32768, "N": 1, "C": 6144, "io": "bf16",
         "gate": "bf16", "h0": False, "mu": -2.0, "fused": True},
        # eight packed prompts that continue from earlier states, fp32 gates, 16 heads of 128
        {"name": "scan packed", "op": "scan", "T": 41131, "N": 8, "C": 2048, "io": "bf16",
         "gate": "f32", "h0": True, "mu": 0.0, "fused": False},
        # the training step's backward pass of the first case
        {"name": "scan grad", "op": "scan_grad", "T": 32768, "N": 1, "C": 6144, "io": "bf16",
         "gate": "bf16", "h0": False, "mu": -2.0, "fused": False},
        # fp32 training of a small layer on short packed sequences, a channel count that no
        # vector divides
        {"name": "scan grad odd", "op": "scan_grad", "T": 4111, "N": 13, "C": 515, "io": "f32",
         "gate": "f32", "h0": True, "mu": 0.0, "fused": False},
        # one token of one sequence: latency
        {"name": "scan step one", "op": "scan_step", "B": 1, "C": 6144, "io": "bf16",
         "gate": "f32", "mu": -2.0},
        # a decode batch of 256 sequences
        {"name": "scan step batch", "op": "scan_step", "B": 256, "C": 6144, "io": "bf16",
         "gate": "bf16", "mu": -2.0},
        # the output norm of a 48-head mixer over a prompt: RMS, gated by silu(z), z a part of
        # the fused input projection
        {"name": "norm prompt", "op": "norm", "T": 32768, "H": 48, "d": 128, "io": "bf16",
         "norm": "rms", "per_head": False, "bias": False, "gated": True, "act": "silu",
         "fused": True},
        # the same place in a decode step of 256 sequences, in the centred form with an affine
        # part of its own for every head and the activation on the result
        {"name": "norm decode", "op": "norm", "T": 256, "H": 48, "d": 128, "io": "bf16",
         "norm": "mean", "per_head": True, "bias": True, "gated": False, "act": "silu",
         "fused": False},
        # the training step's backward pass of the output norm
        {"name": "norm grad", "op": "norm_grad", "T": 32768, "H": 48, "d": 128, "io": "bf16",
         "norm": "rms", "per_head": False, "bias": False, "gated": True, "act": "silu",
         "fused": False},
        # fp32 training of a small layer: few heads, a head size that is no power of two
        {"name": "norm grad small", "op": "norm_grad", "T": 1027, "H": 5, "d": 80, "io": "f32",
         "norm": "mean", "per_head": True, "bias": True, "gated": False, "act": "silu",
         "fused": False},
        # the training step's backward pass through the front end, 16 / 48 heads
        {"name": "front grad", "op": "front_grad", "T": 32768, "N": 1, "Hq": 16, "Hv": 48,
         "io": "bf16", "act": "silu"},
        # a tensor-parallel shard (2 / 6 heads) on short packed sequences, fp32
        {"name": "front grad shard", "op": "front_grad", "T": 4099, "N": 6, "Hq": 2, "Hv": 6,
         "io": "f32", "act": "none"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _fit(rng, lo, hi, width, most):
    """A length in [lo, hi], log-uniform, with length x width <= most."""
    return _log_int(rng, lo, max(lo, min(hi, most // width)))


def draw(rng):
    op = rng.choice(["scan", "scan_grad", "scan_step", "norm", "norm_grad", "front_grad"])
    io = rng.choice(["bf16", "bf16", "f32"])
    most = 32768 * 6144 * 2 // _BYTES[io]
    if op in ("scan", "scan_grad"):
        # whole heads of 128 mostly, sometimes any channel count
        C = 128 * _log_int(rng, 1, 64) if rng.random() < 0.7 else _log_int(rng, 64, 4096)
        T = _fit(rng, 100, 131072, C, most * 2 // 3)
        gate = rng.choice([io, "f32"])
        return {"op": op, "T": T, "N": min(T, _log_int(rng, 1, 64)), "C": C, "io": io,
                "gate": gate, "h0": rng.random() < 0.5, "mu": rng.choice([0.0, -2.0, -4.0]),
                "fused": op == "scan" and gate == io and rng.random() < 0.5}
    if op == "scan_step":
        return {"op": op, "B": _log_int(rng, 1, 512), "C": 128 * _log_int(rng, 1, 48), "io": io,
                "gate": rng.choice([io, "f32"]), "mu": -2.0}
    if op in ("norm", "norm_grad"):
        H = _log_int(rng, 1, 64)
        d = rng.choice([64, 128, 128, 128, 256, 8 * rng.randint(1, 64), rng.randint(16, 300)])
        T = _fit(rng, 1, 65536, H * d, most)
        gated = rng.random() < 0.6
        return {"op": op, "T": T, "H": H, "d": d, "io": io, "norm": rng.choice(["rms", "mean"]),
                "per_head": rng.random() < 0.5, "bias": rng.random() < 0.4, "gated": gated,
                "act": rng.choice(["silu", "silu", "none"]),
                "fused": gated and rng.random() < 0.5}
    Hq = rng.choice([1, 2, 4, 8, 16])
    Hv = Hq * rng.choice([1, 2, 3])
    T = _fit(rng, 64, 65536, (2 * Hq + Hv) * 128, most)
    return {"op": op, "T": T, "N": min(T, _log_int(rng, 1, 64)), "Hq": Hq, "Hv": Hv, "io": io,
            "act": rng.choice(["silu", "none"])}


def work(case):
    op, e = case["op"], _BYTES[case["io"]]
    if op == "scan":
        n = case["T"] * case["C"]
        states = case["N"] * case["C"] * 4 * (2 if case["h0"] else 1)
        return {"bytes": n * (2 * e + _BYTES[case["gate"]]) + states, "flops": 3 * n}
    if op == "scan_grad":
        n = case["T"] * case["C"]
        states = case["N"] * case["C"] * 4 * (3 if case["h0"] else 1)
        return {"bytes": n * (3 * e + 2 * _BYTES[case["gate"]]) + states, "flops": 5 * n}
    if op == "scan_step":
        n = case["B"] * case["C"]
        return {"bytes": n * (2 * e + _BYTES[case["gate"]] + 8), "flops": 3 * n}
    if op == "norm":
        n = case["T"] * case["H"] * case["d"]
        w = case["d"] * (case["H"] if case["per_head"] else 1) * 4 * (2 if case["bias"] else 1)
        return {"bytes": n * e * (3 if case["gated"] else 2) + w, "flops": 10 * n}
    if op == "norm_grad":
        n = case["T"] * case["H"] * case["d"]
        w = case["d"] * (case["H"] if case["per_head"] else 1) * 4 * (2 if case["bias"] else 1)
        return {"bytes": n * e * (5 if case["gated"] else 3) + 2 * w, "flops": 20 * n}
    T, C = case["T"], (2 * case["Hq"] + case["Hv"]) * 128
    return {"bytes": 3 * T * C * e + 6 * T * case["Hv"] * 4 + 2 * C * 16, "flops": 40 * T * C}


# ---------------------------------------------------------------- inputs
def _cu(T, N, seed):
    """N packed lengths that sum to T, empty ones among them, as prefix sums on the host."""
    cuts = np.random.RandomState(seed % (1 << 31)).randint(0, T + 1, max(N - 1, 0))
    if N > 4:
        cuts[0] = cuts[1]  # one empty sequence at least
    return np.concatenate([[0], np.sort(cuts), [T]]).astype(np.int32)


def _gates(gen, shape, mu):
    z = torch.randn(shape, generator=gen, device="cuda") + mu
    return -torch.nn.functional.softplus(z)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)

    op, io = case["op"], _TYPES[case["io"]]
    s = {"case": case}
    if op in ("scan", "scan_grad"):
        T, C, N, gate = case["T"], case["C"], case["N"], _TYPES[case["gate"]]
        s["cu"] = torch.from_numpy(_cu(T, N, seed)).cuda()
        s["h0"] = normal(N, C) if case["h0"] else None
        x, la = normal(T, C, dtype=io), _gates(gen, (T, C), case["mu"]).to(gate)
        if case["fused"]:
            both = torch.stack([x, la], 1)
            x, la = both[:, 0], both[:, 1]
        s["la"] = la
        if op == "scan":
            s["x"] = x
        else:
            s["h"] = _plain_scan(x, la, s["h0"], s["cu"])[0]
            s["dh"] = normal(T, C, dtype=io)
            s["dh_final"] = normal(N, C) if case["h0"] else None
    elif op == "scan_step":
        B, C = case["B"], case["C"]
        s["x"] = normal(B, C, dtype=io)
        s["la"] = _gates(gen, (B, C), case["mu"]).to(_TYPES[case["gate"]])
        s["state"] = normal(B, C)  # running states, updated in place by every step
    elif op in ("norm", "norm_grad"):
        T, H, d = case["T"], case["H"], case["d"]
        s["x"] = normal(T, H, d, dtype=io)
        s["w"] = 1.0 + normal(H, d, scale=0.1) if case["per_head"] else 1.0 + normal(d, scale=0.1)
        s["b"] = normal(*s["w"].shape, scale=0.1) if case["bias"] else None
        s["z"] = None
        if case["gated"]:
            s["z"] = normal(T, 2, H, d, dtype=io)[:, 1] if case["fused"] else \
                normal(T, H, d, dtype=io)
        if op == "norm_grad":
            s["dy"] = normal(T, H, d, dtype=io)
    else:
        T, Hq, Hv = case["T"], case["Hq"], case["Hv"]
        s["cu"] = torch.from_numpy(_cu(T, case["N"], seed)).cuda()
        for name, H in (("q", Hq), ("k", Hq), ("v", Hv)):
            s[name] = normal(T, H, 128, dtype=io)
            s["d" + name] = normal(T, H, 128, dtype=io)
        for name in ("a", "b", "dla", "dbe"):
            s[name] = normal(T, Hv)
        s["w"] = normal((2 * Hq + Hv) * 128, 4, scale=0.5)
    return s


# ---------------------------------------------------------------- plain forms
def _starts(cu, T):
    """The start of the sequence that holds each token, and the last token of each sequence."""
    t = torch.arange(T, device=cu.device)
    n = torch.bucketize(t, cu[1:].long(), right=True)
    return cu.long()[n], n


def _doubling(a, b):
    """All prefixes of h -> a h + b along dim 0, from h = 0, by doubling the span."""
    T, span = a.shape[0], 1
    while span < T:
        b = torch.cat([b[:span], torch.addcmul(b[span:], a[span:], b[:-span])])
        if 2 * span < T:
            a = torch.cat([a[:span], a[span:] * a[:-span]])
        span *= 2
    return b


def _plain_scan(x, la, h0, cu):
    T, N = x.shape[0], cu.numel() - 1
    start, n = _starts(cu, T)
    first = (torch.arange(T, device=x.device) == start)[:, None]
    a, b = torch.exp(la.float()), x.float()
    if h0 is not None:
        b = torch.where(first, torch.addcmul(b, a, h0[n]), b)
    h = _doubling(torch.where(first, 0.0, a), b)
    last = cu[1:].long() - 1
    given = torch.zeros((N, x.shape[1]), device=x.device) if h0 is None else h0
    h_final = torch.where((cu[1:] > cu[:-1])[:, None], h[last.clamp(min=0)], given)
    return h.to(x.dtype), h_final


def _plain_scan_grad(la, h, dh, h0, dh_final, cu):
    T, N = dh.shape[0], cu.numel() - 1
    start, n = _starts(cu, T)
    t = torch.arange(T, device=dh.device)
    last = (t == cu.long()[n + 1] - 1)[:, None]
    a, g = torch.exp(la.float()), dh.float()
    if dh_final is not None:
        g = torch.where(last, g + dh_final[n], g)
    # u_t = a_t g_t is what reaches token t - 1
    u = _doubling(torch.where(last, 0.0, a).flip(0), (a * g).flip(0)).flip(0)
    g = g + torch.where(last, 0.0, torch.cat([u[1:], torch.zeros_like(u[:1])]))
    before = torch.cat([torch.zeros_like(u[:1]), h[:-1].float()])
    entering = 0.0 if h0 is None else h0[n]
    before = torch.where((t == start)[:, None], entering, before)
    empty = (cu[1:] == cu[:-1])[:, None]
    through = torch.zeros((N, dh.shape[1]), device=dh.device) if dh_final is None else dh_final
    dh0 = torch.where(empty, through, u[cu[:-1].long().clamp(max=T - 1)])
    return g.to(dh.dtype), (u * before).to(la.dtype), dh0


def _normed(x, norm):
    x = x.float()
    if norm == "mean":
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS)
    return x * r, r


def _plain_norm(x, w, b, z, norm, act):
    n = _normed(x, norm)[0] * w
    if b is not None:
        n = n + b
    g = n if z is None else z.float()
    g = g * torch.sigmoid(g) if act == "silu" else g
    return (g if z is None else n * g).to(x.dtype)


def _plain_norm_grad(dy, x, w, b, z, norm, act):
    xhat, r = _normed(x, norm)
    n = xhat * w
    if b is not None:
        n = n + b
    g = n if z is None else z.float()
    sg = torch.sigmoid(g)
    value, slope = (g * sg, sg * (1 + g * (1 - sg))) if act == "silu" else (g, torch.ones_like(g))
    dy = dy.float()
    dz = None
    if z is None:
        dn = dy * slope
    else:
        dn, dz = dy * value, (dy * n * slope).to(x.dtype)
    over = 0 if w.dim() == 2 else (0, 1)
    dw, db = (dn * xhat).sum(over), dn.sum(over) if b is not None else None
    dxh = dn * w
    dx = dxh - xhat * (dxh * xhat).mean(-1, keepdim=True)
    if norm == "mean":
        dx = dx - dxh.mean(-1, keepdim=True)
    return (dx * r).to(x.dtype), dw, db, dz


def _plain_front_part(x, w, dout, pos, act, l2):
    """One of q, k, v: x, dout [T, H, 128], w [H 128, 4] -> dx, dw."""
    T = x.shape[0]
    xf, w = x.reshape(T, -1).float(), w.float()

    def back(j):  # x_{t-j} within the sequence
        if j == 0:
            return xf
        moved = torch.cat([torch.zeros_like(xf[:j]), xf[:-j]])[:T]
        return torch.where(pos >= j, moved, 0.0)

    y = back(3) * w[:, 0] + back(2) * w[:, 1] + back(1) * w[:, 2] + xf * w[:, 3]
    s = torch.sigmoid(y)
    u, slope = (y * s, s * (1 + y * (1 - s))) if act == "silu" else (y, 1.0)
    du = dout.float()
    if l2:
        uh = u.view(T, -1, 128)
        r = torch.rsqrt((uh * uh).sum(-1, keepdim=True) + _EPS)
        qh = uh * r
        du = r * (du - qh * (qh * du).sum(-1, keepdim=True))
    dy = du.reshape(T, -1) * slope

    def ahead(j):  # dy_{t+j} of the same sequence
        if j == 0:
            return dy
        return torch.cat([torch.where(pos >= j, dy, 0.0)[j:], torch.zeros_like(dy[:j])])[:T]

    dx = ahead(3) * w[:, 0] + ahead(2) * w[:, 1] + ahead(1) * w[:, 2] + dy * w[:, 3]
    dw = torch.stack([(dy * back(3)).sum(0), (dy * back(2)).sum(0), (dy * back(1)).sum(0),
                      (dy * xf).sum(0)], 1)
    return dx.view(x.shape).to(x.dtype), dw


def _plain_front_grad(s):
    T, Hq = s["q"].shape[0], s["q"].shape[1]
    act = s["case"]["act"]
    pos = (torch.arange(T, device=s["cu"].device) - _starts(s["cu"], T)[0])[:, None]
    wq, wk, wv = s["w"][: Hq * 128], s["w"][Hq * 128: 2 * Hq * 128], s["w"][2 * Hq * 128:]
    dq, dwq = _plain_front_part(s["q"], wq, s["dq"], pos, act, True)
    dk, dwk = _plain_front_part(s["k"], wk, s["dk"], pos, act, True)
    dv, dwv = _plain_front_part(s["v"], wv, s["dv"], pos, act, False)
    be = torch.sigmoid(s["b"])
    return (dq, dk, dv, torch.cat([dwq, dwk, dwv]), -torch.sigmoid(s["a"]) * s["dla"],
            be * (1 - be) * s["dbe"])


# ---------------------------------------------------------------- one pass
@functools.lru_cache(None)
def _framework():
    from linear_attention_12_b200 import gdn
    return gdn


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        gdn = _framework()
    if op == "scan":
        if own:
            return gdn.scan(s["x"], s["la"], s["h0"], s["cu"])
        return _plain_scan(s["x"], s["la"], s["h0"], s["cu"])
    if op == "scan_grad":
        if own:
            return gdn.scan_backward(s["la"], s["h"], s["dh"], s["h0"], s["dh_final"], s["cu"])
        return _plain_scan_grad(s["la"], s["h"], s["dh"], s["h0"], s["dh_final"], s["cu"])
    if op == "scan_step":
        if own:
            h = gdn.scan_step(s["x"], s["la"], s["state"])
        else:
            s["state"].mul_(torch.exp(s["la"].float())).add_(s["x"].float())
            h = s["state"].to(s["x"].dtype)
        return h, s["state"]
    if op == "norm":
        if own:
            return gdn.group_norm(s["x"], s["w"], s["b"], s["z"], norm=c["norm"], act=c["act"],
                                  eps=_EPS)
        return _plain_norm(s["x"], s["w"], s["b"], s["z"], c["norm"], c["act"])
    if op == "norm_grad":
        if own:
            return gdn.group_norm_backward(s["dy"], s["x"], s["w"], s["b"], s["z"],
                                           norm=c["norm"], act=c["act"], eps=_EPS)
        return _plain_norm_grad(s["dy"], s["x"], s["w"], s["b"], s["z"], c["norm"], c["act"])
    if own:
        return gdn.frontend_backward(s["q"], s["k"], s["v"], s["w"], s["a"], s["b"], s["dq"],
                                     s["dk"], s["dv"], s["dla"], s["dbe"], s["cu"], act=c["act"],
                                     eps=_EPS)
    return _plain_front_grad(s)


# ---------------------------------------------------------------- 64 bits
def _exact_scan(s):
    x, la, h0 = s["x"], s["la"], s["h0"]
    cu = s["cu"].tolist()
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    final = torch.zeros((len(cu) - 1, x.shape[1]), dtype=torch.float64, device=x.device)
    if h0 is not None:
        final.copy_(h0)
    a, x = torch.exp(la.double()).unbind(0), x.double().unbind(0)
    rows = out.unbind(0)
    for n in range(len(cu) - 1):
        h = final[n]
        for t in range(cu[n], cu[n + 1]):
            h = torch.addcmul(x[t], a[t], h, out=rows[t])
        final[n] = h
    return out, final


def _exact_scan_grad(s):
    la, h, dh, h0, dh_final = s["la"], s["h"], s["dh"], s["h0"], s["dh_final"]
    cu = s["cu"].tolist()
    N, C = len(cu) - 1, la.shape[1]
    a = torch.exp(la.double())
    g = dh.double()
    before = torch.roll(h, 1, 0).double()
    dh0 = torch.zeros((N, C), dtype=torch.float64, device=la.device)
    ar, gr = a.unbind(0), g.unbind(0)
    for n in range(N):
        lo, hi = cu[n], cu[n + 1]
        if dh_final is not None:
            dh0[n] = dh_final[n]
        if lo == hi:
            continue
        before[lo] = 0.0 if h0 is None else h0[n].double()
        gr[hi - 1].add_(dh0[n])
        for t in range(hi - 1, lo, -1):
            gr[t - 1].addcmul_(ar[t], gr[t])
        dh0[n] = ar[lo] * gr[lo]
    return g, g * a * before, dh0


def _exact_norm(x, w, b, z, norm, act):
    mean = x.mean(-1, keepdim=True) if norm == "mean" else 0.0
    n = (x - mean) / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + _EPS) * w
    n = n if b is None else n + b
    if z is None:
        return torch.nn.functional.silu(n) if act == "silu" else n
    return n * (torch.nn.functional.silu(z) if act == "silu" else z)


def _exact_norm_grad(s, c):
    """By automatic differentiation, a block of tokens at a time."""
    w = s["w"].double().requires_grad_()
    b = None if s["b"] is None else s["b"].double().requires_grad_()
    dx, dz, dw, db = [], [], 0.0, 0.0
    for t in range(0, c["T"], 8192):
        x = s["x"][t:t + 8192].double().requires_grad_()
        z = None if s["z"] is None else s["z"][t:t + 8192].double().requires_grad_()
        y = _exact_norm(x, w, b, z, c["norm"], c["act"])
        leaves = [v for v in (x, w, b, z) if v is not None]
        got = dict(zip(map(id, leaves),
                       torch.autograd.grad(y, leaves, s["dy"][t:t + 8192].double())))
        dx.append(got[id(x)])
        dw = dw + got[id(w)]
        if b is not None:
            db = db + got[id(b)]
        if z is not None:
            dz.append(got[id(z)])
    return (torch.cat(dx), dw, None if b is None else db, torch.cat(dz) if dz else None)


def _exact_front_grad(s, c):
    """By automatic differentiation, one head at a time."""
    cu = s["cu"].tolist()
    outs, weights, at = [], [], 0
    for name in ("q", "k", "v"):
        grads = torch.empty(s[name].shape, dtype=torch.float64, device=s[name].device)
        for head in range(s[name].shape[1]):
            x = s[name][:, head].double().requires_grad_()
            w = s["w"][at:at + 128].double().requires_grad_()
            at += 128
            # every sequence behind three rows of zeros of its own
            padded = []
            for lo, hi in zip(cu[:-1], cu[1:]):
                padded += [x.new_zeros(3, 128), x[lo:hi]]
            p = torch.nn.functional.pad(torch.cat(padded), (0, 0, 0, 3))
            rows = torch.cat([torch.arange(lo, hi, device=x.device) + 3 * n
                              for n, (lo, hi) in enumerate(zip(cu[:-1], cu[1:]))])
            y = sum(p[rows + i] * w[:, i] for i in range(4))
            y = torch.nn.functional.silu(y) if c["act"] == "silu" else y
            if name != "v":
                y = y / torch.sqrt((y ** 2).sum(-1, keepdim=True) + _EPS)
            gx, gw = torch.autograd.grad(y, (x, w), s["d" + name][:, head].double())
            grads[:, head] = gx
            weights.append(gw)
        outs.append(grads)
    a, b = s["a"].double(), s["b"].double()
    be = torch.sigmoid(b)
    return (*outs, torch.cat(weights), -torch.sigmoid(a) * s["dla"].double(),
            be * (1 - be) * s["dbe"].double())


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "scan":
        return _exact_scan(s)
    if op == "scan_grad":
        return _exact_scan_grad(s)
    if op == "scan_step":
        h = s["state"].double() * torch.exp(s["la"].double()) + s["x"].double()
        return h, h
    if op == "norm":
        return torch.cat([
            _exact_norm(s["x"][t:t + 8192].double(), s["w"].double(),
                        None if s["b"] is None else s["b"].double(),
                        None if s["z"] is None else s["z"][t:t + 8192].double(), case["norm"],
                        case["act"]) for t in range(0, case["T"], 8192)])
    if op == "norm_grad":
        return _exact_norm_grad(s, case)
    return _exact_front_grad(s, case)
