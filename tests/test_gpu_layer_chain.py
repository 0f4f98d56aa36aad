"""The operators around a recurrence as a layer uses them: norm with the
residual's addition, a projection, the short convolution on its columns, the linear
attention with its head norm or the selective scan; forward, backward, a prompt and
its tokens; then streams, graphs and a workspace that is handed in.

Bounds.  In fp32 a stage's own error is at most (T + 64) 2^-21 of its terms'
absolute sizes (the attention's products: 2^-13), which are at most some 8 times the
largest value at these sizes; five stages follow each other, each with a gain of
order one, and the gradients pass them twice: 10 x 8 x 2^-15 (T = 40) is under 2^-8
of the largest value, with the attention 10 x 8 x 2^-13 under 2^-6.  A value of
another row, channel or head is wrong by its size."""
import pytest
import torch
import torch.nn.functional as F

import gated_delta_rule_ckda_amd as ck
from parity import log

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
SCAN, ATTN = 2.0 ** -8, 2.0 ** -6


def normal(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g)


def close(name, got, want, bound):
    got, want = got.detach().double().cpu(), want.detach().double()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    off = (got - want).abs().max() / want.abs().max()
    assert off <= bound, (name, float(off))


# ---------------------------------------------------------------- plain layers in fp64

def plain_norm(x, res, w, eps=1e-6):
    r = x + res
    return r / torch.sqrt((r * r).mean(-1, keepdim=True) + eps) * w, r


def plain_conv(x, w, b=None):
    K = w.shape[1]
    p = F.pad(x, (0, 0, K - 1, 0))
    return F.silu(sum(w[:, j] * p[:, j:j + x.shape[1]] for j in range(K)) + (0 if b is None else b))


def plain_scan(x, dt, A, Bm, Cm, D, z, bias):
    d, h, ys = F.softplus(dt + bias), 0, []
    rep = x.shape[2] // Bm.shape[2]
    for t in range(x.shape[1]):
        Bt, Ct = (m[:, t].repeat_interleave(rep, 1) for m in (Bm, Cm))
        h = torch.exp(d[:, t, :, None] * A) * h + (d[:, t] * x[:, t])[..., None] * Bt
        ys.append((h * Ct).sum(-1))
    return (torch.stack(ys, 1) + D * x) * F.silu(z), h


# ---------------------------------------------------------------- a layer with the scan

class ScanLayer:
    """x, res -> y [B,T,C]: norm, projection to x | z | B | C and to dt, convolution, scan."""

    def __init__(self, seed, dm=40, C=72, G=2, N=16, K=4):
        r = normal(seed)
        self.C, self.G, self.N, self.n = C, G, N, G * N
        step = torch.exp(torch.linspace(-6, -1.5, C))
        self.p = dict(wn=1 + 0.2 * r(dm), W=r(dm, 2 * C + 2 * G * N) / dm ** 0.5, Wdt=0.5 * r(dm, C) / dm ** 0.5, wc=0.5 * r(C, K), bc=0.1 * r(C),
                      A=-(1 + torch.arange(N)).float() * torch.exp(0.1 * r(C, N)), D=1 + 0.1 * r(C), bias=torch.log(torch.expm1(step)))

    def split(self, p, lead):
        C, n = self.C, self.n
        heads = lambda t: t.unflatten(lead, (self.G, self.N))  # noqa: E731
        return p[..., :C], p[..., C:2 * C], heads(p[..., 2 * C:2 * C + n]), heads(p[..., 2 * C + n:])

    def plain(self, P, x, res):
        y, r = plain_norm(x, res, P["wn"])
        xs, z, Bm, Cm = self.split(y @ P["W"], 2)
        u = plain_conv(xs, P["wc"], P["bc"])
        return (*plain_scan(u, y @ P["Wdt"], P["A"], Bm, Cm, P["D"], z, P["bias"]), r)

    def weights(self, P, dtype):
        return [P[n].to(dtype) for n in ("W", "Wdt")]

    def forward(self, P, x, res, lens=None, ws=None):
        W, Wdt = self.weights(P, x.dtype)
        y, r = ck.add_norm_fwd(x, res, P["wn"])
        p, dt = y @ W, y @ Wdt
        xs, z, Bm, Cm = self.split(p, 2)
        u, sT = ck.short_conv_fwd(xs, P["wc"], P["bc"], lens=lens)
        u = u.flatten(1, 2)   # [B,1,T,C], one head
        out, hT = ck.selective_scan_fwd(u, dt, P["A"], Bm, Cm, D=P["D"], z=z, dt_bias=P["bias"], lens=lens, workspace=ws)
        return dict(out=out, hT=hT, sT=sT, r=r, y=y, p=p, dt=dt, u=u)

    def backward(self, P, f, dout, dr, dhT, ws=None):
        W, Wdt = self.weights(P, dout.dtype)
        xs, z, Bm, Cm = self.split(f["p"], 2)
        du, ddt, dA, dBm, dCm, dD, dz, dbias, _ = ck.selective_scan_bwd(
            f["u"], f["dt"], P["A"], Bm, Cm, dout, D=P["D"], z=z, dt_bias=P["bias"], dhT=dhT, workspace=ws)
        dxs, dwc, dbc, _ = ck.short_conv_bwd(xs, P["wc"], du.unsqueeze(1), P["bc"])
        dp = torch.cat([dxs, dz, dBm.flatten(2), dCm.flatten(2)], -1)
        flat = lambda t: t.flatten(0, 1)  # noqa: E731
        y = flat(f["y"])
        dy = (flat(dp) @ W.t() + flat(ddt) @ Wdt.t()).view_as(f["y"])
        dx, dres, dwn = ck.add_norm_bwd(f["r"], dy, P["wn"], dsum=dr)
        return dict(x=dx, res=dres, wn=dwn, W=y.t() @ flat(dp), Wdt=y.t() @ flat(ddt), wc=dwc, bc=dbc, A=dA, D=dD, bias=dbias)

    def step(self, P, x, res, conv, H):
        W, Wdt = self.weights(P, x.dtype)
        y, _ = ck.add_norm_fwd(x, res, P["wn"])
        p = y @ W
        xs, z, Bm, Cm = self.split(p, 1)
        u = ck.short_conv_decode_step(xs, P["wc"], conv, P["bc"]).flatten(1)
        return ck.selective_scan_decode_step(u, y @ Wdt, P["A"], Bm, Cm, H, D=P["D"], z=z, dt_bias=P["bias"])


def data(seed, B, T, dm, *more):
    r = normal(seed)
    return [r(B, T, dm), r(B, T, dm), *(r(*s) for s in more)]


def cuda(P, dtype=F32):
    return {n: t.cuda() for n, t in P.items()}


def test_scan_layer_forward_and_gradients():
    L = ScanLayer(1)
    B, T, dm = 2, 40, 40
    x, res, dout, dr, dhT = data(2, B, T, dm, (B, T, L.C), (B, T, dm), (B, L.C, L.N))
    P = cuda(L.p)
    f = L.forward(P, x.cuda(), res.cuda())
    g = L.backward(P, f, dout.cuda(), dr.cuda(), dhT.cuda())
    leaves = {n: t.double().requires_grad_() for n, t in {**L.p, "x": x, "res": res}.items()}
    out, hT, r = L.plain(leaves, leaves["x"], leaves["res"])
    ((out * dout).sum() + (r * dr).sum() + (hT * dhT).sum()).backward()
    torch.cuda.synchronize()
    log("scan layer B=2 T=40")
    for n, want in (("out", out), ("hT", hT), ("r", r)):
        close(n, f[n], want, SCAN)
    for n, t in leaves.items():
        close("d" + n, g[n], t.grad, SCAN)


def test_scan_layer_gradients_against_differences():
    """<gradient, direction> against central differences of the layer in fp64: their own error is some 1e-8."""
    L = ScanLayer(3, C=24, G=1, N=5, K=3)
    B, T, dm = 2, 20, 40
    x, res, dout, dr, dhT = data(4, B, T, dm, (B, T, L.C), (B, T, dm), (B, L.C, L.N))
    P = cuda(L.p)
    g = L.backward(P, L.forward(P, x.cuda(), res.cuda()), dout.cuda(), dr.cuda(), dhT.cuda())
    torch.cuda.synchronize()
    base = {n: t.double() for n, t in {**L.p, "x": x, "res": res}.items()}

    def loss(v):
        out, hT, r = L.plain(v, v["x"], v["res"])
        return (out * dout).sum() + (r * dr).sum() + (hT * dhT).sum()

    r = normal(5)
    for n in base:
        d = r(*base[n].shape).double()
        slope = (loss({**base, n: base[n] + 1e-5 * d}) - loss({**base, n: base[n] - 1e-5 * d})) / 2e-5
        terms = g[n].double().cpu() * d
        assert (slope - terms.sum()).abs() <= SCAN * terms.abs().sum(), n


@pytest.mark.parametrize("lens", [[30, 7, 0], [1, 2, 3]])
def test_scan_layer_prompt_then_tokens(lens):
    """A padded batch of prompts, then tokens one by one, against the whole sequences."""
    L = ScanLayer(6)
    B, T, dm, more = 3, 30, 40, 4
    x, res = data(7, B, T + more, dm)
    P = cuda(L.p)
    xp, rp = x[:, :T].clone(), res[:, :T].clone()
    for i, n in enumerate(lens):
        xp[i, n:], rp[i, n:] = 3.0, float("nan")   # what stands behind a prompt is not read
    f = L.forward(P, xp.cuda(), rp.cuda(), lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    conv, H = f["sT"], f["hT"]
    seqs = [(torch.cat([x[i, :n], x[i, T:]])[None].double(), torch.cat([res[i, :n], res[i, T:]])[None].double()) for i, n in enumerate(lens)]
    want = [L.plain({n: t.double() for n, t in L.p.items()}, *s)[0][0] for s in seqs]
    for s in range(more):
        y = L.step(P, x[:, T + s].contiguous().cuda(), res[:, T + s].contiguous().cuda(), conv, H)
        torch.cuda.synchronize()
        for i, n in enumerate(lens):
            close(f"token {s} of {i}", y[i], want[i][n + s], SCAN)
    for i, n in enumerate(lens):
        if n:
            close(f"prompt {i}", f["out"][i, :n], want[i][:n], SCAN)


# ---------------------------------------------------------------- a layer with the attention

def test_attention_layer_forward_and_gradients():
    """Norm, projection to q | k | v | gate, a convolution of each head-major, linear attention, head norm."""
    B, T, dm, H, Hk, dk, dv = 2, 40, 48, 4, 2, 32, 32
    r = normal(8)
    nq, nv = Hk * dk, H * dv
    P = dict(wn=1 + 0.2 * r(dm), W=r(dm, 2 * nq + 2 * nv) / dm ** 0.5, wq=0.5 * r(nq, 4), wk=0.5 * r(nq, 4), wv=0.5 * r(nv, 3),
             g=-torch.rand(H, generator=torch.Generator().manual_seed(9)) * 0.3, wo=1 + 0.2 * r(H, dv))
    x, res, dout, dr = data(10, B, T, dm, (B, T, H, dv), (B, T, dm))
    at = (0, nq, 2 * nq, 2 * nq + nv, 2 * nq + 2 * nv)
    cut = lambda p: [p[..., a:b] for a, b in zip(at, at[1:])]  # noqa: E731

    leaves = {n: t.double().requires_grad_() for n, t in {**P, "x": x, "res": res}.items()}
    y, rr = plain_norm(leaves["x"], leaves["res"], leaves["wn"])
    pq, pk, pv, pz = cut(y @ leaves["W"])
    heads = lambda t, n: t.unflatten(2, (n, -1)).transpose(1, 2)  # noqa: E731
    q, k, v = (heads(plain_conv(p, leaves[w]), n) for p, w, n in ((pq, "wq", Hk), (pk, "wk", Hk), (pv, "wv", H)))
    S, os = 0, []
    for t in range(T):
        kt, qt = (m[:, :, t].repeat_interleave(H // Hk, 1) for m in (k, q))
        S = torch.exp(leaves["g"])[:, None, None] * S + kt[..., None] * v[:, :, t, None, :]
        os.append((S * qt[..., None]).sum(2))
    o = torch.stack(os, 1)                                                          # [B,T,H,dv]
    want = o / torch.sqrt((o * o).mean(-1, keepdim=True) + 1e-5) * leaves["wo"] * F.silu(pz.unflatten(2, (H, dv)))
    ((want * dout).sum() + (rr * dr).sum()).backward()

    d = cuda(P)
    y, total = ck.add_norm_fwd(x.cuda(), res.cuda(), d["wn"])
    p = y @ d["W"]
    pq, pk, pv, pz = cut(p)
    (q, _), (k, _), (v, _) = (ck.short_conv_fwd(t, d[w], heads=n) for t, w, n in ((pq, "wq", Hk), (pk, "wk", Hk), (pv, "wv", H)))
    o, _ = ck.linattn_fwd(q, k, v, d["g"])
    gate = pz.unflatten(2, (H, dv)).contiguous()
    out = ck.head_norm_fwd(o, d["wo"], gate=gate, rms=True)
    do, dz, dwo, _ = ck.head_norm_bwd(o, dout.cuda(), d["wo"], gate=gate, rms=True)
    dq, dk_, dv_, dg, _ = ck.linattn_bwd(q, k, v, d["g"], do)
    (dpq, dwq, _, _), (dpk, dwk, _, _), (dpv, dwv, _, _) = (
        ck.short_conv_bwd(t, d[w], gr) for t, w, gr in ((pq, "wq", dq), (pk, "wk", dk_), (pv, "wv", dv_)))
    dp = torch.cat([dpq, dpk, dpv, dz.flatten(2)], -1)
    dx, dres, dwn = ck.add_norm_bwd(total, dp @ d["W"].t(), d["wn"], dsum=dr.cuda())
    got = dict(x=dx, res=dres, wn=dwn, W=y.flatten(0, 1).t() @ dp.flatten(0, 1), wq=dwq, wk=dwk, wv=dwv, g=dg, wo=dwo)
    torch.cuda.synchronize()
    log("attention layer B=2 T=40")
    close("out", out, want, ATTN)
    for n, t in leaves.items():
        close("d" + n, got[n], t.grad, ATTN)


# ---------------------------------------------------------------- streams, graphs, workspaces

def layer_case(seed, B, T, dtype=BF, **sizes):
    L = ScanLayer(seed, **sizes)
    x, res, dout, dr, dhT = data(seed + 50, B, T, 40, (B, T, L.C), (B, T, 40), (B, L.C, L.N))
    return L, cuda(L.p), [t.to(dtype).cuda() for t in (x, res, dout, dr)] + [dhT.cuda()]


def train(L, P, d, ws=None):
    f = L.forward(P, d[0], d[1], ws=ws)
    return [f["out"], f["hT"], f["sT"], *L.backward(P, f, *d[2:], ws=ws).values()]


def same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


def serve(L, P, d, conv, H):
    f = L.forward(P, d[0], d[1])
    q, s, _ = ck.add_norm_quant_fwd(d[0], d[1], P["wn"])
    steps = [L.step(P, d[0][:, t].contiguous(), d[1][:, t].contiguous(), conv, H) for t in (0, 1)]
    return [f["out"], f["hT"], f["sT"], q.view(torch.uint8), s, *steps]


# 4 lanes a channel with and without segments, 16 with and without
SHAPES = [dict(B=2, T=70), dict(B=1, T=1400, C=20, G=1), dict(B=800, T=20, C=64, G=1), dict(B=16, T=2060, C=130, G=1)]


@pytest.mark.parametrize("shape", SHAPES)
def test_graph_replays_match_eager(shape):
    """A training step's forward and backward in one graph, replayed with eager work between."""
    shape = dict(shape)
    B, T = shape.pop("B"), shape.pop("T")
    L, P, d = layer_case(20, B, T, **shape)
    want = [t.clone() for t in train(L, P, d)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = train(L, P, d)
    for rep in range(4):
        for t in got:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert same(got, want), rep
        train(L, P, [0.5 * t for t in d])   # eager work between replays
        torch.cuda.synchronize()


def test_serving_graph_replays_match_eager():
    L, P, d = layer_case(21, 3, 33)
    conv0, H0 = normal(1)(3, 3, L.C).to(BF).cuda(), normal(2)(3, L.C, L.N).cuda()
    conv, H = conv0.clone(), H0.clone()
    want = [t.clone() for t in serve(L, P, d, conv, H)] + [conv, H]
    torch.cuda.synchronize()
    cg, Hg = conv0.clone(), H0.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = serve(L, P, d, cg, Hg)
    for rep in range(4):
        for t in got:
            t.zero_()
        cg.copy_(conv0)
        Hg.copy_(H0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert same(got + [cg, Hg], want), rep
        serve(L, P, d, conv0.clone(), H0.clone())
        torch.cuda.synchronize()


def test_graphs_that_share_a_workspace():
    """Two graphs captured with one workspace, replayed in turn: nothing is kept in it between calls."""
    cases = [layer_case(22, 1, 1400, C=20, G=1), layer_case(23, 2, 300)]
    need = max(f(d[0].shape[0], d[0].shape[1], L.C, L.G, L.N, BF) for L, _, d in cases
               for f in (ck.selective_scan_workspace_size, ck.selective_scan_bwd_workspace_size))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    want = [[t.clone() for t in train(*c, ws=ws)] for c in cases]
    torch.cuda.synchronize()
    graphs, got = [], []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(train(*c, ws=ws))
        graphs.append(g)
    for rep in range(3):
        for i in (0, 1):
            for t in got[i]:
                t.fill_(float("nan"))
            ws.fill_(255)
            graphs[i].replay()
            torch.cuda.synchronize()
            assert same(got[i], want[i]), (rep, i)


def test_streams():
    """On a side stream, and two calls at once on two, by the stream argument and as the current stream."""
    cases = [layer_case(24, 1, 1400, C=20, G=1), layer_case(25, 2, 500)]
    want = [train(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(3):
        for i, c in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                got[i] = train(*c)
    torch.cuda.synchronize()
    assert same(got[0], want[0]) and same(got[1], want[1])
    L, P, d = cases[1]
    y, r = ck.add_norm_fwd(d[0], d[1], P["wn"])
    x = torch.nn.functional.pad(d[2], (0, 3))[..., :L.C]
    u, sT = ck.short_conv_fwd(x, P["wc"], P["bc"])
    dx = ck.short_conv_bwd(x, P["wc"], u, P["bc"])
    dn = ck.add_norm_bwd(r, y, P["wn"], dsum=r)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    y2, r2 = ck.add_norm_fwd(d[0], d[1], P["wn"], stream=s)
    u2, sT2 = ck.short_conv_fwd(x, P["wc"], P["bc"], stream=s)
    dx2 = ck.short_conv_bwd(x, P["wc"], u2, P["bc"], stream=s)
    dn2 = ck.add_norm_bwd(r2, y2, P["wn"], dsum=r2, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert same([y, r, u, sT, *dx, *dn], [y2, r2, u2, sT2, *dx2, *dn2])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_tensor_in_several_places(dtype):
    """x is dt, z and dy, Bm is Cm, dhT is h0: the same as with copies."""
    r = normal(30)
    x, Bm, A, h0 = r(2, 100, 33).to(dtype).cuda(), r(2, 100, 1, 16).to(dtype).cuda(), -torch.rand(33, 16).cuda(), r(2, 33, 16).cuda()
    c = lambda t: t.clone()  # noqa: E731
    want = [*ck.selective_scan_fwd(x, c(x), A, Bm, c(Bm), z=c(x), h0=h0),
            *ck.selective_scan_bwd(x, c(x), A, Bm, c(Bm), c(x), z=c(x), h0=h0, dhT=c(h0))]
    got = [*ck.selective_scan_fwd(x, x, A, Bm, Bm, z=x, h0=h0), *ck.selective_scan_bwd(x, x, A, Bm, Bm, x, z=x, h0=h0, dhT=h0)]
    w = r(33, 4).cuda()
    want += ck.short_conv_bwd(x, w, c(x).unsqueeze(1))
    got += ck.short_conv_bwd(x, w, x.unsqueeze(1))
    want += [*ck.add_norm_fwd(x, c(x)), *ck.add_norm_bwd(x, c(x), dsum=c(x))]
    got += [*ck.add_norm_fwd(x, x), *ck.add_norm_bwd(x, x, dsum=x)]
    torch.cuda.synchronize()
    assert same(got, want)


def test_scan_without_channels():
    """No channel: the sums over channels are zero."""
    e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    Bm = torch.ones(2, 30, 3, 16, device="cuda")
    y, hT = ck.selective_scan_fwd(e(2, 30, 0), e(2, 30, 0), e(0, 16), Bm, Bm)
    junk = [torch.full_like(Bm, float("nan")) for _ in range(4)]
    del junk   # (what the gradients' memory held)
    g = ck.selective_scan_bwd(e(2, 30, 0), e(2, 30, 0), e(0, 16), Bm, Bm, e(2, 30, 0))
    torch.cuda.synchronize()
    assert y.shape == (2, 30, 0) and hT.shape == (2, 0, 16)
    assert g[3].shape == g[4].shape == Bm.shape and (g[3] == 0).all() and (g[4] == 0).all()
