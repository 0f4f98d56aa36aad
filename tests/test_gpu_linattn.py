"""The linear attention with a decay for each head on the GPU: forward,
backward and decode step against the fp64 recurrences, elementwise, within
bounds derived in linattn_cases.py; then its states continued, streams, graphs
and the norm behind it."""
import numpy as np
import pytest
import torch

import gated_delta_rule_ckda_amd as ck
import linattn_reference as ref
from linattn_cases import bwd_bounds, check, cuda, fwd_bounds, inputs
from parity import log

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def fwd(d, **kw):
    return ck.linattn_fwd(d["q"], d["k"], d["v"], d["g"], d["h0"], lens=d["lens"], **kw)


def bwd(d, **kw):
    return ck.linattn_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], d["h0"], d["dhT"], lens=d["lens"], **kw)


def run_fwd(x):
    log(f"linattn_fwd q {tuple(x['q'].shape)} v {tuple(x['v'].shape)} g {tuple(x['g'].shape)} {x['q'].dtype}")
    o, hT, bo, bh = fwd_bounds(x)
    got_o, got_h = fwd(cuda(x))
    torch.cuda.synchronize()
    check("o", got_o, o, bo)
    check("hT", got_h, hT, bh)


def run_bwd(x):
    log(f"linattn_bwd q {tuple(x['q'].shape)} v {tuple(x['v'].shape)} g {tuple(x['g'].shape)} {x['q'].dtype}")
    want = bwd_bounds(x)
    got = dict(zip(("dq", "dk", "dv", "dg", "dh0"), bwd(cuda(x))))
    torch.cuda.synchronize()
    for n, (w, b) in want.items():
        check(n, got[n], w, b)


LENGTHS = [1, 2, 15, 16, 17, 63, 64, 65, 128, 129, 200]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", LENGTHS)
def test_forward_lengths(T, dtype):
    run_fwd(inputs(100 + T, 2, 2, 2, T, 64, 32, dtype))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk", [16, 32, 64, 128])
@pytest.mark.parametrize("dv", [16, 32, 64, 128])
def test_forward_widths(dk, dv, dtype):
    run_fwd(inputs(dk * 1000 + dv, 1, 3, 3, 150, dk, dv, dtype))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,H,Hk,decay", [(2, 4, 2, "token"), (1, 6, 1, "head"), (8, 1, 1, "head"), (4, 8, 4, "token")])
def test_forward_heads(B, H, Hk, decay, dtype):
    run_fwd(inputs(B * 100 + H, B, H, Hk, 77, 32, 64, dtype, decay=decay))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("special", ["reset", "lowest", "none", "strong"])
def test_forward_decays(special, dtype):
    run_fwd(inputs(7, 2, 3, 3, 140, 64, 64, dtype, special=special))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_forward_without_state(dtype):
    run_fwd(inputs(9, 2, 2, 2, 100, 128, 128, dtype, state=False))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_forward_lens(dtype):
    run_fwd(inputs(21, 6, 2, 1, 130, 32, 32, dtype, lens=[130, 0, 1, 64, 65, 129]))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_forward_leaves_rows_behind_a_sequence(dtype):
    """Rows at or past lens are not read (NaN there changes nothing) and not written; lengths out of range are clamped."""
    x = inputs(22, 3, 2, 2, 100, 32, 64, dtype, lens=[30, 1000, -5])
    o, hT, bo, bh = fwd_bounds(x)
    d = cuda(x)
    for n in ("q", "k", "v", "g"):
        d[n][0, :, 30:] = float("nan")
        d[n][2] = float("nan")
    out = torch.full((3, 2, 100, 64), 7.0, dtype=dtype, device="cuda")
    got_o, got_h = fwd(d, o=out)
    torch.cuda.synchronize()
    assert (got_o[0, :, 30:] == 7).all() and (got_o[2] == 7).all()
    check("o", got_o[0, :, :30], o[0, :, :30], bo[0, :, :30])
    check("o", got_o[1], o[1], bo[1])
    check("hT", got_h, hT, bh)
    assert torch.equal(got_h[2], d["h0"][2])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [None, [2500, 1300]])
def test_forward_segments(dtype, lens):
    """Few heads and many rows: the sequence is split, its states joined."""
    B, H, Hk, T = 2, 2, 1, 2500
    assert ck.linattn_workspace_size(B, H, T, 32, 32, dtype) > 256
    run_fwd(inputs(31, B, H, Hk, T, 32, 32, dtype, lens=lens))


def test_empty_sequences_and_batches():
    d = cuda(inputs(1, 2, 2, 2, 0, 32, 32, BF))
    o, hT = fwd(d)
    assert o.shape == (2, 2, 0, 32) and torch.equal(hT, d["h0"])
    g = bwd(d)
    assert torch.equal(g[4], d["dhT"])
    h = cuda(inputs(1, 2, 2, 2, 0, 32, 32, BF, decay="head"))
    assert (bwd(h)[3] == 0).all()
    e = cuda(inputs(1, 0, 2, 2, 5, 32, 32, BF, state=False))
    assert fwd(e)[0].shape == (0, 2, 5, 32)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_final_state_in_place_and_continued(dtype):
    """hT = h0 in place, and two parts of a sequence equal the whole."""
    x = inputs(41, 2, 3, 3, 200, 64, 64, dtype)
    o, hT, bo, bh = fwd_bounds(x)
    d = cuda(x)
    S = d["h0"].clone()
    parts = []
    for a, b in ((0, 70), (70, 200)):
        p = {n: d[n][:, :, a:b].contiguous() for n in ("q", "k", "v", "g")}
        parts.append(ck.linattn_fwd(p["q"], p["k"], p["v"], p["g"], S, hT=S)[0])
    torch.cuda.synchronize()
    check("o", torch.cat(parts, 2), o, bo)
    check("hT", S, hT, bh)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 17, 64, 65, 200])
def test_backward_lengths(T, dtype):
    run_bwd(inputs(200 + T, 2, 2, 2, T, 64, 64, dtype))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(16, 16), (16, 128), (128, 16), (32, 64), (128, 128), (64, 32)])
def test_backward_widths(dk, dv, dtype):
    run_bwd(inputs(dk * 1000 + dv + 1, 1, 3, 3, 100, dk, dv, dtype))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,H,Hk,decay", [(2, 4, 2, "token"), (3, 6, 1, "head"), (8, 1, 1, "head"), (2, 8, 4, "token")])
def test_backward_heads(B, H, Hk, decay, dtype):
    run_bwd(inputs(B * 100 + H + 1, B, H, Hk, 77, 32, 64, dtype, decay=decay))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("special", ["reset", "lowest", "none", "strong"])
def test_backward_decays(special, dtype):
    run_bwd(inputs(8, 2, 2, 2, 140, 64, 64, dtype, special=special))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("decay", ["token", "head"])
def test_backward_lens(dtype, decay):
    run_bwd(inputs(23, 6, 2, 1, 130, 32, 32, dtype, decay=decay, lens=[130, 0, 1, 64, 65, 129]))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("state", [True, False])
def test_backward_segments(dtype, state):
    B, H, Hk, T = 1, 2, 1, 2500
    run_bwd(inputs(33, B, H, Hk, T, 32, 32, dtype, state=state, lens=[2333]))


def of_batches(x, keep):
    """The batch entries `keep` of inputs or results: batch entries are independent."""
    return {n: t if t is None or n in ("g", "dg") and t.dim() == 1 else t[keep] for n, t in x.items()}


MANY = [(8, 8, 8), (16, 8, 8), (24, 8, 8), (41, 8, 1), (13, 16, 2)]   # 64 .. 328 heads, whole and broken rounds of units
WIDE = [(16, 128), (128, 128), (64, 128), (128, 64), (32, 64), (64, 64), (128, 16)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", WIDE)
@pytest.mark.parametrize("B,H,Hk", MANY)
def test_many_heads(B, H, Hk, dk, dv, dtype):
    """Calls of many heads take wide slices of the states; two batch entries of each are compared."""
    keep = [0, B - 1]
    x = inputs(B * 1000 + dk + dv, B, H, Hk, 150, dk, dv, dtype)
    log(f"linattn q {tuple(x['q'].shape)} v {tuple(x['v'].shape)} {dtype}")
    d, few = cuda(x), of_batches(x, keep)
    o, hT, bo, bh = fwd_bounds(few)
    want = bwd_bounds(few)
    got_o, got_h = fwd(d)
    only_o, none = fwd(d, want_state=False)
    got = of_batches(dict(zip(("dq", "dk", "dv", "dg", "dh0"), bwd(d))), keep)
    torch.cuda.synchronize()
    assert none is None
    check("o", got_o[keep], o, bo)
    check("hT", got_h[keep], hT, bh)
    check("o without a state", only_o[keep], o, bo)
    for n, (w, b) in want.items():
        check(n, got[n], w, b)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,H,Hk", [(1, 2, 2), (8, 8, 8), (13, 16, 2)])
def test_gradients_without_states(B, H, Hk, dtype):
    """Neither dhT nor dh0: the states of the sweeps are not returned."""
    keep = [0, B - 1]
    x = inputs(B + 61, B, H, Hk, 150, 64, 64, dtype, state=False)
    want = bwd_bounds(of_batches(x, keep))
    got = of_batches(dict(zip(("dq", "dk", "dv", "dg"), bwd(cuda(x), want_dh0=False))), keep)
    torch.cuda.synchronize()
    for n in ("dq", "dk", "dv", "dg"):
        check(n, got[n], *want[n])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(128, 128), (16, 128), (128, 64)])
@pytest.mark.parametrize("lens", [None, [1500, 600]])
def test_segments_of_wide_states(dk, dv, lens, dtype):
    x = inputs(dk + dv, 2, 2, 1, 1500, dk, dv, dtype, lens=lens)
    assert ck.linattn_workspace_size(2, 2, 1500, dk, dv, dtype) > 256
    run_fwd(x)
    run_bwd(x)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,lens", [(1, 100, None), (1, 5000, None), (3, 5000, None), (40, 9, None), (3, 70, [70, 0, 5])])
def test_gradient_of_a_constant_decay(B, T, lens, dtype):
    run_bwd(inputs(B + T, B, 2, 2, T, 16, 16, dtype, decay="head", lens=lens))


def test_backward_against_differences():
    """<gradient, direction> against central differences of the fp64 recurrence."""
    x = inputs(51, 2, 4, 2, 90, 32, 64, F32)
    got = dict(zip(("q", "k", "v", "g", "h0"), bwd(cuda(x))))
    torch.cuda.synchronize()
    r = np.random.default_rng(1)
    y = {n: None if a is None else a.double().numpy() for n, a in x.items()}

    def loss(z):
        o, hT = ref.linattn_fwd(z["q"], z["k"], z["v"], z["g"], z["h0"])
        return (o * z["do"]).sum() + (hT * z["dhT"]).sum()

    for n, grad in got.items():
        d = r.standard_normal(y[n].shape)
        up, down = ({**y, n: y[n] + s * 1e-5 * d} for s in (1, -1))
        slope = (loss(up) - loss(down)) / 2e-5
        terms = np.abs(grad.double().cpu().numpy() * d).sum()
        # the kernel's gradient: its bound is some 2^-13 of sums over absolute terms of like size
        assert abs(slope - (grad.double().cpu().numpy() * d).sum()) <= 2.0 ** -13 * terms, n


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,H,Hk,dk,dv,decay", [(1, 1, 1, 16, 16, "token"), (1, 16, 16, 128, 128, "token"),
                                                (5, 6, 2, 64, 32, "head"), (64, 8, 8, 128, 128, "token"),
                                                (3, 4, 1, 32, 128, "token"), (7, 2, 2, 128, 16, "head")])
def test_decode(N, H, Hk, dk, dv, decay, dtype):
    x = inputs(61, N, H, Hk, 1, dk, dv, dtype, decay=decay)
    one = {n: x[n][:, :, 0].contiguous() for n in ("q", "k", "v")}
    g = x["g"] if decay == "head" else x["g"][:, :, 0].contiguous()
    want_o, want_S = ref.linattn_decode(one["q"], one["k"], one["v"], g, x["h0"])
    abs_o, abs_S = ref.linattn_decode(one["q"].abs(), one["k"].abs(), one["v"].abs(), g, x["h0"].abs())
    S = x["h0"].cuda()
    log(f"linattn_decode N={N} H={H} Hk={Hk} dk={dk} dv={dv} {decay} {dtype}")
    o = ck.linattn_decode_step(one["q"].cuda(), one["k"].cuda(), one["v"].cuda(), g.cuda(), S)
    torch.cuda.synchronize()
    # fp32: the exponential (2 ulp), two roundings a state element, dk additions in o
    check("H", S, want_S, 8 * 2.0 ** -24 * abs_S)
    check("o", o, want_o, torch.finfo(dtype).eps / 2 * np.abs(want_o) + (dk + 16) * 2.0 ** -24 * abs_o)


@pytest.mark.parametrize("special", ["reset", "lowest"])
def test_decode_resets(special):
    x = inputs(62, 4, 4, 4, 1, 32, 32, F32, special=special)
    g = torch.full((4, 4), float("-inf") if special == "reset" else torch.finfo(F32).min)
    S = x["h0"].cuda()
    ck.linattn_decode_step(*(x[n][:, :, 0].contiguous().cuda() for n in ("q", "k", "v")), g.cuda(), S)
    torch.cuda.synchronize()
    want = x["k"][:, :, 0, :, None] * x["v"][:, :, 0, None, :]
    assert torch.equal(S.cpu(), want)


def test_prefill_then_decode_then_norm():
    """As served: a padded batch of prompts through the forward, then tokens
    one by one, each output through the gated norm; against the recurrence over
    prompt and tokens."""
    B, H, Hk, T, dk, dv, steps = 3, 4, 2, 90, 64, 64, 5
    lens = [90, 13, 0]
    x = inputs(71, B, H, Hk, T + steps, dk, dv, BF)
    d = cuda(x)
    first = {n: d[n][:, :, :T].contiguous() for n in ("q", "k", "v", "g")}
    _, S = ck.linattn_fwd(first["q"], first["k"], first["v"], first["g"], d["h0"],
                          lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    w = torch.linspace(0.5, 1.5, H * dv).view(H, dv)
    z = torch.from_numpy(np.random.default_rng(5).standard_normal((B, steps, H, dv)).astype(np.float32)).to(BF)
    _, S_ref, _, bh = fwd_bounds({**x, **{n: x[n][:, :, :T] for n in ("q", "k", "v", "g", "do")},
                                  "lens": torch.tensor(lens, dtype=torch.int32)})
    check("hT", S, S_ref, bh)
    for s in range(steps):
        t = {n: d[n][:, :, T + s].contiguous() for n in ("q", "k", "v", "g")}
        o = ck.linattn_decode_step(t["q"], t["k"], t["v"], t["g"], S)
        y = ck.head_norm_fwd(o.unsqueeze(2), w.cuda(), gate=z[:, s:s + 1].contiguous().cuda(), act="sigmoid", rms=True)
        o_ref, S_ref = ref.linattn_decode(*(x[n][:, :, T + s] for n in ("q", "k", "v", "g")), S_ref)
        y_ref = ref.head_norm(o.unsqueeze(2), w, gate=z[:, s:s + 1], act="sigmoid", rms=True)["y"]
        torch.cuda.synchronize()
        # o: one bf16 rounding, and the prefilled state's error through dk products
        scale = np.abs(o_ref).max()
        check("o", o, o_ref, 2.0 ** -8 * np.abs(o_ref) + 2.0 ** -12 * scale)
        check("y", y, y_ref, 2.0 ** -8 * np.abs(y_ref) + 1e-5)


def test_training_chain():
    """Attention, norm with gate, and back: the loss sum(y c) through both
    backward passes against the fp64 formulas from the kernels' own o."""
    B, H, Hk, T, dk, dv = 2, 4, 2, 150, 32, 64
    x = inputs(81, B, H, Hk, T, dk, dv, F32)
    d = cuda(x)
    r = np.random.default_rng(6)
    z = torch.from_numpy(r.standard_normal((B, T, H, dv)).astype(np.float32))
    c = torch.from_numpy(r.standard_normal((B, T, H, dv)).astype(np.float32))
    w = torch.from_numpy((1 + 0.2 * r.standard_normal((H, dv))).astype(np.float32))
    b = torch.from_numpy((0.2 * r.standard_normal((H, dv))).astype(np.float32))
    o, _ = fwd(d)
    do, dz, dw, db = ck.head_norm_bwd(o, c.cuda(), w.cuda(), b.cuda(), gate=z.cuda())
    got = ck.linattn_bwd(d["q"], d["k"], d["v"], d["g"], do, d["h0"], d["dhT"])
    torch.cuda.synchronize()
    n = ref.head_norm(o, w, b, z, dy=c)
    for name, t in (("dx", do), ("dz", dz), ("dw", dw), ("db", db)):
        scale = np.abs(n[name]).max()
        check(name, t, n[name], np.full(n[name].shape, 1e-5 * scale))
    want = bwd_bounds({**x, "do": do.cpu()})
    for name, t in zip(("dq", "dk", "dv", "dg", "dh0"), got):
        check(name, t, *want[name])


def test_same_call_twice_gives_the_same_bytes():
    d = cuda(inputs(91, 1, 4, 2, 2100, 64, 64, BF))
    a, b = fwd(d), fwd(d)
    ga, gb = bwd(d), bwd(d)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a + tuple(ga), b + tuple(gb)))


def test_side_stream():
    d = cuda(inputs(92, 2, 4, 2, 300, 64, 64, BF, lens=[300, 200]))
    want, want_g = fwd(d), bwd(d)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got, got_g = fwd(d, stream=s), bwd(d, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(tuple(got) + tuple(got_g), tuple(want) + tuple(want_g)))


def test_graph_replays_match_eager():
    """Forward, norm, both backward passes and a decode step in one graph, replayed with eager work between."""
    x = inputs(93, 2, 2, 1, 2048, 32, 32, BF)
    d = cuda(x)
    w = torch.rand(2, 32, device="cuda")
    S0 = d["h0"].clone()
    step = [d[n][:, :, 0].contiguous() for n in ("q", "k", "v", "g")]

    def work(S):
        o, hT = fwd(d)
        y = ck.head_norm_fwd(o, w)
        do, _, dw, db = ck.head_norm_bwd(o, y, w)
        grads = ck.linattn_bwd(d["q"], d["k"], d["v"], d["g"], do, d["h0"], d["dhT"])
        return [o, hT, y, do, dw, db, *grads, ck.linattn_decode_step(*step, S)]

    S = S0.clone()
    want = [t.clone() for t in work(S)] + [S.clone()]
    torch.cuda.synchronize()
    Sg = S0.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = work(Sg)
    for rep in range(4):
        for t in got:
            t.fill_(float("nan"))
        Sg.copy_(S0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got + [Sg], want)):
            assert torch.equal(a, b), (rep, i)
        work(S0.clone())   # eager work between replays
        torch.cuda.synchronize()


def test_two_streams_at_once():
    """Two calls at once, each with its own workspace and outputs."""
    d1, d2 = cuda(inputs(94, 1, 2, 2, 2500, 32, 32, BF)), cuda(inputs(95, 1, 2, 2, 2500, 32, 32, BF))
    want = [bwd(d1), bwd(d2)]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(3):
        got = [bwd(d1, stream=s1), bwd(d2, stream=s2)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_graphs_that_share_a_workspace():
    """Two graphs captured with one workspace, replayed in turn: nothing is kept in it between calls."""
    d1, d2 = cuda(inputs(96, 2, 2, 1, 2048, 32, 64, BF)), cuda(inputs(97, 1, 4, 4, 1500, 64, 32, BF))
    need = max(ck.linattn_bwd_workspace_size(2, 2, 1, 2048, 32, 64, BF), ck.linattn_bwd_workspace_size(1, 4, 4, 1500, 64, 32, BF),
               ck.linattn_workspace_size(2, 2, 2048, 32, 64, BF), ck.linattn_workspace_size(1, 4, 1500, 64, 32, BF))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    both = lambda d: [*fwd(d, workspace=ws), *bwd(d, workspace=ws)]  # noqa: E731
    want = [[t.clone() for t in both(d)] for d in (d1, d2)]
    torch.cuda.synchronize()
    graphs, got = [], []
    for d in (d1, d2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(both(d))
        graphs.append(g)
    for rep in range(3):
        for i in (0, 1):
            for t in got[i]:
                t.fill_(float("nan"))
            ws.fill_(255)
            graphs[i].replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got[i], want[i])), (rep, i)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_tensor_in_several_places(dtype):
    """q is k, do is v, dhT is h0."""
    x = inputs(98, 2, 3, 3, 150, 64, 64, dtype)
    x["k"], x["do"], x["dhT"] = x["q"], x["v"], x["h0"]
    d = cuda(x)
    d["k"], d["do"], d["dhT"] = d["q"], d["v"], d["h0"]
    o, hT, bo, bh = fwd_bounds(x)
    want = bwd_bounds(x)
    got_o, got_h = fwd(d)
    got = dict(zip(("dq", "dk", "dv", "dg", "dh0"), bwd(d)))
    torch.cuda.synchronize()
    check("o", got_o, o, bo)
    check("hT", got_h, hT, bh)
    for n, (w, b) in want.items():
        check(n, got[n], w, b)
