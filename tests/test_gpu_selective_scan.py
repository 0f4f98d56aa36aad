"""The selective scan on the GPU against the fp64 recurrence, elementwise.

Bounds.  fp32 arithmetic.  A step d is off by some 2^-20 relative (softplus: an
exponential, a reciprocal and a series, a few 2^-24 each, and the rounding of dt +
bias), so a decay exp(d A) by |d A| 2^-20 and 2^-23 of its own; a state that has
seen T rows is off by at most T times one row's error, relative to the size m of
its terms' absolute values, and with decays of rate |d A| it remembers some 1 / |d
A| rows, so |d A| T never enters: (T + 64) 2^-21 of the size covers both.
Gradients are sums of products of states and backward states: twice that.  Weight
gradients and those of B and C sum over rows and channels, which adds their count
times 2^-24.  An output's rounding adds half a step of its type."""
import numpy as np
import pytest
import torch

import gated_delta_rule_ckda_amd as ck
import layer_reference as ref
from linattn_cases import check
from parity import log

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def make(seed, B, T, C, G, N, dtype, gate=True, state=True, lens=None, D=True, bias=True, softplus=True):
    r = np.random.default_rng(seed)
    t = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32))  # noqa: E731
    step = torch.from_numpy(np.exp(r.uniform(np.log(1e-3), np.log(0.3), C)).astype(np.float32))
    a = dict(x=t(B, T, C).to(dtype), A=-(1 + torch.arange(N)).float() * torch.exp(0.1 * t(C, N)),
             Bm=t(B, T, G, N).to(dtype), Cm=t(B, T, G, N).to(dtype), D=1 + 0.2 * t(C) if D else None,
             z=t(B, T, C).to(dtype) if gate else None, h0=0.5 * t(B, C, N) if state else None,
             lens=None if lens is None else torch.tensor(lens, dtype=torch.int32))
    if softplus:
        raw = step + torch.log(-torch.expm1(-step))
        a.update(dt=(0.5 * t(B, T, C) + (0 if bias else raw)).to(dtype), dt_bias=raw if bias else None)
    else:
        a.update(dt=(step * torch.rand(B, T, C, generator=torch.Generator().manual_seed(seed))).to(dtype),
                 dt_bias=1e-3 * torch.ones(C) if bias else None)
    return a, t(B, T, C).to(dtype), 0.5 * t(B, C, N) if state else None


def cuda(a):
    return {n: None if t is None else t.cuda() for n, t in a.items()}


def slices(d):
    """Bm, Cm and z as column slices of one projection, at odd offsets, among NaN."""
    B, T, G, N = d["Bm"].shape
    C, n = d["x"].shape[2], G * N
    wide = torch.full((B, T, 2 * n + C + 5), float("nan"), dtype=d["x"].dtype, device="cuda")
    wide[..., 1:1 + n], wide[..., 1 + n:1 + 2 * n] = d["Bm"].flatten(2), d["Cm"].flatten(2)
    out = dict(d, Bm=wide[..., 1:1 + n].unflatten(2, (G, N)), Cm=wide[..., 1 + n:1 + 2 * n].unflatten(2, (G, N)))
    if d["z"] is not None:
        wide[..., 2 + 2 * n:2 + 2 * n + C] = d["z"]
        out["z"] = wide[..., 2 + 2 * n:2 + 2 * n + C]
    return out


NAMES = ("dx", "ddt", "dA", "dBm", "dCm", "dD", "dz", "dbias", "dh0")


def run(seed, B, T, C, G, N, dtype, backward=True, softplus=True, sliced=False, **kw):
    log(f"selective_scan B={B} T={T} C={C} G={G} N={N} {dtype} softplus={softplus} sliced={sliced} {kw}")
    a, dy, dhT = make(seed, B, T, C, G, N, dtype, softplus=softplus, **kw)
    want = ref.selective_scan(**a, softplus=softplus, dy=dy if backward else None, dhT=dhT)
    d = cuda(a)
    if sliced:
        d = slices(d)
    y, hT = ck.selective_scan_fwd(**d, softplus=softplus)
    half, k = torch.finfo(dtype).eps / 2, (T + 64) * 2.0 ** -21
    got = None
    if backward:
        got = ck.selective_scan_bwd(**d, dy=dy.cuda(), dhT=None if dhT is None else dhT.cuda(), softplus=softplus)
    torch.cuda.synchronize()
    check("y", y, want["y"], half * np.abs(want["y"]) + (k + N * 2.0 ** -24) * want["sy"])
    check("hT", hT, want["hT"], k * want["shT"])
    if not backward:
        return
    for name, g in zip(NAMES, got):
        if name == "dz" and a["z"] is None:
            assert g is None
            continue
        rounded = half if name in ("dx", "ddt", "dBm", "dCm", "dz") else 0.0
        count = {"dBm": C // G, "dCm": C // G, "dx": N, "ddt": N, "dz": N, "dh0": 0}.get(name, B * T)
        check(name, g, want[name], rounded * np.abs(want[name]) + (2 * k + count * 2.0 ** -24) * want["s" + name])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 33, 100])
def test_lengths(T, dtype):
    run(T, 2, T, 40, 1, 16, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [1, 3, 8, 15, 16, 17, 31, 32, 33, 48, 63, 64])
def test_states(N, dtype):
    run(N, 1, 37, 36, 1, N, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("C,G", [(1, 1), (3, 1), (31, 1), (33, 1), (64, 2), (70, 2), (6, 6), (100, 4)])
def test_channels_and_groups(C, G, dtype):
    run(C, 2, 21, C, G, 16, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("D,bias,state", [(True, True, True), (False, False, False), (True, False, True), (False, True, False)])
def test_variants(gate, softplus, D, bias, state, dtype):
    run(7, 2, 35, 40, 1, 16, dtype, softplus=softplus, gate=gate, D=D, bias=bias, state=state)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [[50, 0, 1], [16, 17, 50], [99, -1, 32]])
def test_padded(lens, dtype):
    run(5, 3, 50, 40, 2, 16, dtype, lens=lens)
    run(6, 3, 50, 40, 2, 16, dtype, lens=lens, state=False, gate=False)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [5, 16, 32])
def test_column_slices(N, dtype):
    run(N, 2, 30, 35, 1, N, dtype, sliced=True)
    run(N, 2, 19, 44, 2, N, dtype, sliced=True)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,C,N,lens", [(1, 400, 20, 16, None), (2, 777, 40, 16, [777, 300]), (1, 1000, 64, 8, [513]),
                                          (2, 600, 33, 40, [600, 0])])
def test_segments(B, T, C, N, lens, dtype):
    """Few channels and many rows: several segments, some behind a sequence's end."""
    sizes = ck.selective_scan_workspace_size(B, T, C, 1, N, dtype)
    assert sizes > 256   # the sequence does run in segments
    run(T, B, T, C, 1, N, dtype, lens=lens)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_workgroups(dtype):
    """Every CU has one: one segment, several batch entries and groups."""
    run(11, 8, 40, 1200, 3, 4, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,C,G,N,kw", [(1000, 20, 50, 1, 16, {}), (1000, 33, 50, 2, 5, dict(lens=True)),
                                          (1000, 18, 51, 1, 12, dict(gate=False, state=False)), (16, 2060, 130, 1, 16, {}),
                                          (16, 2100, 130, 2, 7, dict(lens=True, gate=False, D=False)),
                                          (48, 700, 70, 1, 15, dict(lens=True, state=False))])
def test_many_channels_or_long_sequences(B, T, C, G, N, kw, dtype):
    """Four lanes a channel (enough channels and rows for every SIMD), with one segment and with several."""
    if kw.get("lens"):
        lens = np.random.default_rng(T).integers(0, T + 1, B)
        lens[:3] = T, 0, 1
        kw = dict(kw, lens=lens.tolist())
    run(T, B, T, C, G, N, dtype, **kw)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("C,G,N", [(1, 1, 16), (40, 2, 16), (33, 1, 1), (5, 5, 3), (12, 1, 8), (7, 1, 17), (9, 3, 64), (4, 1, 33)])
def test_decode_continues_the_forward(C, G, N, dtype):
    T, S = 9, 3
    a, _, _ = make(N, S, T, C, G, N, dtype)
    want = ref.selective_scan(**a)
    d = slices(cuda(a))
    H = d["h0"].clone()
    rows = [ck.selective_scan_decode_step(d["x"][:, t].contiguous(), d["dt"][:, t].contiguous(), d["A"], d["Bm"][:, t], d["Cm"][:, t],
                                          H, D=d["D"], z=d["z"][:, t], dt_bias=d["dt_bias"]) for t in range(T)]
    torch.cuda.synchronize()
    half, k = torch.finfo(dtype).eps / 2, (T + 64) * 2.0 ** -21
    check("y", torch.stack(rows, 1), want["y"], half * np.abs(want["y"]) + (k + N * 2.0 ** -24) * want["sy"])
    check("H", H, want["hT"], k * want["shT"])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("S,C,N", [(515, 512, 16), (517, 510, 13), (129, 512, 64), (515, 2052, 3)])
def test_decode_of_many_sequences(S, C, N, dtype):
    """Two sequences a thread, their number odd: the same bytes as with the sequences in small calls."""
    a, _, _ = make(N, S, 1, C, 1, N, dtype)
    d = {n: t if n in ("A", "D", "dt_bias", "h0") or t is None else t[:, 0].contiguous() for n, t in cuda(a).items() if n != "lens"}
    H = d.pop("h0")
    one = H.clone()
    rest = ("A", "D", "dt_bias")
    want = torch.cat([ck.selective_scan_decode_step(**{n: t if n in rest else t[i:i + 64] for n, t in d.items()}, H=one[i:i + 64])
                      for i in range(0, S, 64)])   # (16-byte aligned pieces)
    y = ck.selective_scan_decode_step(**d, H=H)
    ref_y = ref.selective_scan(**a)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(H, one)
    half, k = torch.finfo(dtype).eps / 2, 65 * 2.0 ** -21
    check("y", y, ref_y["y"][:, 0], half * np.abs(ref_y["y"][:, 0]) + (k + N * 2.0 ** -24) * ref_y["sy"][:, 0])
    check("H", H, ref_y["hT"], k * ref_y["shT"])


def test_state_continues_in_place():
    """Two halves, the second from the first's state, hT in the place of h0, as the whole."""
    a, _, _ = make(2, 2, 64, 40, 1, 16, F32)
    d = cuda(a)
    y, hT = ck.selective_scan_fwd(**d)
    state, parts = d["h0"].clone(), []
    for at in (slice(0, 32), slice(32, 64)):
        half = {n: d[n][:, at].contiguous() for n in ("x", "dt", "Bm", "Cm", "z")}
        parts.append(ck.selective_scan_fwd(**{**d, **half, "h0": state}, hT=state)[0])
    torch.cuda.synchronize()
    assert torch.equal(torch.cat(parts, 1), y) and torch.equal(state, hT)


@pytest.mark.parametrize("lens", [[5, 0], [40, 16]])
def test_rows_behind_a_sequence(lens):
    """Never read, left as they were in outputs that are passed in, else zero."""
    a, dy, _ = make(3, 2, 40, 24, 1, 16, BF, lens=lens)
    d, g = cuda(a), dy.cuda()
    for i, n in enumerate(lens):
        for k in ("x", "dt", "Bm", "Cm", "z"):
            d[k][i, n:] = float("nan")
        g[i, n:] = float("nan")
    y = torch.full((2, 40, 24), 7.0, dtype=BF, device="cuda")
    _, hT = ck.selective_scan_fwd(**d, y=y)
    out = ck.selective_scan_bwd(**d, dy=g)
    torch.cuda.synchronize()
    assert torch.isfinite(y).all() and torch.isfinite(hT).all()
    for i, n in enumerate(lens):
        assert (y[i, n:] == 7).all()
        for k in (0, 1, 3, 4, 6):
            assert (out[k][i, n:] == 0).all()
    assert all(torch.isfinite(t).all() for t in out)


def test_no_rows():
    a, dy, dhT = make(4, 2, 0, 24, 1, 16, F32)
    d = cuda(a)
    y, hT = ck.selective_scan_fwd(**d)
    out = ck.selective_scan_bwd(**d, dy=dy.cuda(), dhT=dhT.cuda())
    torch.cuda.synchronize()
    assert y.shape == (2, 0, 24) and torch.equal(hT, d["h0"]) and torch.equal(out[8].cpu(), dhT)
    assert all((out[k] == 0).all() for k in (2, 5, 7))


@pytest.mark.parametrize("B,T,C,N", [(1, 1500, 20, 16), (1, 1500, 20, 40), (16, 2060, 130, 16), (40, 2060, 130, 16), (2, 30, 24, 16)])
def test_final_state_in_place_of_the_initial_one(B, T, C, N):
    a, _, _ = make(9, B, T, C, 1, N, BF)
    d = cuda(a)
    want = ck.selective_scan_fwd(**d)
    h0 = d["h0"].clone()
    for _ in range(3):
        d["h0"].copy_(h0)
        y, hT = ck.selective_scan_fwd(**d, hT=d["h0"])
        torch.cuda.synchronize()
        assert hT is d["h0"] and torch.equal(y, want[0]) and torch.equal(hT, want[1])


def test_a_channel_with_nan_leaves_the_others():
    """A non-finite input of one channel: the others' outputs, and its own rows before, stay as they were."""
    a, _, _ = make(8, 1, 40, 36, 1, 16, BF)
    d = cuda(a)
    y, hT = ck.selective_scan_fwd(**d)
    d["x"][0, 20, 5] = float("nan")
    y2, h2 = ck.selective_scan_fwd(**d)
    torch.cuda.synchronize()
    others = [c for c in range(36) if c != 5]
    assert torch.equal(y[:, :, others], y2[:, :, others]) and torch.equal(hT[:, others], h2[:, others])
    assert torch.equal(y[:, :20, 5], y2[:, :20, 5]) and torch.isnan(y2[0, 20:, 5]).all()


@pytest.mark.parametrize("T", [2000, 20000])
def test_slow_decays_do_not_drift(T):
    """fp32, a constant step: the decay is 1 - 1e-5 at every row, and what it is
    off by adds up.  By its distance from 1 it is good to 2^-23 of the 1e-5, so a
    state's error is that of T rounded sums, which walk like sqrt T 2^-24 (four
    times that is allowed); a decay rounded to fp32 as such would be off by up to
    2^-25 at every row, T 2^-25 in all."""
    C, N = 32, 16
    step = 1e-5
    d = dict(x=torch.ones(1, T, C), dt=torch.full((1, T, C), step), A=-torch.ones(C, N), Bm=torch.ones(1, T, 1, N), Cm=torch.ones(1, T, 1, N))
    y, hT = ck.selective_scan_fwd(**{k: v.cuda() for k, v in d.items()}, softplus=False, h0=torch.ones(1, C, N).cuda())
    s, a = float(torch.tensor(step)), np.exp(-float(torch.tensor(step)))
    want = a ** T + s * (1 - a ** T) / (1 - a)
    torch.cuda.synchronize()
    assert abs(hT.double().cpu().numpy() / want - 1).max() <= 4 * T ** 0.5 * 2.0 ** -24


def test_same_call_twice_gives_the_same_bytes():
    a, dy, dhT = make(4, 2, 300, 100, 2, 16, BF)
    d = cuda(a)
    out = [ck.selective_scan_bwd(**d, dy=dy.cuda(), dhT=dhT.cuda()) for _ in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(*out))
