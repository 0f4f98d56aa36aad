"""The short causal convolution on the GPU against the fp64 formulas, elementwise.

Bounds.  fp32 arithmetic: a sum of K products and a bias is off by (K + 1) 2^-24
of the sum of absolute values su; SiLU and its slope have slopes of at most 1.1
and 0.5 and their own errors, where bf16 takes the hardware's exponential at an
argument rounded once: (8 + 2 |u|) 2^-23 relative.  Weight gradients sum R rows, R
2^-24 of the absolute terms.  An output's rounding adds half a step of its type."""
import numpy as np
import pytest
import torch

import gated_delta_rule_ckda_amd as ck
import layer_reference as ref
from linattn_cases import check
from parity import log

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def make(seed, B, T, C, K, dtype, state, lens, bias=True):
    r = np.random.default_rng(seed)
    t = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32))  # noqa: E731
    a = dict(x=t(B, T, C).to(dtype), w=0.6 * t(C, K), b=0.2 * t(C) if bias else None,
             s0=t(B, K - 1, C).to(dtype) if state else None, lens=None if lens is None else torch.tensor(lens, dtype=torch.int32))
    return a, t(B, 1, T, C).to(dtype), t(B, K - 1, C).to(dtype) if state else None


def dev(t):
    return None if t is None else t.cuda()


def run(seed, B, H, T, C, K, dtype, silu=True, state=True, lens=None, bias=True, view=None):
    log(f"short_conv B={B} H={H} T={T} C={C} K={K} {dtype} silu={silu} state={state} lens={lens} bias={bias}")
    a, dy, dsT = make(seed, B, T, C, K, dtype, state, lens, bias)
    dy = dy.reshape(B, T, H, C // H).transpose(1, 2).contiguous()
    want = ref.short_conv(**a, heads=H, silu=silu, dy=dy, dsT=dsT)
    d = {n: dev(t) for n, t in a.items()}
    if view is not None:   # a column slice of a wider tensor
        wide = torch.full((B, T, view + C + 3), float("nan"), dtype=dtype, device="cuda")
        wide[..., view:view + C] = d["x"]
        d["x"] = wide[..., view:view + C]
    act = "silu" if silu else None
    y, sT = ck.short_conv_fwd(d["x"], d["w"], d["b"], d["s0"], lens=d["lens"], heads=H, act=act)
    dx, dw, db, ds0 = ck.short_conv_bwd(d["x"], d["w"], dev(dy), d["b"], d["s0"], dev(dsT), lens=d["lens"], act=act)
    torch.cuda.synchronize()
    half, e = torch.finfo(dtype).eps / 2, 2.0 ** -24
    u, su, turn = want["u"], want["su"], want["turn"]
    eu, ea = (K + 1) * e * su, (8 + 2 * np.abs(u)) * 2 * e
    y_err = 1.1 * eu + ea * np.abs(u) if silu else eu
    check("y", y, want["y"], half * np.abs(want["y"]) + turn(y_err))
    assert torch.equal(sT.cpu().double(), torch.from_numpy(want["sT"]))
    eg = np.abs(want["d"]) * (0.5 * eu + ea * (1 + np.abs(u))) * want["live"] if silu else 0.0 * u
    wa, C_ = np.abs(a["w"].double().numpy()), C
    spread = np.zeros((B, T + K - 1, C_))
    for j in range(K):
        spread[:, j:j + T] += wa[:, j] * eg
    for name, got, at in (("dx", dx, slice(K - 1, None)), ("ds0", ds0, slice(None, K - 1))):
        size = want["s" + name]
        check(name, got, want[name], half * np.abs(want[name]) + spread[:, at] + (K + 2) * e * size)
    rows = B * T + 64
    x_all = np.concatenate([np.zeros((B, K - 1, C)) if a["s0"] is None else ref.f64(a["s0"]),
                            np.where(want["live"], ref.f64(a["x"]), 0.0)], 1)
    sw = np.stack([(eg * np.abs(x_all[:, j:j + T])).sum((0, 1)) for j in range(K)], -1)
    check("dw", dw, want["dw"], sw + rows * e * want["sdw"])
    check("db", db, want["db"], eg.sum((0, 1)) + rows * e * want["sdb"])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("silu", [True, False])
def test_taps(K, silu, dtype):
    run(K, 2, 2, 37, 64, K, dtype, silu)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,C", [(1, 1), (1, 2), (1, 7), (1, 31), (1, 513), (1, 1000), (4, 64), (16, 2048), (3, 12), (5, 15),
                                 (2, 20), (1, 1025)])
def test_widths(H, C, dtype):
    run(C, 2, H, 9, C, 4, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 15, 16, 17, 127, 128, 129, 700])
def test_lengths(T, dtype):
    run(T, 1, 2, T, 32, 4, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [[40, 0, 1], [2, 3, 40], [100, -5, 17], [0, 0, 0]])
@pytest.mark.parametrize("state", [True, False])
def test_padded(lens, state, dtype):
    run(3, 3, 2, 40, 48, 4, dtype, state=state, lens=lens)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("view", [0, 1, 5, 8])
def test_column_slice(view, dtype):
    run(view, 2, 2, 21, 64, 4, dtype, view=view)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_slabs(dtype):
    """More slabs than parts of the weights' gradients, and long slabs."""
    run(1, 1500, 1, 3, 8, 3, dtype, bias=False)
    run(2, 3, 1, 3000, 520, 4, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K", [2, 4])
def test_nothing_to_read(K, dtype):
    """No rows: the state goes through; no batch: weight gradients are zero."""
    a, _, dsT = make(1, 2, 0, 16, K, dtype, True, None)
    d = {n: dev(t) for n, t in a.items()}
    y, sT = ck.short_conv_fwd(d["x"], d["w"], d["b"], d["s0"], heads=2)
    dx, dw, db, ds0 = ck.short_conv_bwd(d["x"], d["w"], torch.empty(2, 2, 0, 8, dtype=dtype, device="cuda"), d["b"], d["s0"], dev(dsT))
    torch.cuda.synchronize()
    assert y.shape == (2, 2, 0, 8) and torch.equal(sT, d["s0"]) and torch.equal(ds0.cpu(), dsT)
    assert (dw == 0).all() and (db == 0).all()
    out = ck.short_conv_bwd(torch.empty(0, 5, 16, dtype=dtype, device="cuda"), d["w"],
                            torch.empty(0, 2, 5, 8, dtype=dtype, device="cuda"))
    torch.cuda.synchronize()
    assert (out[1] == 0).all() and (out[2] == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K,H,C", [(4, 2, 64), (3, 1, 37), (2, 1, 1), (4, 32, 4096)])
def test_decode_continues_the_forward(K, H, C, dtype):
    """Row by row, the same values and the same state as the forward over the rows, bit for bit."""
    a, _, _ = make(C, 3, 11, C, K, dtype, True, None)
    d = {n: dev(t) for n, t in a.items()}
    y, sT = ck.short_conv_fwd(d["x"], d["w"], d["b"], d["s0"], heads=H)
    state = d["s0"].clone()
    rows = [ck.short_conv_decode_step(d["x"][:, t], d["w"], state, d["b"], heads=H) for t in range(11)]   # slices of x
    torch.cuda.synchronize()
    assert torch.equal(torch.stack(rows, 2), y) and torch.equal(state, sT)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,C,K", [(601, 1024, 4), (1203, 1024, 3), (2407, 511, 2)])
def test_decode_of_many_sequences(N, C, K, dtype):
    """Several sequences a thread, the last thread with fewer: the same bytes as with the sequences in small calls."""
    a, _, _ = make(C, N, 1, C, K, dtype, True, None)
    x, w, b, state = dev(a["x"])[:, 0].contiguous(), dev(a["w"]), dev(a["b"]), dev(a["s0"])
    one = state.clone()
    want = torch.cat([ck.short_conv_decode_step(x[i:i + 64], w, one[i:i + 64], b) for i in range(0, N, 64)])   # (16-byte aligned pieces)
    y = ck.short_conv_decode_step(x, w, state, b)
    z = ref.short_conv(**a)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(state, one) and torch.equal(state[:, -1], x)
    e, u = 2.0 ** -24, z["u"]
    off = 1.1 * (K + 1) * e * z["su"] + (8 + 2 * np.abs(u)) * 2 * e * np.abs(u)
    check("y", y[:, 0], z["y"][:, 0, 0], torch.finfo(dtype).eps / 2 * np.abs(z["y"][:, 0, 0]) + off[:, 0])


def test_rows_behind_a_sequence_are_left():
    """Outputs passed in keep their rows at or past a length; NaN there is not read."""
    a, dy, _ = make(1, 2, 20, 24, 4, BF, False, [7, 0])
    d = {n: dev(t) for n, t in a.items()}
    d["x"][0, 7:] = float("nan")
    d["x"][1] = float("nan")
    y = torch.full((2, 3, 20, 8), 7.0, dtype=BF, device="cuda")
    ck.short_conv_fwd(d["x"], d["w"], d["b"], lens=d["lens"], heads=3, y=y)
    g = dy.reshape(2, 20, 3, 8).transpose(1, 2).contiguous().cuda()
    g[:, :, 7:] = float("nan")
    g[1] = float("nan")
    dx, dw, db, ds0 = ck.short_conv_bwd(d["x"], d["w"], g, d["b"], lens=d["lens"])
    torch.cuda.synchronize()
    assert (y[0, :, 7:] == 7).all() and (y[1] == 7).all() and torch.isfinite(y).all()
    assert (dx[0, 7:] == 0).all() and (dx[1] == 0).all()
    for t in (dx, dw, db, ds0):
        assert torch.isfinite(t).all()


def test_same_call_twice_gives_the_same_bytes():
    a, dy, _ = make(4, 3, 500, 256, 4, BF, False, None)
    d = {n: dev(t) for n, t in a.items()}
    out = [ck.short_conv_bwd(d["x"], d["w"], dy.cuda(), d["b"]) for _ in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(*out))
