"""The head norm with its output gate on the GPU, forward and backward, against
the fp64 formulas, elementwise.

Bounds.  fp32 arithmetic throughout: a row's mean and centred square sum over D
elements are off by at most D 2^-24 of the sums of absolute values, x - m by
that and a rounding, so n by some (2 D + 8) 2^-24 of (|x| + |m|) s (with
pairwise lane sums far less); the gate's functions by 8 2^-24; the outputs'
rounding adds eps / 2.  dx adds the errors of two means of D products; dw and db
sum R rows, R 2^-24 of the sum of absolute terms."""
import numpy as np
import pytest
import torch

import gated_delta_rule_ckda_amd as ck
import linattn_reference as ref
from linattn_cases import check
from parity import log

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def make(seed, B, H, T, D, dtype, act, shared, offset=0.3):
    r = np.random.default_rng(seed)
    t = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32))  # noqa: E731
    hw = 1 if shared else H
    x = (0.7 * t(B, H, T, D) + offset * t(B, H, T, 1)).to(dtype)
    return dict(x=x, w=1 + 0.2 * t(hw, D), b=0.2 * t(hw, D), gate=None if act is None else t(B, T, H, D).to(dtype)), \
        t(B, T, H, D).to(dtype)


def run(seed, B, H, T, D, dtype, act, rms, shared, eps=1e-5, offset=0.3):
    log(f"head_norm B={B} H={H} T={T} D={D} {dtype} act={act} rms={rms} shared={shared}")
    a, dy = make(seed, B, H, T, D, dtype, act, shared, offset)
    kw = dict(act=act or "silu", rms=rms, eps=eps)
    want = ref.head_norm(**a, dy=dy, **kw)
    d = {n: None if t is None else t.cuda() for n, t in a.items()}
    y = ck.head_norm_fwd(d["x"], d["w"], d["b"], gate=d["gate"], **kw)
    dx, dz, dw, db = ck.head_norm_bwd(d["x"], dy.cuda(), d["w"], d["b"], gate=d["gate"], **kw)
    torch.cuda.synchronize()
    half = torch.finfo(dtype).eps / 2
    w, b = a["w"].double().numpy(), a["b"].double().numpy()
    x = a["x"].double().numpy().transpose(0, 2, 1, 3)
    g = dy.double().numpy()
    # relative errors: of n against size, of the gate
    en = (2 * D + 8) * 2.0 ** -24
    size = (np.abs(x) + np.abs(x).mean(-1, keepdims=True)) * want["rstd"]
    ea = 8 * 2.0 ** -24
    if act is None:
        s, slope = np.ones_like(g), np.zeros_like(g)
    else:
        z = a["gate"].double().numpy()
        sg = 1 / (1 + np.exp(-z))
        s = np.abs(z) * sg + sg if act == "silu" else sg
        slope = sg * (1 + np.abs(z)) + sg
    n_err = en * size
    y_err = (n_err * np.abs(w) + ea * (np.abs(want["n"] * w) + np.abs(b))) * s
    check("y", y, want["y"], half * np.abs(want["y"]) + y_err)
    dn = np.abs(g) * s * np.abs(w)
    mean = lambda t: t.mean(-1, keepdims=True)  # noqa: E731
    dx_abs = dn + mean(dn) + size * mean(dn * size)
    bound = 8 * en * dx_abs * want["rstd"]
    bound = bound.transpose(0, 2, 1, 3)
    check("dx", dx, want["dx"], half * np.abs(want["dx"]) + bound)
    if act is not None:
        err = np.abs(g) * slope * (n_err * np.abs(w) + ea * (np.abs(want["n"] * w) + np.abs(b)))
        check("dz", dz, want["dz"], half * np.abs(want["dz"]) + 2 * err)
    over = (0, 1, 2) if shared else (0, 1)
    rows = B * T * (H if shared else 1)
    fold = (lambda t: t.sum(0, keepdims=True)) if shared else (lambda t: t)
    u = np.abs(g) * s
    add = lambda t: t.sum(over).reshape(w.shape)  # noqa: E731
    check("dw", dw, fold(want["dw"]), add(u * (n_err + (rows + 16) * 2.0 ** -24 * size)))
    check("db", db, fold(want["db"]), add(u * (rows + 16) * 2.0 ** -24))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [1, 2, 7, 8, 15, 16, 17, 24, 32, 64, 100, 127, 128, 130, 200, 255, 256, 264, 511, 520, 1000,
                               1024, 1025, 2047, 2048, 4100, 8184, 8191, 8192])
def test_widths(D, dtype):
    run(D, 2, 1 if D > 256 else 3, 5, D, dtype, "silu", False, False)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", [None, "silu", "sigmoid"])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("shared", [False, True])
def test_variants(act, rms, shared, dtype):
    run(5, 2, 4, 33, 128, dtype, act, rms, shared)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,H,T,D", [(1, 1, 1, 128), (1, 16, 1, 128), (3, 2, 700, 64), (1, 32, 257, 16), (2, 1, 1500, 300),
                                     (1, 70, 3, 32)])
def test_sizes(B, H, T, D, dtype):
    run(B * 1000 + T, B, H, T, D, dtype, "sigmoid", False, H % 2 == 0)


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("B,H,T,D,dtype", [(2, 16, 90, 128, F32), (1, 8, 70, 512, BF), (1, 8, 70, 256, BF), (2, 3, 40, 1025, BF)])
def test_several_slabs_of_several_heads(B, H, T, D, dtype, shared):
    """Both orders of the workgroups (heads or slabs first)."""
    run(D + T, B, H, T, D, dtype, "silu", False, shared)


def test_large_mean_keeps_the_variance():
    """The variance is of centred values: rows far from zero lose nothing but the input's own rounding."""
    run(9, 1, 2, 16, 128, F32, None, False, False, offset=100.0)


def test_constant_rows():
    """Variance zero: n = 0, y = b, dx finite."""
    x = torch.full((1, 2, 3, 64), 5.0, device="cuda")
    b = torch.rand(2, 64, device="cuda")
    y = ck.head_norm_fwd(x, b=b)
    dx, dz, dw, db = ck.head_norm_bwd(x, torch.ones(1, 3, 2, 64, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(y, b.view(1, 1, 2, 64).expand(1, 3, 2, 64)) and dz is None
    assert torch.isfinite(dx).all() and (dw == 0).all()
    assert (db == 6).all()   # without w and b: [1, D], the three rows of both heads


def test_no_rows():
    x = torch.empty(2, 3, 0, 32, device="cuda")
    assert ck.head_norm_fwd(x).shape == (2, 0, 3, 32)
    dx, _, dw, db = ck.head_norm_bwd(x, torch.empty(2, 0, 3, 32, device="cuda"), torch.ones(3, 32, device="cuda"))
    torch.cuda.synchronize()
    assert dx.shape == x.shape and (dw == 0).all() and (db == 0).all()


def test_same_call_twice_gives_the_same_bytes():
    a, dy = make(3, 4, 8, 300, 128, BF, "silu", True)
    d = {n: t.cuda() for n, t in a.items()}
    r = [ck.head_norm_bwd(d["x"], dy.cuda(), d["w"], d["b"], gate=d["gate"]) for _ in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(*r))
