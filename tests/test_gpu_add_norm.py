"""The norm with the residual's addition on the GPU against the fp64 formulas,
elementwise.

Bounds.  fp32 arithmetic: x + res is rounded once (2^-24 |r|), the mean of D
squares by at most D 2^-24 of itself (they have one sign), its root by half that,
so n and y by (D / 2 + 8) 2^-24 of themselves and one rounding of r; the backward's
mean of products by D 2^-24 of its terms.  Outputs add half a step of their type:
of e4m3, half its spacing at the value (2^-3 of the power of two below it, 2^-9
below 2^-6), after y and the scale are off by the above."""
import numpy as np
import pytest
import torch

import gated_delta_rule_ckda_amd as ck
import layer_reference as ref
from linattn_cases import check
from parity import log

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
PAIRS = [(BF, BF), (BF, F32), (F32, F32)]
E = 2.0 ** -24


def tensors(seed, R, D, dtype, rt, weight=True):
    r = np.random.default_rng(seed)
    t = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32))  # noqa: E731
    return t(R, D).to(dtype), None if rt is None else (2 * t(R, D)).to(rt), 1 + 0.2 * t(D) if weight else None, t


def dev(t):
    return None if t is None else t.cuda()


def check_codes(q, scales, y, group, err):
    """Codes and scales of y in 64 bits, whose values the kernel has to a relative error err."""
    R, D = y.shape
    n = group or D
    assert scales.shape == (R, -(-D // n)) and q.dtype == torch.float8_e4m3fn
    top = np.stack([np.abs(y[:, i:i + n]).max(1) for i in range(0, D, n)], 1)
    want = np.where(top == 0, 1.0, top / 448)
    got = scales.double().cpu().numpy()
    assert (np.abs(got - want) <= (err + 2 * E) * want + 2.0 ** -149).all()
    each = np.repeat(want, n, axis=1)[:, :D]
    v = np.abs(y) / each
    spacing = 2.0 ** (np.clip(np.floor(np.log2(np.maximum(v, 2.0 ** -20))), -6, 8) - 3)
    codes = q.double().cpu().numpy()
    bad = ~(np.abs(codes - y / each) <= spacing / 2 + 2 * (err + 4 * E) * v)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], codes[bad][:4], (y / each)[bad][:4])


def run(seed, R, D, dtype, rt, weight=True, eps=1e-6):
    log(f"add_norm R={R} D={D} {dtype} residual={rt} weight={weight}")
    x, res, w, t = tensors(seed, R, D, dtype, rt, weight)
    want = ref.add_norm(x, res, w, eps)
    y, total = ck.add_norm_fwd(dev(x), dev(res), dev(w), eps=eps)
    half, err = torch.finfo(dtype).eps / 2, (D / 2 + 10) * E
    check("y", y, want["y"], (half + err) * np.abs(want["y"]) + E * np.abs(want["rstd"]) * np.abs(want["r"]))
    if rt is None:
        assert total is None
    else:
        check("sum", total, want["r"], torch.finfo(rt).eps / 2 * np.abs(want["r"]))
    for group in (0, 128):
        q, scales, total2 = ck.add_norm_quant_fwd(dev(x), dev(res), dev(w), eps=eps, group=group)
        check_codes(q, scales, want["y"], group, err + 2 * E)
        assert rt is None or torch.equal(total, total2)
    rt = rt or dtype
    s, dy, dsum = (2 * t(R, D)).to(rt), t(R, D).to(dtype), t(R, D).to(rt)
    for more in (dsum, None):
        g = ref.add_norm_bwd(s, dy, w, more, eps)
        dx, dres, dw = ck.add_norm_bwd(dev(s), dev(dy), dev(w), dsum=dev(more), eps=eps)
        torch.cuda.synchronize()
        bound = 3 * (D + 16) * E * g["sdr"]
        check("dx", dx, g["dr"], torch.finfo(dtype).eps / 2 * np.abs(g["dr"]) + bound)
        check("dres", dres, g["dr"], torch.finfo(rt).eps / 2 * np.abs(g["dr"]) + bound)
        check("dw", dw, g["dw"], (D / 2 + R + 80) * E * g["sdw"])


@pytest.mark.parametrize("dtype,rt", PAIRS)
@pytest.mark.parametrize("D", [1, 2, 7, 8, 9, 31, 64, 65, 127, 128, 129, 200, 256, 257, 511, 512, 513, 1000, 1024, 1025, 2047, 2048,
                               2049, 4096, 4100, 8191, 8192])
def test_widths(D, dtype, rt):
    run(D, 5, D, dtype, rt)


@pytest.mark.parametrize("dtype,rt", PAIRS + [(BF, None), (F32, None)])
@pytest.mark.parametrize("R", [1, 2, 3, 33, 300])
def test_rows(R, dtype, rt):
    run(R, R, 96, dtype, rt, weight=R != 3)


@pytest.mark.parametrize("dtype,rt", PAIRS)
def test_many_rows(dtype, rt):
    """Every thread group walks over several rows."""
    run(1, 9001, 40, dtype, rt)
    run(2, 4100, 520, dtype, rt)


def test_both_outputs_and_a_sum_without_residual():
    x, _, w, _ = tensors(1, 6, 200, BF, None)
    y, total = ck.add_norm_fwd(dev(x), None, dev(w), total=torch.empty(6, 200, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(total.cpu(), x.float())
    assert torch.equal(y, ck.add_norm_fwd(dev(x), None, dev(w))[0])


@pytest.mark.parametrize("dtype,rt", PAIRS)
def test_in_place(dtype, rt):
    """The sum in the place of the residual, the gradient in the place of the stream's."""
    x, res, w, _ = tensors(2, 40, 300, dtype, rt)
    y, total = ck.add_norm_fwd(dev(x), dev(res), dev(w))
    stream = dev(res)
    y2, same = ck.add_norm_fwd(dev(x), stream, dev(w), total=stream)
    torch.cuda.synchronize()
    assert same is stream and torch.equal(y, y2) and torch.equal(stream, total)


def test_zero_rows_and_tiny_values():
    """A row of zeros has scale 1 and codes 0; the scale of tiny values may be a subnormal number."""
    x = torch.zeros(4, 256)
    x[1] = 1e-40
    x[2, 128:] = 3.0
    x[3] = torch.linspace(-1, 1, 256) * 1e-38
    q, scales, _ = ck.add_norm_quant_fwd(x.cuda(), eps=1.0)
    torch.cuda.synchronize()
    assert (scales[0] == 1).all() and (q[0].float() == 0).all() and scales[2, 0] == 1 and (q[2, :128].float() == 0).all()
    y = ref.add_norm(x, eps=1.0)["y"]
    codes, s = q.double().cpu().numpy(), scales.double().cpu().numpy()
    assert np.isfinite(codes).all()
    back = codes * np.repeat(s, 128, axis=1)
    # half a step of the codes, and of a subnormal scale half its own step for each unit of a code
    assert (np.abs(back - y) <= np.abs(y) / 16 + 2.0 ** -10 * np.repeat(s, 128, axis=1) + 449 * 2.0 ** -150 + 2.0 ** -149).all()


def test_nan_and_infinity_stay_in_their_rows():
    x = torch.randn(6, 512, generator=torch.Generator().manual_seed(1))
    clean = ck.add_norm_quant_fwd(x.cuda())
    x[2, 7] = float("nan")
    x[4, 300] = float("inf")
    y, _ = ck.add_norm_fwd(x.cuda())
    q, scales, _ = ck.add_norm_quant_fwd(x.cuda())
    torch.cuda.synchronize()
    assert torch.isnan(y[2]).all() and torch.isnan(y[4, 300]) and (y[4, :300] == 0).all()
    assert torch.isnan(q[2].float()).all() and torch.isnan(scales[2]).all()
    rest = [0, 1, 3, 5]
    assert torch.equal(q[rest].view(torch.uint8), clean[0][rest].view(torch.uint8)) and torch.equal(scales[rest], clean[1][rest])


def test_no_rows():
    y, total = ck.add_norm_fwd(torch.empty(0, 64, device="cuda"), torch.empty(0, 64, device="cuda"))
    dx, dres, dw = ck.add_norm_bwd(torch.empty(0, 64, device="cuda"), torch.empty(0, 64, device="cuda"))
    torch.cuda.synchronize()
    assert y.shape == total.shape == dx.shape == (0, 64) and dres is dx and (dw == 0).all()


def test_same_call_twice_gives_the_same_bytes():
    x, res, w, t = tensors(3, 700, 1000, BF, F32)
    dy, dsum = t(700, 1000).to(BF).cuda(), t(700, 1000).cuda()
    out = [ck.add_norm_bwd(dev(res), dy, dev(w), dsum=dsum) for _ in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(*out))
