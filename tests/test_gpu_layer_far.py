"""Tensors of more than 2^31 and 2^32 elements on the GPU: the last rows and sequences, whose
offsets pass 32 bits, against small calls (the same bytes, where a row's arithmetic
does not depend on the others) or the fp64 formulas.  Up to 50 GB of device memory."""
import numpy as np
import pytest
import torch

import gated_delta_rule_ckda_amd as ck
import layer_reference as ref
from linattn_cases import check
from parity import log

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def memory():
    """Each test's memory goes back to the device."""
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.fixture
def new():
    gen = torch.Generator(device="cuda").manual_seed(5)
    return lambda *s, dtype=BF: torch.randn(s, generator=gen, device="cuda", dtype=dtype)


def same(got, want):
    torch.cuda.synchronize()
    assert got.shape == want.shape and torch.equal(got, want)


def test_norm_rows(new):
    R, D, n = (1 << 19) + 3, 8192, 300
    log("add_norm: rows far")
    x, res, w = new(R, D), new(R, D, dtype=F32), 1 + 0.2 * new(D, dtype=F32)
    last = x[-n:].contiguous(), res[-n:].clone(), w
    yn, tn = ck.add_norm_fwd(*last)
    for group in (0, 128):
        q, scales, total = ck.add_norm_quant_fwd(x, res, w, group=group)
        qn, sn, _ = ck.add_norm_quant_fwd(*last, group=group)
        same(q[-n:].view(torch.uint8), qn.view(torch.uint8))
        same(scales[-n:], sn)
        same(total[-n:], tn)
        del q, scales, total
    y, _ = ck.add_norm_fwd(x, res, w, total=res)
    same(y[-n:], yn)
    same(res[-n:], tn)
    del y
    dx, dres, _ = ck.add_norm_bwd(res, x, w, dsum=res)
    dxn, drn, _ = ck.add_norm_bwd(tn, last[0], w, dsum=tn)
    same(dx[-n:], dxn)
    same(dres[-n:], drn)


@pytest.mark.parametrize("heads", [1, 32])
def test_conv_rows(heads, new):
    B, T, C, K, n = 1, (1 << 20) + 37, 4096, 4, 200
    log(f"short_conv: rows far, {heads} heads")
    x, w, b = new(B, T, C), new(C, K, dtype=F32), new(C, dtype=F32)
    last, s0 = x[:, -n:].contiguous(), x[:, T - n - K + 1:T - n].contiguous()
    y, sT = ck.short_conv_fwd(x, w, b, heads=heads)
    yn, sn = ck.short_conv_fwd(last, w, b, s0, heads=heads)
    same(y[:, :, -n:], yn)
    same(sT, sn)
    dx = ck.short_conv_bwd(x, w, y, b)[0]
    same(dx[:, -n:], ck.short_conv_bwd(last, w, yn, b, s0)[0])


def test_conv_step_states(new):
    N, C, K, n = (1 << 18) + 5, 6000, 4, 70
    log("short_conv: states far")
    x, w, b, state = new(N, C), new(C, K, dtype=F32), new(C, dtype=F32), new(N, K - 1, C)
    part = state[-n:].clone()
    y = ck.short_conv_decode_step(x, w, state, b)
    same(y[-n:], ck.short_conv_decode_step(x[-n:].contiguous(), w, part, b))
    same(state[-n:], part)


def test_scan_step_states(new):
    S, C, N, n = (1 << 14) + 1, 4100, 64, 65
    log("selective_scan: states far")
    x, dt, H = new(S, C), new(S, C), new(S, C, N, dtype=F32)
    A, Bm, Cm = -torch.rand(C, N, device="cuda"), new(S, 1, N), new(S, 1, N)
    part = H[-n:].clone()
    y = ck.selective_scan_decode_step(x, dt, A, Bm, Cm, H)
    tail = lambda t: t[-n:].contiguous()  # noqa: E731
    same(y[-n:], ck.selective_scan_decode_step(tail(x), tail(dt), A, tail(Bm), tail(Cm), part))
    same(H[-n:], part)


@pytest.mark.parametrize("T,C,G,N", [((1 << 18) + 5, 8256, 129, 16), ((1 << 19) + 5, 4128, 3, 17)])
def test_scan_rows(T, C, G, N, new):
    """Steps of 0.3 or more and rates of 1 or more: 300 rows leave exp(-90) of a state, so the last 100 rows are those
    of the last 400 alone."""
    tail, keep = 400, 100
    log(f"selective_scan: rows far, T={T} C={C} G={G} N={N}")
    x, dy, Bm, Cm = new(1, T, C), new(1, T, C), new(1, T, G, N), new(1, T, G, N)
    dt = torch.rand((1, T, C), device="cuda", dtype=BF).mul_(0.5).add_(0.3)
    A = -(1 + torch.arange(N, device="cuda")).float() * torch.ones(C, 1, device="cuda")
    each = C // G
    last = slice(T - tail, T)
    half, k = torch.finfo(BF).eps / 2, (tail + 64) * 2.0 ** -21

    def ends(name, got, count, grouped=False):
        for which, c, g in (("first", slice(0, each), slice(0, 1)), ("last", slice(C - each, C), slice(G - 1, G))):
            a = dict(x=x[:, last, c], dt=dt[:, last, c], A=A[c], Bm=Bm[:, last, g], Cm=Cm[:, last, g])
            want = ref.selective_scan(**a, softplus=False, dy=dy[:, last, c] if name != "y" else None)
            v, size = want[name][:, -keep:], want["s" + name][:, -keep:]
            bound = half * np.abs(v) + ((1 if name == "y" else 2) * k + count * 2.0 ** -24) * size
            check(f"{name} {which}", got[:, last, g if grouped else c][:, -keep:].contiguous(), v, bound)

    y, _ = ck.selective_scan_fwd(x, dt, A, Bm, Cm, softplus=False)
    torch.cuda.synchronize()
    ends("y", y, N)
    del y
    dx, ddt, _, dBm, dCm, *_ = ck.selective_scan_bwd(x, dt, A, Bm, Cm, dy, softplus=False)
    torch.cuda.synchronize()
    ends("dx", dx, N)
    ends("ddt", ddt, N)
    ends("dBm", dBm, each, True)
    ends("dCm", dCm, each, True)
