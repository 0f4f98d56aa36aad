"""States under slow constant decays over many chunks: their decay must not
drift, as it does when a factor near 1 is rounded and applied again and again.

With nothing written (v = 0) the state after T rows is exp(T g) h0.  Each
element takes one rounding for each chunk (and segment), 2^-24 of it at most and
to either side, so that the mean error over the elements is that of the decay
itself: the log decays' roundings, (1 + |T g| / ln 2) 2^-23 at most, and those of
a segment's product.  Twice that is allowed.  (A decay of a chunk rounded to
fp32 drifts by up to 2^-24 a chunk, 128 chunks 2^-17.)"""
import math

import numpy as np
import pytest
import torch

import gated_delta_rule_ckda_amd as ck
from parity import log

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
RATES = [-2.0 ** -7, -1.1 * 2.0 ** -9, -2.0 ** -11, -1.7 * 2.0 ** -13, -2.0 ** -14, -1.3 * 2.0 ** -16, 0.0, -2.0 ** -6]


def case(heads, T, d, dtype):
    """Heads of the rates in turn, their log decays as stored, and h0."""
    g = torch.tensor([RATES[i % len(RATES)] for i in range(heads)]).to(dtype)
    r = np.random.default_rng(7)
    h0 = torch.from_numpy((1.0 + r.random((1, heads, d, d))).astype(np.float32))
    return g, h0


def mean_error(S, g, T, h0):
    """Per head: mean relative error of the states against exp(T g) h0 (0 of
    states that have left fp32's range as they must: exp(-128) h0 < 2^-183)."""
    want = torch.exp(T * g.double()).view(1, -1, 1, 1) * h0.double()
    S = S.double().cpu()
    err = ((S - want) / want).mean((0, 2, 3)).numpy()
    gone = want.amax((0, 2, 3)) < 2.0 ** -150
    assert (S[:, gone].abs() <= 2.0 ** -126).all()
    return np.where(gone.numpy(), 0.0, err)


def bound(g, T):
    return 2 * (1 + T * np.abs(g.double().numpy()) / math.log(2)) * 2.0 ** -23


# whole sequences, and segments joined
SIZES = [(64, 4096, 64), (512, 1024, 32), (8, 8192, 64), (2, 8192, 32)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("heads,T,d", SIZES)
def test_forward(heads, T, d, dtype):
    g, h0 = case(heads, T, d, dtype)
    log(f"linattn_fwd slow decays heads {heads} T {T} d {d} {dtype}")
    z = torch.zeros(1, heads, T, d, dtype=dtype, device="cuda")
    _, hT = ck.linattn_fwd(z, z, z, g.cuda(), h0.cuda())
    torch.cuda.synchronize()
    err = np.abs(mean_error(hT, g, T, h0))
    assert (err <= bound(g, T)).all(), (err, bound(g, T))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("heads,T,d", SIZES)
def test_backward(heads, T, d, dtype):
    """dh0 = exp(T g) dhT where nothing is asked (q = do = 0)."""
    g, h0 = case(heads, T, d, dtype)
    log(f"linattn_bwd slow decays heads {heads} T {T} d {d} {dtype}")
    z = torch.zeros(1, heads, T, d, dtype=dtype, device="cuda")
    dh0 = ck.linattn_bwd(z, z, z, g.cuda(), z, None, h0.cuda())[4]
    torch.cuda.synchronize()
    err = np.abs(mean_error(dh0, g, T, h0))
    assert (err <= bound(g, T)).all(), (err, bound(g, T))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode(dtype):
    """4096 single tokens: one rounding each, to either side."""
    steps, d = 4096, 64
    g, h0 = case(len(RATES), steps, d, dtype)
    log(f"linattn_decode_step slow decays steps {steps} d {d} {dtype}")
    z = torch.zeros(1, len(RATES), d, dtype=dtype, device="cuda")
    S, gd, o = h0.cuda(), g.cuda(), torch.empty_like(z)
    for _ in range(steps):
        ck.linattn_decode_step(z, z, z, gd, S, o=o)
    torch.cuda.synchronize()
    err = np.abs(mean_error(S, g, steps, h0))
    assert (err <= bound(g, steps)).all(), (err, bound(g, steps))


@pytest.mark.parametrize("heads,T,d", [(64, 2048, 64), (256, 1024, 128), (8, 4096, 64)])
def test_fp32_state_is_rounded_once_a_chunk(heads, T, d):
    """Without a decay, small writes to large states: an addition a chunk (and
    segment), each off by 2^-24 / sqrt(3) of the state in the rms at most; a
    fifth more is allowed for what is added.  (One for each matrix
    instruction, 16 a chunk, would be four times that.)"""
    r = np.random.default_rng(8)
    t = lambda *s, f=1.0: torch.from_numpy((f * r.standard_normal(s)).astype(np.float32))  # noqa: E731
    k, v, h0 = t(1, heads, T, d, f=d ** -0.5), t(1, heads, T, d), t(1, heads, d, d, f=8.0) + 64.0
    g = torch.zeros(heads)
    log(f"linattn_fwd fp32 states heads {heads} T {T} d {d}")
    _, hT = ck.linattn_fwd(k.cuda(), k.cuda(), v.cuda(), g.cuda(), h0.cuda())
    torch.cuda.synchronize()
    few = [0, 1, heads - 1]
    want = h0[:, few].double() + k[:, few].double().transpose(2, 3) @ v[:, few].double()
    err = (hT.cpu()[:, few].double() - want) / want
    rms = float((err ** 2).mean().sqrt())
    assert rms <= 1.2 * 2.0 ** -24 / math.sqrt(3) * math.sqrt(T / 64), rms
