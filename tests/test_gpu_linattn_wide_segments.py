"""Whole states of 128 columns per workgroup together with segments of the
sequence: what long sequences of some heads run.  Sequences of the whole length
and ones that end in an earlier segment."""
import pytest
import torch

import gated_delta_rule_ckda_amd as ck
from linattn_cases import bwd_bounds, check, cuda, fwd_bounds, inputs
from linattn_decay_cases import BF, accepts
from parity import log

pytestmark = pytest.mark.gpu


def test_forward():
    """16 heads of 128 x 128: 14 segments of 192 rows."""
    B, H, Hk, T, d = 2, 8, 2, 2500, 128
    assert ck.linattn_workspace_size(B, H, T, d, d, BF) > 13 * B * H * d * d * 4
    x = inputs(301, B, H, Hk, T, d, d, BF, lens=[2500, 900])
    log(f"linattn_fwd q {tuple(x['q'].shape)} v {tuple(x['v'].shape)}")
    o, hT, bo, bh = fwd_bounds(x)
    dev = cuda(x)
    args = (dev["q"], dev["k"], dev["v"], dev["g"], dev["h0"])
    got_o, got_h = ck.linattn_fwd(*args, lens=dev["lens"])
    only_o, _ = ck.linattn_fwd(*args, lens=dev["lens"], want_state=False)
    torch.cuda.synchronize()
    check("o", got_o, o, bo)
    check("hT", got_h, hT, bh)
    check("o without a state", only_o, o, bo)


@pytest.mark.parametrize("state", [True, False])
def test_backward(state):
    """4 heads of 128 x 128: 16 segments of 128 rows in both directions."""
    B, H, Hk, T, d = 2, 2, 1, 2048, 128
    assert ck.linattn_bwd_workspace_size(B, H, Hk, T, d, d, BF) > 2 * 15 * B * H * d * d * 4
    x = inputs(302, B, H, Hk, T, d, d, BF, state=state, lens=[2048, 700])
    log(f"linattn_bwd q {tuple(x['q'].shape)} v {tuple(x['v'].shape)}")
    want = bwd_bounds(x)
    dev = cuda(x)
    got = dict(zip(("dq", "dk", "dv", "dg", "dh0"),
                   ck.linattn_bwd(dev["q"], dev["k"], dev["v"], dev["g"], dev["do"], dev["h0"], dev["dhT"], lens=dev["lens"])))
    torch.cuda.synchronize()
    for n, (w, b) in want.items():
        check(n, got[n], w, b)
    wrong = accepts(x, want["dg"][0], got["dg"].double().cpu().numpy())
    assert wrong is None, wrong
