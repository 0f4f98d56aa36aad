"""The gradient of the log decays on the GPU, within bounds relative to itself
(linattn_decay_cases.py): ordinary, strong, mixed and reset decays."""
import pytest
import torch

import gated_delta_rule_ckda_amd as ck
from linattn_cases import cuda
from linattn_decay_cases import BF, F32, KINDS, SIZES, accepts, case, exact
from parity import log

pytestmark = pytest.mark.gpu


def gradient(x):
    log(f"linattn_bwd dg q {tuple(x['q'].shape)} v {tuple(x['v'].shape)} g {tuple(x['g'].shape)} {x['q'].dtype}")
    d = cuda(x)
    dg = ck.linattn_bwd(d["q"], d["k"], d["v"], d["g"], d["do"], d["h0"], d["dhT"], lens=d["lens"])[3]
    torch.cuda.synchronize()
    return dg.double().cpu().numpy()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", SIZES)
def test_decay_gradient(size, kind, dtype):
    for state in (False, True):
        x = case(21, *size, dtype, kind, state=state)
        wrong = accepts(x, exact(x), gradient(x))
        assert wrong is None, (state, wrong)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", [-0.003, -0.05, -0.3, -3.0, -10.0])
@pytest.mark.parametrize("size", [(1, 2, 1, 4500, 32, 32), (3, 2, 2, 1100, 16, 16)])
def test_gradient_of_a_constant_decay(size, kind, dtype):
    x = case(22, *size, dtype, kind, decay="head", state=size[0] > 1)
    wrong = accepts(x, exact(x), gradient(x))
    assert wrong is None, wrong


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["ordinary", "reset", -6.0])
def test_lengths(kind, dtype):
    """Sequences that end inside, at and behind chunk borders, and empty ones."""
    x = case(23, 8, 2, 1, 200, 32, 64, dtype, kind, state=True, lens=[200, 0, 1, 63, 64, 65, 128, 130])
    wrong = accepts(x, exact(x), gradient(x))
    assert wrong is None, wrong


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["ordinary", "mixed", -6.0])
def test_segments(kind, dtype):
    """One head whose sweeps run in segments, whole and ending in an earlier segment."""
    for lens in (None, [1205]):
        x = case(24, 1, 1, 1, 2500, 64, 64, dtype, kind, state=True, lens=lens)
        wrong = accepts(x, exact(x), gradient(x))
        assert wrong is None, (lens, wrong)


def test_large_states_behind_strong_decays():
    """States so large that their pair is all there is, through a product of decays of e^-30 a chunk."""
    x = case(25, 1, 1, 1, 192, 16, 16, F32, -0.4, state=True)
    x = {**x, "h0": 1e12 * x["h0"], "dhT": 1e12 * x["dhT"], **{n: 1e-12 * x[n] for n in ("q", "k", "v", "do")}}
    wrong = accepts(x, exact(x), gradient(x))
    assert wrong is None, wrong
