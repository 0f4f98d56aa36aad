"""A workspace that overlaps an input is refused, as one that overlaps an output
is: the kernels write it before they have read the inputs.  Fake addresses."""
import pytest

import gated_delta_rule_ckda_amd as ck
from test_linattn_abi import at, bwd, fwd, norm_bwd


@pytest.mark.parametrize("off", [0, 256])
@pytest.mark.parametrize("i,name", enumerate(("q", "k", "v", "g", "h0", "lens")))
def test_forward(i, name, off):
    assert fwd(ws=at(i, -off), B=1, H=2, Hk=1, T=4096) == ck.ERR_ALIAS   # runs in segments
    assert f"workspace overlaps {name}".encode() in ck.lib().ckda_last_error()


@pytest.mark.parametrize("off", [0, 256])
@pytest.mark.parametrize("i,name", enumerate(("q", "k", "v", "g", "h0", "lens", "do", "dhT")))
def test_backward(i, name, off):
    assert bwd(ws=at(i, -off)) == ck.ERR_ALIAS
    assert f"workspace overlaps {name}".encode() in ck.lib().ckda_last_error()


@pytest.mark.parametrize("off", [0, 256])
@pytest.mark.parametrize("i,name", enumerate(("x", "z", "w", "b", "dy")))
def test_head_norm_backward(i, name, off):
    assert norm_bwd(ws=at(i, -off)) == ck.ERR_ALIAS
    assert f"workspace overlaps {name}".encode() in ck.lib().ckda_last_error()
