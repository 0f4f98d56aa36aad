"""Limits of the sizes and strides that the short convolution, the selective scan
and the residual norm take (CPU).  Calls on fake addresses that are let through a
check here end at a later one, so that nothing reaches the device."""
import pytest

import gated_delta_rule_ckda_amd as ck
from test_layer_abi import at, scan, scan_bwd, scan_dec


@pytest.mark.parametrize("kw", [dict(ldbc=1 << 24), dict(ldz=1 << 24), dict(ldbc=2 ** 31 - 1, ldz=2 ** 31 - 1)])
def test_a_scan_step_takes_any_row_stride(kw):
    """One token's rows of a [S, T, W] tensor are T W apart; the forward's and the backward's tiles have an offset limit."""
    assert scan(**kw) == ck.ERR_DIM and b"row strides" in ck.lib().ckda_last_error()
    assert scan_bwd(**kw) == ck.ERR_DIM and b"row strides" in ck.lib().ckda_last_error()
    assert scan_dec(**kw, y=at(8)) == ck.ERR_ALIAS   # the check behind the sizes'
    assert scan_dec(**{**kw, "ldbc": 31}) == ck.ERR_DIM and b"ldbc" in ck.lib().ckda_last_error()
    assert scan_dec(**{**kw, "ldz": 63}) == ck.ERR_DIM and b"ldz" in ck.lib().ckda_last_error()
