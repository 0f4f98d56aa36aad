"""Limits of the sizes and strides that the short convolution, the selective scan
and the residual norm take (CPU).  Calls on fake addresses that are let through a
check here end at a later one, so that nothing reaches the device."""
import pytest
import torch

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


F32, BF = torch.float32, torch.bfloat16


def wide(*shape, dtype=BF):
    """A tensor of any shape in one element's memory."""
    return torch.zeros(1, dtype=dtype).expand(shape)


N33 = 2 ** 32 + 5   # as a 32-bit size: 5


@pytest.mark.parametrize("shape", [(N33, 1), (N33, 16), (2 ** 31, 1), (2 ** 17, 2 ** 15, 8)])
def test_more_rows_than_the_abi_counts_are_refused(shape):
    """The norm takes every leading dimension as rows: their product is a 32-bit size too, and 2^32 + 5 rows were 5."""
    x, w = wide(*shape), torch.zeros(shape[-1])
    for call in (lambda: ck.add_norm_fwd(x, x, w), lambda: ck.add_norm_fwd(x), lambda: ck.add_norm_quant_fwd(x, x, w),
                 lambda: ck.add_norm_bwd(x, x, w)):
        with pytest.raises(ValueError, match="rows .*more than 2"):
            call()
    assert shape != (2 ** 31, 1) or pytest.raises(ValueError, ck.add_norm_fwd, x[:-1]).match("GPU tensor")


def test_sizes_that_the_abi_cannot_hold_are_refused():
    w, A = torch.zeros(1, 4), torch.zeros(1, 16)
    big, one = wide(1, N33, 1), wide(N33, 1)
    bc, bc1 = wide(1, N33, 1, 16), wide(N33, 1, 16)
    for call in (lambda: ck.short_conv_fwd(big, w), lambda: ck.short_conv_bwd(big, w, wide(1, 1, N33, 1)),
                 lambda: ck.short_conv_decode_step(one, w, wide(N33, 3, 1)), lambda: ck.selective_scan_fwd(big, big, A, bc, bc),
                 lambda: ck.selective_scan_bwd(big, big, A, bc, bc, big),
                 lambda: ck.selective_scan_decode_step(one, one, A, bc1, bc1, wide(N33, 1, 16, dtype=F32)),
                 lambda: ck.head_norm_fwd(wide(1, 1, N33, 16)), lambda: ck.decode_step(*[wide(N33, 1, 16)] * 4, wide(N33, 1), wide(N33, 1, 16, 16))):
        with pytest.raises(ValueError, match="more than 2\\^31 - 1 of a dimension"):
            call()
