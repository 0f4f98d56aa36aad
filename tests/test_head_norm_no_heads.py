"""A head norm without heads (or rows): empty outputs, and gradients of shared
weights that are zero."""
import pytest
import torch

import gated_delta_rule_ckda_amd as ck
from test_linattn_abi import at, norm_bwd


def test_gradients_of_shared_weights_are_launched():
    """Without heads but with [1, D] gradients to write a call is no empty one: its arguments are checked."""
    assert norm_bwd(H=0, wheads=1, flags=0, z=None, ws=None) == ck.ERR_WORKSPACE
    assert norm_bwd(H=0, wheads=0, flags=0, z=None, ws=None) == 0          # weights of no heads: nothing to write
    assert norm_bwd(H=0, wheads=1, flags=0, z=None, dw=None, db=None, ws=None) == 0
    assert norm_bwd(H=0, wheads=1, flags=0, z=None, dw=at(9, 64)) == ck.ERR_ALIAS


@pytest.mark.parametrize("shape", [(2, 0, 5, 64), (0, 4, 5, 64), (2, 4, 0, 64)])
def test_weights_of_each_head_or_shared_are_taken(shape):
    """Shapes pass the binding's checks up to the device, also [0, D] weights of no heads."""
    B, H, T, D = shape
    x = torch.empty(shape)
    for heads in (H, 1):
        w = torch.empty(heads, D)
        with pytest.raises(ValueError, match="x must be a GPU tensor"):
            ck.head_norm_fwd(x, w, w)


@pytest.mark.gpu
@pytest.mark.parametrize("shared", [True, False])
@pytest.mark.parametrize("shape", [(2, 0, 5, 64), (0, 4, 5, 64), (2, 4, 0, 64)])
def test_no_rows(shape, shared):
    B, H, T, D = shape
    x, dy = torch.empty(shape, device="cuda"), torch.empty(B, T, H, D, device="cuda")
    w = torch.ones(1 if shared else H, D, device="cuda")
    junk = [torch.full((1, D), 7.0, device="cuda") for _ in range(8)]   # what fresh gradients may find in memory
    del junk
    assert ck.head_norm_fwd(x, w, w).shape == (B, T, H, D)
    dx, dz, dw, db = ck.head_norm_bwd(x, dy, w, w)
    torch.cuda.synchronize()
    assert dx.shape == shape and dz is None and dw.shape == db.shape == w.shape
    assert (dw == 0).all() and (db == 0).all()
