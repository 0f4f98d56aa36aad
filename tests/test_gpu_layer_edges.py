"""Documented calls of the short convolution, the selective scan and the residual
norm on the GPU that the operators' own tests do not make."""
import pytest
import torch

import gated_delta_rule_ckda_amd as ck
from test_gpu_selective_scan import cuda, make

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
def test_scan_step_on_tokens_far_apart(dtype):
    """Bm, Cm and z of the last token of a long projection: rows 2^24 elements and more apart."""
    S, T, C, G, N = 3, 16384, 40, 2, 16
    a, _, _ = make(1, S, 1, C, G, N, dtype)
    d = {n: t if n in ("A", "D", "dt_bias", "h0") else t[:, 0].contiguous() for n, t in cuda(a).items() if n != "lens"}
    n, W = G * N, 1031
    wide = torch.full((S, T, W), float("nan"), dtype=dtype, device="cuda")
    wide[:, -1, 3:3 + n], wide[:, -1, 3 + n:3 + 2 * n], wide[:, -1, 500:500 + C] = d["Bm"].flatten(1), d["Cm"].flatten(1), d["z"]
    far = dict(d, Bm=wide[:, -1, 3:3 + n].unflatten(1, (G, N)), Cm=wide[:, -1, 3 + n:3 + 2 * n].unflatten(1, (G, N)),
               z=wide[:, -1, 500:500 + C])
    assert far["Bm"].stride(0) == T * W > 1 << 24
    want, got = d.pop("h0"), far.pop("h0").clone()
    y_want, y = ck.selective_scan_decode_step(**d, H=want), ck.selective_scan_decode_step(**far, H=got)
    torch.cuda.synchronize()
    assert torch.equal(y, y_want) and torch.equal(got, want)
