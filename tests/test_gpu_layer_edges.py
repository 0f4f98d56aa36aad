"""Documented calls of the short convolution, the selective scan and the residual
norm on the GPU that the operators' own tests do not make."""
import numpy as np
import pytest
import torch

import gated_delta_rule_ckda_amd as ck
import test_gpu_add_norm as norm
import test_gpu_short_conv as conv
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


# ---------------------------------------------------------------- the C ABI on the device

CODE = {BF: ck.DTYPE_BF16, F32: ck.DTYPE_F32}


def abi(name, *args):
    """An entry point on device tensors (None: NULL), on the current stream."""
    ptr = [a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args]
    status = getattr(ck.lib(), name)(*ptr, torch.cuda.current_stream().cuda_stream)
    assert status == 0, ck.lib().ckda_last_error()


def workspace(nbytes):
    """Of a call whose results must not depend on what it holds."""
    return torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda"), nbytes


def nan(t):
    return torch.full_like(t, float("nan"))


def same(got, want):
    torch.cuda.synchronize()
    for name in got:
        assert torch.equal(got[name], want[name]), name


def subsets(names):
    """Each name alone, all but each, and all."""
    one = [{n} for n in names]
    rest = [set(names) - {n} for n in names]
    return [x for i, x in enumerate(one + rest + [set(names)]) if x and x not in (one + rest)[:i]]


# ---------------------------------------------------------------- residual norm

@pytest.mark.parametrize("dtype,rt", norm.PAIRS + [(BF, None), (F32, None)])
@pytest.mark.parametrize("R,D", [(5, 1), (40, 300), (9001, 40), (4100, 520), (2100, 2048), (3, 8192)])
@pytest.mark.parametrize("group", [0, 128])
def test_norm_both_outputs_of_one_call(group, R, D, dtype, rt):
    """y and the codes from one call are those of two calls; the sum as well, with a residual or without."""
    x, res, w, _ = norm.tensors(R + D, R, D, dtype, rt)
    x, res, w = norm.dev(x), norm.dev(res), norm.dev(w)
    want = dict(zip(("q", "scales", "sum"), ck.add_norm_quant_fwd(x, res, w, group=group)))
    want["y"], _ = ck.add_norm_fwd(x, res, w)
    want["q"] = want["q"].view(torch.uint8)
    if rt is None:
        want["sum"] = x.float()
    got = {n: torch.full_like(t, 77 if n == "q" else float("nan")) for n, t in want.items()}
    abi("ckda_add_norm_fwd", x, res, w, got["y"], got["q"], got["scales"], got["sum"], R, D, group, CODE[dtype], CODE[want["sum"].dtype], 1e-6)
    same(got, want)


@pytest.mark.parametrize("dtype,rt", norm.PAIRS)
@pytest.mark.parametrize("R,D", [(1, 7), (40, 300), (9001, 40), (4100, 520), (2100, 2048), (3, 8192)])
def test_norm_gradients_in_place_and_one_by_one(R, D, dtype, rt):
    """dres in the place of dsum, and every choice of dx, dres and dw: the same bytes as all of them apart."""
    _, s, w, t = norm.tensors(R + D, R, D, dtype, rt)
    s, w, dy, dsum = s.cuda(), w.cuda(), t(R, D).to(dtype).cuda(), t(R, D).to(rt).cuda()
    want = dict(zip(("dx", "dres", "dw"), ck.add_norm_bwd(s, dy, w, dsum=dsum)))
    nbytes = ck.lib().ckda_add_norm_bwd_workspace_size(R, D, CODE[dtype], CODE[rt])
    size = (R, D, CODE[dtype], CODE[rt], 1e-6)
    for keep in ({"dx"}, {"dres"}, {"dx", "dw"}, {"dres", "dw"}, {"dx", "dres"}, {"dx", "dres", "dw"}):
        for place in (False, True) if "dres" in keep else (False,):
            more = dsum.clone()
            got = {n: more if place and n == "dres" else nan(want[n]) for n in keep}
            abi("ckda_add_norm_bwd", s, w, dy, more, got.get("dx"), got.get("dres"), got.get("dw"), *size, *workspace(nbytes))
            same(got, want)


# ---------------------------------------------------------------- short convolution

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,H,T,C,K,lens", [(3, 2, 40, 24, 4, [40, 0, 2]), (2, 1, 700, 37, 3, None), (1, 1, 1, 5, 2, None),
                                            (2, 1, 0, 12, 4, None)])
def test_conv_without_some_outputs(B, H, T, C, K, lens, dtype):
    a, dy, dsT = conv.make(T, B, T, C, K, dtype, True, lens)
    d = {n: conv.dev(t) for n, t in a.items()}
    dy, dsT = dy.reshape(B, T, H, C // H).transpose(1, 2).contiguous().cuda(), dsT.cuda()
    y, _ = ck.short_conv_fwd(**d, heads=H)
    y2, none = ck.short_conv_fwd(**d, heads=H, want_state=False)
    assert none is None
    same(dict(y=y2), dict(y=y))
    want = dict(zip(("dx", "dw", "db", "ds0"), ck.short_conv_bwd(**d, dy=dy, dsT=dsT)))
    nbytes = ck.lib().ckda_short_conv_bwd_workspace_size(B, T, C, K, CODE[dtype])
    for drop in subsets(("dw", "db", "ds0")):
        got = {n: nan(t) for n, t in want.items() if n not in drop}
        abi("ckda_short_conv_bwd", d["x"], d["w"], d["b"], d["s0"], d["lens"], dy, dsT, got["dx"], *[got.get(n) for n in ("dw", "db", "ds0")],
            B, T, C, H, K, C, CODE[dtype], ck.CONV_SILU | ck.PAD_ZERO, *workspace(nbytes))
        same(got, want)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,C", [(1, 37), (2, 24)])
def test_conv_gradients_behind_a_sequence_are_left(H, C, dtype):
    B, T, K, lens = 4, 300, 4, [300, 0, 2, 131]
    a, dy, dsT = conv.make(H, B, T, C, K, dtype, True, lens)
    d = {n: conv.dev(t) for n, t in a.items()}
    dy, dsT = dy.reshape(B, T, H, C // H).transpose(1, 2).contiguous().cuda(), dsT.cuda()
    want = dict(zip(("dx", "dw", "db", "ds0"), ck.short_conv_bwd(**d, dy=dy, dsT=dsT)))
    for i, n in enumerate(lens):
        want["dx"][i, n:] = 7
    got = {n: torch.full_like(t, 7) for n, t in want.items()}
    nbytes = ck.lib().ckda_short_conv_bwd_workspace_size(B, T, C, K, CODE[dtype])
    abi("ckda_short_conv_bwd", d["x"], d["w"], d["b"], d["s0"], d["lens"], dy, dsT, *got.values(), B, T, C, H, K, C, CODE[dtype],
        ck.CONV_SILU, *workspace(nbytes))
    same(got, want)


# ---------------------------------------------------------------- selective scan

# one segment and several, with 16 lanes a channel and with 4; 64 states; nothing but states
SCANS = [(2, 50, 40, 2, 16), (1, 1500, 20, 1, 16), (1000, 20, 50, 1, 16), (16, 2060, 130, 1, 16), (1, 600, 33, 1, 64), (2, 0, 24, 1, 16)]
OUT = ("dx", "ddt", "dA", "dBm", "dCm", "dD", "dz", "dbias", "dh0")


def scan_bwd(d, dy, dhT, out, flags):
    B, T, C = d["x"].shape
    G, N = d["Bm"].shape[2:]
    code = CODE[d["x"].dtype]
    nbytes = ck.selective_scan_bwd_workspace_size(B, T, C, G, N, code)
    abi("ckda_selective_scan_bwd", *[d[n] for n in ("x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "h0", "lens")], dy, dhT,
        *[out.get(n) for n in OUT], B, T, C, G, N, G * N, C, code, ck.SCAN_SOFTPLUS | flags, *workspace(nbytes))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,C,G,N", SCANS)
@pytest.mark.parametrize("gate", [True, False])
def test_scan_without_some_outputs(gate, B, T, C, G, N, dtype):
    a, dy, dhT = make(N, B, T, C, G, N, dtype, gate=gate)
    d, dy, dhT = cuda(a), dy.cuda(), dhT.cuda()
    y, _ = ck.selective_scan_fwd(**d)
    y2, none = ck.selective_scan_fwd(**d, want_state=False)
    assert none is None
    same(dict(y=y2), dict(y=y))
    want = {n: t for n, t in zip(OUT, ck.selective_scan_bwd(**d, dy=dy, dhT=dhT)) if t is not None}
    some = ck.selective_scan_bwd(**d, dy=dy, dhT=dhT, want_dh0=False)
    assert some[8] is None
    same({n: t for n, t in zip(OUT, some) if t is not None}, want)
    for drop in subsets(("dA", "dD", "dbias", "dh0")):
        got = {n: nan(t) for n, t in want.items() if n not in drop}
        scan_bwd(d, dy, dhT, got, ck.PAD_ZERO)
        same(got, want)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,C,G,N", SCANS[:5])
def test_scan_gradients_behind_a_sequence_are_left(B, T, C, G, N, dtype):
    lens = np.random.default_rng(T).integers(0, T + 1, B)
    lens[:3] = [T // 3 if B == 1 else T, 0, 1][:B]
    a, dy, dhT = make(N, B, T, C, G, N, dtype, lens=lens.tolist())
    d, dy, dhT = cuda(a), dy.cuda(), dhT.cuda()
    want = dict(zip(OUT, ck.selective_scan_bwd(**d, dy=dy, dhT=dhT)))
    behind = torch.arange(T, device="cuda") >= d["lens"][:, None]
    for n in ("dx", "ddt", "dBm", "dCm", "dz"):
        assert (want[n][behind] == 0).all()
        want[n][behind] = 7
    got = {n: torch.full_like(t, 7) for n, t in want.items()}
    scan_bwd(d, dy, dhT, got, 0)
    same(got, want)
