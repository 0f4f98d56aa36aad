"""Refusals of the short convolution's, the selective scan's and the residual
norm's entry points: the C ABI on fake addresses (nothing reaches the device) and
the binding on CPU tensors (shapes are checked first, then the device)."""
import pytest
import torch

import gated_delta_rule_ckda_amd as ck

BASE, MB = 0x7F0000000000, 1 << 20   # fake, never-dereferenced device addresses
BIG = 1 << 50


def at(i, off=0):
    return BASE + i * 65536 * MB + off


def addresses(names, kw):
    return [kw.get(n, at(i)) for i, n in enumerate(names)]


def conv(**kw):
    p = addresses(("x", "w", "b", "s0", "lens", "y", "sT"), kw)
    C = kw.get("C", 64)
    return ck.lib().ckda_short_conv_fwd(*p, kw.get("B", 2), kw.get("T", 20), C, kw.get("H", 2), kw.get("K", 4),
                                        kw.get("ldx", C), kw.get("dtype", 1), kw.get("flags", 1), None)


def conv_bwd(**kw):
    p = addresses(("x", "w", "b", "s0", "lens", "dy", "dsT", "dx", "dw", "db", "ds0", "ws"), kw)
    B, T, C, K, dt = kw.get("B", 2), kw.get("T", 20), kw.get("C", 64), kw.get("K", 4), kw.get("dtype", 1)
    need = ck.lib().ckda_short_conv_bwd_workspace_size(B, T, C, K, dt)
    return ck.lib().ckda_short_conv_bwd(*p[:11], B, T, C, kw.get("H", 2), K, kw.get("ldx", C), dt, kw.get("flags", 33), p[11],
                                        kw.get("ws_bytes", need), None)


def conv_dec(**kw):
    p = addresses(("x", "w", "b", "state", "y"), kw)
    C = kw.get("C", 64)
    return ck.lib().ckda_short_conv_decode_step(*p, kw.get("B", 2), C, kw.get("K", 4), kw.get("ldx", C), kw.get("dtype", 1),
                                                kw.get("flags", 1), None)


CONV = [(ck.ERR_DIM, dict(B=-1)), (ck.ERR_DIM, dict(C=-64)), (ck.ERR_DIM, dict(ldx=63)), (ck.ERR_UNSUPPORTED, dict(K=1)),
        (ck.ERR_UNSUPPORTED, dict(K=5)), (ck.ERR_UNSUPPORTED, dict(dtype=2)), (ck.ERR_FLAGS, dict(flags=2)),
        (ck.ERR_FLAGS, dict(flags=64)), (ck.ERR_NULL, dict(x=None)), (ck.ERR_NULL, dict(w=None)), (ck.ERR_DIM, dict(x=at(0, 1))),
        (ck.ERR_DIM, dict(w=at(1, 4))), (ck.ERR_DIM, dict(b=at(2, 8))), (ck.ERR_DIM, dict(C=(1 << 24) + 2))]
SEQ = [(ck.ERR_DIM, dict(T=-1)), (ck.ERR_DIM, dict(H=3)), (ck.ERR_DIM, dict(H=0)), (ck.ERR_DIM, dict(s0=at(3, 2))),
       (ck.ERR_DIM, dict(lens=at(4, 2)))]


@pytest.mark.parametrize("status,kw", CONV + SEQ + [
    (ck.ERR_NULL, dict(y=None)), (ck.ERR_DIM, dict(y=at(5, 8))), (ck.ERR_ALIAS, dict(y=at(0))), (ck.ERR_ALIAS, dict(y=at(4))),
    (ck.ERR_ALIAS, dict(sT=at(3))), (ck.ERR_ALIAS, dict(sT=at(5, 64))), (ck.ERR_ALIAS, dict(y=at(0, 128 * 39), ldx=128)),
    (ck.ERR_DIM, dict(T=2 ** 31 - 1)), (ck.ERR_DIM, dict(B=1 << 25, T=1)), (ck.ERR_DIM, dict(B=1 << 20, T=1 << 20))])
def test_conv_fwd_refusals(status, kw):
    assert conv(**kw) == status
    assert b"ckda_short_conv_fwd" in ck.lib().ckda_last_error()


@pytest.mark.parametrize("status,kw", CONV + SEQ + [
    *[(ck.ERR_NULL, {n: None}) for n in ("dy", "dx")], (ck.ERR_WORKSPACE, dict(ws=None)), (ck.ERR_WORKSPACE, dict(ws_bytes=64)),
    (ck.ERR_WORKSPACE, dict(ws=at(11, 128))), (ck.ERR_ALIAS, dict(dx=at(5))), (ck.ERR_ALIAS, dict(dw=at(1))),
    (ck.ERR_ALIAS, dict(db=at(8))), (ck.ERR_ALIAS, dict(ds0=at(6))), (ck.ERR_ALIAS, dict(ds0=at(11))),
    (ck.ERR_ALIAS, dict(ws=at(0))), (ck.ERR_DIM, dict(B=1 << 25, T=1, ws_bytes=BIG))])
def test_conv_bwd_refusals(status, kw):
    assert conv_bwd(**kw) == status
    assert b"ckda_short_conv_bwd" in ck.lib().ckda_last_error()


@pytest.mark.parametrize("status,kw", CONV + [
    (ck.ERR_FLAGS, dict(flags=32)), *[(ck.ERR_NULL, {n: None}) for n in ("state", "y")], (ck.ERR_DIM, dict(state=at(3, 8))),
    (ck.ERR_ALIAS, dict(state=at(0))), (ck.ERR_ALIAS, dict(y=at(3))), (ck.ERR_ALIAS, dict(y=at(0))),
    (ck.ERR_DIM, dict(B=1 << 27))])
def test_conv_decode_refusals(status, kw):
    assert conv_dec(**kw) == status
    assert b"ckda_short_conv_decode_step" in ck.lib().ckda_last_error()


def scan_tail(kw, B=None):
    C, G, N = kw.get("C", 64), kw.get("G", 2), kw.get("N", 16)
    head = (kw.get("B", 2),) if B is None else (kw.get("B", 2), kw.get("T", 20))
    return (*head, C, G, N, kw.get("ldbc", max(G * N, 0)), kw.get("ldz", C), kw.get("dtype", 1))


SCAN_IN = ("x", "dt", "A", "Bm", "Cm", "D", "z", "bias")


def scan(**kw):
    p = addresses((*SCAN_IN, "h0", "lens", "y", "hT", "ws"), kw)
    t = scan_tail(kw, 1)
    need = ck.lib().ckda_selective_scan_fwd_workspace_size(*t[:5], t[7])
    return ck.lib().ckda_selective_scan_fwd(*p[:12], *t, kw.get("flags", 1), p[12], kw.get("ws_bytes", need), None)


BWD = (*SCAN_IN, "h0", "lens", "dy", "dhT", "dx", "ddt", "dA", "dBm", "dCm", "dD", "dz", "dbias", "dh0", "ws")


def scan_bwd(**kw):
    p = addresses(BWD, kw)
    t = scan_tail(kw, 1)
    need = ck.lib().ckda_selective_scan_bwd_workspace_size(*t[:5], t[7])
    return ck.lib().ckda_selective_scan_bwd(*p[:21], *t, kw.get("flags", 33), p[21], kw.get("ws_bytes", need), None)


def scan_dec(**kw):
    p = addresses((*SCAN_IN, "H", "y"), kw)
    return ck.lib().ckda_selective_scan_decode_step(*p, *scan_tail(kw), kw.get("flags", 1), None)


SCAN = [(ck.ERR_DIM, dict(B=-1)), (ck.ERR_DIM, dict(C=-2)), (ck.ERR_DIM, dict(G=0)), (ck.ERR_DIM, dict(G=3)),
        (ck.ERR_UNSUPPORTED, dict(N=0)), (ck.ERR_UNSUPPORTED, dict(N=65)), (ck.ERR_UNSUPPORTED, dict(dtype=-1)),
        (ck.ERR_DIM, dict(ldbc=31)), (ck.ERR_DIM, dict(ldz=63)), (ck.ERR_FLAGS, dict(flags=2)), (ck.ERR_FLAGS, dict(flags=17)),
        *[(ck.ERR_NULL, {n: None}) for n in ("x", "dt", "A", "Bm", "Cm")], (ck.ERR_DIM, dict(x=at(0, 2))),
        (ck.ERR_DIM, dict(A=at(2, 4))), (ck.ERR_DIM, dict(Bm=at(3, 1))), (ck.ERR_DIM, dict(Cm=at(4, 1))),
        (ck.ERR_DIM, dict(z=at(6, 1))), (ck.ERR_DIM, dict(bias=at(7, 4))), (ck.ERR_DIM, dict(C=(1 << 24) + 2))]


@pytest.mark.parametrize("status,kw", SCAN + [
    (ck.ERR_DIM, dict(T=-1)), (ck.ERR_NULL, dict(y=None)), (ck.ERR_WORKSPACE, dict(ws=None)), (ck.ERR_WORKSPACE, dict(ws_bytes=255)),
    (ck.ERR_WORKSPACE, dict(ws=at(12, 16))), (ck.ERR_DIM, dict(lens=at(9, 1))), (ck.ERR_DIM, dict(h0=at(8, 4))),
    (ck.ERR_ALIAS, dict(y=at(0))), (ck.ERR_ALIAS, dict(y=at(6))), (ck.ERR_ALIAS, dict(hT=at(8, 64))), (ck.ERR_ALIAS, dict(hT=at(2))),
    (ck.ERR_ALIAS, dict(y=at(12))), (ck.ERR_ALIAS, dict(y=at(3, 64 * 100), ldbc=256)), (ck.ERR_ALIAS, dict(ws=at(0))),
    (ck.ERR_DIM, dict(B=1 << 20, C=1 << 12, T=1)), (ck.ERR_DIM, dict(B=1 << 23, C=64, T=1)), (ck.ERR_DIM, dict(T=2 ** 31 - 1))])
def test_scan_fwd_refusals(status, kw):
    assert scan(**kw) == status
    assert b"ckda_selective_scan_fwd" in ck.lib().ckda_last_error()


@pytest.mark.parametrize("status,kw", SCAN + [
    *[(ck.ERR_NULL, {n: None}) for n in ("dy", "dx", "ddt", "dBm", "dCm", "dz")], (ck.ERR_WORKSPACE, dict(ws=None)),
    (ck.ERR_WORKSPACE, dict(ws_bytes=1000)), (ck.ERR_WORKSPACE, dict(ws=at(21, 8))), (ck.ERR_ALIAS, dict(dx=at(10))),
    (ck.ERR_ALIAS, dict(ddt=at(12))), (ck.ERR_ALIAS, dict(dA=at(2))), (ck.ERR_ALIAS, dict(dBm=at(3))), (ck.ERR_ALIAS, dict(dCm=at(15))),
    (ck.ERR_ALIAS, dict(dD=at(21))), (ck.ERR_ALIAS, dict(dz=at(6))), (ck.ERR_ALIAS, dict(dbias=at(7))), (ck.ERR_ALIAS, dict(dh0=at(8))),
    (ck.ERR_DIM, dict(B=1 << 23, C=64, T=1, ws_bytes=BIG)), (ck.ERR_DIM, dict(B=1 << 10, T=1 << 20, ws_bytes=BIG))])
def test_scan_bwd_refusals(status, kw):
    assert scan_bwd(**kw) == status
    assert b"ckda_selective_scan_bwd" in ck.lib().ckda_last_error()


@pytest.mark.parametrize("status,kw", SCAN + [
    (ck.ERR_FLAGS, dict(flags=32)), *[(ck.ERR_NULL, {n: None}) for n in ("H", "y")], (ck.ERR_DIM, dict(H=at(8, 8))),
    (ck.ERR_ALIAS, dict(H=at(2))), (ck.ERR_ALIAS, dict(y=at(8))), (ck.ERR_ALIAS, dict(y=at(1))), (ck.ERR_DIM, dict(B=1 << 24))])
def test_scan_decode_refusals(status, kw):
    assert scan_dec(**kw) == status
    assert b"ckda_selective_scan_decode_step" in ck.lib().ckda_last_error()


def norm(**kw):
    p = addresses(("x", "res", "w", "y", "q", "scales", "sum"), kw)
    return ck.lib().ckda_add_norm_fwd(*p, kw.get("R", 4), kw.get("D", 64), kw.get("group", 0), kw.get("dtype", 1),
                                      kw.get("res_dtype", 0), kw.get("eps", 1e-6), None)


def norm_bwd(**kw):
    p = addresses(("sum", "w", "dy", "dsum", "dx", "dres", "dw", "ws"), kw)
    R, D, dt, rt = kw.get("R", 4), kw.get("D", 64), kw.get("dtype", 1), kw.get("res_dtype", 0)
    need = ck.lib().ckda_add_norm_bwd_workspace_size(R, D, dt, rt)
    return ck.lib().ckda_add_norm_bwd(*p[:7], R, D, dt, rt, kw.get("eps", 1e-6), p[7], kw.get("ws_bytes", need), None)


NORM = [(ck.ERR_DIM, dict(R=-1)), (ck.ERR_DIM, dict(D=0)), (ck.ERR_UNSUPPORTED, dict(D=8193)), (ck.ERR_UNSUPPORTED, dict(dtype=2)),
        (ck.ERR_UNSUPPORTED, dict(dtype=0, res_dtype=1)), (ck.ERR_UNSUPPORTED, dict(res_dtype=3)), (ck.ERR_DIM, dict(eps=0.0)),
        (ck.ERR_DIM, dict(eps=-1.0)), (ck.ERR_DIM, dict(eps=float("nan"))), (ck.ERR_DIM, dict(eps=float("inf")))]


@pytest.mark.parametrize("status,kw", NORM + [
    (ck.ERR_UNSUPPORTED, dict(group=64)), (ck.ERR_UNSUPPORTED, dict(group=-128)), (ck.ERR_NULL, dict(x=None)),
    (ck.ERR_NULL, dict(y=None, q=None, scales=None)), (ck.ERR_NULL, dict(scales=None)), (ck.ERR_NULL, dict(q=None)),
    (ck.ERR_DIM, dict(x=at(0, 8))), (ck.ERR_DIM, dict(q=at(4, 8))), (ck.ERR_DIM, dict(sum=at(6, 4))), (ck.ERR_ALIAS, dict(y=at(0))),
    (ck.ERR_ALIAS, dict(q=at(3))), (ck.ERR_ALIAS, dict(scales=at(2))), (ck.ERR_ALIAS, dict(sum=at(1, 16))), (ck.ERR_ALIAS, dict(sum=at(0)))])
def test_norm_refusals(status, kw):
    assert norm(**kw) == status
    assert b"ckda_add_norm_fwd" in ck.lib().ckda_last_error()


@pytest.mark.parametrize("status,kw", NORM + [
    *[(ck.ERR_NULL, {n: None}) for n in ("sum", "dy")], (ck.ERR_NULL, dict(dx=None, dres=None)), (ck.ERR_WORKSPACE, dict(ws=None)),
    (ck.ERR_WORKSPACE, dict(ws_bytes=8)), (ck.ERR_WORKSPACE, dict(ws=at(7, 64))), (ck.ERR_DIM, dict(dy=at(2, 2))),
    (ck.ERR_ALIAS, dict(dx=at(2))), (ck.ERR_ALIAS, dict(dres=at(0))), (ck.ERR_ALIAS, dict(dres=at(3, 16))), (ck.ERR_ALIAS, dict(dw=at(1))),
    (ck.ERR_ALIAS, dict(dx=at(7)))])
def test_norm_bwd_refusals(status, kw):
    assert norm_bwd(**kw) == status
    assert b"ckda_add_norm_bwd" in ck.lib().ckda_last_error()


def test_empty_calls_are_ok():
    none = dict.fromkeys(("x", "w", "b", "s0", "y", "sT", "dy", "dsT", "dx", "dw", "db", "ds0", "state", "ws"))
    assert conv(B=0, **{k: v for k, v in none.items()}) == 0 and conv(C=0, H=1, **none) == 0 and conv(T=0, **none) == 0
    assert conv_bwd(B=0, **none) == 0 and conv_bwd(T=0, **none) == 0 and conv_dec(B=0, **none) == 0
    empty = dict.fromkeys(BWD + ("hT", "H", "y"))
    assert scan(B=0, **empty) == 0 and scan(C=0, ldz=0, **empty) == 0 and scan(T=0, **empty) == 0
    assert scan_bwd(B=0, **empty) == 0 and scan_bwd(C=0, T=0, ldz=0, **empty) == 0 and scan_dec(B=0, **empty) == 0
    assert norm(R=0, x=None, y=None, q=None, scales=None) == 0 and norm_bwd(R=0, dw=None) == 0
    assert ck.lib().ckda_last_error() == b""


def test_scan_bwd_without_channels_needs_the_sums_over_them():
    assert scan_bwd(C=0, ldz=0, dBm=None) == ck.ERR_NULL and scan_bwd(C=0, ldz=0, dCm=None) == ck.ERR_NULL


def test_workspace_sizes():
    L = ck.lib()
    c, f, b, n = (L.ckda_short_conv_bwd_workspace_size, L.ckda_selective_scan_fwd_workspace_size,
                  L.ckda_selective_scan_bwd_workspace_size, L.ckda_add_norm_bwd_workspace_size)
    assert c(2, 20, 64, 5, 1) == 0 and c(-1, 20, 64, 4, 1) == 0 and c(0, 20, 64, 4, 1) == 256 and c(4, 4096, 2048, 4, 1) % (5 * 2048 * 4) == 0
    assert f(4, 4096, 2048, 1, 16, 1) == 256                     # a workgroup for every CU: no segments
    assert f(1, 4096, 64, 1, 16, 1) > 256 and f(1, 100, 64, 1, 65, 1) == 0 and f(1, 100, 64, 3, 16, 1) == 0
    assert b(4, 4096, 2048, 1, 16, 1) >= 4 * 256 * 2048 * 16 * 4 and b(0, 5, 64, 1, 16, 1) == 256 and b(1, 5, 64, 1, 16, 4) == 0
    assert n(10, 64, 1, 0) > 0 and n(10, 64, 0, 1) == 0 and n(10, 8193, 1, 1) == 0 and n(0, 64, 1, 1) == 256


# ---------------------------------------------------------------- binding

F32, BF = torch.float32, torch.bfloat16


def t(*s, dtype=BF):
    return torch.zeros(*s, dtype=dtype)


B, T, C, H, K, G, N = 2, 6, 12, 3, 4, 2, 5


def conv_args(**over):
    a = dict(x=t(B, T, C), w=t(C, K, dtype=F32), b=t(C, dtype=F32), s0=t(B, K - 1, C), lens=t(B, dtype=torch.int32))
    return {**a, **over}


@pytest.mark.parametrize("over", [dict(x=t(B, C)), dict(w=t(C + 1, K, dtype=F32)), dict(w=t(C, dtype=F32)), dict(b=t(C + 1, dtype=F32)),
                                  dict(s0=t(B, K, C)), dict(lens=t(B + 1, dtype=torch.int32)), dict(heads=5), dict(act="relu")])
def test_conv_binding_shapes(over):
    a = conv_args(**over)
    with pytest.raises(ValueError, match="shape|divide|act|dimensions"):
        ck.short_conv_fwd(**a)
    heads = a.pop("heads", H)
    with pytest.raises(ValueError, match="shape|divide|act|dimensions"):
        ck.short_conv_bwd(**a, dy=t(B, heads, T, 4))


def test_conv_binding_good_shapes_reach_the_device_check():
    with pytest.raises(ValueError, match="GPU tensor"):
        ck.short_conv_fwd(**conv_args(), heads=H)
    with pytest.raises(ValueError, match="GPU tensor"):
        ck.short_conv_bwd(**conv_args(), dy=t(B, H, T, C // H))
    with pytest.raises(ValueError, match="shape"):
        ck.short_conv_decode_step(t(B, C), t(C, K, dtype=F32), t(B, K, C))
    with pytest.raises(ValueError, match="GPU tensor"):
        ck.short_conv_decode_step(t(B, C), t(C, K, dtype=F32), t(B, K - 1, C))


def scan_args(**over):
    a = dict(x=t(B, T, C), dt=t(B, T, C), A=t(C, N, dtype=F32), Bm=t(B, T, G, N), Cm=t(B, T, G, N), D=t(C, dtype=F32), z=t(B, T, C),
             dt_bias=t(C, dtype=F32), h0=t(B, C, N, dtype=F32), lens=t(B, dtype=torch.int32))
    return {**a, **over}


@pytest.mark.parametrize("over", [dict(x=t(B, T)), dict(dt=t(B, T + 1, C)), dict(A=t(C, N + 1, dtype=F32)), dict(Bm=t(B, T, N)),
                                  dict(Bm=t(B, T, 5, N), Cm=t(B, T, 5, N)), dict(D=t(1, dtype=F32)), dict(h0=t(B, N, C, dtype=F32)),
                                  dict(lens=t(3, dtype=torch.int32)), dict(dt_bias=t(C + 1, dtype=F32))])
def test_scan_binding_shapes(over):
    with pytest.raises(ValueError, match="shape|divide|dimensions"):
        ck.selective_scan_fwd(**scan_args(**over))
    with pytest.raises(ValueError, match="shape|divide|dimensions"):
        ck.selective_scan_bwd(**scan_args(**over), dy=t(B, T, C))


def test_scan_binding_good_shapes_reach_the_device_check():
    with pytest.raises(ValueError, match="GPU tensor"):
        ck.selective_scan_fwd(**scan_args())
    with pytest.raises(ValueError, match="GPU tensor"):
        ck.selective_scan_bwd(**scan_args(), dy=t(B, T, C))
    a = scan_args()
    one = {k: a[k][:, 0].contiguous() for k in ("x", "dt", "Bm", "Cm", "z")}
    with pytest.raises(ValueError, match="GPU tensor"):
        ck.selective_scan_decode_step(**one, A=a["A"], H=a["h0"])
    with pytest.raises(ValueError, match="shape"):
        ck.selective_scan_decode_step(**one, A=a["A"], H=a["h0"][:1])


def test_norm_binding_shapes():
    x, w = t(4, C), t(C, dtype=F32)
    for kw in (dict(res=t(4, C + 1)), dict(w=t(C + 1, dtype=F32)), dict(total=t(5, C)), dict(res=t(4, C), total=t(3, C))):
        with pytest.raises(ValueError, match="shape"):
            ck.add_norm_fwd(x, **kw)
    with pytest.raises(TypeError, match="residual"):
        ck.add_norm_fwd(x.float(), t(4, C), w)
    with pytest.raises(ValueError, match="group"):
        ck.add_norm_quant_fwd(x, group=32)
    with pytest.raises(ValueError, match="shape"):
        ck.add_norm_bwd(t(4, C, dtype=F32), t(5, C), w)
    for call in (lambda: ck.add_norm_fwd(x, x, w), lambda: ck.add_norm_bwd(x, x, w)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
