"""Refusals of the linear attention's and the head norm's entry points: the C
ABI on fake addresses (nothing reaches the device) and the binding on CPU
tensors (shapes are checked first, then the device)."""
import ctypes

import pytest
import torch

import gated_delta_rule_ckda_amd as ck

BASE, MB = 0x7F0000000000, 1 << 20   # fake, never-dereferenced device addresses
INT_MAX = 2 ** 31 - 1


def at(i, off=0):
    return BASE + i * 1024 * MB + off


def fwd(**kw):
    B, H, Hk, T = kw.get("B", 2), kw.get("H", 4), kw.get("Hk", 2), kw.get("T", 64)
    dk, dv, dt, fl = kw.get("dk", 64), kw.get("dv", 64), kw.get("dtype", 1), kw.get("flags", 0)
    p = {n: kw.get(n, at(i)) for i, n in enumerate(("q", "k", "v", "g", "h0", "lens", "o", "hT", "ws"))}
    need = ck.lib().ckda_linattn_fwd_workspace_size(B, H, T, dk, dv, dt)
    return ck.lib().ckda_linattn_fwd(p["q"], p["k"], p["v"], p["g"], p["h0"], p["lens"], p["o"], p["hT"], B, H, Hk, T, dk,
                                     dv, dt, fl, p["ws"], kw.get("ws_bytes", need), None)


BWD = ("q", "k", "v", "g", "h0", "lens", "do", "dhT", "dq", "dk_", "dv_", "dg", "dh0", "ws")


def bwd(**kw):
    B, H, Hk, T = kw.get("B", 2), kw.get("H", 4), kw.get("Hk", 2), kw.get("T", 64)
    dk, dv, dt, fl = kw.get("dk", 64), kw.get("dv", 64), kw.get("dtype", 1), kw.get("flags", 0)
    p = [kw.get(n, at(i)) for i, n in enumerate(BWD)]
    need = ck.lib().ckda_linattn_bwd_workspace_size(B, H, Hk, T, dk, dv, dt)
    return ck.lib().ckda_linattn_bwd(*p[:13], B, H, Hk, T, dk, dv, dt, fl, p[13], kw.get("ws_bytes", need), None)


def dec(**kw):
    N, H, Hk = kw.get("N", 2), kw.get("H", 4), kw.get("Hk", 2)
    p = [kw.get(n, at(i)) for i, n in enumerate(("q", "k", "v", "g", "S", "o"))]
    return ck.lib().ckda_linattn_decode_step(*p, N, H, Hk, kw.get("dk", 64), kw.get("dv", 64), kw.get("dtype", 1),
                                             kw.get("flags", 0), None)


def norm(**kw):
    B, H, T, D = kw.get("B", 2), kw.get("H", 4), kw.get("T", 8), kw.get("D", 64)
    p = [kw.get(n, at(i)) for i, n in enumerate(("x", "z", "w", "b", "y"))]
    return ck.lib().ckda_head_norm_fwd(*p, B, H, T, D, kw.get("wheads", H), kw.get("dtype", 1), kw.get("flags", 2),
                                       kw.get("eps", 1e-5), None)


def norm_bwd(**kw):
    B, H, T, D = kw.get("B", 2), kw.get("H", 4), kw.get("T", 8), kw.get("D", 64)
    wh, dt = kw.get("wheads", H), kw.get("dtype", 1)
    p = [kw.get(n, at(i)) for i, n in enumerate(("x", "z", "w", "b", "dy", "dx", "dz", "dw", "db", "ws"))]
    need = ck.lib().ckda_head_norm_bwd_workspace_size(B, H, T, D, wh, dt)
    return ck.lib().ckda_head_norm_bwd(*p[:9], B, H, T, D, wh, dt, kw.get("flags", 2), kw.get("eps", 1e-5), p[9],
                                       kw.get("ws_bytes", need), None)


SIZES = [(ck.ERR_DIM, dict(B=-1)), (ck.ERR_DIM, dict(H=-4)), (ck.ERR_DIM, dict(Hk=3)), (ck.ERR_DIM, dict(Hk=0)),
         (ck.ERR_UNSUPPORTED, dict(dtype=2)), (ck.ERR_UNSUPPORTED, dict(dk=96)), (ck.ERR_UNSUPPORTED, dict(dv=256)),
         (ck.ERR_FLAGS, dict(flags=1)), (ck.ERR_FLAGS, dict(flags=48))]


@pytest.mark.parametrize("status,kw", SIZES + [
    (ck.ERR_DIM, dict(T=-1)), (ck.ERR_NULL, dict(q=None)), (ck.ERR_NULL, dict(k=None)), (ck.ERR_NULL, dict(v=None)),
    (ck.ERR_NULL, dict(g=None)), (ck.ERR_NULL, dict(o=None)), (ck.ERR_WORKSPACE, dict(ws=None)),
    (ck.ERR_WORKSPACE, dict(ws_bytes=255)), (ck.ERR_WORKSPACE, dict(ws=at(8, 128))), (ck.ERR_DIM, dict(q=at(0, 8))),
    (ck.ERR_DIM, dict(h0=at(4, 4))), (ck.ERR_DIM, dict(lens=at(5, 2))), (ck.ERR_DIM, dict(T=1 << 25, dk=128)),
    (ck.ERR_ALIAS, dict(o=at(2))), (ck.ERR_ALIAS, dict(o=at(5))), (ck.ERR_ALIAS, dict(hT=at(4, 64))),
    (ck.ERR_ALIAS, dict(hT=at(6))), (ck.ERR_ALIAS, dict(o=at(8))), (ck.ERR_ALIAS, dict(hT=at(0))),
    (ck.ERR_DIM, dict(B=1 << 20, H=1 << 12, Hk=1, T=1)),
])
def test_fwd_refusals(status, kw):
    assert fwd(**kw) == status
    assert b"ckda_linattn_fwd" in ck.lib().ckda_last_error()


@pytest.mark.parametrize("status,kw", SIZES + [
    (ck.ERR_DIM, dict(T=-1)), *[(ck.ERR_NULL, {n: None}) for n in ("q", "k", "v", "g", "do", "dq", "dk_", "dv_", "dg")],
    (ck.ERR_WORKSPACE, dict(ws=None)), (ck.ERR_WORKSPACE, dict(ws_bytes=1000)), (ck.ERR_WORKSPACE, dict(ws=at(13, 64))),
    (ck.ERR_DIM, dict(do=at(6, 2))), (ck.ERR_DIM, dict(lens=at(5, 1))), (ck.ERR_ALIAS, dict(dq=at(0))),
    (ck.ERR_ALIAS, dict(dk_=at(8))), (ck.ERR_ALIAS, dict(dh0=at(7))), (ck.ERR_ALIAS, dict(dg=at(3))),
    (ck.ERR_ALIAS, dict(dv_=at(13, 256))), (ck.ERR_ALIAS, dict(dq=at(5))), (ck.ERR_DIM, dict(T=1 << 23)),
    (ck.ERR_DIM, dict(B=1 << 16, H=1 << 12, Hk=1, T=1)),
])
def test_bwd_refusals(status, kw):
    assert bwd(**kw) == status
    assert b"ckda_linattn_bwd" in ck.lib().ckda_last_error()


@pytest.mark.parametrize("status,kw", [(s, {**k, **({"N": k["B"]} if "B" in k else {})}) for s, k in SIZES] + [
    *[(ck.ERR_NULL, {n: None}) for n in ("q", "k", "v", "g", "S", "o")], (ck.ERR_DIM, dict(S=at(4, 8))),
    (ck.ERR_ALIAS, dict(o=at(4))), (ck.ERR_ALIAS, dict(S=at(1))), (ck.ERR_ALIAS, dict(o=at(3))),
    (ck.ERR_DIM, dict(N=1 << 20, H=1 << 10)),
])
def test_decode_refusals(status, kw):
    assert dec(**kw) == status
    assert b"ckda_linattn_decode_step" in ck.lib().ckda_last_error()


@pytest.mark.parametrize("call,kw", [
    (fwd, dict(B=1 << 16, H=1 << 8, Hk=1, T=1)), (bwd, dict(B=1 << 14, H=1 << 8, Hk=1 << 8, T=1)),
    (bwd, dict(B=1 << 10, H=1 << 4, Hk=1 << 3, T=1 << 16)), (dec, dict(N=1 << 14, H=1 << 10, Hk=1)),
])
def test_launch_grid(call, kw):
    """Sizes whose launches would have 2^32 threads or more are refused before any of them."""
    assert call(**kw, ws_bytes=1 << 50) == ck.ERR_DIM if call is not dec else call(**kw) == ck.ERR_DIM
    assert b"launch grid" in ck.lib().ckda_last_error()


NORM = [(ck.ERR_DIM, dict(B=-1)), (ck.ERR_DIM, dict(D=0)), (ck.ERR_UNSUPPORTED, dict(D=8193)),
        (ck.ERR_DIM, dict(wheads=2)), (ck.ERR_DIM, dict(wheads=0)), (ck.ERR_UNSUPPORTED, dict(dtype=5)),
        (ck.ERR_FLAGS, dict(flags=8)), (ck.ERR_FLAGS, dict(flags=6)), (ck.ERR_FLAGS, dict(flags=0)),
        (ck.ERR_FLAGS, dict(flags=2, z=None)), (ck.ERR_DIM, dict(eps=0.0)), (ck.ERR_DIM, dict(eps=-1.0)),
        (ck.ERR_DIM, dict(eps=float("nan"))), (ck.ERR_DIM, dict(eps=float("inf"))), (ck.ERR_NULL, dict(x=None)),
        (ck.ERR_DIM, dict(x=at(0, 4))), (ck.ERR_DIM, dict(w=at(2, 4))), (ck.ERR_DIM, dict(B=1 << 16, T=1 << 15)),
        (ck.ERR_DIM, dict(H=65536))]


@pytest.mark.parametrize("status,kw", NORM + [(ck.ERR_NULL, dict(y=None)), (ck.ERR_ALIAS, dict(y=at(0))),
                                              (ck.ERR_ALIAS, dict(y=at(1))), (ck.ERR_ALIAS, dict(y=at(3)))])
def test_norm_refusals(status, kw):
    assert norm(**kw) == status
    assert b"ckda_head_norm_fwd" in ck.lib().ckda_last_error()


@pytest.mark.parametrize("status,kw", NORM + [
    *[(ck.ERR_NULL, {n: None}) for n in ("dy", "dx", "dz")], (ck.ERR_WORKSPACE, dict(ws=None)),
    (ck.ERR_WORKSPACE, dict(ws_bytes=8)), (ck.ERR_WORKSPACE, dict(ws=at(9, 16))), (ck.ERR_ALIAS, dict(dx=at(0))),
    (ck.ERR_ALIAS, dict(dz=at(4))), (ck.ERR_ALIAS, dict(db=at(7))), (ck.ERR_ALIAS, dict(dw=at(9)))])
def test_norm_bwd_refusals(status, kw):
    assert norm_bwd(**kw) == status
    assert b"ckda_head_norm_bwd" in ck.lib().ckda_last_error()


def test_empty_calls_are_ok():
    L = ck.lib()
    assert fwd(B=0, q=None, k=None, v=None, g=None, o=None, h0=None, hT=None, ws=None) == 0
    assert fwd(H=0, Hk=0) == 0
    assert fwd(T=0, hT=None, q=None, k=None, v=None, g=None, o=None, ws=None) == 0
    assert bwd(B=0) == 0 and bwd(H=0, Hk=0) == 0
    assert dec(N=0, q=None, S=None) == 0
    assert norm(T=0, x=None, y=None) == 0
    assert norm_bwd(B=0, dw=None, db=None) == 0
    assert L.ckda_last_error() == b""


def test_workspace_sizes():
    L = ck.lib()
    f, b, n = L.ckda_linattn_fwd_workspace_size, L.ckda_linattn_bwd_workspace_size, L.ckda_head_norm_bwd_workspace_size
    assert f(4, 16, 4096, 128, 128, 1) >= 256
    assert f(1, 1, 64, 96, 128, 1) == 0 and f(-1, 1, 64, 64, 64, 1) == 0 and f(1, 1, 64, 64, 64, 3) == 0
    # few heads and many rows: fp32 states and a decay for every segment
    few = f(1, 2, 65536, 64, 64, 1)
    assert few > 2 * 2 * 64 * 64 * 4 and few % 256 == 0
    assert b(2, 4, 3, 64, 64, 64, 1) == 0 and b(2, 4, 2, 64, 48, 64, 1) == 0
    # shared heads add the heads' fp32 parts of dq and dk
    assert b(2, 4, 2, 64, 64, 64, 1) - b(2, 4, 4, 64, 64, 64, 1) == 2 * 2 * 4 * 64 * 64 * 4
    assert n(2, 4, 8, 64, 4, 1) > 0 and n(2, 4, 8, 64, 3, 1) == 0 and n(2, 4, 8, 9000, 4, 1) == 0
    assert n(0, 4, 8, 64, 4, 1) == 256


# ---------------------------------------------------------------- binding

B, H, Hk, T, DK, DV = 2, 4, 2, 10, 16, 32


def t(*s, dtype=torch.bfloat16):
    return torch.zeros(*s, dtype=dtype)


def args(**over):
    a = dict(q=t(B, Hk, T, DK), k=t(B, Hk, T, DK), v=t(B, H, T, DV), g=t(B, H, T), do=t(B, H, T, DV),
             h0=t(B, H, DK, DV, dtype=torch.float32), dhT=t(B, H, DK, DV, dtype=torch.float32),
             lens=t(B, dtype=torch.int32))
    a.update(over)
    return a


def py_fwd(**over):
    a = args(**over)
    ck.linattn_fwd(a["q"], a["k"], a["v"], a["g"], a["h0"], lens=a["lens"])


def py_bwd(**over):
    a = args(**over)
    ck.linattn_bwd(a["q"], a["k"], a["v"], a["g"], a["do"], a["h0"], a["dhT"], lens=a["lens"])


WRONG = [("q", (B, 3, T, DK)), ("k", (B, Hk, T, DK + 1)), ("k", (B, H, T, DK)), ("v", (B, H, T + 1, DV)), ("g", (B, H)),
         ("g", (H + 1,)), ("g", (B, H, T, 1)), ("h0", (B, H, DV, DK)), ("lens", (B + 1,)), ("q", (B, T, DK))]


@pytest.mark.parametrize("call", [py_fwd, py_bwd])
@pytest.mark.parametrize("name,shape", WRONG)
def test_binding_rejects_wrong_shapes(call, name, shape):
    dt = dict(h0=torch.float32, lens=torch.int32).get(name, torch.bfloat16)
    with pytest.raises(ValueError, match="shape|dimensions|divide"):
        call(**{name: t(*shape, dtype=dt)})


@pytest.mark.parametrize("call", [py_fwd, py_bwd])
def test_binding_good_shapes_reach_the_device_check(call):
    with pytest.raises(ValueError, match="GPU tensor"):
        call()
    with pytest.raises(ValueError, match="GPU tensor"):
        call(g=t(H))


def test_binding_norm_shapes():
    x, z, w = t(B, H, T, DV), t(B, T, H, DV), t(H, DV, dtype=torch.float32)
    for kw in (dict(w=t(3, DV, dtype=torch.float32)), dict(w=w, b=w[:1]), dict(gate=x), dict(act="relu"),
               dict(w=t(DV, dtype=torch.float32)), dict(b=t(H, DV + 1, dtype=torch.float32))):
        with pytest.raises(ValueError, match="shape|act"):
            ck.head_norm_fwd(x, **kw)
        with pytest.raises(ValueError, match="shape|act"):
            ck.head_norm_bwd(x, z, **kw)
    with pytest.raises(ValueError, match="shape"):
        ck.head_norm_bwd(x, x)
    for kw in (dict(), dict(w=w, b=w), dict(w=w[:1], gate=z)):
        with pytest.raises(ValueError, match="GPU tensor"):
            ck.head_norm_fwd(x, **kw)


def test_binding_decode_shapes():
    q, v, g, S = t(B, Hk, DK), t(B, H, DV), t(B, H), t(B, H, DK, DV, dtype=torch.float32)
    for a in ((q, q, v, t(B, H, 1), S), (q, q[:1], v, g, S), (t(B, 3, DK), q, v, g, S), (q, q, v, g, S[:1])):
        with pytest.raises(ValueError, match="shape|divide"):
            ck.linattn_decode_step(*a)
    with pytest.raises(ValueError, match="GPU tensor"):
        ck.linattn_decode_step(q, q, v, t(H), S)
