"""The 64-bit statements of tests/layer_reference.py against central differences,
on the CPU."""
import numpy as np
import pytest

import layer_reference as ref


def arr(r, *s):
    return r.standard_normal(s)


def differences(f, x, eps=1e-6):
    g = np.zeros_like(x)
    flat, out = x.reshape(-1), g.reshape(-1)
    for i in range(flat.size):
        keep = flat[i]
        flat[i] = keep + eps
        hi = f()
        flat[i] = keep - eps
        lo = f()
        flat[i] = keep
        out[i] = (hi - lo) / (2 * eps)
    return g


def agree(got, want):
    assert np.abs(got - want).max() <= 1e-7 * max(1.0, np.abs(want).max())


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("K,T,lens", [(4, 6, [6, 3]), (2, 5, None), (3, 1, [1, 0]), (4, 2, [2, 1])])
def test_short_conv(K, T, lens, silu):
    r = np.random.default_rng(K * 10 + T)
    B, H, C = 2, 2, 4
    a = dict(x=arr(r, B, T, C), w=arr(r, C, K), b=arr(r, C), s0=arr(r, B, K - 1, C))
    lens = None if lens is None else np.array(lens)
    dy, dsT = arr(r, B, H, T, C // H), arr(r, B, K - 1, C)

    def loss():
        o = ref.short_conv(**a, lens=lens, heads=H, silu=silu)
        return (o["y"] * dy).sum() + (o["sT"] * dsT).sum()

    g = ref.short_conv(**a, lens=lens, heads=H, silu=silu, dy=dy, dsT=dsT)
    for name, key in (("x", "dx"), ("w", "dw"), ("b", "db"), ("s0", "ds0")):
        agree(g[key], differences(loss, a[name]))


@pytest.mark.parametrize("softplus,gate", [(True, True), (False, False)])
@pytest.mark.parametrize("G,lens", [(1, None), (2, [4, 0])])
def test_selective_scan(G, lens, softplus, gate):
    r = np.random.default_rng(G)
    B, T, C, N = 2, 4, 4, 3
    a = dict(x=arr(r, B, T, C), dt=0.3 * arr(r, B, T, C) + (0.0 if softplus else 1.0), A=-np.exp(0.3 * arr(r, C, N)),
             Bm=arr(r, B, T, G, N), Cm=arr(r, B, T, G, N), D=arr(r, C), z=arr(r, B, T, C) if gate else None,
             dt_bias=0.3 * arr(r, C), h0=arr(r, B, C, N))
    lens = None if lens is None else np.array(lens)
    dy, dhT = arr(r, B, T, C), arr(r, B, C, N)

    def loss():
        o = ref.selective_scan(**a, lens=lens, softplus=softplus)
        return (o["y"] * dy).sum() + (o["hT"] * dhT).sum()

    g = ref.selective_scan(**a, lens=lens, softplus=softplus, dy=dy, dhT=dhT)
    for name, key in (("x", "dx"), ("dt", "ddt"), ("A", "dA"), ("Bm", "dBm"), ("Cm", "dCm"), ("D", "dD"), ("z", "dz"),
                      ("dt_bias", "dbias"), ("h0", "dh0")):
        if a[name] is not None:
            agree(g[key], differences(loss, a[name]))
            assert (g["s" + key] >= np.abs(g[key]) * (1 - 1e-12)).all()


def test_add_norm():
    r = np.random.default_rng(1)
    a = dict(x=arr(r, 3, 7), res=arr(r, 3, 7), w=arr(r, 7))
    dy, dsum = arr(r, 3, 7), arr(r, 3, 7)

    def loss():
        o = ref.add_norm(**a, eps=1e-3)
        return (o["y"] * dy).sum() + (o["r"] * dsum).sum()

    g = ref.add_norm_bwd(a["x"] + a["res"], dy, a["w"], dsum, eps=1e-3)
    agree(g["dr"], differences(loss, a["x"]))
    agree(g["dr"], differences(loss, a["res"]))
    agree(g["dw"], differences(loss, a["w"]))


def test_e4m3_values():
    import torch
    codes = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(codes, ref.e4m3_values())
