"""Plain fp64 statements of the short causal convolution, the selective scan and
the norm with the residual's addition, for the tests: row by row from the
formulas (numpy), gradients written out.  Nothing here is chunked and nothing is
shared with the library.

Beside each result stands its size: the same formula with the absolute value of
every term, which rounding errors are relative to."""
import numpy as np


def f64(x):
    return None if x is None else np.asarray(x.detach().cpu().double().numpy() if hasattr(x, "detach") else x, np.float64)


def lengths(lens, B, T):
    return np.full(B, T) if lens is None else np.clip(np.asarray(lens.cpu() if hasattr(lens, "cpu") else lens), 0, T)


def sigmoid(z):
    return 1.0 / (1.0 + np.exp(-z))


# ---------------------------------------------------------------- short convolution

def short_conv(x, w, b=None, s0=None, lens=None, heads=1, silu=True, dy=None, dsT=None):
    """dict of y [B,H,T,Dh], sT, u and su (the sums before the activation and their
    sizes, [B,T,C]); with dy also dx, dw, db, ds0, g (dy times the slope) and the
    sizes sdx, sdw, sdb, sds0 (of g's magnitudes)."""
    x, w, b, s0, dy, dsT = (f64(t) for t in (x, w, b, s0, dy, dsT))
    B, T, C = x.shape
    K = w.shape[1]
    n = lengths(lens, B, T)
    live = (np.arange(T) < n[:, None])[..., None]
    past = np.concatenate([np.zeros((B, K - 1, C)) if s0 is None else s0, np.where(live, x, 0.0)], 1)
    u, su = np.zeros((B, T, C)), np.zeros((B, T, C))
    for t in range(T):
        for j in range(K):
            u[:, t] += w[:, j] * past[:, t + j]
            su[:, t] += np.abs(w[:, j] * past[:, t + j])
    if b is not None:
        u, su = u + b, su + np.abs(b)
    y = np.where(live, u * sigmoid(u) if silu else u, 0.0)
    turn = lambda v: v.reshape(B, T, heads, C // heads).transpose(0, 2, 1, 3)  # noqa: E731
    out = dict(y=turn(y), u=u, su=su, turn=turn, live=live, sT=np.stack([past[i, n[i]:n[i] + K - 1] for i in range(B)]))
    if dy is None:
        return out
    d = dy.transpose(0, 2, 1, 3).reshape(B, T, C)
    sg = sigmoid(u)
    g = np.where(live, d * (sg * (1 + u * (1 - sg)) if silu else 1.0), 0.0)
    dpast, size = np.zeros_like(past), np.zeros_like(past)
    dw, sdw = np.zeros_like(w), np.zeros_like(w)
    for t in range(T):
        for j in range(K):
            dpast[:, t + j] += w[:, j] * g[:, t]
            size[:, t + j] += np.abs(w[:, j] * g[:, t])
            dw[:, j] += (g[:, t] * past[:, t + j]).sum(0)
            sdw[:, j] += np.abs(g[:, t] * past[:, t + j]).sum(0)
    if dsT is not None:
        for i in range(B):
            dpast[i, n[i]:n[i] + K - 1] += dsT[i]
            size[i, n[i]:n[i] + K - 1] += np.abs(dsT[i])
    out.update(dx=dpast[:, K - 1:], ds0=dpast[:, :K - 1], sdx=size[:, K - 1:], sds0=size[:, :K - 1], dw=dw, sdw=sdw,
               db=g.sum((0, 1)), sdb=np.abs(g).sum((0, 1)), g=g, d=d)
    return out


# ---------------------------------------------------------------- selective scan

def selective_scan(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, h0=None, lens=None, softplus=True, dy=None, dhT=None):
    """dict of y, hT and their sizes sy, shT; with dy also dx, ddt, dA, dBm, dCm, dD,
    dz, dbias, dh0 and their sizes (s before the name)."""
    x, dt, A, Bm, Cm, D, z, bias, h0, dy, dhT = (f64(t) for t in (x, dt, A, Bm, Cm, D, z, dt_bias, h0, dy, dhT))
    B, T, C = x.shape
    G, N = Bm.shape[2:]
    n = lengths(lens, B, T)
    live = np.arange(T) < n[:, None]
    raw = dt if bias is None else dt + bias
    d = np.logaddexp(raw, 0.0) if softplus else raw
    Dv = np.zeros(C) if D is None else D
    group = np.arange(C) // (C // G)
    Bc, Cc = Bm[:, :, group], Cm[:, :, group]                     # [B, T, C, N]
    zero = np.zeros((B, C, N))
    h, m = (zero, zero) if h0 is None else (h0, np.abs(h0))
    hs, ms = [h], [m]                                             # states and their sizes, before row 0 first
    for t in range(T):
        on = live[:, t, None, None]
        a = np.exp(d[:, t, :, None] * A)
        add = (d[:, t] * x[:, t])[..., None] * Bc[:, t]
        h, m = np.where(on, a * h + add, h), np.where(on, a * m + np.abs(add), m)
        hs.append(h)
        ms.append(m)
    on = live[..., None]
    after, sizes = np.stack(hs[1:], 1) if T else np.zeros((B, 0, C, N)), np.stack(ms[1:], 1) if T else np.zeros((B, 0, C, N))
    pre, spre = (after * Cc).sum(-1) + Dv * x, (sizes * np.abs(Cc)).sum(-1) + np.abs(Dv * x)
    gate, slope = (1.0, None) if z is None else (z * sigmoid(z), sigmoid(z) * (1 + z * (1 - sigmoid(z))))
    out = dict(y=np.where(on, pre * gate, 0.0), sy=np.where(on, spre * np.abs(gate), 0.0), hT=h, shT=m)
    if dy is None:
        return out
    ds = np.where(on, dy * gate, 0.0)
    R, sR = (zero, zero) if dhT is None else (dhT, np.abs(dhT))
    names = ("dx", "ddt", "dA", "dBm", "dCm")
    g = {k: np.zeros_like(v) for k, v in zip(names, (x, x, A, Bm, Cm))}
    g.update({"s" + k: np.zeros_like(v) for k, v in zip(names, (x, x, A, Bm, Cm))})
    fold = lambda v: v.reshape(B, G, C // G, N).sum(2)  # noqa: E731
    for t in range(T - 1, -1, -1):
        m3 = live[:, t, None, None]
        a = np.where(m3, np.exp(d[:, t, :, None] * A), 1.0)
        add = ds[:, t, :, None] * Cc[:, t]
        R, sR = R + np.where(m3, add, 0.0), sR + np.where(m3, np.abs(add), 0.0)
        dx_ = (d[:, t] * x[:, t])[..., None]
        for s, r, hb, ha, mul in (("", R, hs[t], hs[t + 1], lambda v: v), ("s", sR, ms[t], ms[t + 1], np.abs)):
            r = np.where(m3, r, 0.0)
            u = (r * mul(Bc[:, t])).sum(-1)
            q = a * r * hb
            v = (q * mul(A)).sum(-1)
            g[s + "dx"][:, t] = mul(d[:, t]) * u + mul(Dv * ds[:, t])
            g[s + "ddt"][:, t] = mul(x[:, t]) * u + v
            g[s + "dA"] += (mul(d[:, t])[..., None] * q).sum(0)
            g[s + "dBm"][:, t] = fold(r * mul(dx_))
            g[s + "dCm"][:, t] = fold(mul(ds[:, t, :, None]) * ha * m3)
        R, sR = a * R, a * sR
    if softplus:
        g["ddt"], g["sddt"] = g["ddt"] * sigmoid(raw), g["sddt"] * sigmoid(raw)
    g.update(dD=(ds * x).sum((0, 1)), sdD=np.abs(ds * x).sum((0, 1)), dbias=g["ddt"].sum((0, 1)), sdbias=g["sddt"].sum((0, 1)),
             dh0=R, sdh0=sR)
    if z is not None:
        g.update(dz=np.where(on, dy * pre * slope, 0.0),
                 sdz=np.where(on, np.abs(dy) * spre * sigmoid(z) * (1 + np.abs(z)), 0.0))
    out.update(g)
    return out


# ---------------------------------------------------------------- norm with the residual's addition

def add_norm(x, res=None, w=None, eps=1e-6):
    """dict of r, n, rstd, y."""
    x, res, w = f64(x), f64(res), f64(w)
    r = x if res is None else x + res
    rstd = 1.0 / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    return dict(r=r, n=r * rstd, rstd=rstd, y=r * rstd * (1.0 if w is None else w))


def add_norm_bwd(r, dy, w=None, dsum=None, eps=1e-6):
    """dict of dr, dw and their sizes."""
    r, dy, w, dsum = f64(r), f64(dy), f64(w), f64(dsum)
    rstd = 1.0 / np.sqrt((r * r).mean(-1, keepdims=True) + eps)
    n = r * rstd
    dn = dy * (1.0 if w is None else w)
    more = 0.0 if dsum is None else dsum
    over = tuple(range(r.ndim - 1))
    return dict(dr=more + rstd * (dn - n * (dn * n).mean(-1, keepdims=True)), dw=(dy * n).sum(over),
                sdr=np.abs(more) + rstd * (np.abs(dn) + np.abs(n) * np.abs(dn * n).mean(-1, keepdims=True)),
                sdw=np.abs(dy * n).sum(over))


def e4m3_values():
    """The finite values >= 0 of e4m3: exponents 2^-6 .. 2^8 with three bits, and steps of 2^-9 below."""
    v = [i * 2.0 ** -9 for i in range(8)] + [(1 + f / 8) * 2.0 ** e for e in range(-6, 9) for f in range(8)]
    return np.array(sorted(v))[:-1]   # the last pattern is NaN
