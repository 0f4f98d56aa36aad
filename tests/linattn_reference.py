"""Plain fp64 statements of the linear attention with a decay for each head and
of the head norm, for the tests: the recurrences step by step (numpy), and the
norm with its gradients from the formulas.  Nothing here is chunked and nothing
is shared with the library."""
import numpy as np


def _f64(x):
    return None if x is None else np.asarray(x.detach().cpu().double().numpy() if hasattr(x, "detach") else x, np.float64)


def _setup(q, k, g, T, B, H, lens):
    r = H // q.shape[1]
    q, k = np.repeat(q, r, axis=1), np.repeat(k, r, axis=1)
    if g.ndim == 1:
        g = np.broadcast_to(g.reshape(1, H, 1), (B, H, T))
    live = np.arange(T) < (np.full(B, T) if lens is None else np.clip(lens, 0, T)).reshape(B, 1)   # [B, T]
    return q, k, np.exp(g), live


def linattn_fwd(q, k, v, g, h0=None, lens=None):
    """(o, hT); rows of o at or past a sequence's length are zero."""
    q, k, v, g, h0 = (_f64(x) for x in (q, k, v, g, h0))
    B, H, T, dv = v.shape
    lens = None if lens is None else np.asarray(lens.cpu() if hasattr(lens, "cpu") else lens)
    q, k, a, live = _setup(q, k, g, T, B, H, lens)
    S = np.zeros((B, H, q.shape[-1], dv)) if h0 is None else h0.copy()
    o = np.zeros((B, H, T, dv))
    for t in range(T):
        b = live[:, t]
        S[b] = a[b, :, t, None, None] * S[b] + k[b, :, t, :, None] * v[b, :, t, None, :]
        o[b, :, t] = np.einsum("bhij,bhi->bhj", S[b], q[b, :, t])
    return o, S


def linattn_bwd(q, k, v, g, do, h0=None, dhT=None, lens=None):
    """dict of dq, dk, dv, dg, dh0, and qdq, kdk: the dot products q_t . dq_t
    and k_t . dk_t of every head."""
    q, k, v, g, do, h0, dhT = (_f64(x) for x in (q, k, v, g, do, h0, dhT))
    B, H, T, dv_ = v.shape
    Hk, dk_, per_head = q.shape[1], q.shape[-1], g.ndim == 1
    lens = None if lens is None else np.asarray(lens.cpu() if hasattr(lens, "cpu") else lens)
    q, k, a, live = _setup(q, k, g, T, B, H, lens)
    S = [np.zeros((B, H, dk_, dv_)) if h0 is None else h0.copy()]
    for t in range(T):
        n = S[-1].copy()
        b = live[:, t]
        n[b] = a[b, :, t, None, None] * n[b] + k[b, :, t, :, None] * v[b, :, t, None, :]
        S.append(n)
    R = np.zeros_like(S[0]) if dhT is None else dhT.copy()
    dq, dk, dv, dg = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), np.zeros((B, H, T))
    for t in range(T - 1, -1, -1):
        b = live[:, t]
        R[b] += q[b, :, t, :, None] * do[b, :, t, None, :]
        dq[b, :, t] = np.einsum("bhij,bhj->bhi", S[t + 1][b], do[b, :, t])
        dk[b, :, t] = np.einsum("bhij,bhj->bhi", R[b], v[b, :, t])
        dv[b, :, t] = np.einsum("bhij,bhi->bhj", R[b], k[b, :, t])
        R[b] *= a[b, :, t, None, None]
        dg[b, :, t] = np.einsum("bhij,bhij->bh", R[b], S[t][b])
    fold = lambda x: x.reshape(B, Hk, H // Hk, T, dk_).sum(2)  # noqa: E731
    flow = np.zeros((B, H)) if dhT is None else np.einsum("bhij,bhij->bh", dhT, S[-1])
    return dict(dq=fold(dq), dk=fold(dk), dv=dv, dg=dg.sum((0, 2)) if per_head else dg, dh0=R,
                qdq=(q * dq).sum(-1), kdk=(k * dk).sum(-1), flow=flow)


def linattn_decode(q, k, v, g, S):
    """(o, new state)."""
    q, k, v, g, S = (_f64(x) for x in (q, k, v, g, S))
    r = v.shape[1] // q.shape[1]
    q, k = np.repeat(q, r, axis=1), np.repeat(k, r, axis=1)
    a = np.exp(g)
    S = (a.reshape(1, -1, 1, 1) if g.ndim == 1 else a[..., None, None]) * S + k[..., :, None] * v[..., None, :]
    return np.einsum("nhij,nhi->nhj", S, q), S


def _act(z, act):
    sg = 1.0 / (1.0 + np.exp(-z))
    return (z * sg, sg * (1 + z * (1 - sg))) if act == "silu" else (sg, sg * (1 - sg))


def head_norm(x, w=None, b=None, gate=None, act="silu", rms=False, eps=1e-5, dy=None):
    """y [B,T,H,D]; with dy also the gradients: dict of y, n, rstd, dx, dz, dw,
    db (dw, db [H,D], not yet summed over heads)."""
    x, w, b, gate, dy = (_f64(t) for t in (x, w, b, gate, dy))
    u = x.transpose(0, 2, 1, 3)
    D = u.shape[-1]
    if not rms:
        u = u - u.mean(-1, keepdims=True)
    rstd = 1.0 / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    n = u * rstd
    w = np.ones((1, D)) if w is None else w
    b = np.zeros((1, D)) if b is None else b
    s, slope = (np.ones_like(n), np.zeros_like(n)) if gate is None else _act(gate, act)
    out = dict(y=(n * w + b) * s, n=n, rstd=rstd)
    if dy is not None:
        f = dy * s
        dn = f * w
        dx = dn - n * (dn * n).mean(-1, keepdims=True)
        if not rms:
            dx = dx - dn.mean(-1, keepdims=True)
        out.update(dx=(dx * rstd).transpose(0, 2, 1, 3), dz=dy * (n * w + b) * slope, dw=(f * n).sum((0, 1)),
                   db=f.sum((0, 1)), dn=dn)
    return out
