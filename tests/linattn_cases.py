"""Inputs and elementwise error bounds for the linear attention's GPU tests.

Bounds.  Every output is a sum of products of inputs and decays; A, the same
sum over absolute values (the fp64 reference run on absolute inputs), bounds
the effect of relative errors of its terms.  For bf16 inputs a term carries one
factor split into two bf16 terms (2^-16), for the states three (2^-24); all
sums are fp32, at most T + 512 additions deep (2^-24 each); a decay factor
2^(x - y) is off by at most (1 + Y) 2^-23 with Y the largest sum of log2 decays
in a 64-row chunk, at most 200 (beyond, the factor is 0 in fp32).  The output's
own rounding adds eps / 2 of its value.  Twice the sum of these is allowed for
second-order terms."""
import math

import numpy as np
import torch

import linattn_reference as ref


def inputs(seed, B, H, Hk, T, dk, dv, dtype, decay="token", state=True, lens=None, special=None):
    """dict of CPU tensors q, k, v, g, h0, lens, do, dhT.  decay "token" or
    "head"; special: "reset" (some log decays -inf), "lowest" (some at the
    type's lowest value), "none" (all zero), "strong" (around -6)."""
    r = np.random.default_rng(seed)
    t = lambda *s, f=1.0: torch.from_numpy((f * r.standard_normal(s)).astype(np.float32))  # noqa: E731
    g = -torch.exp(t(*((H,) if decay == "head" else (B, H, T)), f=1.2) - 3.0)
    if special == "none":
        g = torch.zeros_like(g)
    elif special == "strong":
        g = g - 6.0
    elif special in ("reset", "lowest"):
        hit = torch.from_numpy(r.random(g.shape) < 0.1)
        g = torch.where(hit, torch.tensor(-math.inf if special == "reset" else torch.finfo(dtype).min), g)
    x = dict(q=t(B, Hk, T, dk, f=dk ** -0.5), k=t(B, Hk, T, dk, f=dk ** -0.5), v=t(B, H, T, dv), g=g, do=t(B, H, T, dv))
    x = {n: a.to(dtype) for n, a in x.items()}
    x["h0"] = t(B, H, dk, dv, f=0.5) if state else None
    x["dhT"] = t(B, H, dk, dv, f=0.5) if state else None
    x["lens"] = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    return x


def absolute(x):
    return {n: a if n in ("g", "lens") or a is None else a.abs() for n, a in x.items()}


def _slack(x, split):
    T = x["v"].shape[2]
    g = x["g"].double().clamp(min=-1000.0)
    per_chunk = 64 * float(g.abs().max()) if g.numel() else 0.0
    y = min(200.0, per_chunk * 1.4426950408889634)
    return 2 * (split + (1 + y) * 2.0 ** -23 + (T + 512) * 2.0 ** -24)


def fwd_bounds(x):
    """(o, hT, bound of o, bound of hT) in fp64."""
    kw = dict(h0=x["h0"], lens=x["lens"])
    o, hT = ref.linattn_fwd(x["q"], x["k"], x["v"], x["g"], **kw)
    m = absolute(x)
    oa, ha = ref.linattn_fwd(m["q"], m["k"], m["v"], m["g"], h0=m["h0"], lens=m["lens"])
    dt = x["q"].dtype
    bf = dt == torch.bfloat16
    eps = torch.finfo(dt).eps / 2
    return (o, hT, eps * np.abs(o) + _slack(x, 2.0 ** -16 if bf else 0.0) * oa,
            2.0 ** -24 * np.abs(hT) + _slack(x, 2.0 ** -24 if bf else 0.0) * ha)


def bwd_bounds(x):
    """dict name -> (gradient, bound) in fp64."""
    run = lambda y: ref.linattn_bwd(y["q"], y["k"], y["v"], y["g"], y["do"], y["h0"], y["dhT"], y["lens"])  # noqa: E731
    got, mag = run(x), run(absolute(x))
    dt = x["q"].dtype
    bf = dt == torch.bfloat16
    eps = torch.finfo(dt).eps / 2
    c, cs = _slack(x, 2.0 ** -16 if bf else 0.0), _slack(x, 2.0 ** -24 if bf else 0.0)
    out = {n: (got[n], eps * np.abs(got[n]) + c * mag[n]) for n in ("dq", "dk", "dv")}
    out["dh0"] = (got["dh0"], 2.0 ** -24 * np.abs(got["dh0"]) + cs * mag["dh0"])
    # dg_t = flow + sum_{u >= t} (q_u . dq_u - k_u . dk_u): errors of the terms add up
    run_abs = (mag["qdq"] + mag["kdk"])[:, :, ::-1].cumsum(2)[:, :, ::-1] + mag["flow"][..., None]
    if x["g"].dim() == 1:
        run_abs = run_abs.sum((0, 2))
    out["dg"] = (got["dg"], eps * np.abs(got["dg"]) + c * run_abs)
    return out


def check(name, got, want, bound, tiny=1e-30):
    got = got.detach().double().cpu().numpy()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    bad = ~(np.abs(got - want) <= bound + tiny)
    assert not bad.any(), (name, int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4], bound[bad][:4])


def cuda(x):
    return {n: None if a is None else a.cuda() for n, a in x.items()}
