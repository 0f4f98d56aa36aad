"""Inputs and bounds for the decay gradient of the linear attention, relative to
the gradient itself.

dg_t is a sum of products; every one of them carries relative errors of its own
and passes gate t.  With bf16 inputs a product of the kernels' has one factor in
two bf16 terms, off by at most 2^-17; with fp32 inputs it is a sum of up to 128
rounded terms (2^-24 each, 2^-20.5 if all went as random steps of full size).
Of a head's rows at most T such errors, independent of each other, come together
in one gate, so that the errors' rms stays below sqrt(T) times that of the
gradient's rms, and so does a single row's below 6 times that (six standard
deviations).  Rounding to the inputs' type adds eps / 2 of the value.  A constant
decay's gradient is the sum over its T rows, off by at most T times the rows' rms
error (Cauchy and Schwarz).  Where a log decay is below fp32's range (-104) the
factor is 0 and so is the gradient, exactly: nothing passes."""
import math

import numpy as np
import torch

import linattn_reference as ref
from linattn_cases import inputs

BF, F32 = torch.bfloat16, torch.float32
NOTHING = -104.0   # exp of anything below is 0 in fp32


def decays(x, kind, seed):
    """x with log decays of a kind: a number (the same everywhere), "mixed"
    (ordinary ones, one in twenty -12) or "reset" (one in twenty -inf)."""
    g = x["g"]
    r = np.random.default_rng(seed)
    if not isinstance(kind, str):
        g = torch.full_like(g, kind)
    elif kind != "ordinary":
        hit = torch.from_numpy(r.random(g.shape) < 0.05)
        g = torch.where(hit, torch.tensor(-12.0 if kind == "mixed" else -math.inf, dtype=g.dtype), g)
    return {**x, "g": g}


def case(seed, B, H, Hk, T, dk, dv, dtype, kind, decay="token", state=False, lens=None):
    x = inputs(seed, B, H, Hk, T, dk, dv, dtype, decay=decay, state=state, lens=lens)
    return decays(x, kind, seed + 1)


def exact(x):
    """The gradient row by row, [B,H,T], from the fp64 recurrence."""
    B, H, T = x["v"].shape[:3]
    g = x["g"].view(1, -1, 1).expand(B, H, T) if x["g"].dim() == 1 else x["g"]
    return ref.linattn_bwd(x["q"], x["k"], x["v"], g, x["do"], x["h0"], x["dhT"], x["lens"])["dg"]


def accepts(x, rows, got):
    """None, or what is wrong with `got` (numpy, the shape of g) for the exact rows."""
    T = rows.shape[2]
    dt = x["q"].dtype
    half = torch.finfo(dt).eps / 2
    part = (2.0 ** -17 if dt == BF else 2.0 ** -20.5) * math.sqrt(T)
    count = np.full(rows.shape[0], T) if x["lens"] is None else np.clip(x["lens"].numpy(), 0, T)
    rms = np.sqrt((rows ** 2).sum(2) / np.maximum(count, 1)[:, None])   # [B,H]
    if got.ndim == 1:
        want = rows.sum((0, 2))
        bound = half * np.abs(want) + (part * rms * count[:, None]).sum(0)
        bad = ~(np.abs(got - want) <= bound)
        return f"{bad.sum()} heads: {got[bad][:3]} want {want[bad][:3]} bound {bound[bad][:3]}" if bad.any() else None
    err = np.abs(got - rows)
    bad = ~(err <= half * np.abs(rows) + 6 * part * rms[..., None] + 1e-37)
    if bad.any():
        return f"{bad.sum()} rows: {got[bad][:3]} want {rows[bad][:3]} rms {rms.max()}"
    over = np.sqrt((np.maximum(err - half * np.abs(rows), 0) ** 2).sum(2) / np.maximum(count, 1)[:, None]) > part * rms
    if over.any():
        return f"rms error above {part} of the gradient's in {over.sum()} heads"
    nothing = x["g"].double().numpy() < NOTHING
    if (got[nothing] != 0).any():
        return f"{(got[nothing] != 0).sum()} gradients where nothing passes, up to {np.abs(got[nothing]).max()}"
    return None


KINDS = ["ordinary", "mixed", "reset", -0.003, -0.3, -3.0, -6.0, -10.0, -16.0, -40.0]
# T of one round of chunks, of more than 1024 rows and of several rounds (4096 rows each)
SIZES = [(1, 2, 1, 77, 128, 128), (2, 2, 2, 300, 64, 32), (1, 2, 2, 1100, 16, 64), (1, 2, 1, 4500, 32, 32)]
