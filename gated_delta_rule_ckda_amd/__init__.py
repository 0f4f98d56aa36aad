"""MI355X (gfx950) CKDA / KDA kernels: Python binding of the C ABI in include/ckda.h.

Only argument marshalling happens here: torch supplies device memory and the
current HIP stream, and every step of the computation runs in the HIP
kernels of libckda.so.  There is no fallback: if the library is missing or
fails to load, every call raises.

    o, hT = chunk_fwd(q, k, v, alpha, beta, h0=None, chunk=64)
    o = decode_step(q, k, v, alpha, beta, H)          # H updated in place

    o, hT = linattn_fwd(q, k, v, g, h0=None)          # linear attention, a decay for each head
    y = head_norm_fwd(o, w, b, gate=z)                # norm and output gate, token-major

    y, total = add_norm_fwd(x, residual, w)           # rms norm ahead of the projections (add_norm_quant_fwd: 8 bits)
    q, sT = short_conv_fwd(x, w, heads=H)             # short causal convolution, head-major
    y, hT = selective_scan_fwd(x, dt, A, Bm, Cm)      # diagonal recurrence, a decay for each channel and state

With fuse=FUSE_GATES | FUSE_NORM_K (| FUSE_NORM_Q) the kernels first apply the
per-token prologue: alpha and beta are logits, keys (queries) are normalised.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libckda.so")

DTYPE_F32, DTYPE_BF16 = 0, 1
STATUS = {0: "CKDA_OK", 1: "CKDA_ERR_NULL", 2: "CKDA_ERR_DIM", 3: "CKDA_ERR_UNSUPPORTED",
          4: "CKDA_ERR_ALIAS", 5: "CKDA_ERR_HIP", 6: "CKDA_ERR_WORKSPACE", 7: "CKDA_ERR_FLAGS"}
(ERR_NULL, ERR_DIM, ERR_UNSUPPORTED, ERR_ALIAS, ERR_HIP, ERR_WORKSPACE, ERR_FLAGS) = range(1, 8)
FUSE_GATES, FUSE_NORM_K, FUSE_NORM_Q = 1, 2, 4       # CKDA_FUSE_*
GATE_SCALAR = 8                                      # CKDA_GATE_SCALAR
DECAY_HEAD = 16                                      # CKDA_DECAY_HEAD
NORM_RMS, NORM_GATE_SILU, NORM_GATE_SIGMOID = 1, 2, 4   # CKDA_NORM_*
CONV_SILU, SCAN_SOFTPLUS, PAD_ZERO = 1, 1, 32        # CKDA_CONV_SILU, CKDA_SCAN_SOFTPLUS, CKDA_PAD_ZERO
EXPORTS = ("ckda_chunk_fwd_workspace_size", "ckda_chunk_fwd", "ckda_chunk_fwd_noalloc", "ckda_chunk_fwd_timed",
           "ckda_chunk_fwd_ex",
           "ckda_chunk_fwd_gather", "ckda_decode_step", "ckda_decode_step_ex", "ckda_decode_step_gather",
           "ckda_deltaproduct2_fwd", "ckda_deltaproduct2_decode_step", "ckda_chunk_bwd",
           "ckda_chunk_bwd_workspace_size", "ckda_chunk_bwd_ex", "ckda_chunk_bwd_ex_workspace_size",
           "ckda_deltaproduct2_bwd", "ckda_deltaproduct2_bwd_workspace_size",
           "ckda_linattn_fwd", "ckda_linattn_fwd_workspace_size", "ckda_linattn_bwd", "ckda_linattn_bwd_workspace_size",
           "ckda_linattn_decode_step", "ckda_head_norm_fwd", "ckda_head_norm_bwd", "ckda_head_norm_bwd_workspace_size",
           "ckda_short_conv_fwd", "ckda_short_conv_bwd", "ckda_short_conv_bwd_workspace_size", "ckda_short_conv_decode_step",
           "ckda_selective_scan_fwd", "ckda_selective_scan_fwd_workspace_size", "ckda_selective_scan_bwd",
           "ckda_selective_scan_bwd_workspace_size", "ckda_selective_scan_decode_step",
           "ckda_add_norm_fwd", "ckda_add_norm_bwd", "ckda_add_norm_bwd_workspace_size",
           "ckda_status_string", "ckda_last_error", "ckda_abi_version")

_lib = None


class CkdaError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"{STATUS.get(status, status)}: {detail}")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded libckda.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with gated_delta_rule_ckda_amd/build.py "
                               "(or __graft_entry__.build())")
        L = ctypes.CDLL(LIB_PATH)
        vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.ckda_chunk_fwd_workspace_size.argtypes = [i] * 7
        L.ckda_chunk_fwd_workspace_size.restype = sz
        L.ckda_chunk_fwd.argtypes = [vp] * 8 + [i] * 7 + [vp, sz, vp]
        L.ckda_chunk_fwd.restype = i
        L.ckda_chunk_fwd_noalloc.argtypes = [vp] * 8 + [i] * 7 + [vp]
        L.ckda_chunk_fwd_noalloc.restype = i
        L.ckda_chunk_fwd_timed.argtypes = [vp] * 8 + [i] * 7 + [vp, sz, vp, vp, vp, vp]
        L.ckda_chunk_fwd_timed.restype = i
        L.ckda_chunk_fwd_ex.argtypes = [vp] * 8 + [i] * 8 + [vp, sz, vp]
        L.ckda_chunk_fwd_ex.restype = i
        L.ckda_chunk_fwd_gather.argtypes = [vp] * 8 + [i] * 4 + [vp] + [i] * 5 + [vp, sz, vp]
        L.ckda_chunk_fwd_gather.restype = i
        L.ckda_decode_step_gather.argtypes = [vp] * 7 + [i] * 3 + [vp] + [i] * 4 + [vp]
        L.ckda_decode_step_gather.restype = i
        L.ckda_deltaproduct2_fwd.argtypes = [vp] * 8 + [i] * 8 + [vp, sz, vp]
        L.ckda_deltaproduct2_fwd.restype = i
        L.ckda_deltaproduct2_decode_step.argtypes = [vp] * 7 + [i] * 6 + [vp]
        L.ckda_deltaproduct2_decode_step.restype = i
        L.ckda_chunk_bwd_workspace_size.argtypes = [i] * 6
        L.ckda_chunk_bwd_workspace_size.restype = sz
        L.ckda_chunk_bwd.argtypes = [vp] * 14 + [i] * 6 + [vp, sz, vp]
        L.ckda_chunk_bwd.restype = i
        L.ckda_chunk_bwd_ex_workspace_size.argtypes = [i] * 7
        L.ckda_chunk_bwd_ex_workspace_size.restype = sz
        L.ckda_chunk_bwd_ex.argtypes = [vp] * 14 + [i] * 7 + [vp, sz, vp]
        L.ckda_chunk_bwd_ex.restype = i
        L.ckda_deltaproduct2_bwd_workspace_size.argtypes = [i] * 6
        L.ckda_deltaproduct2_bwd_workspace_size.restype = sz
        L.ckda_deltaproduct2_bwd.argtypes = [vp] * 14 + [i] * 6 + [vp, sz, vp]
        L.ckda_deltaproduct2_bwd.restype = i
        L.ckda_decode_step.argtypes = [vp] * 7 + [i] * 5 + [vp]
        L.ckda_decode_step.restype = i
        L.ckda_decode_step_ex.argtypes = [vp] * 7 + [i] * 6 + [vp]
        L.ckda_decode_step_ex.restype = i
        f = ctypes.c_float
        L.ckda_linattn_fwd_workspace_size.argtypes = [i] * 6
        L.ckda_linattn_fwd_workspace_size.restype = sz
        L.ckda_linattn_fwd.argtypes = [vp] * 8 + [i] * 8 + [vp, sz, vp]
        L.ckda_linattn_fwd.restype = i
        L.ckda_linattn_bwd_workspace_size.argtypes = [i] * 7
        L.ckda_linattn_bwd_workspace_size.restype = sz
        L.ckda_linattn_bwd.argtypes = [vp] * 13 + [i] * 8 + [vp, sz, vp]
        L.ckda_linattn_bwd.restype = i
        L.ckda_linattn_decode_step.argtypes = [vp] * 6 + [i] * 7 + [vp]
        L.ckda_linattn_decode_step.restype = i
        L.ckda_head_norm_fwd.argtypes = [vp] * 5 + [i] * 7 + [f, vp]
        L.ckda_head_norm_fwd.restype = i
        L.ckda_head_norm_bwd_workspace_size.argtypes = [i] * 6
        L.ckda_head_norm_bwd_workspace_size.restype = sz
        L.ckda_head_norm_bwd.argtypes = [vp] * 9 + [i] * 7 + [f, vp, sz, vp]
        L.ckda_head_norm_bwd.restype = i
        L.ckda_short_conv_fwd.argtypes = [vp] * 7 + [i] * 8 + [vp]
        L.ckda_short_conv_fwd.restype = i
        L.ckda_short_conv_bwd_workspace_size.argtypes = [i] * 5
        L.ckda_short_conv_bwd_workspace_size.restype = sz
        L.ckda_short_conv_bwd.argtypes = [vp] * 11 + [i] * 8 + [vp, sz, vp]
        L.ckda_short_conv_bwd.restype = i
        L.ckda_short_conv_decode_step.argtypes = [vp] * 5 + [i] * 6 + [vp]
        L.ckda_short_conv_decode_step.restype = i
        L.ckda_selective_scan_fwd_workspace_size.argtypes = [i] * 6
        L.ckda_selective_scan_fwd_workspace_size.restype = sz
        L.ckda_selective_scan_fwd.argtypes = [vp] * 12 + [i] * 9 + [vp, sz, vp]
        L.ckda_selective_scan_fwd.restype = i
        L.ckda_selective_scan_bwd_workspace_size.argtypes = [i] * 6
        L.ckda_selective_scan_bwd_workspace_size.restype = sz
        L.ckda_selective_scan_bwd.argtypes = [vp] * 21 + [i] * 9 + [vp, sz, vp]
        L.ckda_selective_scan_bwd.restype = i
        L.ckda_selective_scan_decode_step.argtypes = [vp] * 10 + [i] * 8 + [vp]
        L.ckda_selective_scan_decode_step.restype = i
        L.ckda_add_norm_fwd.argtypes = [vp] * 7 + [i] * 5 + [f, vp]
        L.ckda_add_norm_fwd.restype = i
        L.ckda_add_norm_bwd_workspace_size.argtypes = [i] * 4
        L.ckda_add_norm_bwd_workspace_size.restype = sz
        L.ckda_add_norm_bwd.argtypes = [vp] * 7 + [i] * 4 + [f, vp, sz, vp]
        L.ckda_add_norm_bwd.restype = i
        L.ckda_status_string.argtypes = [i]
        L.ckda_status_string.restype = ctypes.c_char_p
        L.ckda_last_error.argtypes = []
        L.ckda_last_error.restype = ctypes.c_char_p
        L.ckda_abi_version.argtypes = []
        L.ckda_abi_version.restype = i
        _lib = L
    return _lib


def _check(status: int):
    if status != 0:
        raise CkdaError(status, lib().ckda_last_error().decode())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    if t.dtype == torch.float32:
        return DTYPE_F32
    raise TypeError(f"inputs must be bfloat16 or float32, got {t.dtype}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _require(ts, dtype):
    for name, t in ts.items():
        if not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.dtype != dtype:
            raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")


def _shapes(expect):
    """Raise ValueError unless every given tensor has exactly its expected
    shape.  The C ABI receives bare pointers and cannot see shapes, so this is
    the only guard against a wrong-shaped tensor turning into out-of-bounds
    device reads or writes; it runs before anything else touches the
    tensors.  `expect` maps a name to (tensor or None, shape tuple)."""
    for name, (t, shape) in expect.items():
        if t is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


INT_MAX = 2 ** 31 - 1   # of the C ABI's sizes; ctypes would wrap a larger one around


def _dims(t, n, name):
    shape = t.shape
    if len(shape) != n:
        raise ValueError(f"{name} must have {n} dimensions, got shape {tuple(shape)}")
    if t.numel() > INT_MAX and max(shape) > INT_MAX:   # (the count first: small calls wait for the host)
        raise ValueError(f"{name} has shape {tuple(shape)}, with more than 2^31 - 1 of a dimension")
    return shape


def _scratch(nbytes, device, stream):
    """A temporary uint8 workspace for one call.  It is allocated from torch's
    caching allocator; when the kernels run on another stream than the
    current one, the allocation is tied to that stream too, so that it is not
    handed out again before those kernels are done with it."""
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    if stream is not None and stream != torch.cuda.current_stream(device):
        ws.record_stream(stream)
    return ws


def workspace_size(B, H, T, dk, dv, chunk, dtype) -> int:
    code = dtype if isinstance(dtype, int) else _dtype_code(torch.empty(0, dtype=dtype))
    return int(lib().ckda_chunk_fwd_workspace_size(B, H, T, dk, dv, chunk, code))


def chunk_fwd(q, k, v, alpha, beta, h0=None, chunk=64, workspace=None, o=None, hT=None,
              want_state=True, stream=None, events=None, fuse=0, idx=None):
    """Chunkwise forward.  q, k, alpha [B,H,T,dk]; v [B,H,T,dv]; beta [B,H,T];
    h0 [B,H,dk,dv] fp32 or None.  Returns (o [B,H,T,dv], hT [B,H,dk,dv] fp32 or None).

    `workspace` (uint8 GPU tensor of at least workspace_size() bytes), `o` and
    `hT` may be passed in to avoid allocations (e.g. in timed loops).
    `events`, three recorded-once torch.cuda.Event objects (or None), are
    recorded before the Gram kernel, between the kernels and after the
    state-pass kernel (ckda_chunk_fwd_timed).  `fuse` (FUSE_* bits) applies
    the per-token prologue (ckda_chunk_fwd_ex); it cannot be combined with
    `events`.  `idx` ([H, dk] int32 GPU tensor) gathers each head's retained
    key channels from full-width q, k, alpha rows [B,H,T,dk_in] inside the
    kernels (ckda_chunk_fwd_gather); states then have dk rows."""
    B, H, T, dk = _dims(q, 4, "q")
    dk_in = dk
    if idx is not None:
        if idx.dim() != 2 or idx.shape[0] != H:
            raise ValueError(f"idx must be [H, dk], got {tuple(idx.shape)}")
        dk = idx.shape[1]
    dv = _dims(v, 4, "v")[-1]
    scalar = bool(fuse & GATE_SCALAR)
    _shapes(dict(k=(k, (B, H, T, dk_in)), v=(v, (B, H, T, dv)),
                 alpha=(alpha, (B, H, T) if scalar else (B, H, T, dk_in)), beta=(beta, (B, H, T)),
                 h0=(h0, (B, H, dk, dv)), o=(o, (B, H, T, dv)), hT=(hT, (B, H, dk, dv))))
    _require(dict(q=q, k=k, v=v, alpha=alpha, beta=beta), q.dtype)
    if idx is not None:
        _require(dict(idx=idx), torch.int32)
    code = _dtype_code(q)
    if h0 is not None:
        _require(dict(h0=h0), torch.float32)
    if o is not None:
        _require(dict(o=o), q.dtype)
    if hT is not None:
        _require(dict(hT=hT), torch.float32)
    need = workspace_size(B, H, T, dk, dv, chunk, code)
    if need == 0:
        raise CkdaError(ERR_UNSUPPORTED, f"unsupported sizes dk={dk} dv={dv} chunk={chunk}")
    if workspace is None:
        workspace = _scratch(need, q.device, stream)
    if o is None:
        o = torch.empty((B, H, T, dv), dtype=q.dtype, device=q.device)
    if hT is None and want_state:
        hT = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(h0), _ptr(o), _ptr(hT),
            B, H, T, dk, dv, chunk, code, _ptr(workspace), workspace.numel() * workspace.element_size(),
            _stream(stream))
    if idx is not None:
        if events is not None:
            raise ValueError("events are recorded by the plain forward only")
        _check(lib().ckda_chunk_fwd_gather(*args[:11], dk_in, _ptr(idx), *args[11:15], int(fuse), *args[15:]))
    elif fuse:
        if events is not None:
            raise ValueError("events are recorded by the plain forward only (fuse=0)")
        args = args[:15] + (int(fuse),) + args[15:]
        _check(lib().ckda_chunk_fwd_ex(*args))
    elif events is None:
        _check(lib().ckda_chunk_fwd(*args))
    else:
        handles = [None if e is None else ctypes.c_void_p(e.cuda_event) for e in events]
        _check(lib().ckda_chunk_fwd_timed(*args, *handles))
    return o, hT


def chunk_fwd_noalloc(q, k, v, alpha, beta, h0, o, hT=None, chunk=64, stream=None):
    """ckda_chunk_fwd_noalloc: the chunkwise forward with no workspace and no
    allocation (for callers that cannot allocate, e.g. under graph capture).
    The caller passes the outputs o [B,H,T,dv] and hT [B,H,dk,dv] fp32 (or
    None).  Calls that overlap in time on one GPU share its fixed scratch and
    race; calls on one stream are safe.  Returns (o, hT)."""
    B, H, T, dk = _dims(q, 4, "q")
    dv = _dims(v, 4, "v")[-1]
    if o is None:
        raise ValueError("o is required (this entry point allocates nothing)")
    _shapes(dict(k=(k, (B, H, T, dk)), v=(v, (B, H, T, dv)), alpha=(alpha, (B, H, T, dk)), beta=(beta, (B, H, T)),
                 h0=(h0, (B, H, dk, dv)), o=(o, (B, H, T, dv)), hT=(hT, (B, H, dk, dv))))
    _require(dict(q=q, k=k, v=v, alpha=alpha, beta=beta, o=o), q.dtype)
    for name, t in (("h0", h0), ("hT", hT)):
        if t is not None:
            _require({name: t}, torch.float32)
    _check(lib().ckda_chunk_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(h0), _ptr(o),
                                        _ptr(hT), B, H, T, dk, dv, chunk, _dtype_code(q), _stream(stream)))
    return o, hT


def decode_step(q, k, v, alpha, beta, H, o=None, stream=None, fuse=0, idx=None):
    """One decode step.  q, k, alpha [N,Hh,dk]; v [N,Hh,dv]; beta [N,Hh];
    H [N,Hh,dk,dv] fp32 updated in place.  Returns o [N,Hh,dv].  `fuse`
    (FUSE_* bits) applies the per-token prologue first (ckda_decode_step_ex).
    `idx` ([Hh, dk] int32) gathers retained key channels from rows of dk_in
    (ckda_decode_step_gather)."""
    N, Hh, dk = _dims(q, 3, "q")
    dk_in = dk
    if idx is not None:
        if idx.dim() != 2 or idx.shape[0] != Hh:
            raise ValueError(f"idx must be [H, dk], got {tuple(idx.shape)}")
        dk = idx.shape[1]
    dv = _dims(v, 3, "v")[-1]
    scalar = bool(fuse & GATE_SCALAR)
    _shapes(dict(k=(k, (N, Hh, dk_in)), v=(v, (N, Hh, dv)), alpha=(alpha, (N, Hh) if scalar else (N, Hh, dk_in)),
                 beta=(beta, (N, Hh)), H=(H, (N, Hh, dk, dv)), o=(o, (N, Hh, dv))))
    _require(dict(q=q, k=k, v=v, alpha=alpha, beta=beta), q.dtype)
    _require(dict(H=H), torch.float32)
    if idx is not None:
        _require(dict(idx=idx), torch.int32)
    if o is not None:
        _require(dict(o=o), q.dtype)
    code = _dtype_code(q)
    if o is None:
        o = torch.empty((N, Hh, dv), dtype=q.dtype, device=q.device)
    ptrs = (_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(H), _ptr(o))
    if idx is not None:
        _check(lib().ckda_decode_step_gather(*ptrs, N, Hh, dk_in, _ptr(idx), dk, dv, code, int(fuse), _stream(stream)))
    elif fuse:
        _check(lib().ckda_decode_step_ex(*ptrs, N, Hh, dk, dv, code, int(fuse), _stream(stream)))
    else:
        _check(lib().ckda_decode_step(*ptrs, N, Hh, dk, dv, code, _stream(stream)))
    return o


def deltaproduct2_fwd(q, k, v, beta, alpha=None, h0=None, chunk=64, workspace=None, o=None, hT=None,
                      want_state=True, stream=None, fuse=0):
    """DeltaProduct_2 forward (ckda_deltaproduct2_fwd): q [B,H,T,dk];
    k [B,H,T,2,dk]; v [B,H,T,2,dv]; beta [B,H,T,2]; alpha [B,H,T] scalar
    gates or None (ungated); h0 [B,H,dk,dv] fp32 or None.  Returns (o, hT)."""
    B, H, T, dk = _dims(q, 4, "q")
    dv = _dims(v, 5, "v")[-1]
    _shapes(dict(k=(k, (B, H, T, 2, dk)), v=(v, (B, H, T, 2, dv)), beta=(beta, (B, H, T, 2)),
                 alpha=(alpha, (B, H, T)), h0=(h0, (B, H, dk, dv)), o=(o, (B, H, T, dv)), hT=(hT, (B, H, dk, dv))))
    ts = dict(q=q, k=k, v=v, beta=beta)
    if alpha is not None:
        ts["alpha"] = alpha
    if o is not None:
        ts["o"] = o
    _require(ts, q.dtype)
    code = _dtype_code(q)
    for name, t in (("h0", h0), ("hT", hT)):
        if t is not None:
            _require({name: t}, torch.float32)
    need = workspace_size(B, H, 2 * T, dk, dv, chunk, code)
    if need == 0:
        raise CkdaError(ERR_UNSUPPORTED, f"unsupported sizes dk={dk} dv={dv} chunk={chunk}")
    if workspace is None:
        workspace = _scratch(need, q.device, stream)
    if o is None:
        o = torch.empty((B, H, T, dv), dtype=q.dtype, device=q.device)
    if hT is None and want_state:
        hT = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    _check(lib().ckda_deltaproduct2_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(h0), _ptr(o),
                                        _ptr(hT), B, H, T, dk, dv, chunk, code, int(fuse), _ptr(workspace),
                                        workspace.numel() * workspace.element_size(), _stream(stream)))
    return o, hT


def deltaproduct2_decode_step(q, k, v, beta, H, alpha=None, o=None, stream=None, fuse=0):
    """One DeltaProduct_2 decode step: q [N,Hh,dk]; k [N,Hh,2,dk];
    v [N,Hh,2,dv]; beta [N,Hh,2]; alpha [N,Hh] or None; H fp32 in place."""
    N, Hh, dk = _dims(q, 3, "q")
    dv = _dims(v, 4, "v")[-1]
    _shapes(dict(k=(k, (N, Hh, 2, dk)), v=(v, (N, Hh, 2, dv)), beta=(beta, (N, Hh, 2)), alpha=(alpha, (N, Hh)),
                 H=(H, (N, Hh, dk, dv)), o=(o, (N, Hh, dv))))
    ts = dict(q=q, k=k, v=v, beta=beta)
    if alpha is not None:
        ts["alpha"] = alpha
    if o is not None:
        ts["o"] = o
    _require(ts, q.dtype)
    _require(dict(H=H), torch.float32)
    code = _dtype_code(q)
    if o is None:
        o = torch.empty((N, Hh, dv), dtype=q.dtype, device=q.device)
    _check(lib().ckda_deltaproduct2_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(H), _ptr(o),
                                                N, Hh, dk, dv, code, int(fuse), _stream(stream)))
    return o


def bwd_workspace_size(B, H, T, dk, dv, dtype) -> int:
    code = dtype if isinstance(dtype, int) else _dtype_code(torch.empty(0, dtype=dtype))
    return int(lib().ckda_chunk_bwd_workspace_size(B, H, T, dk, dv, code))


def bwd_ex_workspace_size(B, H, T, dk, dv, dtype, flags) -> int:
    code = dtype if isinstance(dtype, int) else _dtype_code(torch.empty(0, dtype=dtype))
    return int(lib().ckda_chunk_bwd_ex_workspace_size(B, H, T, dk, dv, code, int(flags)))


def chunk_bwd(q, k, v, alpha, beta, do, h0=None, dhT=None, want_dh0=True, workspace=None, stream=None, fuse=0):
    """Backward of chunk_fwd (ckda_chunk_bwd): given do = dL/do [B,H,T,dv]
    (input dtype) and dhT = dL/dH_T [B,H,dk,dv] fp32 or None, returns fp32
    (dq, dk, dv, dalpha, dbeta, dh0 or None).  With `fuse` (FUSE_* and
    GATE_SCALAR bits, ckda_chunk_bwd_ex) the inputs are those of the fused
    forward and the gradients are with respect to them: logits, raw keys
    and queries; with GATE_SCALAR alpha and dalpha are [B,H,T]."""
    B, H, T, dk = _dims(q, 4, "q")
    dv = _dims(v, 4, "v")[-1]
    _shapes(dict(k=(k, (B, H, T, dk)), alpha=(alpha, (B, H, T) if fuse & GATE_SCALAR else (B, H, T, dk)),
                 beta=(beta, (B, H, T)), do=(do, (B, H, T, dv)), h0=(h0, (B, H, dk, dv)), dhT=(dhT, (B, H, dk, dv))))
    _require(dict(q=q, k=k, v=v, alpha=alpha, beta=beta, do=do), q.dtype)
    code = _dtype_code(q)
    if h0 is not None:
        _require(dict(h0=h0), torch.float32)
    if dhT is not None:
        _require(dict(dhT=dhT), torch.float32)
    need = bwd_ex_workspace_size(B, H, T, dk, dv, code, fuse) if fuse else bwd_workspace_size(B, H, T, dk, dv, code)
    if need == 0:
        raise CkdaError(ERR_UNSUPPORTED, f"unsupported sizes dk={dk} dv={dv} or flags {fuse}")
    if workspace is None:
        workspace = _scratch(need, q.device, stream)
    f32 = dict(dtype=torch.float32, device=q.device)
    gq, gk = (torch.empty((B, H, T, dk), **f32) for _ in range(2))
    galpha = torch.empty((B, H, T) if fuse & GATE_SCALAR else (B, H, T, dk), **f32)
    gv = torch.empty((B, H, T, dv), **f32)
    gbeta = torch.empty((B, H, T), **f32)
    gh0 = torch.empty((B, H, dk, dv), **f32) if want_dh0 else None
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(h0), _ptr(do), _ptr(dhT),
            _ptr(gq), _ptr(gk), _ptr(gv), _ptr(galpha), _ptr(gbeta), _ptr(gh0), B, H, T, dk, dv, code)
    tail = (_ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    if fuse:
        _check(lib().ckda_chunk_bwd_ex(*args, int(fuse), *tail))
    else:
        _check(lib().ckda_chunk_bwd(*args, *tail))
    return gq, gk, gv, galpha, gbeta, gh0


def deltaproduct2_bwd(q, k, v, alpha, beta, do, h0=None, dhT=None, want_dh0=True, workspace=None, stream=None):
    """Backward of deltaproduct2_fwd (ckda_deltaproduct2_bwd): q [B,H,T,dk],
    k [B,H,T,2,dk], v [B,H,T,2,dv], beta [B,H,T,2], alpha [B,H,T] or None,
    do [B,H,T,dv] (input dtype), dhT fp32 or None.  Returns fp32 (dq, dk, dv,
    dalpha or None, dbeta, dh0 or None) in the inputs' shapes."""
    B, H, T, dk = _dims(q, 4, "q")
    dv = _dims(v, 5, "v")[-1]
    _shapes(dict(k=(k, (B, H, T, 2, dk)), v=(v, (B, H, T, 2, dv)), beta=(beta, (B, H, T, 2)),
                 alpha=(alpha, (B, H, T)), do=(do, (B, H, T, dv)), h0=(h0, (B, H, dk, dv)),
                 dhT=(dhT, (B, H, dk, dv))))
    ts = dict(q=q, k=k, v=v, beta=beta, do=do)
    if alpha is not None:
        ts["alpha"] = alpha
    _require(ts, q.dtype)
    code = _dtype_code(q)
    for name, t in (("h0", h0), ("dhT", dhT)):
        if t is not None:
            _require({name: t}, torch.float32)
    need = int(lib().ckda_deltaproduct2_bwd_workspace_size(B, H, T, dk, dv, code))
    if need == 0:
        raise CkdaError(ERR_UNSUPPORTED, f"unsupported sizes dk={dk} dv={dv}")
    if workspace is None:
        workspace = _scratch(need, q.device, stream)
    f32 = dict(dtype=torch.float32, device=q.device)
    gq = torch.empty((B, H, T, dk), **f32)
    gk = torch.empty((B, H, T, 2, dk), **f32)
    gv = torch.empty((B, H, T, 2, dv), **f32)
    galpha = torch.empty((B, H, T), **f32) if alpha is not None else None
    gbeta = torch.empty((B, H, T, 2), **f32)
    gh0 = torch.empty((B, H, dk, dv), **f32) if want_dh0 else None
    _check(lib().ckda_deltaproduct2_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(h0), _ptr(do),
                                        _ptr(dhT), _ptr(gq), _ptr(gk), _ptr(gv), _ptr(galpha), _ptr(gbeta), _ptr(gh0),
                                        B, H, T, dk, dv, code, _ptr(workspace),
                                        workspace.numel() * workspace.element_size(), _stream(stream)))
    return gq, gk, gv, galpha, gbeta, gh0


# ---------------------------------------------------------------- linear attention, head norm

def _tensors(device, expect):
    """Checks of shape, dtype, contiguity and device for `expect`, a list of
    (name, tensor or None, shape, dtype); all tensors must be on `device`, a
    GPU.  The C ABI cannot see any of these."""
    index = device.index if device.type == "cuda" else -2
    for _, t, shape, dtype in expect:
        if t is not None and (t.shape != shape or t.dtype != dtype or t.get_device() != index or not t.is_contiguous()):
            break
    else:
        return
    for name, t, shape, _ in expect:   # shapes first
        if t is not None and t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    for name, t, _, dtype in expect:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor")
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.dtype != dtype:
            raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")


def _run(device, stream, fn, *args):
    """fn(*args, stream handle) with `device` current: on `stream`, or on the
    device's current stream."""
    if stream is None:
        # (the handle itself: a Stream object costs some 3 us, a third of a small call)
        handle = torch._C._cuda_getCurrentRawStream(device.index)
    elif stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors are on {device}")
    else:
        handle = stream.cuda_stream
    if device.index == torch._C._cuda_getDevice():
        status = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            status = fn(*args, handle)
    if status:
        _check(status)


def _workspace_arg(workspace, need, device, stream):
    """The caller's workspace, or a temporary one of `need` bytes, and its
    (pointer, bytes); the tensor is to be kept until the call is made."""
    if workspace is None:
        workspace = _fresh((need,), torch.uint8, device, stream)
    elif not workspace.is_cuda or workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous GPU tensor on {device}")
    return workspace, (workspace.data_ptr(), workspace.numel() * workspace.element_size())


def _fresh(shape, dtype, device, stream):
    """A new tensor for one call, made on the stream the kernels run on, so
    that its memory cannot still be in use by earlier work of another stream;
    also tied to the current stream, where the caller may use it before it is
    freed."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    if stream == current:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(current)
    return t


def _zero(tensors, stream):
    """Zeroes the tensors in one launch, on the stream the kernels run on."""
    if stream is None:
        torch._foreach_zero_(tensors)
    else:
        with torch.cuda.stream(stream):
            torch._foreach_zero_(tensors)


def _linattn_dims(q, v, g, lead):
    """(B, H, Hk, T, dk, dv, flags) of q [B,Hk,T,dk] and v [B,H,T,dv] (lead 2),
    or of a decode step's q [N,Hk,dk] and v [N,H,dv] (lead 1, T = 1)."""
    sq, sv = _dims(q, lead + 2, "q"), _dims(v, lead + 2, "v")
    H, Hk = sv[1], sq[1]
    if Hk < 1 or H % Hk:
        raise ValueError(f"q has {Hk} heads, which do not divide the {H} heads of v")
    return sv[0], H, Hk, sv[2] if lead == 2 else 1, sq[-1], sv[-1], DECAY_HEAD if g.dim() == 1 else 0


def linattn_workspace_size(B, H, T, dk, dv, dtype) -> int:
    code = dtype if isinstance(dtype, int) else _dtype_code(torch.empty(0, dtype=dtype))
    return int(lib().ckda_linattn_fwd_workspace_size(B, H, T, dk, dv, code))


def linattn_bwd_workspace_size(B, H, Hk, T, dk, dv, dtype) -> int:
    code = dtype if isinstance(dtype, int) else _dtype_code(torch.empty(0, dtype=dtype))
    return int(lib().ckda_linattn_bwd_workspace_size(B, H, Hk, T, dk, dv, code))


def linattn_fwd(q, k, v, g, h0=None, lens=None, workspace=None, o=None, hT=None, want_state=True, stream=None):
    """Linear attention with a decay for each head (ckda_linattn_fwd):
    H_t = exp(g_t) H_{t-1} + k_t v_t^T, o_t = H_t^T q_t.

    q, k [B,Hk,T,dk]; v [B,H,T,dv], Hk dividing H (head h uses query and key
    head h // (H / Hk)); g [B,H,T] log decays, or [H] constants; h0
    [B,H,dk,dv] fp32 or None; lens [B] int32 GPU tensor of sequence lengths or
    None.  Returns (o [B,H,T,dv], hT [B,H,dk,dv] fp32 or None).  Rows of o at
    or past a sequence's length are left as they were (zero if o is not given).
    `workspace` (uint8, linattn_workspace_size() bytes), `o` and `hT` may be
    passed in to avoid allocations; hT may be h0."""
    B, H, Hk, T, dk, dv, flags = _linattn_dims(q, v, g, 2)
    dev, dt, f32 = q.device, q.dtype, torch.float32
    _tensors(dev, [("q", q, (B, Hk, T, dk), dt), ("k", k, (B, Hk, T, dk), dt), ("v", v, (B, H, T, dv), dt),
                   ("g", g, (H,) if flags else (B, H, T), dt), ("h0", h0, (B, H, dk, dv), f32),
                   ("lens", lens, (B,), torch.int32), ("o", o, (B, H, T, dv), dt), ("hT", hT, (B, H, dk, dv), f32)])
    code = _dtype_code(q)
    L = lib()
    need = L.ckda_linattn_fwd_workspace_size(B, H, T, dk, dv, code)
    if need == 0:
        raise CkdaError(ERR_UNSUPPORTED, f"unsupported sizes B={B} H={H} T={T} dk={dk} dv={dv}")
    workspace, ws = _workspace_arg(workspace, need, dev, stream)
    if o is None:
        o = _fresh((B, H, T, dv), dt, dev, stream)
        if lens is not None:
            _zero([o], stream)
    if hT is None and want_state:
        hT = _fresh((B, H, dk, dv), f32, dev, stream)
    _run(dev, stream, L.ckda_linattn_fwd, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), _ptr(h0), _ptr(lens),
         o.data_ptr(), _ptr(hT), B, H, Hk, T, dk, dv, code, flags, *ws)
    return o, hT


def linattn_bwd(q, k, v, g, do, h0=None, dhT=None, lens=None, want_dh0=True, workspace=None, stream=None):
    """Backward of linattn_fwd (ckda_linattn_bwd): given do = dL/do [B,H,T,dv]
    and dhT = dL/dH_T [B,H,dk,dv] fp32 or None, returns (dq, dk, dv, dg, dh0 or
    None): dq, dk [B,Hk,T,dk], dv [B,H,T,dv] and dg (the shape of g, with
    respect to the log decays) in the inputs' dtype, dh0 fp32.  Rows at or past
    a sequence's length have zero gradients."""
    B, H, Hk, T, dk, dv, flags = _linattn_dims(q, v, g, 2)
    dev, dt, f32 = q.device, q.dtype, torch.float32
    _tensors(dev, [("q", q, (B, Hk, T, dk), dt), ("k", k, (B, Hk, T, dk), dt), ("v", v, (B, H, T, dv), dt),
                   ("g", g, (H,) if flags else (B, H, T), dt), ("do", do, (B, H, T, dv), dt),
                   ("h0", h0, (B, H, dk, dv), f32), ("dhT", dhT, (B, H, dk, dv), f32),
                   ("lens", lens, (B,), torch.int32)])
    code = _dtype_code(q)
    L = lib()
    need = L.ckda_linattn_bwd_workspace_size(B, H, Hk, T, dk, dv, code)
    if need == 0:
        raise CkdaError(ERR_UNSUPPORTED, f"unsupported sizes B={B} H={H} T={T} dk={dk} dv={dv}")
    workspace, ws = _workspace_arg(workspace, need, dev, stream)
    gq, gk = (_fresh((B, Hk, T, dk), dt, dev, stream) for _ in range(2))
    gv = _fresh((B, H, T, dv), dt, dev, stream)
    gg = _fresh(g.shape, dt, dev, stream)
    if lens is not None:
        _zero([gq, gk, gv, gg], stream)
    gh0 = _fresh((B, H, dk, dv), f32, dev, stream) if want_dh0 else None
    _run(dev, stream, L.ckda_linattn_bwd, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), _ptr(h0), _ptr(lens),
         do.data_ptr(), _ptr(dhT), gq.data_ptr(), gk.data_ptr(), gv.data_ptr(), gg.data_ptr(), _ptr(gh0), B, H, Hk, T, dk,
         dv, code, flags, *ws)
    return gq, gk, gv, gg, gh0


def linattn_decode_step(q, k, v, g, H, o=None, stream=None):
    """One token of linattn_fwd (ckda_linattn_decode_step): q, k [N,Hk,dk];
    v [N,Hh,dv]; g [N,Hh] or [Hh]; H [N,Hh,dk,dv] fp32 updated in place.
    Returns o [N,Hh,dv]."""
    N, Hh, Hk, _, dk, dv, flags = _linattn_dims(q, v, g, 1)
    dev, dt = q.device, q.dtype
    _tensors(dev, [("q", q, (N, Hk, dk), dt), ("k", k, (N, Hk, dk), dt), ("v", v, (N, Hh, dv), dt),
                   ("g", g, (Hh,) if flags else (N, Hh), dt), ("H", H, (N, Hh, dk, dv), torch.float32),
                   ("o", o, (N, Hh, dv), dt)])
    code = _dtype_code(q)
    if o is None:
        o = _fresh((N, Hh, dv), dt, dev, stream)
    _run(dev, stream, lib().ckda_linattn_decode_step, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(),
         H.data_ptr(), o.data_ptr(), N, Hh, Hk, dk, dv, code, flags)
    return o


_ACTS = {"silu": NORM_GATE_SILU, "sigmoid": NORM_GATE_SIGMOID}


def _norm_args(x, w, b, gate, act, rms):
    """(B, H, T, D, wheads, flags) of head_norm_fwd's arguments."""
    B, H, T, D = _dims(x, 4, "x")
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    wheads = None
    for name, t in (("w", w), ("b", b)):
        if t is not None:
            if t.dim() != 2 or t.shape[0] not in (1, H) or wheads not in (None, t.shape[0]):
                raise ValueError(f"{name} must be [H, D] or [1, D] (w and b alike), got shape {tuple(t.shape)}")
            wheads = t.shape[0]
    return B, H, T, D, 1 if wheads is None else wheads, (NORM_RMS if rms else 0) | (_ACTS[act] if gate is not None else 0)


def head_norm_fwd(x, w=None, b=None, gate=None, act="silu", rms=False, eps=1e-5, y=None, stream=None):
    """Norm of the attention's output rows with an output gate
    (ckda_head_norm_fwd): y = (n w + b) act(gate), n the layer norm of each row
    of x (rms: without the mean).

    x [B,H,T,D], head-major; gate [B,T,H,D], token-major, or None; w, b [H,D],
    or [1,D] for all heads, fp32, or None; act "silu" or "sigmoid" (of the
    gate).  Returns y [B,T,H,D], token-major."""
    B, H, T, D, wheads, flags = _norm_args(x, w, b, gate, act, rms)
    dev, dt, f32 = x.device, x.dtype, torch.float32
    _tensors(dev, [("x", x, (B, H, T, D), dt), ("gate", gate, (B, T, H, D), dt), ("w", w, (wheads, D), f32),
                   ("b", b, (wheads, D), f32), ("y", y, (B, T, H, D), dt)])
    code = _dtype_code(x)
    if y is None:
        y = _fresh((B, T, H, D), dt, dev, stream)
    _run(dev, stream, lib().ckda_head_norm_fwd, x.data_ptr(), _ptr(gate), _ptr(w), _ptr(b), y.data_ptr(), B, H, T, D,
         wheads, code, flags, eps)
    return y


def head_norm_bwd(x, dy, w=None, b=None, gate=None, act="silu", rms=False, eps=1e-5, workspace=None, stream=None):
    """Backward of head_norm_fwd (ckda_head_norm_bwd): given dy [B,T,H,D],
    returns (dx [B,H,T,D], dgate [B,T,H,D] or None, dw, db): dx and dgate in
    x's dtype, dw and db fp32 in the shape of w and b ([1,D] without either:
    the gradients at w = 1, b = 0)."""
    B, H, T, D, wheads, flags = _norm_args(x, w, b, gate, act, rms)
    dev, dt, f32 = x.device, x.dtype, torch.float32
    _tensors(dev, [("x", x, (B, H, T, D), dt), ("dy", dy, (B, T, H, D), dt), ("gate", gate, (B, T, H, D), dt),
                   ("w", w, (wheads, D), f32), ("b", b, (wheads, D), f32)])
    code = _dtype_code(x)
    L = lib()
    need = L.ckda_head_norm_bwd_workspace_size(B, H, T, D, wheads, code)
    if need == 0:
        raise CkdaError(ERR_UNSUPPORTED, f"unsupported sizes D={D}")
    workspace, ws = _workspace_arg(workspace, need, dev, stream)
    dx = _fresh((B, H, T, D), dt, dev, stream)
    dz = _fresh((B, T, H, D), dt, dev, stream) if gate is not None else None
    dw, db = (_fresh((wheads, D), f32, dev, stream) for _ in range(2))
    _run(dev, stream, L.ckda_head_norm_bwd, x.data_ptr(), _ptr(gate), _ptr(w), _ptr(b), dy.data_ptr(), dx.data_ptr(),
         _ptr(dz), dw.data_ptr(), db.data_ptr(), B, H, T, D, wheads, code, flags, eps, *ws)
    return dx, dz, dw, db


# ---------------------------------------------------------------- around the recurrence in a layer

def _like(t, stream):
    """_fresh in the shape and type of `t`, which is contiguous (0.5 us less than by shape, dtype and device)."""
    return torch.empty_like(t) if stream is None else _fresh(t.shape, t.dtype, t.device, stream)


def _beside(t, shape, stream):
    """_fresh in the type of `t`, on its device."""
    return t.new_empty(shape) if stream is None else _fresh(shape, t.dtype, t.device, stream)


def _slice_of(device, name, t, shape, dtype, rows, width):
    """Row stride of t, a column slice of a contiguous tensor: of `shape`, whose
    first `rows` dimensions count rows and whose others are `width` elements next
    to each other."""
    if t.shape == shape and t.dtype == dtype and t.get_device() == device.index:   # the usual ones first
        if t.is_contiguous():
            return width
        st = t.stride()
        ld = st[rows - 1]
        if (st[-1] == 1 and width <= ld <= INT_MAX and (rows == 1 or st[0] == ld * shape[1])
                and (len(st) == rows + 1 or st[-2] == shape[-1])):
            return ld
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.is_contiguous():
        return width
    inner = 1
    for size, stride in zip(reversed(t.shape[rows:]), reversed(t.stride()[rows:])):
        if size != 1 and stride != inner:
            raise ValueError(f"the columns of {name} must be contiguous")
        inner *= size
    ld = None
    count = 1   # rows below the dimension
    for size, stride in zip(reversed(t.shape[:rows]), reversed(t.stride()[:rows])):
        if size != 1:
            if ld is None and stride % count == 0:
                ld = stride // count
            if ld is None or stride != ld * count:
                raise ValueError(f"{name} must be a column slice of a contiguous tensor")
        count *= size
    ld = width if ld is None else ld
    if ld < width or ld > INT_MAX:
        raise ValueError(f"{name} must be a column slice of a contiguous tensor")
    return ld


def _conv_args(x, w, b, heads, act, lead):
    """(lead sizes, C, K, flags, Dh) of short_conv_fwd's arguments."""
    sx = _dims(x, lead + 1, "x")
    C, K = sx[-1], _dims(w, 2, "w")[1]
    if act not in (None, "silu"):
        raise ValueError(f"act must be None or 'silu', got {act!r}")
    if heads < 1 or C % heads:
        raise ValueError(f"{heads} heads do not divide the {C} channels of x")
    return sx[:lead], C, K, CONV_SILU if act else 0, C // heads


def short_conv_fwd(x, w, b=None, s0=None, lens=None, heads=1, act="silu", y=None, sT=None, want_state=True, stream=None):
    """Short causal convolution (ckda_short_conv_fwd): y_t = act(b + sum_j w_j
    x_{t-K+1+j}) for each channel, K = 2, 3 or 4.

    x [B,T,C], which may be a column slice of a wider projection; w [C,K] and b
    [C] fp32, b or None; s0 [B,K-1,C] the inputs before the first row, or None;
    lens [B] int32 GPU tensor of sequence lengths or None; act "silu" or None.
    Returns (y [B,heads,T,C/heads], the last inputs sT [B,K-1,C] or None).  Rows
    of y at or past a sequence's length are zero, or left as they were where y is
    passed in."""
    (B, T), C, K, flags, Dh = _conv_args(x, w, b, heads, act, 2)
    dev, dt, f32 = x.device, x.dtype, torch.float32
    _tensors(dev, [("w", w, (C, K), f32), ("b", b, (C,), f32), ("s0", s0, (B, K - 1, C), dt), ("lens", lens, (B,), torch.int32),
                   ("y", y, (B, heads, T, Dh), dt), ("sT", sT, (B, K - 1, C), dt)])
    ldx = _slice_of(dev, "x", x, (B, T, C), dt, 2, C)
    code = _dtype_code(x)
    if y is None:
        y = _beside(x, (B, heads, T, Dh), stream)
        flags |= PAD_ZERO
    if sT is None and want_state:
        sT = _beside(x, (B, K - 1, C), stream) if s0 is None else _like(s0, stream)
    _run(dev, stream, lib().ckda_short_conv_fwd, x.data_ptr(), w.data_ptr(), _ptr(b), _ptr(s0), _ptr(lens), y.data_ptr(),
         _ptr(sT), B, T, C, heads, K, ldx, code, flags)
    return y, sT


def short_conv_bwd(x, w, dy, b=None, s0=None, dsT=None, lens=None, act="silu", workspace=None, stream=None):
    """Backward of short_conv_fwd (ckda_short_conv_bwd): given dy
    [B,heads,T,C/heads] and dsT [B,K-1,C] or None, returns (dx [B,T,C], dw [C,K],
    db [C], ds0 [B,K-1,C]): dx and ds0 in x's dtype, dw and db fp32.  Rows at or
    past a sequence's length have zero gradients."""
    heads = _dims(dy, 4, "dy")[1]
    (B, T), C, K, flags, Dh = _conv_args(x, w, b, heads, act, 2)
    dev, dt, f32 = x.device, x.dtype, torch.float32
    _tensors(dev, [("w", w, (C, K), f32), ("b", b, (C,), f32), ("s0", s0, (B, K - 1, C), dt), ("lens", lens, (B,), torch.int32),
                   ("dy", dy, (B, heads, T, Dh), dt), ("dsT", dsT, (B, K - 1, C), dt)])
    ldx = _slice_of(dev, "x", x, (B, T, C), dt, 2, C)
    code = _dtype_code(x)
    L = lib()
    need = L.ckda_short_conv_bwd_workspace_size(B, T, C, K, code)
    if need == 0:
        raise CkdaError(ERR_UNSUPPORTED, f"unsupported sizes B={B} T={T} C={C} K={K}")
    workspace, ws = _workspace_arg(workspace, need, dev, stream)
    dx, ds0 = _beside(x, (B, T, C), stream), _beside(x, (B, K - 1, C), stream)
    dw, db = _like(w, stream), _beside(w, (C,), stream)
    _run(dev, stream, L.ckda_short_conv_bwd, x.data_ptr(), w.data_ptr(), _ptr(b), _ptr(s0), _ptr(lens), dy.data_ptr(),
         _ptr(dsT), dx.data_ptr(), dw.data_ptr(), db.data_ptr(), ds0.data_ptr(), B, T, C, heads, K, ldx, code,
         flags | PAD_ZERO, *ws)
    return dx, dw, db, ds0


def short_conv_decode_step(x, w, state, b=None, heads=1, act="silu", y=None, stream=None):
    """One token of short_conv_fwd (ckda_short_conv_decode_step): x [N,C], which
    may be a column slice; state [N,K-1,C] (the last inputs) updated in place.
    Returns y [N,heads,C/heads]."""
    (N,), C, K, flags, Dh = _conv_args(x, w, b, heads, act, 1)
    dev, dt, f32 = x.device, x.dtype, torch.float32
    _tensors(dev, [("w", w, (C, K), f32), ("b", b, (C,), f32), ("state", state, (N, K - 1, C), dt), ("y", y, (N, heads, Dh), dt)])
    ldx = _slice_of(dev, "x", x, (N, C), dt, 1, C)
    code = _dtype_code(x)
    if y is None:
        y = _beside(x, (N, heads, Dh), stream)
    _run(dev, stream, lib().ckda_short_conv_decode_step, x.data_ptr(), w.data_ptr(), _ptr(b), state.data_ptr(), y.data_ptr(),
         N, C, K, ldx, code, flags)
    return y


def selective_scan_workspace_size(B, T, C, G, N, dtype) -> int:
    code = dtype if isinstance(dtype, int) else _dtype_code(torch.empty(0, dtype=dtype))
    return int(lib().ckda_selective_scan_fwd_workspace_size(B, T, C, G, N, code))


def selective_scan_bwd_workspace_size(B, T, C, G, N, dtype) -> int:
    code = dtype if isinstance(dtype, int) else _dtype_code(torch.empty(0, dtype=dtype))
    return int(lib().ckda_selective_scan_bwd_workspace_size(B, T, C, G, N, code))


def _scan_args(x, dt, A, Bm, Cm, D, z, dt_bias, more, lead):
    """Checks of the selective scan's tensors; (lead sizes, C, G, N, ldbc, ldz)."""
    sx, sb = _dims(x, lead + 1, "x"), _dims(Bm, lead + 2, "Bm")
    rows, C, (G, N) = sx[:lead], sx[-1], sb[lead:]
    if G < 1 or C % G:
        raise ValueError(f"{G} groups of Bm do not divide the {C} channels of x")
    dev, t, f32 = x.device, x.dtype, torch.float32
    _tensors(dev, [("x", x, (*rows, C), t), ("dt", dt, (*rows, C), t), ("A", A, (C, N), f32), ("D", D, (C,), f32),
                   ("dt_bias", dt_bias, (C,), f32), *more(rows, C, N)])
    ldbc = _slice_of(dev, "Bm", Bm, (*rows, G, N), t, lead, G * N)
    if _slice_of(dev, "Cm", Cm, (*rows, G, N), t, lead, G * N) != ldbc:
        raise ValueError("Bm and Cm must have the same row stride")
    ldz = C if z is None else _slice_of(dev, "z", z, (*rows, C), t, lead, C)
    return rows, C, G, N, ldbc, ldz


def selective_scan_fwd(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, h0=None, lens=None, softplus=True, workspace=None,
                       y=None, hT=None, want_state=True, stream=None):
    """Selective scan (ckda_selective_scan_fwd): d = softplus(dt + dt_bias), h_t =
    exp(d A) h_{t-1} + d x_t B_t for each channel and state, y_t = (C_t . h_t + D
    x_t) silu(z_t).

    x, dt [B,T,C]; A [C,N] fp32; Bm, Cm [B,T,G,N] (G dividing C; N up to 64);
    D, dt_bias [C] fp32 or None; z [B,T,C] or None (no gate); h0 [B,C,N] fp32 or
    None; lens [B] int32 GPU tensor of sequence lengths or None; Bm, Cm and z may
    be column slices of a wider projection (Bm and Cm of the same).  Returns
    (y [B,T,C], hT [B,C,N] fp32 or None).  Rows of y at or past a sequence's length
    are zero, or left as they were where y is passed in.  hT may be h0."""
    f32 = torch.float32
    (B, T), C, G, N, ldbc, ldz = _scan_args(x, dt, A, Bm, Cm, D, z, dt_bias, lambda r, C, N: [
        ("h0", h0, (r[0], C, N), f32), ("lens", lens, (r[0],), torch.int32), ("y", y, (*r, C), x.dtype),
        ("hT", hT, (r[0], C, N), f32)], 2)
    dev, code, flags = x.device, _dtype_code(x), SCAN_SOFTPLUS if softplus else 0
    L = lib()
    need = L.ckda_selective_scan_fwd_workspace_size(B, T, C, G, N, code)
    if need == 0:
        raise CkdaError(ERR_UNSUPPORTED, f"unsupported sizes B={B} T={T} C={C} G={G} N={N}")
    workspace, ws = _workspace_arg(workspace, need, dev, stream)
    if y is None:
        y = _like(x, stream)
        flags |= PAD_ZERO
    if hT is None and want_state:
        hT = _beside(A, (B, C, N), stream) if h0 is None else _like(h0, stream)
    _run(dev, stream, L.ckda_selective_scan_fwd, x.data_ptr(), dt.data_ptr(), A.data_ptr(), Bm.data_ptr(), Cm.data_ptr(),
         _ptr(D), _ptr(z), _ptr(dt_bias), _ptr(h0), _ptr(lens), y.data_ptr(), _ptr(hT), B, T, C, G, N, ldbc, ldz, code,
         flags, *ws)
    return y, hT


def selective_scan_bwd(x, dt, A, Bm, Cm, dy, D=None, z=None, dt_bias=None, h0=None, dhT=None, lens=None, softplus=True,
                       want_dh0=True, workspace=None, stream=None):
    """Backward of selective_scan_fwd (ckda_selective_scan_bwd): given dy [B,T,C]
    and dhT [B,C,N] fp32 or None, returns (dx, ddt, dA, dBm, dCm, dD, dz or None,
    ddt_bias, dh0 or None): dx, ddt, dz [B,T,C] and dBm, dCm [B,T,G,N] in x's dtype,
    the others fp32 (dD and ddt_bias also where D and dt_bias are None: the
    gradients at zero).  Rows at or past a sequence's length have zero gradients."""
    f32 = torch.float32
    (B, T), C, G, N, ldbc, ldz = _scan_args(x, dt, A, Bm, Cm, D, z, dt_bias, lambda r, C, N: [
        ("h0", h0, (r[0], C, N), f32), ("lens", lens, (r[0],), torch.int32), ("dy", dy, (*r, C), x.dtype),
        ("dhT", dhT, (r[0], C, N), f32)], 2)
    dev, code = x.device, _dtype_code(x)
    L = lib()
    need = L.ckda_selective_scan_bwd_workspace_size(B, T, C, G, N, code)
    if need == 0:
        raise CkdaError(ERR_UNSUPPORTED, f"unsupported sizes B={B} T={T} C={C} G={G} N={N}")
    workspace, ws = _workspace_arg(workspace, need, dev, stream)
    dx, ddt, dA = _like(x, stream), _like(dt, stream), _like(A, stream)
    dz = None if z is None else _like(x, stream)
    dBm = _beside(x, (B, T, G, N), stream)
    dCm = _like(dBm, stream)
    dD = _beside(A, (C,), stream)
    dbias = _like(dD, stream)
    dh0 = _beside(A, (B, C, N), stream) if want_dh0 else None
    _run(dev, stream, L.ckda_selective_scan_bwd, x.data_ptr(), dt.data_ptr(), A.data_ptr(), Bm.data_ptr(), Cm.data_ptr(),
         _ptr(D), _ptr(z), _ptr(dt_bias), _ptr(h0), _ptr(lens), dy.data_ptr(), _ptr(dhT), dx.data_ptr(), ddt.data_ptr(),
         dA.data_ptr(), dBm.data_ptr(), dCm.data_ptr(), dD.data_ptr(), _ptr(dz), dbias.data_ptr(), _ptr(dh0), B, T, C, G, N,
         ldbc, ldz, code, (SCAN_SOFTPLUS if softplus else 0) | PAD_ZERO, *ws)
    return dx, ddt, dA, dBm, dCm, dD, dz, dbias, dh0


def selective_scan_decode_step(x, dt, A, Bm, Cm, H, D=None, z=None, dt_bias=None, softplus=True, y=None, stream=None):
    """One token of selective_scan_fwd (ckda_selective_scan_decode_step): x, dt, z
    [S,C]; Bm, Cm [S,G,N]; H [S,C,N] fp32 updated in place.  Returns y [S,C]."""
    (S,), C, G, N, ldbc, ldz = _scan_args(x, dt, A, Bm, Cm, D, z, dt_bias, lambda r, C, N: [
        ("H", H, (r[0], C, N), torch.float32), ("y", y, (r[0], C), x.dtype)], 1)
    dev, code = x.device, _dtype_code(x)
    if y is None:
        y = _like(x, stream)
    _run(dev, stream, lib().ckda_selective_scan_decode_step, x.data_ptr(), dt.data_ptr(), A.data_ptr(), Bm.data_ptr(),
         Cm.data_ptr(), _ptr(D), _ptr(z), _ptr(dt_bias), H.data_ptr(), y.data_ptr(), S, C, G, N, ldbc, ldz, code,
         SCAN_SOFTPLUS if softplus else 0)
    return y


def _add_norm_args(x, res, w, total, more=lambda shape, D: ()):
    """(rows, D, residual's dtype) of x [..., D] with a residual of the same shape."""
    shape, t = x.shape, x.dtype
    if len(shape) < 1 or shape[-1] < 1:
        raise ValueError(f"x must have rows of at least one element, got shape {tuple(shape)}")
    D = shape[-1]
    R = x.numel() // D
    if R > INT_MAX:
        raise ValueError(f"x has {R} rows (shape {tuple(shape)}), more than 2^31 - 1")
    rt = res.dtype if res is not None else t if total is None else total.dtype
    if rt != t and rt != torch.float32:
        raise TypeError(f"the residual must be {t} or float32, got {rt}")
    _tensors(x.device, [("x", x, shape, t), ("res", res, shape, rt), ("w", w, (D,), torch.float32), ("total", total, shape, rt),
                        *more(shape, D)])
    return R, D, rt


def add_norm_fwd(x, res=None, w=None, eps=1e-6, y=None, total=None, stream=None):
    """Root-mean-square norm with the residual's addition (ckda_add_norm_fwd): r =
    x + res, y = r / sqrt(mean r^2 + eps) w over the last dimension.

    x [...,D]; res of the same shape, in x's dtype or fp32, or None; w [D] fp32 or
    None.  Returns (y in x's dtype, r in the residual's dtype; None without res
    unless `total` is passed in).  total may be res."""
    R, D, rt = _add_norm_args(x, res, w, total, lambda shape, D: [("y", y, shape, x.dtype)])
    dev, code = x.device, _dtype_code(x)
    if y is None:
        y = _like(x, stream)
    if total is None and res is not None:
        total = _like(res, stream)
    _run(dev, stream, lib().ckda_add_norm_fwd, x.data_ptr(), _ptr(res), _ptr(w), y.data_ptr(), None, None, _ptr(total), R, D,
         0, code, DTYPE_BF16 if rt == torch.bfloat16 else DTYPE_F32, eps)
    return y, total


def add_norm_quant_fwd(x, res=None, w=None, eps=1e-6, group=128, q=None, scales=None, total=None, stream=None):
    """add_norm_fwd with its output in 8 bits: returns (q [...,D] float8_e4m3fn,
    scales [..., groups] fp32, r or None), where q scales stands for y: one scale
    for each 128 columns of a row (group=128; the last may have fewer) or for the
    whole row (group=0), max |y| / 448."""
    if group not in (0, 128):
        raise ValueError(f"group must be 128 or 0 (a row), got {group}")
    e4m3 = torch.float8_e4m3fn
    groups = lambda shape, D: (*shape[:-1], -(-D // group) if group else 1)  # noqa: E731
    R, D, rt = _add_norm_args(x, res, w, total, lambda shape, D: [("q", q, shape, e4m3), ("scales", scales, groups(shape, D), torch.float32)])
    dev, code = x.device, _dtype_code(x)
    if q is None:
        q = _fresh(x.shape, e4m3, dev, stream)
    if scales is None:
        scales = _fresh(groups(x.shape, D), torch.float32, dev, stream)
    if total is None and res is not None:
        total = _like(res, stream)
    _run(dev, stream, lib().ckda_add_norm_fwd, x.data_ptr(), _ptr(res), _ptr(w), None, q.data_ptr(), scales.data_ptr(),
         _ptr(total), R, D, group, code, DTYPE_BF16 if rt == torch.bfloat16 else DTYPE_F32, eps)
    return q, scales, total


def add_norm_bwd(total, dy, w=None, dsum=None, eps=1e-6, workspace=None, stream=None):
    """Backward of add_norm_fwd (ckda_add_norm_bwd) from its r (`total`), dy (x's
    dtype) and dsum (the gradient of r from what follows, in r's dtype, or None).
    Returns (dx in dy's dtype, dres in total's dtype, dw [D] fp32); where the dtypes
    are the same dx and dres are one tensor."""
    R, D, rt = _add_norm_args(dy, total, w, dsum)
    dev, code, L = dy.device, _dtype_code(dy), lib()
    rcode = DTYPE_BF16 if rt == torch.bfloat16 else DTYPE_F32
    need = L.ckda_add_norm_bwd_workspace_size(R, D, code, rcode)
    if need == 0:
        raise CkdaError(ERR_UNSUPPORTED, f"unsupported sizes D={D}")
    workspace, ws = _workspace_arg(workspace, need, dev, stream)
    dx, dw = _like(dy, stream), _fresh((D,), torch.float32, dev, stream)
    dres = dx if rt == dy.dtype else _like(total, stream)
    _run(dev, stream, L.ckda_add_norm_bwd, total.data_ptr(), _ptr(w), dy.data_ptr(), _ptr(dsum), dx.data_ptr(),
         None if dres is dx else dres.data_ptr(), dw.data_ptr(), R, D, code, rcode, eps, *ws)
    return dx, dres, dw
