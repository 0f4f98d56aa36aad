"""The linear attention with a decay for each head, and the head norm that
follows it: cases to measure, their plain forms and their values in 64 bits.

`own` says which side `run` takes: the plain form (elementary torch operations
in 32 bits, decay sums and long sums in 64), or this repository's kernels
through gated_delta_rule_ckda_amd."""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
CHUNK = 64


# ------------------------------------------------------------------ cases

def _la(name, op, B, H, Hk, T, dk, dv, dtype, decay, state, pad):
    return dict(name=name, op=op, B=B, H=H, Hk=Hk, T=T, dk=dk, dv=dv, dtype=dtype, decay=decay, state=state, pad=pad)


def _norm(name, op, B, H, T, D, dtype, gate, rms, shared):
    return dict(name=name, op=op, B=B, H=H, T=T, D=D, dtype=dtype, gate=gate, rms=rms, shared=shared)


def listed():
    return [
        # one short prompt of one user: latency
        _la("fwd_prompt", "fwd", 1, 16, 16, 77, 128, 128, BF16, "token", False, False),
        # a training step's forward pass, at the sizes of the repository's own forward workload
        _la("fwd_train", "fwd", 4, 16, 16, 4096, 128, 128, BF16, "token", False, False),
        # one long document, keys and queries shared by groups of four heads: few heads, many tokens
        _la("fwd_long_grouped", "fwd", 1, 16, 4, 32768, 128, 128, BF16, "token", True, False),
        # a padded batch continued from earlier states in full precision, one constant decay for each head
        _la("fwd_padded_f32", "fwd", 3, 8, 8, 1000, 64, 128, F32, "head", True, True),
        # a training step's backward pass
        _la("bwd_train", "bwd", 4, 16, 16, 4096, 128, 128, BF16, "token", False, False),
        # backward of a padded batch with shared keys, constant decays and states: truncated backpropagation
        _la("bwd_grouped_odd", "bwd", 2, 12, 4, 777, 64, 128, BF16, "head", True, True),
        # backward in full precision
        _la("bwd_f32", "bwd", 1, 8, 8, 1023, 64, 64, F32, "token", False, False),
        # one user's next token: latency
        _la("decode_one", "decode", 1, 16, 16, 1, 128, 128, BF16, "token", True, False),
        # a full serving batch's next tokens, at the sizes of the repository's own decode workload
        _la("decode_batch", "decode", 256, 32, 32, 1, 128, 128, BF16, "token", True, False),
        # a training step's norm and output gate after the attention
        _norm("norm_fwd_train", "norm_fwd", 4, 16, 4096, 128, BF16, "silu", False, False),
        # its backward pass, as a root mean square norm with a sigmoid gate and one weight for all heads
        _norm("norm_bwd_train", "norm_bwd", 4, 16, 4096, 128, BF16, "sigmoid", True, True),
        # an ordinary layer norm over rows of an odd width in full precision, backward
        _norm("norm_bwd_odd_f32", "norm_bwd", 2, 1, 1000, 2047, F32, "none", False, False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "decode", "norm_fwd", "norm_bwd"])
    dtype = rng.choice([BF16, BF16, F32])
    if op in ("norm_fwd", "norm_bwd"):
        wide = rng.random() < 0.4
        H = 1 if wide else rng.randint(1, 32)
        D = _log(rng, 17, 8192) if wide else rng.choice([16, 32, 64, 128, 128])
        T = _log(rng, 1, 8192)
        B = _log(rng, 1, 8)
        B = max(1, min(B, 33_000_000 // (H * T * D)))
        T = min(T, 33_000_000 // (H * D))
        return dict(op=op, B=B, H=H, T=T, D=D, dtype=dtype, gate=rng.choice(["none", "silu", "sigmoid"]),
                    rms=rng.random() < 0.5, shared=rng.random() < 0.5)
    Hk = rng.choice([1, 2, 4, 8, 16])
    H = Hk * rng.choice([1, 1, 2, 3])
    dk, dv = rng.choice([16, 32, 64, 128]), rng.choice([16, 32, 64, 128, 128])
    decay = rng.choice(["token", "head"])
    if op == "decode":
        return dict(op=op, B=_log(rng, 1, 256), H=min(H, 32), Hk=min(H, 32) if H > 32 else Hk, T=1, dk=dk, dv=dv,
                    dtype=dtype, decay=decay, state=True, pad=False)
    T = _log(rng, 2 if op == "bwd" else 1, 16384)
    B = max(1, min(_log(rng, 1, 8), (262144 // (2 if dtype == F32 else 1)) // (H * T)))
    return dict(op=op, B=B, H=H, Hk=Hk, T=T, dk=dk, dv=dv, dtype=dtype, decay=decay, state=rng.random() < 0.5,
                pad=rng.random() < 0.4)


# ------------------------------------------------------------------ inputs

def _type(case):
    return torch.bfloat16 if case["dtype"] == BF16 else torch.float32


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = _type(case)

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(shape, generator=gen, device=dev) * scale).to(dtype)

    s = dict(case=case)
    B, H, T = case["B"], case["H"], case["T"]
    if case["op"] in ("norm_fwd", "norm_bwd"):
        D, Hw = case["D"], 1 if case["shared"] else H
        s["x"] = normal(B, H, T, D, scale=0.7) + normal(B, H, T, 1, scale=0.3)
        s["gate"] = normal(B, T, H, D) if case["gate"] != "none" else None
        s["w"] = 1.0 + normal(Hw, D, scale=0.2, dtype=torch.float32)
        s["b"] = normal(Hw, D, scale=0.2, dtype=torch.float32)
        if case["op"] == "norm_bwd":
            s["dy"] = normal(B, T, H, D)
        return s
    Hk, dk, dv = case["Hk"], case["dk"], case["dv"]
    if case["op"] == "decode":
        lead = (B,)
        tail = ()
    else:
        lead, tail = (B,), (T,)
    s["q"] = normal(*lead, Hk, *tail, dk, scale=dk ** -0.5)
    s["k"] = torch.nn.functional.normalize(normal(*lead, Hk, *tail, dk, dtype=torch.float32), dim=-1).to(dt)
    s["v"] = normal(*lead, H, *tail, dv)
    if case["decay"] == "head":
        # constant decays from 1 - 2^-2 to 1 - 2^-10 over the heads, jittered
        e = torch.linspace(2, 10, H, device=dev) + torch.rand(H, generator=gen, device=dev)
        s["g"] = torch.log1p(-torch.exp2(-e)).to(dt)
    else:
        # per-token log decays, log-normal around a memory of some 25 tokens: from hundreds of tokens to a few
        s["g"] = (-torch.exp(torch.randn((*lead, H, *tail), generator=gen, device=dev) * 1.2 - 3.2)).to(dt)
    if case["op"] == "decode":
        s["H"] = normal(B, H, dk, dv, dtype=torch.float32, scale=0.5)
        return s
    s["h0"] = normal(B, H, dk, dv, dtype=torch.float32, scale=0.5) if case["state"] else None
    s["lens"] = None
    if case["pad"]:
        lens = torch.randint(0, T + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
        lens[0] = T   # the batch is padded to its longest sequence
        s["lens"] = lens
    if case["op"] == "bwd":
        s["do"] = normal(B, H, T, dv)
        s["dhT"] = normal(B, H, dk, dv, dtype=torch.float32, scale=0.5) if case["state"] else None
    return s


# ------------------------------------------------------------------ plain forms

def _chunked(q, k, v, g, h0):
    """o_t = H_t^T q_t, H_t = exp(g_t) H_{t-1} + k_t v_t^T over chunks; q, k, v
    float32 [B,H,T,.], g float64 [B,H,T].  Returns (o, final state)."""
    B, H, T, dk = q.shape
    dv, n = v.shape[-1], max(1, -(-T // CHUNK))
    pad = n * CHUNK - T
    q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, pad)).view(B, H, n, CHUNK, -1) for x in (q, k, v))
    c = torch.nn.functional.pad(g.clamp(min=-1e4), (0, pad)).view(B, H, n, CHUNK).cumsum(-1)
    causal = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    G = torch.exp((c.unsqueeze(-1) - c.unsqueeze(-2)).masked_fill(~causal, -math.inf)).float()
    o = ((q @ k.transpose(-1, -2)) * G) @ v
    total = c[..., -1]                                             # log decay of a whole chunk
    own_state = (k * torch.exp(total.unsqueeze(-1) - c).float().unsqueeze(-1)).transpose(-1, -2) @ v
    # state before chunk i: sum over j < i of the chunks' own states, decayed by chunks j + 1 .. i - 1, and h0
    e = torch.nn.functional.pad(total.cumsum(-1), (1, 0))          # log decay before chunk i, i = 0 .. n
    earlier = torch.ones(n + 1, n, dtype=torch.bool, device=q.device).tril(-1)
    M = torch.exp((e.unsqueeze(-1) - e[..., 1:].unsqueeze(-2)).masked_fill(~earlier, -math.inf)).float()
    states = (M @ own_state.view(B, H, n, dk * dv)).view(B, H, n + 1, dk, dv)
    if h0 is not None:
        states = states + torch.exp(e).float()[..., None, None] * h0.unsqueeze(2)
    o = o + torch.exp(c).float().unsqueeze(-1) * (q @ states[:, :, :-1])
    return o.reshape(B, H, n * CHUNK, dv)[:, :, :T], states[:, :, -1]


def _rows(s, x):
    """x in float32 with the rows behind each sequence's length zeroed."""
    x = x.float()
    if s["lens"] is None:
        return x
    T = x.shape[2]
    inside = torch.arange(T, device=x.device) < s["lens"].view(-1, 1)
    inside = inside.view(x.shape[0], 1, T, *([1] * (x.dim() - 3)))
    return torch.where(inside, x, torch.zeros((), device=x.device))


def _decays(s):
    """Log decays in float64, [B,H,T], 0 behind each sequence's length."""
    c = s["case"]
    g = s["g"]
    if c["decay"] == "head":
        g = g.view(1, -1, 1).expand(c["B"], -1, c["T"])
    return _rows(s, g).double()


def _heads(s, x):
    return x.repeat_interleave(s["case"]["H"] // s["case"]["Hk"], dim=1)


def _plain_fwd(s):
    q, k, v = _heads(s, _rows(s, s["q"])), _heads(s, _rows(s, s["k"])), _rows(s, s["v"])
    o, hT = _chunked(q, k, v, _decays(s), s["h0"])
    return _rows(s, o).to(s["q"].dtype), hT


def _plain_bwd(s):
    c, dt = s["case"], s["q"].dtype
    B, H, Hk, T = c["B"], c["H"], c["Hk"], c["T"]
    q, k, v, do = _heads(s, _rows(s, s["q"])), _heads(s, _rows(s, s["k"])), _rows(s, s["v"]), _rows(s, s["do"])
    g = _decays(s)
    turn = lambda x: None if x is None else x.transpose(-1, -2)  # noqa: E731
    dq, hT = _chunked(do, v, k, g, turn(s["h0"]))
    back = lambda x: x.flip(2)  # noqa: E731
    later = back(torch.nn.functional.pad(g[:, :, 1:], (0, 1)))     # decay between a token and the next one
    dk, _ = _chunked(back(v), back(do), back(q), later, turn(s["dhT"]))
    dv, R1 = _chunked(back(k), back(q), back(do), later, s["dhT"])
    dk, dv = back(dk), back(dv)
    dh0 = torch.exp(g[:, :, 0]).float()[..., None, None] * R1
    # what passes gate t: queries from t on, less keys from t on, and the final state
    flow = (q.double() * dq.double()).sum(-1) - (k.double() * dk.double()).sum(-1)
    dg = flow.flip(2).cumsum(2).flip(2)
    if s["dhT"] is not None:
        dg = dg + (s["dhT"].double() * turn(hT).double()).sum((-1, -2)).unsqueeze(-1)
    dg = _masked64(s, dg)
    if c["decay"] == "head":
        dg = dg.sum((0, 2))
    fold = lambda x: _rows(s, x).view(B, Hk, H // Hk, T, -1).sum(2).to(dt)  # noqa: E731
    out = [fold(dq), fold(dk), _rows(s, dv).to(dt), dg.to(dt)]
    return out + [dh0] if c["state"] else out


def _masked64(s, x):
    if s["lens"] is None:
        return x
    inside = torch.arange(x.shape[2], device=x.device) < s["lens"].view(-1, 1)
    return torch.where(inside.unsqueeze(1), x, torch.zeros((), device=x.device, dtype=x.dtype))


def _plain_decode(s):
    c = s["case"]
    r = c["H"] // c["Hk"]
    q, k, v = (x.float() for x in (s["q"].repeat_interleave(r, 1), s["k"].repeat_interleave(r, 1), s["v"]))
    a = torch.exp(s["g"].float())
    H = s["H"]
    H.mul_(a[..., None, None]).add_(k.unsqueeze(-1) * v.unsqueeze(-2))
    return (q.unsqueeze(-2) @ H).squeeze(-2).to(s["q"].dtype), H


def _act(z, gate):
    sg = torch.sigmoid(z)
    return z * sg if gate == "silu" else sg


def _act_slope(z, gate):
    sg = torch.sigmoid(z)
    return sg * (1 + z * (1 - sg)) if gate == "silu" else sg * (1 - sg)


EPS = 1e-5


def _normed(x, rms):
    """(n, 1 / deviation) of the rows of x in float32."""
    m = 0.0 if rms else x.mean(-1, keepdim=True)
    r = torch.rsqrt(((x - m) ** 2).mean(-1, keepdim=True) + EPS)
    return (x - m) * r, r


def _plain_norm_fwd(s):
    c = s["case"]
    n, _ = _normed(s["x"].float().transpose(1, 2), c["rms"])
    y = n * s["w"] + s["b"]
    if s["gate"] is not None:
        y = y * _act(s["gate"].float(), c["gate"])
    return y.to(s["x"].dtype).contiguous()


def _plain_norm_bwd(s):
    c, dt = s["case"], s["x"].dtype
    n, r = _normed(s["x"].float().transpose(1, 2), c["rms"])
    dy = s["dy"].float()
    out = []
    if s["gate"] is not None:
        z = s["gate"].float()
        out = [(dy * (n * s["w"] + s["b"]) * _act_slope(z, c["gate"])).to(dt)]
        dy = dy * _act(z, c["gate"])
    dn = dy * s["w"]
    dx = dn - n * (dn * n).mean(-1, keepdim=True)
    if not c["rms"]:
        dx = dx - dn.mean(-1, keepdim=True)
    over = (0, 1, 2) if c["shared"] else (0, 1)
    dw, db = (dy * n).sum(over), dy.sum(over)
    if c["shared"]:
        dw, db = dw.unsqueeze(0), db.unsqueeze(0)
    return [(dx * r).to(dt).transpose(1, 2).contiguous()] + out + [dw, db]


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"fwd": _plain_fwd, "bwd": _plain_bwd, "decode": _plain_decode, "norm_fwd": _plain_norm_fwd,
                "norm_bwd": _plain_norm_bwd}[op](s)
    import gated_delta_rule_ckda_amd as ck
    if op == "fwd":
        return ck.linattn_fwd(s["q"], s["k"], s["v"], s["g"], s["h0"], lens=s["lens"])
    if op == "bwd":
        out = ck.linattn_bwd(s["q"], s["k"], s["v"], s["g"], s["do"], s["h0"], s["dhT"], lens=s["lens"],
                             want_dh0=c["state"])
        return out if c["state"] else out[:4]
    if op == "decode":
        return ck.linattn_decode_step(s["q"], s["k"], s["v"], s["g"], s["H"]), s["H"]
    kw = dict(gate=s["gate"], act="silu" if c["gate"] == "none" else c["gate"], rms=c["rms"], eps=EPS)
    if op == "norm_fwd":
        return ck.head_norm_fwd(s["x"], s["w"], s["b"], **kw)
    dx, dgate, dw, db = ck.head_norm_bwd(s["x"], s["dy"], s["w"], s["b"], **kw)
    return [dx, dw, db] if dgate is None else [dx, dgate, dw, db]


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    es = 2 if case["dtype"] == BF16 else 4
    B, H, T = case["B"], case["H"], case["T"]
    if case["op"] in ("norm_fwd", "norm_bwd"):
        D = case["D"]
        n = B * H * T * D
        back = case["op"] == "norm_bwd"
        tensors = (3 if back else 2) + (0 if case["gate"] == "none" else 2 if back else 1)
        weights = (4 if back else 2) * (1 if case["shared"] else H) * D * 4
        return {"bytes": tensors * n * es + weights, "flops": (24 if back else 10) * n}
    Hk, dk, dv = case["Hk"], case["dk"], case["dv"]
    # rows that count: a padded batch has one whole sequence, and the others have half its length in the mean
    tokens = T * (B + 1) / 2 if case["pad"] else B * T
    shared, each = tokens * Hk * dk * es, tokens * H * dv * es     # one of q, k; one of v, o
    decays = (H if case["decay"] == "head" else tokens * H) * es
    state = B * H * dk * dv * 4
    lens = 4 * B if case["pad"] else 0
    if case["op"] == "fwd":
        return {"bytes": 2 * shared + 2 * each + decays + lens + (2 if case["state"] else 1) * state,
                "flops": 4 * tokens * H * dk * dv}
    if case["op"] == "decode":
        return {"bytes": 2 * shared + 2 * each + decays + 2 * state, "flops": 5 * tokens * H * dk * dv}
    return {"bytes": 4 * shared + 3 * each + 2 * decays + lens + (3 if case["state"] else 0) * state,
            "flops": 12 * tokens * H * dk * dv}


# ------------------------------------------------------------------ values in 64 bits

def exact(case, seed):
    if case["T"] * (3 if case["op"] == "bwd" else 1) > 40000:
        return None
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        return _exact_norm(case, s)
    r = case["H"] // case["Hk"]
    wide = lambda x: torch.cat([x[:, i // r:i // r + 1] for i in range(case["H"])], 1).double()  # noqa: E731
    q, k, v = wide(s["q"]), wide(s["k"]), s["v"].double()
    if op == "decode":
        a = torch.exp(s["g"].double())
        a = a.view(1, -1, 1, 1) if case["decay"] == "head" else a[:, :, None, None]
        H = a * s["H"].double() + k[:, :, :, None] * v[:, :, None, :]
        return (q[:, :, :, None] * H).sum(2), H
    return _exact_fwd(case, s, q, k, v) if op == "fwd" else _exact_bwd(case, s, q, k, v)


def _exact_setup(case, s, q, v):
    """Per-token decays [B,H,T,1,1], the running state, and which rows count [B,T]."""
    B, H, T = case["B"], case["H"], case["T"]
    a = torch.exp(s["g"].double())
    a = a.view(1, H, 1).expand(B, H, T) if case["decay"] == "head" else a
    lens = torch.full((B,), T, device=q.device) if s["lens"] is None else s["lens"]
    live = torch.arange(T, device=q.device).view(1, T) < lens.view(B, 1)
    a = torch.where(live.view(B, 1, T), a, torch.ones_like(a))
    h0 = s["h0"].double() if s["h0"] is not None else q.new_zeros(B, H, case["dk"], case["dv"])
    return a.view(B, H, T, 1, 1), h0, live.view(B, 1, T, 1)


def _exact_fwd(case, s, q, k, v):
    a, H, live = _exact_setup(case, s, q, v)
    k = torch.where(live, k, torch.zeros_like(k))
    o = torch.zeros_like(v)
    for t in range(case["T"]):
        H = torch.addcmul(a[:, :, t] * H, k[:, :, t, :, None], v[:, :, t, None, :])
        o[:, :, t] = torch.matmul(q[:, :, t, None, :], H)[:, :, 0]
    return torch.where(live, o, torch.zeros_like(o)), H


def _exact_bwd(case, s, q, k, v):
    T, step = case["T"], 64
    a, H, live = _exact_setup(case, s, q, v)
    zero = lambda x: torch.where(live, x, torch.zeros_like(x))  # noqa: E731
    q, k, v, do = zero(q), zero(k), zero(v), zero(s["do"].double())
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg = q.new_zeros(q.shape[:3])
    kept = []                                       # the state before every 64th token
    for t in range(T):
        if t % step == 0:
            kept.append(H)
        H = torch.addcmul(a[:, :, t] * H, k[:, :, t, :, None], v[:, :, t, None, :])
        dq[:, :, t] = torch.matmul(H, do[:, :, t, :, None])[..., 0]
    R = s["dhT"].double() if s["dhT"] is not None else torch.zeros_like(H)   # dL/dH_t from later tokens
    for first in range((T - 1) // step * step, -1, -step):
        before = [kept.pop()]
        for t in range(first, min(T, first + step) - 1):
            before.append(torch.addcmul(a[:, :, t] * before[-1], k[:, :, t, :, None], v[:, :, t, None, :]))
        for t in range(min(T, first + step) - 1, first - 1, -1):
            R = torch.addcmul(R, q[:, :, t, :, None], do[:, :, t, None, :])
            dk[:, :, t] = torch.matmul(R, v[:, :, t, :, None])[..., 0]
            dv[:, :, t] = torch.matmul(k[:, :, t, None, :], R)[:, :, 0]
            R = a[:, :, t] * R                      # dL/dH_{t-1}: with respect to log a, <R, H_{t-1}>
            dg[:, :, t] = (R * before.pop()).sum((-1, -2))
    dg = torch.where(live[..., 0], dg, torch.zeros_like(dg))
    B, H_, Hk = case["B"], case["H"], case["Hk"]
    dq, dk = (zero(x).view(B, Hk, H_ // Hk, T, -1).sum(2) for x in (dq, dk))
    out = [dq, dk, dv, dg.sum((0, 2)) if case["decay"] == "head" else dg]
    return out + [R] if case["state"] else out


def _exact_norm(case, s):
    """From the definition, with gradients by automatic differentiation in 64 bits."""
    back = case["op"] == "norm_bwd"
    x = s["x"].double().requires_grad_(back)
    w, b = s["w"].double().requires_grad_(back), s["b"].double().requires_grad_(back)
    z = None if s["gate"] is None else s["gate"].double().requires_grad_(back)
    u = x.permute(0, 2, 1, 3)
    if not case["rms"]:
        u = u - u.sum(-1, keepdim=True) / case["D"]
    y = u / torch.sqrt((u * u).sum(-1, keepdim=True) / case["D"] + EPS) * w + b
    if z is not None:
        y = y / (1 + torch.exp(-z)) * (z if case["gate"] == "silu" else 1.0)
    if not back:
        return y
    wanted = [x, w, b] if z is None else [x, z, w, b]
    return list(torch.autograd.grad(y, wanted, s["dy"].double()))
