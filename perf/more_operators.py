"""What stands around a recurrence in a layer: the norm with the residual's
addition, the short causal convolution, and the selective scan (a diagonal
recurrence whose decay differs for every channel and state).  Cases to measure,
their plain forms and their values in 64 bits.

`own` says which side `run` takes: the plain form (elementary torch operations
in 32 bits), or this repository's kernels through gated_delta_rule_ckda_amd."""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
EPS = 1e-6
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases

def _conv(name, op, B, H, T, C, K, dtype, silu, state, pad):
    return dict(name=name, op=op, B=B, H=H, T=T, C=C, K=K, dtype=dtype, silu=silu, state=state, pad=pad)


def _scan(name, op, B, T, C, G, N, dtype, gate, state, pad):
    return dict(name=name, op=op, B=B, T=T, C=C, G=G, N=N, dtype=dtype, gate=gate, state=state, pad=pad)


def _norm(name, op, R, D, dtype, res, group):
    return dict(name=name, op=op, R=R, D=D, dtype=dtype, res=res, group=group)


def listed():
    return [
        # the convolution before the queries of one user's short prompt, 16 heads of 128 channels: latency
        _conv("conv_fwd_prompt", "conv_fwd", 1, 16, 77, 2048, 4, BF16, True, True, False),
        # a training step's forward pass, at the sizes of the repository's own forward workload
        _conv("conv_fwd_train", "conv_fwd", 4, 16, 4096, 2048, 4, BF16, True, False, False),
        # its backward pass
        _conv("conv_bwd_train", "conv_bwd", 4, 16, 4096, 2048, 4, BF16, True, False, False),
        # a full serving batch's next tokens: 256 sequences of the repository's own decode workload's 32 x 128 channels
        _conv("conv_decode_batch", "conv_decode", 256, 32, 1, 4096, 4, BF16, True, True, False),
        # a training step's forward pass with the gate, one state vector of 16 for each of 2048 channels
        _scan("scan_fwd_train", "scan_fwd", 4, 4096, 2048, 1, 16, BF16, True, False, False),
        # one long document continued from a state: few channels, many tokens
        _scan("scan_fwd_long", "scan_fwd", 1, 32768, 1024, 1, 16, BF16, True, True, False),
        # a training step's backward pass
        _scan("scan_bwd_train", "scan_bwd", 4, 4096, 2048, 1, 16, BF16, True, False, False),
        # backward of a padded batch in full precision, odd sizes, two groups, states: truncated backpropagation
        _scan("scan_bwd_odd_f32", "scan_bwd", 3, 777, 500, 2, 16, F32, True, True, True),
        # a full serving batch's next tokens
        _scan("scan_decode_batch", "scan_decode", 256, 1, 4096, 1, 16, BF16, True, True, False),
        # a training step's norm ahead of a projection in 8 bits, one scale for 128 columns, residual in full precision
        _norm("norm_fwd_8bit", "norm_quant", 16384, 2048, BF16, F32, 128),
        # one user's next token: latency
        _norm("norm_fwd_one", "norm_fwd", 1, 2048, BF16, BF16, 0),
        # a training step's backward pass, the gradient of the residual stream carried in full precision
        _norm("norm_bwd_train", "norm_bwd", 16384, 2048, BF16, F32, 0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    kind = rng.choice(["conv", "conv", "scan", "scan", "norm"])
    dtype = rng.choice([BF16, BF16, F32])
    if kind == "norm":
        op = rng.choice(["norm_fwd", "norm_quant", "norm_bwd"])
        D = _log(rng, 64, 8192)
        R = min(_log(rng, 1, 32768), 33_000_000 // D)
        return dict(op=op, R=R, D=D, dtype=dtype, res=rng.choice([None, dtype, F32]) if op != "norm_bwd" else
                    rng.choice([dtype, F32]), group=rng.choice([0, 128]) if op == "norm_quant" else 0)
    if kind == "conv":
        op = rng.choice(["conv_fwd", "conv_fwd", "conv_bwd", "conv_bwd", "conv_decode"])
        H = rng.choice([1, 1, 4, 16, 24])
        C = H * rng.choice([16, 32, 64, 128, 128]) if H > 1 else _log(rng, 30, 6000)
        T = 1 if op == "conv_decode" else _log(rng, 1, 16384)
        B = _log(rng, 1, 256 if op == "conv_decode" else 8)
        B = max(1, min(B, 33_000_000 // (C * T)))
        T = min(T, 33_000_000 // C)
        return dict(op=op, B=B, H=H, T=T, C=C, K=rng.choice([2, 3, 4, 4]), dtype=dtype, silu=rng.random() < 0.7,
                    state=op == "conv_decode" or rng.random() < 0.5, pad=op != "conv_decode" and rng.random() < 0.4)
    op = rng.choice(["scan_fwd", "scan_fwd", "scan_bwd", "scan_bwd", "scan_decode"])
    G, N = rng.choice([1, 1, 2, 4]), rng.choice([8, 16, 16, 16, 32, 64])
    C = G * _log(rng, 20, 4096 // G)
    T = 1 if op == "scan_decode" else _log(rng, 1, 16384)
    B = _log(rng, 1, 256 if op == "scan_decode" else 8)
    most = 500_000_000 // N
    B = max(1, min(B, most // (C * T)))
    return dict(op=op, B=B, T=min(T, most // C), C=C, G=G, N=N, dtype=dtype, gate=rng.random() < 0.7,
                state=op == "scan_decode" or rng.random() < 0.5, pad=op != "scan_decode" and rng.random() < 0.4)


# ------------------------------------------------------------------ inputs

def _type(name):
    return {BF16: torch.bfloat16, F32: torch.float32, None: None}[name]


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = _type(case["dtype"])

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(shape, generator=gen, device=dev) * scale).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    s = dict(case=case)
    op = case["op"]
    if op.startswith("norm"):
        R, D = case["R"], case["D"]
        s["w"] = 1.0 + normal(D, scale=0.2, dtype=torch.float32)
        if op == "norm_bwd":
            s["sum"] = normal(R, D, dtype=_type(case["res"])) * 2
            s["dsum"] = normal(R, D, dtype=_type(case["res"]))
            s["dy"] = normal(R, D)
        else:
            s["x"] = normal(R, D)
            s["res"] = None if case["res"] is None else normal(R, D, dtype=_type(case["res"])) * 2
        return s
    B, T, C = case["B"], case["T"], case["C"]
    s["lens"] = None
    if case["pad"]:
        lens = torch.randint(0, T + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
        lens[0] = T   # the batch is padded to its longest sequence
        s["lens"] = lens
    if op.startswith("conv"):
        H, K = case["H"], case["K"]
        lead = (B,) if op == "conv_decode" else (B, T)
        s["x"] = normal(*lead, C)
        s["w"] = (uniform(C, K) * 2 - 1) / math.sqrt(K) * 1.7
        s["b"] = normal(C, scale=0.2, dtype=torch.float32)
        s["s0"] = normal(B, K - 1, C) if case["state"] else None
        if op == "conv_bwd":
            s["dy"] = normal(B, H, T, C // H)
            s["dsT"] = normal(B, K - 1, C) if case["state"] else None
        return s
    G, N = case["G"], case["N"]
    lead = (B,) if op == "scan_decode" else (B, T)
    s["x"] = normal(*lead, C, scale=0.7)
    # steps between 1e-3 and 1e-1 over the channels, spread by the token; the states' rates from 1 to N
    step = torch.exp(uniform(C) * math.log(100.0) + math.log(1e-3))
    s["bias"] = step + torch.log(-torch.expm1(-step))              # softplus(bias) = step
    s["dt"] = normal(*lead, C, scale=0.7)
    s["A"] = -torch.arange(1, N + 1, device=dev, dtype=torch.float32) * torch.exp(normal(C, N, scale=0.1, dtype=torch.float32))
    both = normal(*lead, 2 * G * N)                                # one projection's output, side by side
    s["Bm"] = both[..., :G * N].unflatten(-1, (G, N))
    s["Cm"] = both[..., G * N:].unflatten(-1, (G, N))
    s["D"] = 1.0 + normal(C, scale=0.2, dtype=torch.float32)
    s["z"] = normal(*lead, C) if case["gate"] else None
    if op == "scan_decode":
        s["H"] = normal(B, C, N, dtype=torch.float32, scale=0.5)
        return s
    s["h0"] = normal(B, C, N, dtype=torch.float32, scale=0.5) if case["state"] else None
    if op == "scan_bwd":
        s["dy"] = normal(B, T, C)
        s["dhT"] = normal(B, C, N, dtype=torch.float32, scale=0.5) if case["state"] else None
    return s


# ------------------------------------------------------------------ plain forms

def _inside(s):
    """[B,T,1]: which rows are part of their sequence, or None for all."""
    if s["lens"] is None:
        return None
    T = s["case"]["T"]
    return (torch.arange(T, device=s["lens"].device) < s["lens"].view(-1, 1)).unsqueeze(-1)


def _rows(inside, x):
    return x if inside is None else torch.where(inside, x, torch.zeros((), device=x.device, dtype=x.dtype))


def _silu(u):
    return u * torch.sigmoid(u)


def _silu_slope(u):
    g = torch.sigmoid(u)
    return g * (1 + u * (1 - g))


def _heads(x, H):
    return x.unflatten(-1, (H, -1)).transpose(1, 2).contiguous()


def _conv_rows(s):
    """The state's rows and the sequence's in float32, [B, K - 1 + T, C], and the rows of its end."""
    c = s["case"]
    x = _rows(_inside(s), s["x"].float())
    head = s["s0"].float() if s["s0"] is not None else x.new_zeros(c["B"], c["K"] - 1, c["C"])
    n = torch.full((c["B"],), c["T"], device=x.device) if s["lens"] is None else s["lens"].long()
    return torch.cat([head, x], 1), n.view(-1, 1, 1) + torch.arange(c["K"] - 1, device=x.device).view(1, -1, 1)


def _conv_sums(s, rows):
    c = s["case"]
    return s["b"] + sum(rows[:, j:j + c["T"]] * s["w"][:, j] for j in range(c["K"]))


def _plain_conv_fwd(s):
    c, dt = s["case"], s["x"].dtype
    rows, end = _conv_rows(s)
    u = _conv_sums(s, rows)
    y = _rows(_inside(s), _silu(u) if c["silu"] else u)
    return _heads(y.to(dt), c["H"]), rows.gather(1, end.expand(-1, -1, c["C"])).to(dt)


def _plain_conv_bwd(s):
    c, dt = s["case"], s["x"].dtype
    K, T = c["K"], c["T"]
    rows, end = _conv_rows(s)
    g = s["dy"].float().transpose(1, 2).flatten(2)
    if c["silu"]:
        g = g * _silu_slope(_conv_sums(s, rows))
    g = _rows(_inside(s), g)
    drows = sum(torch.nn.functional.pad(g * s["w"][:, j], (0, 0, j, K - 1 - j)) for j in range(K))
    if s["dsT"] is not None:
        drows.scatter_add_(1, end.expand(-1, -1, c["C"]), s["dsT"].float())
    dw = torch.stack([(g * rows[:, j:j + T]).sum((0, 1)) for j in range(K)], -1)
    out = [drows[:, K - 1:].to(dt), dw, g.sum((0, 1))]
    return out + [drows[:, :K - 1].to(dt)] if c["state"] else out


def _plain_conv_decode(s):
    c = s["case"]
    rows = torch.cat([s["s0"], s["x"].unsqueeze(1)], 1)
    u = s["b"] + (rows.float() * s["w"].t()).sum(1)
    s["s0"].copy_(rows[:, 1:])
    return (_silu(u) if c["silu"] else u).to(s["x"].dtype).unflatten(-1, (c["H"], -1)), s["s0"]


def _linear_scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dimension 1 from zero, and the running
    products of a: log2 T steps of twice the reach."""
    reach = 1
    while reach < a.shape[1]:
        b = torch.cat([b[:, :reach], torch.addcmul(b[:, reach:], a[:, reach:], b[:, :-reach])], 1)
        a = torch.cat([a[:, :reach], a[:, reach:] * a[:, :-reach]], 1)
        reach *= 2
    return b, a


def _steps(s):
    return torch.nn.functional.softplus(s["dt"].float() + s["bias"], threshold=1e9)


def _each(s, m):
    """[..., G, N] -> float32 [..., C, N]."""
    return m.float().repeat_interleave(s["case"]["C"] // s["case"]["G"], dim=-2)


def _plain_states(s, step, x):
    """Decays and states [B,T,C,N] and the state before each row."""
    a = torch.exp(step.unsqueeze(-1) * s["A"])
    inside = _inside(s)
    Bm = _rows(None if inside is None else inside.unsqueeze(-1), _each(s, s["Bm"]))
    h, products = _linear_scan(a, (step * x).unsqueeze(-1) * Bm)
    if s["h0"] is not None:
        h = torch.addcmul(h, products, s["h0"].unsqueeze(1))
    return a, h


def _plain_scan_fwd(s):
    inside = _inside(s)
    x, step = _rows(inside, s["x"].float()), _rows(inside, _steps(s))
    _, h = _plain_states(s, step, x)
    y = (h * _each(s, s["Cm"])).sum(-1) + s["D"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return _rows(inside, y).to(s["x"].dtype), h[:, -1].contiguous()


def _plain_scan_bwd(s):
    c, dt = s["case"], s["x"].dtype
    inside = _inside(s)
    wide = None if inside is None else inside.unsqueeze(-1)
    x, step = _rows(inside, s["x"].float()), _rows(inside, _steps(s))
    a, h = _plain_states(s, step, x)
    dy, Cm = s["dy"].float(), _rows(wide, _each(s, s["Cm"]))
    ds, dz = dy, None
    if s["z"] is not None:
        z = s["z"].float()
        dz = _rows(inside, dy * ((h * Cm).sum(-1) + s["D"] * x) * _silu_slope(z)).to(dt)
        ds = dy * _silu(z)
    ds = _rows(inside, ds)
    fold = lambda v: v.unflatten(2, (c["G"], -1)).sum(3).to(dt)  # noqa: E731
    dCm = fold(ds.unsqueeze(-1) * h)
    # R_t = a_{t+1} R_{t+1} + ds_t C_t, from the last row on
    last = torch.zeros_like(a[:, :1]) if s["dhT"] is None else s["dhT"].unsqueeze(1)
    later = torch.cat([torch.ones_like(last), a[:, 1:].flip(1)], 1)
    R, products = _linear_scan(later, (ds.unsqueeze(-1) * Cm).flip(1))
    R = torch.addcmul(R, products, last).flip(1)
    del products, later, Cm
    first = torch.zeros_like(h[:, :1]) if s["h0"] is None else s["h0"].unsqueeze(1)
    through = R * a * torch.cat([first, h[:, :-1]], 1)              # with respect to log a
    del h
    dBm = _rows(wide, fold(R * (step * x).unsqueeze(-1)))
    p = (R * _each(s, s["Bm"])).sum(-1)
    dx = _rows(inside, step * p + s["D"] * ds)
    dstep = x * p + (through * s["A"]).sum(-1)
    draw_ = _rows(inside, dstep * torch.sigmoid(s["dt"].float() + s["bias"]))
    dA = (through * step.unsqueeze(-1)).sum((0, 1))
    out = [dx.to(dt), draw_.to(dt), dA, dBm, dCm, (ds * x).sum((0, 1)), dz, draw_.sum((0, 1))]
    return out + [(a * R)[:, 0].contiguous()] if c["state"] else out


def _plain_scan_decode(s):
    x, step = s["x"].float(), _steps(s)
    H = s["H"]
    H.mul_(torch.exp(step.unsqueeze(-1) * s["A"])).add_((step * x).unsqueeze(-1) * _each(s, s["Bm"]))
    y = (H * _each(s, s["Cm"])).sum(-1) + s["D"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return y.to(s["x"].dtype), H


def _plain_norm_fwd(s):
    c = s["case"]
    r = s["x"].float()
    if s["res"] is not None:
        r = r + s["res"].float()
    y = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * s["w"]
    total = [] if s["res"] is None else [r.to(s["res"].dtype)]
    if c["op"] == "norm_fwd":
        return [y.to(s["x"].dtype)] + total
    D, n = c["D"], c["group"] or c["D"]
    groups = torch.nn.functional.pad(y, (0, -D % n)).unflatten(-1, (-1, n))
    scale = groups.abs().amax(-1, keepdim=True) / E4M3_MAX
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    codes = (groups / scale).flatten(-2)[..., :D].to(torch.float8_e4m3fn)
    return [codes.contiguous(), scale.squeeze(-1)] + total


def _plain_norm_bwd(s):
    r, dy = s["sum"].float(), s["dy"].float()
    inv = torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS)
    n = r * inv
    dn = dy * s["w"]
    dr = s["dsum"].float() + inv * (dn - n * (dn * n).mean(-1, keepdim=True))
    return [dr.to(s["dy"].dtype), dr.to(s["sum"].dtype), (dy * n).sum(0)]


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"conv_fwd": _plain_conv_fwd, "conv_bwd": _plain_conv_bwd, "conv_decode": _plain_conv_decode,
                "scan_fwd": _plain_scan_fwd, "scan_bwd": _plain_scan_bwd, "scan_decode": _plain_scan_decode,
                "norm_fwd": _plain_norm_fwd, "norm_quant": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd}[op](s)
    import gated_delta_rule_ckda_amd as ck
    if op.startswith("conv"):
        act = "silu" if c["silu"] else None
        if op == "conv_fwd":
            return ck.short_conv_fwd(s["x"], s["w"], s["b"], s["s0"], lens=s["lens"], heads=c["H"], act=act)
        if op == "conv_decode":
            return ck.short_conv_decode_step(s["x"], s["w"], s["s0"], s["b"], heads=c["H"], act=act), s["s0"]
        out = ck.short_conv_bwd(s["x"], s["w"], s["dy"], s["b"], s["s0"], s["dsT"], lens=s["lens"], act=act)
        return out if c["state"] else out[:3]
    if op == "scan_fwd":
        return ck.selective_scan_fwd(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], D=s["D"], z=s["z"], dt_bias=s["bias"],
                                     h0=s["h0"], lens=s["lens"])
    if op == "scan_decode":
        return ck.selective_scan_decode_step(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["H"], D=s["D"], z=s["z"],
                                             dt_bias=s["bias"]), s["H"]
    if op == "scan_bwd":
        out = ck.selective_scan_bwd(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["dy"], D=s["D"], z=s["z"],
                                    dt_bias=s["bias"], h0=s["h0"], dhT=s["dhT"], lens=s["lens"], want_dh0=c["state"])
        return out if c["state"] else out[:8]
    if op == "norm_bwd":
        return ck.add_norm_bwd(s["sum"], s["dy"], s["w"], dsum=s["dsum"], eps=EPS)
    if op == "norm_fwd":
        y, total = ck.add_norm_fwd(s["x"], s["res"], s["w"], eps=EPS)
        return [y] if total is None else [y, total]
    codes, scale, total = ck.add_norm_quant_fwd(s["x"], s["res"], s["w"], eps=EPS, group=c["group"])
    return [codes, scale] if total is None else [codes, scale, total]


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    es = 2 if case["dtype"] == BF16 else 4
    op = case["op"]
    if op.startswith("norm"):
        R, D = case["R"], case["D"]
        rs = {None: 0, BF16: 2, F32: 4}[case["res"]]
        if op == "norm_bwd":   # dy, sum, dsum; the gradient in both types
            return {"bytes": R * D * (2 * es + 3 * rs) + 8 * D, "flops": 10 * R * D}
        out = es if op == "norm_fwd" else 1
        scales = 0 if op == "norm_fwd" else 4 * R * (1 if not case["group"] else -(-D // case["group"]))
        return {"bytes": R * D * (es + 2 * rs + out) + 4 * D + scales, "flops": 6 * R * D}
    B, T, C = case["B"], case["T"], case["C"]
    # rows that count: a padded batch has one whole sequence, and the others have half its length in the mean
    rows = T * (B + 1) / 2 if case["pad"] else B * T
    lens = 4 * B if case["pad"] else 0
    if op.startswith("conv"):
        K = case["K"]
        state = B * (K - 1) * C * es
        weights = (K + 1) * C * 4
        act = 4 if case["silu"] else 0
        if op == "conv_bwd":
            return {"bytes": 3 * rows * C * es + 2 * weights + lens + (3 * state if case["state"] else 0),
                    "flops": (6 * K + 2 * act) * rows * C}
        return {"bytes": 2 * rows * C * es + weights + lens + (2 if case["state"] else 1) * state,
                "flops": (2 * K + act) * rows * C}
    G, N = case["G"], case["N"]
    each, shared, state = rows * C * es, rows * G * N * es, B * C * N * 4
    weights = (C * N + 2 * C) * 4
    gate = 1 if case["gate"] else 0
    if op == "scan_bwd":
        return {"bytes": (5 + 2 * gate) * each + 4 * shared + 2 * weights + lens + (3 * state if case["state"] else 0),
                "flops": 22 * rows * C * N}
    states = 2 if op == "scan_decode" or case["state"] else 1
    return {"bytes": (3 + gate) * each + 2 * shared + weights + lens + states * state, "flops": 7 * rows * C * N}


# ------------------------------------------------------------------ values in 64 bits

def exact(case, seed):
    op = case["op"]
    if case.get("T", 1) * (3 if op == "scan_bwd" else 1) > 60000:
        return None
    s = prepare(case, seed)
    w = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    if op.startswith("norm"):
        return _exact_norm(case, w)
    return _exact_conv(case, w) if op.startswith("conv") else _exact_scan(case, w)


def _exact_norm(c, w):
    if c["op"] == "norm_bwd":
        r, v = w["sum"].requires_grad_(), w["w"].requires_grad_()
        y = r / torch.sqrt((r * r).sum(-1, keepdim=True) / c["D"] + EPS) * v
        dr, dv = torch.autograd.grad(y, [r, v], w["dy"])
        dr = dr + w["dsum"]
        return [dr, dr, dv]
    r = w["x"] if w["res"] is None else w["x"] + w["res"]
    y = r / torch.sqrt((r * r).sum(-1, keepdim=True) / c["D"] + EPS) * w["w"]
    total = [] if w["res"] is None else [r]
    if c["op"] == "norm_fwd":
        return [y] + total
    n = c["group"] or c["D"]
    pieces = [y[:, i:i + n] for i in range(0, c["D"], n)]
    scales = [p.abs().max(-1).values / E4M3_MAX for p in pieces]
    return [torch.cat([p / q[:, None] for p, q in zip(pieces, scales)], 1), torch.stack(scales, 1)] + total


def _exact_conv(c, w):
    """Tap by tap from the definition, gradients by automatic differentiation in 64 bits."""
    B, H, T, C, K = c["B"], c["H"], c["T"], c["C"], c["K"]
    back = c["op"] == "conv_bwd"
    state = w["s0"] if w["s0"] is not None else torch.zeros(B, K - 1, C, dtype=torch.float64, device=w["x"].device)
    x = w["x"].view(B, T, C)
    lens = torch.full((B,), T, device=x.device) if w["lens"] is None else w["lens"].long()
    live = (torch.arange(T, device=x.device).view(1, T, 1) < lens.view(B, 1, 1)).double()
    leaves = [t.requires_grad_(back) for t in (x, w["w"], w["b"], state)]
    past = torch.cat([state, x * live], 1)
    u = w["b"].expand(B, T, C)
    for tap in range(K):
        u = u + w["w"][:, tap] * past[:, tap:T + tap]
    y = u / (1 + torch.exp(-u)) if c["silu"] else u
    y = (y * live).reshape(B, T, H, C // H).permute(0, 2, 1, 3)
    ends = torch.stack([past[i, int(lens[i]):int(lens[i]) + K - 1] for i in range(B)])
    if not back:
        return (y[:, :, 0], ends) if c["op"] == "conv_decode" else (y, ends)
    loss = (y * w["dy"]).sum() + ((ends * w["dsT"]).sum() if w["dsT"] is not None else 0)
    grads = list(torch.autograd.grad(loss, leaves))
    return grads if c["state"] else grads[:3]


def _exact_scan(c, w):
    """Row after row from the definition."""
    B, T, C, G, N = c["B"], c["T"], c["C"], c["G"], c["N"]
    step = torch.logaddexp(w["dt"] + w["bias"], torch.zeros((), dtype=torch.float64, device=w["dt"].device)).view(B, T, C)
    x, A, D = w["x"].view(B, T, C), w["A"], w["D"]
    z = None if w["z"] is None else w["z"].view(B, T, C)
    group = torch.arange(C, device=x.device) // (C // G)
    Bm, Cm = w["Bm"].reshape(B, T, G, N), w["Cm"].reshape(B, T, G, N)
    lens = torch.full((B,), T, device=x.device) if w["lens"] is None else w["lens"].long()
    live = torch.arange(T, device=x.device).view(1, T) < lens.view(B, 1)
    back = c["op"] == "scan_bwd"
    first = w["H"] if c["op"] == "scan_decode" else w["h0"]
    h = torch.zeros(B, C, N, dtype=torch.float64, device=x.device) if first is None else first
    start, kept, s = h, [], torch.zeros_like(x)
    for t in range(T):
        new = torch.exp(step[:, t, :, None] * A) * h + (step[:, t] * x[:, t])[..., None] * Bm[:, t, group]
        h = torch.where(live[:, t, None, None], new, h)
        s[:, t] = torch.einsum("bcn,bcn->bc", h, Cm[:, t, group])
        if back:
            kept.append(h)
    pre = s + D * x
    g = None if z is None else 1 / (1 + torch.exp(-z))
    on = live[..., None].double()
    if not back:
        y = (pre if z is None else pre * z * g) * on
        return (y[:, 0], h) if c["op"] == "scan_decode" else (y, h)
    dy = w["dy"]
    dz = None if z is None else dy * pre * g * (1 + z * (1 - g)) * on
    ds = (dy if z is None else dy * z * g) * on
    dx, dstep = D * ds, torch.zeros_like(x)
    dA, dB, dC = torch.zeros_like(A), torch.zeros_like(Bm), torch.zeros_like(Cm)
    R = torch.zeros_like(h) if w["dhT"] is None else w["dhT"]
    for t in range(T - 1, -1, -1):
        m = live[:, t, None, None]
        R = torch.where(m, R + ds[:, t, :, None] * Cm[:, t, group], R)
        dC[:, t] = (ds[:, t, :, None] * kept[t]).reshape(B, G, C // G, N).sum(2)
        active = torch.where(m, R, torch.zeros_like(R))
        dB[:, t] = (active * (step[:, t] * x[:, t])[..., None]).reshape(B, G, C // G, N).sum(2)
        p = (active * Bm[:, t, group]).sum(-1)
        dx[:, t] += step[:, t] * p
        back_one = torch.where(m, R * torch.exp(step[:, t, :, None] * A), R)
        q = torch.where(m, back_one, torch.zeros_like(R)) * (kept[t - 1] if t else start)
        dA += (q * step[:, t, :, None]).sum(0)
        dstep[:, t] = x[:, t] * p + (q * A).sum(-1)
        R = back_one
    ddt = dstep / (1 + torch.exp(-(w["dt"] + w["bias"])))
    out = [dx, ddt, dA, dB, dC, (ds * x).sum((0, 1)), dz, ddt.sum((0, 1))]
    return out + [R] if c["state"] else out
