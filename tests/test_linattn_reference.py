"""The fp64 reference of the linear attention and the head norm (used by the GPU
tests): its gradients against central differences of its forward, and the
chunk-free recurrence against the explicit sum over all pairs."""
import numpy as np
import pytest

import linattn_reference as ref


def _inputs(seed, B=2, H=4, Hk=2, T=9, dk=3, dv=5, head_decay=False):
    r = np.random.default_rng(seed)
    g = -r.exponential(0.5, (H,) if head_decay else (B, H, T))
    return dict(q=r.normal(size=(B, Hk, T, dk)), k=r.normal(size=(B, Hk, T, dk)), v=r.normal(size=(B, H, T, dv)), g=g,
                h0=r.normal(size=(B, H, dk, dv))), r.normal(size=(B, H, T, dv)), r.normal(size=(B, H, dk, dv))


def _loss(x, do, dhT, lens):
    o, hT = ref.linattn_fwd(x["q"], x["k"], x["v"], x["g"], x["h0"], lens)
    return (o * do).sum() + (hT * dhT).sum()


@pytest.mark.parametrize("head_decay", [False, True])
@pytest.mark.parametrize("lens", [None, [9, 4], [1, 0]])
def test_linattn_gradients_match_central_differences(head_decay, lens):
    x, do, dhT = _inputs(3, head_decay=head_decay)
    lens = None if lens is None else np.array(lens)
    got = ref.linattn_bwd(x["q"], x["k"], x["v"], x["g"], do, x["h0"], dhT, lens)
    r = np.random.default_rng(7)
    for name in x:
        d = r.normal(size=x[name].shape)
        step = 1e-5
        up, down = ({**x, name: x[name] + s * step * d} for s in (1, -1))
        slope = (_loss(up, do, dhT, lens) - _loss(down, do, dhT, lens)) / (2 * step)
        # truncation ~ step^2, rounding ~ 1e-16 |L| / step
        assert abs(slope - (got["d" + name] * d).sum()) <= 1e-6 * max(1.0, abs(slope)), name


def test_linattn_equals_the_sum_over_pairs():
    x, _, _ = _inputs(5, T=7)
    o, _ = ref.linattn_fwd(x["q"], x["k"], x["v"], x["g"], x["h0"])
    q, k = np.repeat(x["q"], 2, 1), np.repeat(x["k"], 2, 1)
    for t in range(7):
        want = np.einsum("bhi,bhij->bhj", q[:, :, t], x["h0"]) * np.exp(x["g"][:, :, :t + 1].sum(2))[..., None]
        for s in range(t + 1):
            c = np.exp(x["g"][:, :, s + 1:t + 1].sum(2)) * (q[:, :, t] * k[:, :, s]).sum(-1)
            want = want + c[..., None] * x["v"][:, :, s]
        assert np.allclose(o[:, :, t], want, rtol=1e-12, atol=1e-12)


def test_decay_gradient_is_the_running_sum_of_the_dots():
    """dg_t = <dhT, H_T> + sum_{u >= t} (q_u . dq_u - k_u . dk_u)."""
    x, do, dhT = _inputs(8)
    got = ref.linattn_bwd(x["q"], x["k"], x["v"], x["g"], do, x["h0"], dhT)
    run = (got["qdq"] - got["kdk"])[:, :, ::-1].cumsum(2)[:, :, ::-1] + got["flow"][..., None]
    assert np.allclose(run, got["dg"], rtol=1e-11, atol=1e-11)


def test_decode_steps_equal_the_forward():
    x, _, _ = _inputs(11, T=5)
    o, hT = ref.linattn_fwd(x["q"], x["k"], x["v"], x["g"], x["h0"])
    S = x["h0"]
    for t in range(5):
        ot, S = ref.linattn_decode(x["q"][:, :, t], x["k"][:, :, t], x["v"][:, :, t], x["g"][:, :, t], S)
        assert np.allclose(ot, o[:, :, t], rtol=1e-13, atol=1e-13)
    assert np.allclose(S, hT, rtol=1e-13, atol=1e-13)


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("act", [None, "silu", "sigmoid"])
def test_head_norm_gradients_match_central_differences(rms, act):
    r = np.random.default_rng(4)
    B, H, T, D = 2, 3, 4, 6
    x = dict(x=r.normal(size=(B, H, T, D)), w=r.normal(size=(H, D)), b=r.normal(size=(H, D)),
             gate=None if act is None else r.normal(size=(B, T, H, D)))
    dy = r.normal(size=(B, T, H, D))
    kw = dict(act=act or "silu", rms=rms, eps=1e-5)
    got = ref.head_norm(x["x"], x["w"], x["b"], x["gate"], dy=dy, **kw)
    for name, grad in (("x", "dx"), ("w", "dw"), ("b", "db"), ("gate", "dz")):
        if x[name] is None:
            continue
        d, step = r.normal(size=x[name].shape), 1e-5
        ys = [ref.head_norm(**{**x, name: x[name] + s * step * d}, **kw)["y"] for s in (1, -1)]
        slope = ((ys[0] - ys[1]) * dy).sum() / (2 * step)
        assert abs(slope - (got[grad] * d).sum()) <= 1e-6 * max(1.0, abs(slope)), name
