"""The bounds of the decay gradient's tests reject what is wrong: each wrong
gradient below is planted in the fp64 one, on the CPU."""
import numpy as np
import pytest

from linattn_decay_cases import BF, F32, KINDS, SIZES, accepts, case, exact


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", SIZES[:3])
def test_wrong_gradients_are_rejected(size, kind, dtype):
    for state in (False, True):
        x = case(11, *size, dtype, kind, state=state)
        rows = exact(x)
        assert accepts(x, rows, rows) is None
        wrong = {"zero": 0 * rows, "sign": -rows, "shifted": np.roll(rows, 1, axis=2), "off by 2%": 1.02 * rows}
        if state:
            wrong["without dhT"] = exact({**x, "dhT": None})
        # a share of the neighbours' size in every row: what a difference of long sums leaves
        r = np.random.default_rng(1)
        wrong["noise"] = rows + 0.05 * np.sqrt((rows ** 2).mean(2, keepdims=True)) * r.standard_normal(rows.shape)
        for name, got in wrong.items():
            assert accepts(x, rows, got) is not None, (name, state)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", [-0.003, -0.3, -3.0, -10.0])
def test_wrong_gradients_of_constant_decays_are_rejected(kind, dtype):
    for size in SIZES[1:3]:
        x = case(12, *size, dtype, kind, decay="head")
        rows = exact(x)
        want = rows.sum((0, 2))
        assert accepts(x, rows, want) is None
        for name, got in {"zero": 0 * want, "sign": -want, "off by 10%": 1.1 * want}.items():
            assert accepts(x, rows, got) is not None, name


def test_a_reset_has_no_gradient():
    x = case(13, 1, 2, 1, 77, 32, 32, F32, "reset", state=True)
    rows = exact(x)
    bad = rows.copy()
    hit = np.isneginf(x["g"].numpy())
    assert hit.any() and (rows[hit] == 0).all()
    bad[hit] = 1e-9
    assert accepts(x, rows, bad) is not None
