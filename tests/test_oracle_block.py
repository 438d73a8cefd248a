"""The float64 forms of the block's operators: closed cases, and gradients
against central differences (bars as in test_oracle_tower)."""
import numpy as np
import pytest

from oracle import tower
from test_oracle_tower import _differences, _near


@pytest.mark.parametrize("weighted", [False, True])
def test_rms_norm_gradients_against_differences(weighted):
    rng = np.random.default_rng(3)
    h, dout, dres = (rng.normal(size=(4, 7)) for _ in range(3))
    w = 1 + 0.3 * rng.normal(size=7) if weighted else None

    def loss():
        return float((tower.rms_norm(h, w, 1e-3)["out"] * dout).sum() + (h * dres).sum())

    r = tower.rms_norm(h, w, 1e-3, dout, dres)
    _near(r["dx"], _differences(loss, h))
    if weighted:
        _near(r["dweight"], _differences(loss, w))


def test_rms_norm_closed_cases():
    h = np.array([[3.0, -4.0, 0.0, 0.0], [2.0, 2.0, 2.0, -2.0]])
    r = tower.rms_norm(h, np.array([1.0, 2.0, 3.0, 4.0]), 0.0)
    assert np.allclose(r["rstd"], [0.4, 0.5]) and np.allclose(r["out"], [[1.2, -3.2, 0, 0], [1, 2, 3, -4]])
    q, s = tower.rms_norm_quantized(h, None, 0.0)
    # 1.2 / 1.6 * 127 = 95.25
    assert q.tolist() == [[95, -127, 0, 0], [127, 127, 127, -127]] and np.allclose(s, [1.6 / 127, 1 / 127])
    q, s = tower.rms_norm_quantized(np.zeros((1, 5)), None, 1e-6)
    assert not q.any() and s[0] == 0


def test_residual_sums_are_rounded_to_their_type():
    x, res = np.array([[1.0, 2.0 ** -9, 3 * 2.0 ** -9]]), np.array([[2.0 ** -30, 1.0, 1.0]])
    assert tower.residual_sum(x, res, "f32").tolist() == [[1.0, 1 + 2.0 ** -9, 1 + 3 * 2.0 ** -9]]
    # bf16 holds 1 and 1 + 2^-7: 1 + 2^-9 is nearer to the first, 1 + 3 2^-9 to the second; a tie goes to even
    assert tower.residual_sum(x, res, "bf16").tolist() == [[1.0, 1.0, 1 + 2.0 ** -7]]
    tie = tower.residual_sum(np.array([[2.0 ** -8, 3 * 2.0 ** -8]]), np.ones((1, 2)), "bf16")
    assert tie.tolist() == [[1.0, 1 + 2.0 ** -6]]


def test_rotation():
    rng = np.random.default_rng(4)
    x, dout = rng.normal(size=(5, 3, 8)), rng.normal(size=(5, 3, 8))
    angle = rng.normal(size=(5, 4)) * 10
    c, s = np.cos(angle), np.sin(angle)
    out, mag = tower.rotate_heads(x, c, s)
    # lengths of the pairs stay, the inverse undoes it, and it is the gradient
    assert np.allclose(out[..., :4] ** 2 + out[..., 4:] ** 2, x[..., :4] ** 2 + x[..., 4:] ** 2)
    assert np.allclose(tower.rotate_heads(out, c, s, True)[0], x) and (mag >= np.abs(out) - 1e-15).all()
    _near(tower.rotate_heads(dout, c, s, True)[0], _differences(lambda: float((tower.rotate_heads(x, c, s)[0] * dout).sum()), x))
    # a quarter turn takes (a, b) to (-b, a)
    quarter = tower.rotate_heads(x, np.zeros((5, 4)), np.ones((5, 4)))[0]
    assert np.allclose(quarter, np.concatenate((-x[..., 4:], x[..., :4]), axis=2))


@pytest.mark.parametrize("bias", [False, True])
def test_mlp_gradients_against_differences(bias):
    rng = np.random.default_rng(5)
    x, wg, wu, wd = (rng.normal(size=s) for s in ((4, 3), (5, 3), (5, 3), (3, 5)))
    b = [rng.normal(size=n) for n in (5, 5, 3)] if bias else [None] * 3
    dout = rng.normal(size=x.shape)

    def loss():
        return float((tower.gated_mlp(x, wg, wu, wd, *b)["out"] * dout).sum())

    r = tower.gated_mlp(x, wg, wu, wd, *b, dout)
    names = [("dx", x), ("dw_gate", wg), ("dw_up", wu), ("dw_down", wd)] + list(zip(("db_gate", "db_up", "db_down"), b))
    for name, t in names:
        if t is not None:
            _near(r[name], _differences(loss, t))


def test_mlp_closed_cases():
    one = np.ones((1, 1))
    # silu(0) = 0; silu(1) = 1 / (1 + 1 / e); far gates are the value itself, or nothing
    for g, silu in ((0.0, 0.0), (1.0, 1 / (1 + np.exp(-1.0))), (900.0, 900.0), (-900.0, 0.0)):
        r = tower.gated_mlp(g * one, one, 2 * one, 3 * one, dout=one)
        assert np.allclose(r["out"], 3 * silu * 2 * g) and np.isfinite(r["dx"]).all()
