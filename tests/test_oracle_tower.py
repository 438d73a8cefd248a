"""The float64 forms of the vision tower's operators: closed cases, and
gradients against central differences.

A central difference of step t has a truncation error of t^2 / 6 times the
third derivative and a rounding error of about 2^-52 |f| / t; with t = 2^-17
and sums of order 10 both are below 1e-9, against a bar of 1e-7 of the
gradient's largest entry plus 1e-8."""
import numpy as np
import pytest

from oracle import tower

T = 2.0 ** -17


def _differences(f, x):
    g = np.zeros_like(x)
    flat, out = x.reshape(-1), g.reshape(-1)
    for i in range(flat.size):
        keep = flat[i]
        flat[i] = keep + T
        hi = f()
        flat[i] = keep - T
        lo = f()
        flat[i] = keep
        out[i] = (hi - lo) / (2 * T)
    return g


def _near(got, want):
    assert np.abs(got - want).max() <= 1e-7 * np.abs(want).max() + 1e-8


@pytest.mark.parametrize("window,use_sink", [(-1, False), (-1, True), (2, True), (0, True)])
def test_attention_gradients_against_differences(window, use_sink):
    rng = np.random.default_rng(5)
    cu = [0, 1, 1, 5, 12]
    q, k, v = (rng.normal(size=(12, h, 3)) for h in (4, 2, 2))
    dout = rng.normal(size=q.shape)
    sink = rng.normal(size=4) if use_sink else None

    def loss():
        return float((tower.chunk_attention(q, k, v, cu, window, None, sink)["out"] * dout).sum())

    r = tower.chunk_attention(q, k, v, cu, window, None, sink, dout)
    for name, x in (("dq", q), ("dk", k), ("dv", v)) + ((("dsink", sink),) if use_sink else ()):
        _near(r[name], _differences(loss, x))


def test_attention_closed_cases():
    rng = np.random.default_rng(6)
    q, k, v = (rng.normal(size=(9, 2, 4)) for _ in range(3))
    # a window of zero sees the row itself alone
    r = tower.chunk_attention(q, k, v, [0, 9], 0)
    assert np.allclose(r["out"], v, atol=1e-15)
    # equal keys: the mean of the chunk's values, lse = logit + log n
    k[:] = k[:1]
    r = tower.chunk_attention(q, k, v, [0, 4, 9])
    assert np.allclose(r["out"][:4], v[:4].mean(axis=0), atol=1e-15)
    assert np.allclose(r["lse"][:, 4:], 0.5 * np.einsum("rhd,hd->hr", q[4:], k[0]) + np.log(5), atol=1e-14)
    # a sink of -inf takes key 0 away: alone in its band, nothing is left
    r = tower.chunk_attention(q, k, v, [0, 9], 0, None, np.array([-np.inf, 0.0]), np.ones_like(q))
    assert (r["out"][0, 0] == 0).all() and r["lse"][0, 0] == -np.inf and np.isfinite(r["dq"]).all()
    assert np.allclose(r["out"][0, 1], v[0, 1])


def test_norm_gradients_against_differences():
    rng = np.random.default_rng(7)
    x, dout = rng.normal(1.0, 2.0, (5, 7)), rng.normal(size=(5, 7))
    w, b = rng.normal(size=7), rng.normal(size=7)

    def loss():
        return float((tower.layer_norm(x, w, b, 1e-3)["out"] * dout).sum())

    r = tower.layer_norm(x, w, b, 1e-3, dout)
    for name, t in (("dx", x), ("dweight", w), ("dbias", b)):
        _near(r[name], _differences(loss, t))


def test_norm_closed_cases():
    r = tower.layer_norm(np.array([[3.0, 3.0], [1.0, -1.0]]), None, None, 0.25)
    assert (r["out"][0] == 0).all() and r["rstd"][0] == 2.0
    assert np.allclose(r["out"][1], np.array([1, -1]) / np.sqrt(1.25))


def test_quantized_closed_cases():
    # scale 1 / 127 * 127 = 1: values are their own quotients, ties go to even
    x = np.array([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5], [0, 0, 0, 0, 0, 0], [1, 2, np.nan, 0, 0, 0], [np.inf, 1, 0, 0, 0, 0]])
    q, s = tower.quantize_rows(x)
    assert q[0].tolist() == [127, 0, 2, 2, 0, -2] and s[0] == 1
    assert (q[1:] == 0).all() and s[1] == 0 and np.isnan(s[2:]).all()
    out, _ = tower.quantized_linear(q[:1], s[:1], np.array([[1, 2, 0, 0, 0, 0]]), np.array([0.5]), np.array([3.0]))
    assert out.tolist() == [[66.5]]
