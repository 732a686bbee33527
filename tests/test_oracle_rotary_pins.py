"""The rotary and head norm oracle, pinned to things that do not restate its formulas."""
import numpy as np
import pytest

from oracle import rotary_oracle as ro

R = np.random.default_rng


@pytest.mark.parametrize("inter", [False, True])
def test_turn_is_a_complex_product(inter):
    r = R(0)
    x, p, f = r.standard_normal((5, 3, 14)), np.array([0, 1, -7, 40, 9]), 0.3 ** np.arange(5)
    y = ro.turn(x, p, f, inter, 1.3)
    a, b = ro.columns(5, inter)
    z = (x[..., a] + 1j * x[..., b]) * 1.3 * np.exp(1j * p[:, None, None] * f)
    np.testing.assert_allclose(y[..., a] + 1j * y[..., b], z, rtol=1e-13)
    np.testing.assert_array_equal(y[..., 10:], x[..., 10:])


@pytest.mark.parametrize("inter", [False, True])
def test_products_depend_on_distance_alone(inter):
    r = R(1)
    q, k, f = r.standard_normal((1, 1, 16)), r.standard_normal((1, 1, 16)), 10000.0 ** -(np.arange(8) / 8)
    at = lambda i, j: float((ro.turn(q, [i], f, inter) * ro.turn(k, [j], f, inter)).sum())  # noqa: E731
    assert abs(at(3, 10) - at(1003, 1010)) < 1e-9
    assert abs(at(3, 10) - at(3, 11)) > 1e-3


def test_turned_back_is_the_input():
    r = R(2)
    x, f = r.standard_normal((4, 2, 12)), 0.5 ** np.arange(4)
    np.testing.assert_allclose(ro.turn(ro.turn(x, [1, 2, 3, 4], f), [1, 2, 3, 4], f, back=True), x, atol=1e-14)


def test_known_quarter_turn():
    x = np.array([[[1.0, 2.0, 3.0, 4.0]]])
    np.testing.assert_allclose(ro.turn(x, [1], [np.pi / 2, 0.0], False), [[[-3.0, 2.0, 1.0, 4.0]]], atol=1e-15)
    np.testing.assert_allclose(ro.turn(x, [1], [np.pi / 2, 0.0], True), [[[-2.0, 1.0, 3.0, 4.0]]], atol=1e-15)


def test_norm_has_unit_mean_square_and_ignores_scale():
    x = R(3).standard_normal((3, 2, 9))
    y, _ = ro.norm(x, None, 0.0)
    np.testing.assert_allclose((y * y).mean(-1), 1.0)
    np.testing.assert_allclose(ro.norm(7.0 * x, None, 0.0)[0], y)


@pytest.mark.parametrize("inter", [False, True])
def test_gradients_against_differences(inter):
    r = R(4)
    x, w, dy = r.standard_normal((3, 2, 10)), 1 + 0.3 * r.standard_normal(10), r.standard_normal((3, 2, 10))
    p, f, eps = [0, 5, 900], 0.4 ** np.arange(3), 0.05
    loss = lambda x, w: float((dy * ro.turn(ro.norm(x, w, eps)[0], p, f, inter, 0.8)).sum())  # noqa: E731
    dx, dw = ro.norm_bwd(x, w, ro.turn(dy, p, f, inter, 0.8, back=True), eps)
    h = 1e-6
    for t, g, of in ((x, dx, lambda t: loss(t, w)), (w, dw, lambda t: loss(x, t))):
        for i in np.ndindex(t.shape):
            up, down = t.copy(), t.copy()
            up[i] += h
            down[i] -= h
            assert abs((of(up) - of(down)) / (2 * h) - g[i]) < 1e-8
