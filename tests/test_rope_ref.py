"""Pins of the 64-bit reference of the per-head norm and rotary positions."""
import numpy as np
import pytest

import rope_ref


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 4, 8])
@pytest.mark.parametrize("norm", [False, True])
def test_gradients_are_the_differences(interleaved, rot, norm):
    rng = np.random.default_rng(7)
    rows, heads, d, eps, h = 3, 2, 8, 1e-3, 1e-6
    x, dy = rng.normal(size=(2, rows, heads, d))
    gain = 1 + 0.3 * rng.normal(size=d) if norm else None
    ang = rng.uniform(-7, 7, size=(rows, rot // 2))
    args = (ang, interleaved, norm, eps)
    dx, dg, _ = rope_ref.backward(dy, x, gain, *args)

    def loss(x, gain):
        return (rope_ref.forward(x, gain, *args) * dy).sum()

    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        assert (loss(x + e, gain) - loss(x - e, gain)) / (2 * h) == pytest.approx(dx[i], abs=1e-7)
    if norm:
        for i in range(d):
            e = np.zeros(d)
            e[i] = h
            assert (loss(x, gain + e) - loss(x, gain - e)) / (2 * h) == pytest.approx(dg[i],
                                                                                      abs=1e-7)


@pytest.mark.parametrize("interleaved", [False, True])
def test_products_depend_on_relative_positions(interleaved):
    rng = np.random.default_rng(3)
    freq = np.array([1.0, 0.1, 0.01, 0.001])
    axis = [0, 1, 1, 0]
    q, k = rng.normal(size=(2, 1, 1, 8))

    def score(pq, pk):
        a = rope_ref.angles(np.array(pq)[:, None], freq, axis)
        b = rope_ref.angles(np.array(pk)[:, None], freq, axis)
        return (rope_ref.turn(q, a, interleaved) * rope_ref.turn(k, b, interleaved)).sum()

    assert score((5, 9), (2, 3)) == pytest.approx(score((105, 1009), (102, 1003)), abs=1e-10)
    assert score((5, 9), (2, 3)) != pytest.approx(score((6, 9), (2, 3)), abs=1e-3)
    # a quarter turn: (1, 0) goes to (0, 1)
    e, f = rope_ref.pair_columns(2, interleaved)
    x = np.zeros((1, 1, 2))
    x[..., e] = 1.0
    y = rope_ref.turn(x, np.array([[np.pi / 2]]), interleaved)
    assert y[0, 0, f[0]] == pytest.approx(1.0) and y[0, 0, e[0]] == pytest.approx(0.0)
