"""The feed-forward oracle against hand-worked values and differences (no GPU)."""

import math

import numpy as np
import pytest

from oracle import ffn as of

ACTS = ("silu", "gelu", "gelu_tanh")


def test_activations_by_hand():
    assert of.act(0.0, "silu") == 0.0 and of.slope(0.0, "silu") == 0.5
    np.testing.assert_allclose(of.act(1.0, "silu"), 1.0 / (1.0 + math.exp(-1.0)), rtol=1e-15)
    np.testing.assert_allclose(of.act(1.0, "gelu"), 0.8413447460685429, rtol=1e-14)  # Phi(1)
    np.testing.assert_allclose(of.act(-2.0, "gelu"), -2.0 * 0.022750131948179195, rtol=1e-12)
    assert abs(of.act(1.0, "gelu_tanh") - of.act(1.0, "gelu")) < 2e-4  # the tanh form is near it
    for name in ACTS:
        assert abs(of.act(40.0, name) - 40.0) < 1e-12 and abs(of.act(-40.0, name)) < 1e-12


@pytest.mark.parametrize("name", ACTS)
def test_slopes_against_differences(name):
    x, h = np.linspace(-6.0, 6.0, 241), 1e-5
    d = (of.act(x + h, name) - of.act(x - h, name)) / (2 * h)
    np.testing.assert_allclose(of.slope(x, name), d, rtol=0, atol=1e-9)


def test_runs():
    assert of.runs(10) == [(0, 10)]
    assert of.runs(10, [0, 4, 4, 9]) == [(0, 4), (4, 4), (4, 9)]
    assert of.runs(10, [-2, 4, 3, 99], [1, 5, -1]) == [(0, 1), (4, 4), (4, 4)]
    assert of.runs(10, [2, 8], [3]) == [(2, 5)]


@pytest.mark.parametrize("name", ACTS)
def test_gradients_against_differences(name):
    rng = np.random.default_rng(0)
    x, dy = rng.normal(size=(7, 5)), rng.normal(size=(7, 3))
    up, down = rng.normal(size=(2, 8, 5)), rng.normal(size=(2, 3, 4))
    off, cnt = [0, 3, 6], [2, 3]
    y, z = of.forward(x, up, down, name, off, cnt)
    assert (y[2] == 0).all() and (y[6] == 0).all()
    grads = of.backward(dy, x, up, down, z, name, off, cnt)
    for a, g in zip((x, up, down), grads):
        flat = a.reshape(-1)
        for i in range(flat.size):
            keep = flat[i]
            v = []
            for h in (1e-6, -1e-6):
                flat[i] = keep + h
                v.append((of.forward(x, up, down, name, off, cnt)[0] * dy).sum())
            flat[i] = keep
            assert abs((v[0] - v[1]) / 2e-6 - g.reshape(-1)[i]) < 1e-7


def test_int8_rows_by_hand():
    x = np.array([[254.0, 1.0, 3.0, -5.0, 127.0], [0.0, 0.0, 0.0, 0.0, 0.0], [1.0, np.nan, 0.0, 0.0, 0.0],
                  [1.0, -np.inf, 0.0, 0.0, 0.0], [-2.0, 1.0, 0.5, 2.0, -1.0]])
    codes, scales = of.int8_rows(x)
    # 127 x / 254 = x / 2: ties go to the even code
    assert codes[0].tolist() == [127, 0, 2, -2, 64] and scales[0] == 2.0
    assert (codes[1:4] == 0).all() and scales[1] == 0.0 and np.isnan(scales[2:4]).all()
    assert codes[4].tolist() == [-127, 64, 32, 127, -64]  # 63.5 and 31.75
