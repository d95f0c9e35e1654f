"""Pins for oracle.balance at logits far from 0, where 1 - s of a float64 sigmoid has no bits left."""

import numpy as np

from oracle import balance


def test_score_rest():
    assert np.allclose(balance.score_rest([0.0, np.log(3.0), 50.0, 700.0, -800.0, np.inf, -np.inf], "sigmoid"),
                       [0.5, 0.25, np.exp(-50.0), np.exp(-700.0), 1.0, 0.0, 1.0], rtol=1e-14, atol=0)
    assert balance.score_rest([3.0, -np.inf], "softmax").tolist() == [1.0, 1.0]


def test_gradient_of_large_logits():
    # two experts with s = 1 to the last bit: p = 1/2, a = E c / (k n^2) = 2, 0: p (a - 1) e^-l
    grad, size = balance.balance_grad(1.0, np.array([[60.0, 80.0]]), np.array([[0]]), "sigmoid")
    assert np.allclose(grad, [[0.5 * np.exp(-60.0), -0.5 * np.exp(-80.0)]], rtol=1e-14, atol=0)
    assert np.allclose(size, [[1.5, 0.5]])
