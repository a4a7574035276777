"""Pins of the plain 64-bit forms in oracle/layer.py at the edges of their
definitions (no GPU)."""
import numpy as np

from oracle import layer


def test_infinite_and_nan_logits():
    inf, top = np.inf, float(np.finfo(np.float32).max)
    x = np.array([[1.0, inf, 2.0, inf], [np.nan, -inf, 3.0, inf], [inf, top, 0.0, -inf]])
    s = [layer.scores_of(r, layer.SOFTMAX) for r in x]
    assert np.array_equal(s[0], [0, 0.5, 0, 0.5]) and np.array_equal(s[1], [0, 0, 0, 1])
    assert np.array_equal(s[2], [0.5, 0.5, 0, 0])
    assert np.array_equal(layer.scores_of(x[1], layer.SIGMOID)[[0, 1, 3]], [0, 0, 1])
    r = layer.route(x, 2, layer.SOFTMAX)
    assert r["experts"].tolist() == [[1, 3], [3, 2], [0, 1]]
    assert np.array_equal(r["weights"], [[0.5, 0.5], [1, 0], [0.5, 0.5]])
    d, _ = layer.route_backward(x, r["experts"], np.ones((3, 2)), layer.SOFTMAX, False)
    assert np.array_equal(d, np.zeros((3, 4)))
