"""The plain forms of the rotation, the norm, its operands and the adapters
(oracle/layer.py) against what is known of them apart from their formulas."""
import numpy as np
import torch

from oracle import layer


def test_rotation_is_a_turn_of_the_plane():
    rng = np.random.default_rng(0)
    x = layer.bf16_round(rng.standard_normal((5, 2, 32)))
    f = (10.0 ** -np.arange(8) / 3).astype(np.float32)
    pos = np.array([0, 1, 7, 4096, 131071])
    for inter in (False, True):
        y = layer.rotate(x, pos, f, inter)
        assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 16:], x[..., 16:])
        z = x[..., 0:16:2] + 1j * x[..., 1:16:2] if inter else x[..., :8] + 1j * x[..., 8:16]
        w = z * np.exp(1j * pos[:, None, None] * f.astype(np.float64))
        got = y[..., 0:16:2] + 1j * y[..., 1:16:2] if inter else y[..., :8] + 1j * y[..., 8:16]
        assert np.all(np.abs(got.real - w.real) <= 2.0 ** -8 * np.abs(w.real) + 1e-12)
        assert np.all(np.abs(got.imag - w.imag) <= 2.0 ** -8 * np.abs(w.imag) + 1e-12)


def test_scores_after_the_rotation_go_by_the_distance():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 64))
    f = (1e4 ** (-np.arange(32) / 32)).astype(np.float32)

    def score(a, b):
        return np.sum(layer.rotate(q, [a], f) * layer.rotate(k, [b], f))

    # two roundings of 2^-8 of each product
    tol = 2.0 ** -6.9 * np.sum(np.abs(q) + np.abs(np.roll(q, 32, -1))) * np.abs(k).max() * 2
    assert abs(score(5, 3) - score(100005, 100003)) <= tol


def test_positions():
    assert layer.token_positions([0, 2, 2, 3], [5, 9, 1], 4).tolist() == [3, 4, 0, 0]


def test_norm_gradient_by_differences():
    rng = np.random.default_rng(2)
    x, w, dy = rng.standard_normal((3, 10)), rng.standard_normal(10), rng.standard_normal((3, 10))
    h, r, y = layer.rms_norm(x, w, 1e-3)
    assert np.allclose((y / w).std(1) ** 2 + (y / w).mean(1) ** 2, 1.0, atol=1e-2)
    dx, dw, *_ = layer.rms_norm_backward(h, w, r, dy)

    def loss(x, w):
        return np.sum(layer.rms_norm(x, w, 1e-3)[2] * dy)

    for i, j in ((0, 0), (1, 4), (2, 9)):
        d = np.zeros_like(x)
        d[i, j] = 1e-6
        assert abs((loss(x + d, w) - loss(x - d, w)) / 2e-6 - dx[i, j]) < 1e-7
        assert abs((loss(x, w + d[i]) - loss(x, w - d[i])) / 2e-6 - dw[j]) < 1e-7


def test_mxfp8_against_torch():
    rng = np.random.default_rng(3)
    x = layer.bf16_round(rng.standard_normal((40, 96)) * 2.0 ** rng.integers(-20, 20, (40, 1)))
    x[0], x[1] = 0.0, -0.0
    x[2, :32] = 448.0 * 2.0 ** 5              # a block whose largest value is the format's
    x[3, :32] = 449.0
    codes, sc, val = layer.mxfp8_quantize(x)
    f = 2.0 ** (sc.astype(np.float64) - 127)
    b = torch.from_numpy(x.reshape(40, 3, 32) / f[..., None]).float().to(torch.float8_e4m3fn)
    assert np.array_equal(b.view(torch.uint8).numpy().reshape(codes.shape), codes)
    assert np.array_equal(val, (b.double().numpy() * f[..., None]).reshape(val.shape))
    assert sc[2, 0] == 127 + 5 and sc[0, 0] == 0
    top = np.abs(b.double().numpy()).max(-1)[sc > 0]
    assert np.all((top > 216) & (top <= 448))


def test_adapters():
    rng = np.random.default_rng(4)
    x, a, b = rng.standard_normal((6, 16)), rng.standard_normal((3, 8, 16)), rng.standard_normal((3, 5, 8))
    y = rng.standard_normal((6, 5))
    out, *_ = layer.lora(x, a, b, [0, 2, 2, 5], [2, 0, -1], [1, 1, 0.5], y)
    assert np.allclose(out[:2], y[:2] + 0.5 * x[:2] @ (b[2] @ a[2]).T)
    assert np.array_equal(out[2:], y[2:])


def test_sinks_stay_visible():
    """All keys alike but the first: its value enters in proportion."""
    cache = np.zeros((4, 1, layer.kv_page_bytes(1, 16, 64)), np.uint8)
    table, off, lens = np.array([[0, 1, 2, 3]]), [0, 1], np.array([60])
    k, v = np.zeros((60, 1, 64)), np.zeros((60, 1, 64))
    v[0] = 4.0
    layer.kv_append(1, cache, 16, [0, 60], table, lens, k, v)
    q = np.ones((1, 1, 64))
    assert np.all(layer.attention(1, cache, 16, off, table, lens, q, window=7)[0] == 0)
    assert np.allclose(layer.attention(1, cache, 16, off, table, lens, q, window=7, sinks=1)[0], 4.0 / 8)
    assert np.allclose(layer.attention(1, cache, 16, off, table, lens, q, window=7, sinks=3)[0], 4.0 / 10)
    assert np.allclose(layer.attention(1, cache, 16, off, table, lens, q, window=100, sinks=3)[0], 4.0 / 60)
