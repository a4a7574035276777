"""Pins of the plain 64-bit forms in oracle/layer.py (no GPU): the cache's
quantizer against the pinned C quantizer, its layout as a bijection, attention
and the router against closed forms, and the gradients against differences."""
import numpy as np
import pytest

from oracle import layer

RNG = np.random.default_rng(7)


def _bf16(x):
    return layer.bf16_round(x)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** -100, 2.0 ** 90])
def test_cache_quantizer_is_the_pinned_one(orc, fmt, scale):
    x = _bf16(RNG.standard_normal((37, 128)) * scale * np.exp(RNG.standard_normal((37, 1))))
    x[3] = 0.0
    x[4, ::2] = -0.0
    bits = (x.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    ref = orc.quantize(fmt, bits)
    t = ref["tscale"][0] if fmt == 0 else None
    codes, sc, _ = layer.kv_quantize(fmt, x, t)
    assert np.array_equal(codes[:, 0::2] | (codes[:, 1::2] << 4), ref["q"])
    assert np.array_equal(sc, ref["scales"])


@pytest.mark.parametrize("fmt,page,dim", [(0, 16, 64), (0, 32, 128), (1, 16, 128), (1, 64, 256)])
def test_every_bit_of_a_page_has_one_owner(fmt, page, dim):
    kb, kh, vb, vh, ks, vs = layer.kv_places(fmt, page, dim)
    nb = layer.kv_page_bytes(fmt, page, dim)
    half = np.concatenate([(2 * b + s // 4).ravel() for b, s in ((kb, kh), (vb, vh))]
                          + [(2 * x + i).ravel() for x in (ks, vs) for i in (0, 1)])
    assert np.array_equal(np.sort(half), np.arange(2 * nb))
    # no byte is shared by two tokens
    for b in (kb, vb):
        assert all(len(np.intersect1d(b[0], b[s])) == 0 for s in range(1, page))


@pytest.mark.parametrize("fmt", [0, 1])
def test_append_then_read(fmt):
    H, D, page = 2, 64, 16
    offsets, lens = np.array([0, 3, 3, 20]), np.array([18, 5, 17])
    table = np.array([[4, 0], [2, -1], [1, 3]], np.int32)
    k, v = _bf16(RNG.standard_normal((2, 20, H, D)))
    t = np.array([0.002, 0.004], np.float32) if fmt == 0 else None
    cache = RNG.integers(0, 256, (5, H, layer.kv_page_bytes(fmt, page, D)), dtype=np.uint8)
    before = cache.copy()
    layer.kv_append(fmt, cache, page, offsets, table, lens, k, v, t, t)
    gk, gv = layer.kv_read(fmt, cache, page, offsets, table, lens, 20, D, t, t)
    for g, x in ((gk, k), (gv, v)):
        want = layer.kv_quantize(fmt, x, None if t is None else t[None])[2]
        assert np.array_equal(g, _bf16(want))
    assert np.array_equal(cache[2], before[2])       # the sequence without new tokens


def test_attention_closed_forms():
    """One key: its value.  Equal scores: the mean of the values seen.  A window
    of one: each token's own value.  Nothing seen: zero."""
    fmt, H, D, page, n = 1, 1, 64, 16, 9
    table = np.array([[1, 0]], np.int32)
    k, v = _bf16(RNG.standard_normal((2, n, H, D)))
    cache = np.zeros((2, H, layer.kv_page_bytes(fmt, page, D)), np.uint8)
    off, lens = np.array([0, n]), np.array([n])
    layer.kv_append(fmt, cache, page, off, table, lens, k, v)
    _, vals = layer.kv_read(fmt, cache, page, off, table, lens, n, D)
    q = np.zeros((n, 2, D))
    o, _, _ = layer.attention(fmt, cache, page, off, table, lens, q)
    want = np.cumsum(vals[:, 0], 0) / np.arange(1, n + 1)[:, None]
    assert np.allclose(o[:, 0], want, atol=1e-12) and np.array_equal(o[:, 0], o[:, 1])
    q = RNG.standard_normal((n, 2, D))
    o, _, _ = layer.attention(fmt, cache, page, off, table, lens, q, window=1)
    assert np.allclose(o[:, 1], vals[:, 0], atol=1e-12)
    o, _, _ = layer.attention(fmt, cache, page, off, np.array([[-1, 0]], np.int32), lens, q)
    assert np.all(o == 0)


def test_route_by_hand():
    x = np.array([[0.0, 2.0, 2.0, 1.0], [3.0, 0.0, 1.0, 2.0]])
    r = layer.route(x, 2)
    assert r["experts"].tolist() == [[1, 2], [0, 3]]
    assert np.allclose(r["weights"], [[0.5, 0.5], [1 / (1 + np.exp(-1)), 1 / (1 + np.exp(1))]])
    assert r["offsets"].tolist() == [0, 1, 2, 3, 4]
    assert r["row_src"].tolist() == [1, 0, 0, 1] and r["row_of"].tolist() == [[1, 2], [0, 3]]
    # groups: {0, 1} and {2, 3}; the second has the larger pair in row 0 with this bias
    r = layer.route(x, 1, layer.SIGMOID, np.array([0, 0, 0, 0.5]), 2, 1, renorm=False)
    assert r["experts"].tolist() == [[3], [3]]
    assert np.allclose(r["weights"][:, 0], 1 / (1 + np.exp([-1.0, -2.0])))


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(score, renorm):
    x = RNG.standard_normal((5, 12))
    r = layer.route(x, 3, score, renorm=renorm)
    dw = RNG.standard_normal((5, 3))
    d, _ = layer.route_backward(x, r["experts"], dw, score, renorm)
    h = 1e-6
    for e in range(12):
        up, dn = x.copy(), x.copy()
        up[:, e] += h
        dn[:, e] -= h
        diff = (layer.route_weights(up, r["experts"], score, renorm)
                - layer.route_weights(dn, r["experts"], score, renorm)) / (2 * h)
        assert np.allclose((diff * dw).sum(1), d[:, e], atol=1e-8)


def test_combine_gradient_against_differences():
    y, w = RNG.standard_normal((12, 5)), RNG.standard_normal((4, 3))
    row_of = RNG.permutation(12).reshape(4, 3)
    do = RNG.standard_normal((4, 5))
    d_y, d_w, _ = layer.combine_backward(y, row_of, w, do)
    h = 1e-6

    def f(y, w):
        return (layer.combine(y, row_of, w)[0] * do).sum()

    for i in np.ndindex(y.shape):
        e = np.zeros_like(y)
        e[i] = h
        assert abs((f(y + e, w) - f(y - e, w)) / (2 * h) - d_y[i]) < 1e-8
    for i in np.ndindex(w.shape):
        e = np.zeros_like(w)
        e[i] = h
        assert abs((f(y, w + e) - f(y, w - e)) / (2 * h) - d_w[i]) < 1e-8
