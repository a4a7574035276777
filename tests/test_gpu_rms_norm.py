"""GPU: the root-mean-square norm, its quantized operands, its gradient and an
operand's values.

y is the 64-bit value rounded once to F32 (and from there to BF16): against the
unrounded 64-bit form that is 2^-24 of it, and the BF16 value the same but for
one in 2^28, so that BF16 outputs and codes are compared bit for bit."""
import numpy as np
import pytest
import torch

import fp4_w4a4_quantized_amd as fq
from gpu_helpers import need_gpu, say
from oracle import layer

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
TYPES = {torch.bfloat16: fq.OUT_BF16, torch.float32: fq.OUT_F32}


def dev(a, dt=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(dt)


def host(t):
    return t.double().cpu().numpy()


def case(rows, cols, dt, residual, seed=0, wdt=None, mult=1.0):
    rng = np.random.default_rng(seed + rows * 31 + cols)

    def values(*shape):
        a = rng.standard_normal(shape)
        return layer.bf16_round(a) if dt == torch.bfloat16 else a.astype(np.float32).astype(np.float64)

    x = values(rows, cols) * mult
    res = values(rows, cols) * mult if residual else None
    if residual and cols > 8:
        res[:, ::7] = values(rows, len(range(0, cols, 7))) * 16 * mult
    w = values(cols)
    return x, res, w


def strided(a, dt, pad):
    """A view whose rows lie cols + pad elements apart."""
    t = torch.zeros(a.shape[0], a.shape[1] + pad, device="cuda", dtype=dt)
    t[:, :a.shape[1]] = dev(a, dt)
    return t[:, :a.shape[1]]


def none(a, *f):
    return None if a is None else f[0](a, *f[1:])


SIZES = [(1, 1), (3, 7), (2, 64), (5, 511), (1, 4096), (9, 2049), (2, 8200), (3, 20000), (2, 32768)]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_norm(dt, rows, cols):
    need_gpu()
    say(f"norm {dt} {rows} x {cols}")
    for residual in (False, True):
        x, res, w = case(rows, cols, dt, residual)
        h, r, y = layer.rms_norm(x, w, 1e-6, res, dt == torch.bfloat16)
        for ydt in (torch.bfloat16, torch.float32):
            for pad in (0, 3):
                f = fq.rms_norm(strided(x, dt, pad), dev(w, dt), 1e-6, none(res, strided, dt, pad + 2), TYPES[ydt])
                if residual:
                    assert np.array_equal(host(f["h"]), h)
                assert np.all(np.abs(host(f["rstd"])[:, None] - r) <= (E + 2.0 ** -50) * r)
                got = host(f["y"])
                if ydt == torch.bfloat16:
                    assert np.array_equal(got, layer.bf16_round(y))
                else:
                    assert np.all(np.abs(got - y) <= (E + 2.0 ** -48) * np.abs(y) + 2.0 ** -149)


def test_many_rows():
    """Rows enough for one wave each, and more groups of them than workgroups."""
    need_gpu()
    for rows, cols in ((2048, 96), (2051, 4096), (9001, 33)):
        say(f"many rows {rows} x {cols}")
        x, res, w = case(rows, cols, torch.bfloat16, True)
        h, r, y = layer.rms_norm(x, w, 1e-5, res)
        f = fq.rms_norm(dev(x, torch.bfloat16), dev(w), 1e-5, dev(res, torch.bfloat16))
        assert np.array_equal(host(f["h"]), h) and np.array_equal(host(f["y"]), layer.bf16_round(y))


def test_weight_types_and_in_place():
    need_gpu()
    x, res, w = case(6, 300, torch.bfloat16, True)
    w32 = np.random.default_rng(1).standard_normal(300).astype(np.float32).astype(np.float64)
    for wt in (w, w32):
        h, r, y = layer.rms_norm(x, wt, 1e-6, res)
        f = fq.rms_norm(dev(x, torch.bfloat16), dev(wt), 1e-6, dev(res, torch.bfloat16))
        assert np.array_equal(host(f["y"]), layer.bf16_round(y))
    # h over the residual, y over x
    tx, tr, rstd = dev(x, torch.bfloat16), dev(res, torch.bfloat16), torch.empty(6, device="cuda")
    fq.rms_norm_into(tx, dev(w32), 1e-6, tr, tr, tx, rstd)
    assert np.array_equal(host(tr), h) and np.array_equal(host(tx), layer.bf16_round(y))
    assert np.all(np.abs(host(rstd)[:, None] - r) <= (E + 2.0 ** -50) * r)


def test_rows_of_zeros_and_of_extreme_values():
    """Zeros (eps alone), values whose squares leave F32 on either side, one NaN:
    it stays in its row."""
    need_gpu()
    for dt in (torch.bfloat16, torch.float32):
        x, _, w = case(6, 256, dt, False)
        x[0], x[1] = 0.0, -0.0
        x[2] *= 2.0 ** 100
        x[3] *= 2.0 ** -100
        h, r, y = layer.rms_norm(x, w, 1e-6, None)
        for eps in (1e-6, 0.0):
            h, r, y = layer.rms_norm(x[2:], w, eps, None)
            t = dev(x, dt)
            t[5, 7] = float("nan")
            got = host(fq.rms_norm(t, dev(w, dt), eps, y_dtype=fq.OUT_F32)["y"])
            if eps:
                assert np.all(got[:2] == 0)
            assert np.all(np.abs(got[2:5] - y[:3]) <= (E + 2.0 ** -48) * np.abs(y[:3]) + 2.0 ** -149)
            assert np.all(np.isnan(got[5]))


@pytest.mark.parametrize("cols", [256, 2080, 9024])
def test_products_beyond_f32(cols):
    """h w leaves F32 on either side where y does not."""
    need_gpu()
    for dt, big, wbig in ((torch.bfloat16, 100, 60), (torch.bfloat16, -100, -60), (torch.float32, 100, 60)):
        say(f"norm products beyond f32 {dt} {cols} 2^{big} 2^{wbig}")
        x, _, w = case(4, cols, dt, False)
        x, w = x * 2.0 ** big, w * 2.0 ** wbig
        h, r, y = layer.rms_norm(x, w, 0.0, None)
        assert np.abs(y).max() < 2.0 ** 70 and (np.abs(x * w).max() > 2.0 ** 128 or np.abs(x * w).max() < 2.0 ** -149)
        f = fq.rms_norm(dev(x, dt), dev(w, dt), 0.0, y_dtype=fq.OUT_F32)
        assert np.all(np.abs(host(f["y"]) - y) <= (E + 2.0 ** -48) * np.abs(y) + 2.0 ** -149)
        want = fq.quantize(fq.MXFP4, dev(layer.bf16_round(y), torch.bfloat16))
        same_operand(fq.rms_norm_quantize(fq.MXFP4, dev(x, dt), dev(w, dt), 0.0), want, fq.MXFP4, 0, 4, cols)


# ---- quantized operands -------------------------------------------------------

def same_operand(a, b, fmt, layout, rows, cols):
    if layout == fq.TILED:                 # (padding rows hold anything)
        assert torch.equal(fq.dequantize(fmt, a, fq.OUT_F32), fq.dequantize(fmt, b, fq.OUT_F32))
        rc = rows // 16 * 16 * cols // 2
        assert torch.equal(a["q"][:rc], b["q"][:rc])
        rs = rows // 64 * 64 * cols // fq.BLOCK[fmt]
        assert torch.equal(a["scales"][:rs], b["scales"][:rs])
    else:
        assert torch.equal(a["q"], b["q"]) and torch.equal(a["scales"], b["scales"])
    assert fmt == fq.MXFP4 or torch.equal(a["tscale"], b["tscale"])
    if b["resid"] is not None:
        assert torch.equal(a["resid"], b["resid"])


@pytest.mark.parametrize("fmt", [fq.NVFP4, fq.MXFP4])
@pytest.mark.parametrize("layout", [fq.ROWMAJOR, fq.TILED])
@pytest.mark.parametrize("rows,cols", [(1, 128), (3, 256), (64, 2048), (70, 4096), (2100, 384), (5, 8320), (4, 18432), (2, 32768)])
def test_operand_is_the_quantizers(fmt, layout, rows, cols):
    need_gpu()
    say(f"norm into operand fmt {fmt} layout {layout} {rows} x {cols}")
    rng = np.random.default_rng(cols)
    for dt, residual, nc in ((torch.bfloat16, True, 16), (torch.bfloat16, False, 0), (torch.float32, True, 40)):
        x, res, w = case(rows, cols, dt, residual)
        h, r, y = layer.rms_norm(x, w, 1e-6, res, dt == torch.bfloat16)
        yb = dev(layer.bf16_round(y), torch.bfloat16)
        chan = dev(np.sort(rng.permutation(cols)[:nc])).int() if nc else None
        want = fq.quantize(fmt, yb, chan_idx=chan, layout=layout)
        a = fq.rms_norm_quantize(fmt, dev(x, dt), dev(w, dt), 1e-6, none(res, dev, dt), chan_idx=chan, layout=layout,
                                 y_dtype=fq.OUT_BF16 if residual else None, rstd=residual)
        same_operand(a, want, fmt, layout, rows, cols)
        if residual:
            assert np.array_equal(host(a["h"]), h) and torch.equal(a["y"], yb)
            assert np.all(np.abs(host(a["rstd"])[:, None] - r) <= (E + 2.0 ** -50) * r)
        if fmt == fq.NVFP4:                # one pass, with the scale that the two found
            b = fq.rms_norm_quantize(fmt, dev(x, dt), dev(w, dt), 1e-6, none(res, dev, dt), tscale=want["tscale"],
                                     chan_idx=chan, layout=layout)
            same_operand(b, want, fmt, layout, rows, cols)


def test_narrow_and_strided():
    """Sixteen columns (NVFP4), and rows of odd strides."""
    need_gpu()
    for fmt, cols in ((0, 16), (0, 48), (1, 32), (1, 96)):
        x, res, w = case(11, cols, torch.bfloat16, True)
        h, r, y = layer.rms_norm(x, w, 1e-6, res)
        a = fq.rms_norm_quantize(fmt, strided(x, torch.bfloat16, 5), dev(w), 1e-6, strided(res, torch.bfloat16, 1))
        same_operand(a, fq.quantize(fmt, dev(layer.bf16_round(y), torch.bfloat16)), fmt, 0, 11, cols)


@pytest.mark.parametrize("rows,cols", [(1, 32), (5, 4096), (2100, 96), (3, 9600)])
def test_mxfp8(rows, cols):
    need_gpu()
    say(f"norm into MXFP8 {rows} x {cols}")
    for dt in (torch.bfloat16, torch.float32):
        x, res, w = case(rows, cols, dt, True)
        w[:32] *= 2.0 ** -120                          # a block of very small values
        h, r, y = layer.rms_norm(x, w, 1e-6, res, dt == torch.bfloat16)
        codes, sc, val = layer.mxfp8_quantize(layer.bf16_round(y))
        a = fq.rms_norm_quantize(fq.MXFP8, dev(x, dt), dev(w), 1e-6, dev(res, dt))
        assert np.array_equal(a["q"].cpu().numpy(), codes) and np.array_equal(a["scales"].cpu().numpy(), sc)
        assert np.array_equal(host(fq.dequantize(fq.MXFP8, a, fq.OUT_F32)), val)


def test_zero_tensors_and_no_rows():
    need_gpu()
    for fmt in (0, 1, 2):
        x, w = torch.zeros(3, 64, device="cuda"), torch.ones(64, device="cuda")
        a = fq.rms_norm_quantize(fmt, x, w)
        assert torch.all(fq.dequantize(fmt, a) == 0)
        a = fq.rms_norm_quantize(fmt, x[:0], w)
        assert a["q"].shape[0] == 0 and fq.dequantize(fmt, a).shape == (0, 64)
        if fmt == 0:
            assert a["tscale"].item() == 1.0
    f = fq.rms_norm(x[:0], w)
    dx, dw = fq.rms_norm_backward(f["h"], w, f["rstd"], x[:0])
    assert dx.shape == (0, 64) and torch.all(dw == 0)


# ---- an operand's values --------------------------------------------------------

@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("layout", [fq.ROWMAJOR, fq.TILED])
def test_dequantize(fmt, layout):
    need_gpu()
    for rows, cols in ((1, 128), (17, 640), (130, 1024)):
        rng = np.random.default_rng(rows)
        x = layer.bf16_round(rng.standard_normal((rows, cols)) * 2.0 ** rng.integers(-9, 9, (rows, 1)))
        a = fq.quantize(fmt, dev(x, torch.bfloat16), layout=layout)
        t = None if fmt else a["tscale"].cpu().numpy()[0]
        val = layer.kv_quantize(fmt, x, t)[2]
        assert np.array_equal(host(fq.dequantize(fmt, a, fq.OUT_F32)), val.astype(np.float32).astype(np.float64))
        assert np.array_equal(host(fq.dequantize(fmt, a)), layer.bf16_round(val))
        if layout == fq.ROWMAJOR:
            a = {k: a[k] for k in ("q", "scales", "tscale")}
            assert np.array_equal(host(fq.dequantize(fmt, a)), layer.bf16_round(val))


# ---- the gradient ---------------------------------------------------------------

@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", SIZES + [(700, 130), (1030, 4100)])
def test_gradient(dt, rows, cols):
    """d_x: u and g are off by 2 and 1 units of 2^-24; a lane's part of the mean has
    at most 64 terms, the lanes' and waves' sums nine levels and eight terms:
    (64 + 9 + 8 + 3) units of the sum of absolute terms; the difference and the
    products four more of what they take in.  d_weight: rows / 512 terms in a
    workgroup, 512 / 16 + 16 after it, and u's and the product's three units."""
    need_gpu()
    say(f"norm gradient {dt} {rows} x {cols}")
    half = 2.0 ** -8 if dt == torch.bfloat16 else E
    for residual in (False, True):
        x, res, w = case(rows, cols, dt, residual)
        dy, dh, _ = case(rows, cols, dt, residual, seed=7)
        f = fq.rms_norm(dev(x, dt), dev(w, dt), 1e-5, none(res, dev, dt))
        h, r, _ = layer.rms_norm(x, w, 1e-5, res, dt == torch.bfloat16)
        want, want_w, mean, total = layer.rms_norm_backward(h, w, r, dy, dh)
        for pad in (0, 1):
            dx, dw = fq.rms_norm_backward(f["h"] if not pad else strided(h, dt, 3), dev(w, dt), f["rstd"],
                                          strided(dy, dt, pad), none(dh, strided, dt, pad))
            u, g = np.abs(h * r), np.abs(w * dy)
            s = np.abs((w * dy * h * r).mean(1, keepdims=True))
            tol = r * (4 * E * g + u * (8 * E * s + 84 * E * mean)) + 4 * E * np.abs(want)
            tol = tol + half * (np.abs(want) + tol) + 2.0 ** -149
            err = np.abs(host(dx) - want)
            assert np.all(err <= tol), f"d_x {np.max(err / tol):.2f} of the bound"
            n = -(-rows // 512) + 48 + 3
            tol = n * E * total + 2.0 ** -149
            err = np.abs(host(dw) - want_w)
            assert np.all(err <= tol), f"d_weight {np.max(err / tol):.2f} of the bound"


def test_gradient_in_place_and_repeated():
    need_gpu()
    x, res, w = case(40, 1000, torch.bfloat16, True)
    dy, dh, _ = case(40, 1000, torch.bfloat16, True, seed=7)
    b = torch.bfloat16
    f = fq.rms_norm(dev(x, b), dev(w), 1e-5, dev(res, b))
    args = f["h"], dev(w), f["rstd"]
    dx, dw = fq.rms_norm_backward(*args, dev(dy, b), dev(dh, b))
    dx2, dw2 = fq.rms_norm_backward(*args, dev(dy, b), dev(dh, b))
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    for over in (0, 1):
        tdy, tdh, out = dev(dy, b), dev(dh, b), torch.empty(1000, device="cuda")
        fq.rms_norm_backward_into(*args, tdy, tdh, tdy if over else tdh, out)
        assert torch.equal(tdy if over else tdh, dx) and torch.equal(out, dw)


def test_gradient_by_differences():
    """The gradient of sum(y c) in F32 against differences in 64 bits of the
    definition: the formula's error is 2^-20 of the row's scale, the differences'
    1e-6 of it."""
    need_gpu()
    x, res, w = case(3, 50, torch.float32, True)
    c = np.random.default_rng(9).standard_normal((3, 50)).astype(np.float32).astype(np.float64)
    f = fq.rms_norm(dev(x), dev(w), 1e-3, dev(res))
    dx, dw = fq.rms_norm_backward(f["h"], dev(w), f["rstd"], dev(c))
    h = host(f["h"])

    def loss(h, w):
        return np.sum(h / np.sqrt((h * h).mean(1, keepdims=True) + 1e-3) * w * c)

    for i, j in ((0, 0), (1, 17), (2, 49)):
        d = np.zeros((3, 50))
        d[i, j] = 1e-5
        assert abs((loss(h + d, w) - loss(h - d, w)) / 2e-5 - host(dx)[i, j]) < 1e-5
        assert abs((loss(h, w + d[i]) - loss(h, w - d[i])) / 2e-5 - host(dw)[j]) < 1e-5


def test_captured_and_on_a_stream():
    """Norm, operand (two passes) and gradient captured together; replays with
    other inputs against the eager calls, on another stream too."""
    need_gpu()
    b = torch.bfloat16
    x, res, w = case(70, 512, b, True)
    dy, dh, _ = case(70, 512, b, True, seed=7)
    tx, tr, tw, ty, th = dev(x, b), dev(res, b), dev(w), dev(dy, b), dev(dh, b)

    def call(stream=None):
        a = fq.rms_norm_quantize(0, tx, tw, 1e-6, tr, rstd=True, layout=fq.TILED, stream=stream)
        dx, dw = fq.rms_norm_backward(a["h"], tw, a["rstd"], ty, th, stream=stream)
        return a["h"], fq.dequantize(0, a, stream=stream), a["tscale"], dx, dw

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    for seed in (1, 2, 3):
        x, res, _ = case(70, 512, b, True, seed=seed)
        tx.copy_(dev(x, b))
        tr.copy_(dev(res, b))
        want = call()
        g.replay()
        torch.cuda.synchronize()
        for p, q in zip(out, want):
            assert torch.equal(p, q)
        s.wait_stream(torch.cuda.current_stream())
        other = call(stream=s)
        s.synchronize()
        for p, q in zip(other, want):
            assert torch.equal(p, q)
