"""GPU: the norm into an operand for batches of no rows, of more rows than a pass has
workgroups (1024, each with a row, or four rows of up to 1024 columns, at a time),
and with tensor scales far from the values, bit for bit against the quantizer's
operand of the BF16 y and the plain 64-bit form (which test_gpu_rms_norm.py
derives)."""
import numpy as np
import pytest
import torch

import fp4_w4a4_quantized_amd as fq
from gpu_helpers import need_gpu, say
from oracle import layer
from test_gpu_rms_norm import case, dev, host, none, same_operand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [fq.NVFP4, fq.MXFP4])
@pytest.mark.parametrize("layout", [fq.ROWMAJOR, fq.TILED])
def test_no_rows_with_channels(fmt, layout):
    need_gpu()
    x, w = torch.zeros(0, 128, device="cuda", dtype=torch.bfloat16), torch.ones(128, device="cuda")
    chan = torch.arange(0, 128, 9, device="cuda", dtype=torch.int32)
    for residual in (None, x):
        a = fq.rms_norm_quantize(fmt, x, w, residual=residual, chan_idx=chan, layout=layout, y_dtype=fq.OUT_BF16,
                                 rstd=True)
        assert a["rows"] == 0 and a["resid"].shape == (0, chan.numel()) and a["y"].shape == (0, 128)
        assert fq.dequantize(fmt, a).shape == (0, 128) and (fmt or a["tscale"].item() == 1.0)


@pytest.mark.parametrize("fmt", [fq.NVFP4, fq.MXFP4])
def test_no_rows_through_the_product(fmt):
    """The norm's operand and the quantizer's into the compensated product."""
    need_gpu()
    x, w = torch.zeros(0, 128, device="cuda", dtype=torch.bfloat16), torch.ones(128, device="cuda")
    chan = torch.arange(0, 128, 16, device="cuda", dtype=torch.int32)
    b = fq.quantize(fmt, torch.ones(64, 128, device="cuda", dtype=torch.bfloat16))
    for a in (fq.rms_norm_quantize(fmt, x, w, chan_idx=chan), fq.quantize(fmt, x, chan_idx=chan)):
        assert a["resid"].shape == (0, 8) and fq.gemm(fmt, a, b, chan_idx=chan).shape == (0, 64)


# two turns of rows and more: a wave a row; four waves, loads of the next row ahead;
# four and eight waves without; and the second turn of one row alone
TURNS = [(8201, 128), (4101, 1024), (2100, 1152), (1025, 2048), (1100, 4224), (1040, 8320), (1026, 16512)]


@pytest.mark.parametrize("fmt", [fq.NVFP4, fq.MXFP4])
@pytest.mark.parametrize("layout", [fq.ROWMAJOR, fq.TILED])
@pytest.mark.parametrize("rows,cols", TURNS)
def test_rows_in_several_turns(fmt, layout, rows, cols):
    need_gpu()
    say(f"norm turns fmt {fmt} layout {layout} {rows} x {cols}")
    b = torch.bfloat16
    x, res, w = case(rows, cols, b, True)
    h, r, y = layer.rms_norm(x, w, 1e-6, res)
    yb = dev(layer.bf16_round(y), b)
    chan = dev(np.sort(np.random.default_rng(cols).permutation(cols)[:24])).int()
    args = dev(x, b), dev(w), 1e-6, dev(res, b)
    for ch in (chan, None):
        want = fq.quantize(fmt, yb, chan_idx=ch, layout=layout)
        a = fq.rms_norm_quantize(fmt, *args, chan_idx=ch, layout=layout, y_dtype=fq.OUT_BF16, rstd=True)
        same_operand(a, want, fmt, layout, rows, cols)
        assert np.array_equal(host(a["h"]), h) and torch.equal(a["y"], yb)
        assert np.all(np.abs(host(a["rstd"])[:, None] - r) <= (2.0 ** -24 + 2.0 ** -50) * r)
        if fmt == fq.NVFP4:
            b1 = fq.rms_norm_quantize(fmt, *args, tscale=want["tscale"], chan_idx=ch, layout=layout)
            same_operand(b1, want, fmt, layout, rows, cols)


@pytest.mark.parametrize("rows,cols", [(8201, 96), (2100, 1152), (1100, 4224)])
def test_rows_in_several_turns_mxfp8(rows, cols):
    need_gpu()
    say(f"norm turns MXFP8 {rows} x {cols}")
    x, res, w = case(rows, cols, torch.bfloat16, True)
    h, r, y = layer.rms_norm(x, w, 1e-6, res)
    codes, sc, _ = layer.mxfp8_quantize(layer.bf16_round(y))
    a = fq.rms_norm_quantize(fq.MXFP8, dev(x, torch.bfloat16), dev(w), 1e-6, dev(res, torch.bfloat16))
    assert np.array_equal(host(a["h"]), h)
    assert np.array_equal(a["q"].cpu().numpy(), codes) and np.array_equal(a["scales"].cpu().numpy(), sc)


@pytest.mark.parametrize("rows,cols", [(8201, 128), (2100, 1152), (1100, 4224)])
def test_the_largest_value_in_any_turn(rows, cols):
    """The tensor's largest magnitude in the first row, in a later turn's and in the
    last one: the tensor scale sees every workgroup's maximum."""
    need_gpu()
    b = torch.bfloat16
    x, _, w = case(rows, cols, b, False)
    w[-1] = 40.0
    for row in (0, 1, rows // 2, rows - 1):
        t = x.copy()
        t[:, -1] *= 0.01
        t[row, -1] = -64.0
        y = layer.bf16_round(layer.rms_norm(layer.bf16_round(t), w, 1e-6)[2])
        assert np.abs(y).max() == np.abs(y[row, -1])
        a = fq.rms_norm_quantize(fq.NVFP4, dev(t, b), dev(w), 1e-6)
        assert a["tscale"].item() == np.float32(np.abs(y).max()) / np.float32(2688)
        same_operand(a, fq.quantize(fq.NVFP4, dev(y, b)), fq.NVFP4, fq.ROWMAJOR, rows, cols)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1023, 33), (5000, 130), (9001, 96)])
def test_gradient_of_many_rows(dt, rows, cols):
    """d_weight: rows / n terms in each of n workgroups (a quarter of the rows, 256 to
    1024 of them), n / 16 and 16 of those sums after it, and u's and the product's three
    units of 2^-24."""
    need_gpu()
    say(f"norm gradient {dt} {rows} x {cols}")
    x, res, w = case(rows, cols, dt, True)
    dy, dh, _ = case(rows, cols, dt, True, seed=7)
    h, r, _ = layer.rms_norm(x, w, 1e-5, res, dt == torch.bfloat16)
    f = fq.rms_norm(dev(x, dt), dev(w, dt), 1e-5, dev(res, dt))
    want, want_w, mean, total = layer.rms_norm_backward(h, w, r, dy, dh)
    dx, dw = fq.rms_norm_backward(f["h"], dev(w, dt), f["rstd"], dev(dy, dt), dev(dh, dt))
    e = 2.0 ** -24
    u, g = np.abs(h * r), np.abs(w * dy)
    s = np.abs((w * dy * h * r).mean(1, keepdims=True))
    tol = r * (4 * e * g + u * (8 * e * s + 84 * e * mean)) + 4 * e * np.abs(want)
    tol = tol + (2.0 ** -8 if dt == torch.bfloat16 else e) * (np.abs(want) + tol) + 2.0 ** -149
    assert np.all(np.abs(host(dx) - want) <= tol)
    n = min(max(rows // 4, 256), 1024)
    units = -(-rows // n) + -(-n // 16) + 16 + 3
    assert np.all(np.abs(host(dw) - want_w) <= units * e * total + 2.0 ** -149)


# ---- tensor scales far from the values ------------------------------------------

def check_scale(y, a, chan, t, layout, rows, cols):
    """The operand a of y (BF16 values) under the scale t, against the 64-bit encoder."""
    with np.errstate(over="ignore"):
        codes, sc, val = layer.kv_quantize(fq.NVFP4, y, np.full(rows, t, np.float32))
    assert np.array_equal(host(fq.dequantize(fq.NVFP4, a, fq.OUT_F32)), val)
    if layout == fq.ROWMAJOR:
        assert np.array_equal(a["q"].cpu().numpy(), codes[:, ::2] | codes[:, 1::2] << 4)
        assert np.array_equal(a["scales"].cpu().numpy(), sc)
    d = (y - val).astype(np.float32)[:, chan]
    assert np.array_equal(host(a["resid"].view(torch.bfloat16)), layer.bf16_round(d))


def with_zeros(x):
    """Rows and blocks of zeros of either sign, and single ones."""
    x[0, :40], x[1], x[2, 16:64] = 0.0, -0.0, -0.0
    x[3, ::5] = -0.0
    return x


@pytest.mark.parametrize("layout", [fq.ROWMAJOR, fq.TILED])
@pytest.mark.parametrize("rows,cols", [(70, 256), (1100, 1152), (4100, 128)])
def test_given_scales_far_from_the_values(layout, rows, cols):
    """Values past 2688 times the scale saturate, however far; scales on either side
    of where the encoder's divisions are replaced (2^-80 .. 2^80)."""
    need_gpu()
    b = torch.bfloat16
    x, _, w = case(rows, cols, b, False)
    x = with_zeros(x)
    y = layer.bf16_round(layer.rms_norm(x, w, 1e-6)[2])
    chan = np.sort(np.random.default_rng(1).permutation(cols)[:32])
    own = np.abs(y).max() / 2688.0
    for f in (own / 64, own / 7, own * 64, own * 5000, 2.0 ** -20, 2.0 ** -60, 2.0 ** -80, 2.0 ** -80 * (1 - 2.0 ** -24),
              2.0 ** -90, 2.0 ** -126, 2.0 ** -140, 2.0 ** 60, 2.0 ** 80, 2.0 ** 80 * (1 + 2.0 ** -23), 2.0 ** 90,
              2.0 ** 120):
        t = np.float32(f)
        say(f"norm given scale {t} layout {layout} {rows} x {cols}")
        a = fq.rms_norm_quantize(fq.NVFP4, dev(x, b), dev(w), 1e-6, tscale=dev([t]), chan_idx=dev(chan).int(),
                                 layout=layout)
        check_scale(y, a, chan, t, layout, rows, cols)


@pytest.mark.parametrize("layout", [fq.ROWMAJOR, fq.TILED])
@pytest.mark.parametrize("e", [-126, -100, -73, -68, 68, 88, 93, 100, 124])
def test_own_scales_of_extreme_values(layout, e):
    """y near 2^e: the tensor scale lies on either side of the encoder's range, or is
    a subnormal number."""
    need_gpu()
    b, rows, cols = torch.bfloat16, 66, 384
    x, _, w = case(rows, cols, b, False)
    x, w = with_zeros(x), layer.bf16_round(w * 0.25) * 2.0 ** e
    y = layer.bf16_round(layer.rms_norm(x, w, 1e-6)[2])
    assert np.isfinite(y).all() and np.abs(y).max() > 0
    chan = np.sort(np.random.default_rng(1).permutation(cols)[:32])
    c = dev(chan).int()
    a = fq.rms_norm_quantize(fq.NVFP4, dev(x, b), dev(w), 1e-6, chan_idx=c, layout=layout)
    t = np.float32(np.abs(y).max()) / np.float32(2688)
    assert a["tscale"].item() == t
    check_scale(y, a, chan, t, layout, rows, cols)
    same_operand(a, fq.quantize(fq.NVFP4, dev(y, b), chan_idx=c, layout=layout), fq.NVFP4, layout, rows, cols)
