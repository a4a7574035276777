"""GPU: the norm into an operand for batches of no rows."""
import pytest
import torch

import fp4_w4a4_quantized_amd as fq
from gpu_helpers import need_gpu

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
