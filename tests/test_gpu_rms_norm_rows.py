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
