"""GPU: sizes that the calls around the products do not take are refused before
memory is asked for their results."""
import pytest
import torch

import fp4_w4a4_quantized_amd as fq
from gpu_helpers import need_gpu, say

pytestmark = pytest.mark.gpu

BF, I32 = dict(device="cuda", dtype=torch.bfloat16), dict(device="cuda", dtype=torch.int32)
z = torch.zeros


def refused(why, f, *args, **kw):
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    with pytest.raises(fq.Fp4qError, match=why):
        f(*args, **kw)
    assert torch.cuda.max_memory_allocated() == before


def test_refused_sizes_take_no_memory():
    """(The adapters' result would have 35 TB, the channels' residual 550 GB.)"""
    need_gpu()
    say("sizes refused")
    off, ad = z(2, **I32), z(1, **I32)
    refused("unsupported", fq.lora, z(1 << 24, 8, **BF), z(1, 8, 8, **BF), z(1, 1 << 20, 8, **BF), off, ad)
    refused("unsupported", fq.lora, z(4096, 12, **BF), z(1, 8, 12, **BF), z(1, 1 << 20, 8, **BF), off, ad)
    w = z(128, device="cuda")
    refused("invalid", fq.rms_norm_quantize, fq.NVFP4, z(1 << 18, 128, **BF), w, chan_idx=z(1 << 20, **I32))
    x, w = z(64, 32784, **BF), z(32784, device="cuda")
    refused("unsupported", fq.rms_norm, x, w, residual=x)
    refused("unsupported", fq.rms_norm_quantize, fq.NVFP4, x, w, residual=x)
    refused("unsupported", fq.rms_norm_backward, x, w, z(64, device="cuda"), x)


def test_refused_rotation_takes_no_memory():
    need_gpu()
    cache = z(4, 1, fq.kv_page_bytes(1, 16, 64), device="cuda", dtype=torch.uint8)
    where = [fq.MXFP4, cache, 16, z(2, **I32), z(1, 1, **I32), z(1, **I32)]
    x = z(1 << 25, 1, 64, **BF)
    refused("unsupported", fq.kv_append_rotated, *where, x, x, x, z(8, device="cuda"))
