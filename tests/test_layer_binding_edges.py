"""The native module of the calls between the FP4 linear layers (no GPU): sizes
that are refused are refused before memory is asked for."""
import pytest
import torch

import fp4_w4a4_quantized_amd as fq

I32 = dict(dtype=torch.int32)


@pytest.mark.parametrize("k", [33, 2 ** 31 - 1, 0])
def test_a_route_without_room(k):
    """(26 TB of results for the largest k; a host tensor is refused after the
    other checks of the module)"""
    with pytest.raises(ValueError, match="a tensor on the GPU is needed"):
        fq.route(torch.zeros(1000, 64), k)


def test_a_read_without_room():
    cache = torch.zeros(4, 2, fq.kv_page_bytes(1, 16, 64), dtype=torch.uint8)
    where = [1, cache, 16, torch.zeros(3, **I32), torch.zeros(2, 3, **I32), torch.zeros(2, **I32)]
    for rows in (2 ** 31, 2 ** 40, 2 ** 62):
        with pytest.raises(ValueError, match="a tensor on the GPU is needed"):
            fq.kv_read(*where, rows, 64)


def test_an_attention_without_room():
    cache = torch.zeros(4, 2, fq.kv_page_bytes(1, 16, 64), dtype=torch.uint8)
    where = [1, cache, 16, torch.zeros(3, **I32), torch.zeros(2, 3, **I32), torch.zeros(2, **I32)]
    for max_new, max_len in ((3, 2 ** 62), (2 ** 62, 20), (2 ** 40, 2 ** 40)):
        with pytest.raises(ValueError, match="a tensor on the GPU is needed"):
            fq.kv_attention(*where, torch.zeros(5, 4, 64, dtype=torch.bfloat16), max_new, max_len)
