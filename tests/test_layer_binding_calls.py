"""The native module of the calls between the FP4 linear layers (no GPU): a call made
while another one's arguments are being read."""
import threading

import pytest
import torch

import fp4_w4a4_quantized_amd as fq
from test_layer_binding import BF, cache_args, z

GPU = "a tensor on the GPU is needed"


class Number:
    """A number that makes another call when it is read."""

    def __init__(self, value, apart):
        self.value, self.apart, self.calls = value, apart, 0

    def call(self):
        with pytest.raises(ValueError, match="y: a tensor"):
            fq.combine(None, None, None)
        self.calls += 1

    def __index__(self):
        if self.apart:
            t = threading.Thread(target=self.call)
            t.start()
            t.join()
        else:
            self.call()
        return self.value

    def __float__(self):
        return float(self.__index__())


@pytest.mark.parametrize("apart", [False, True])
def test_a_call_within_a_call(apart):
    """A host tensor that was seen before the inner call is still refused."""
    q = z(5, 4, 64, **BF)
    for f in (lambda n: fq.kv_attention(*cache_args(), q, 3, n),
              lambda n: fq.kv_attention(*cache_args(), q, n, 20, window=8, sinks=2),
              lambda n: fq.rms_norm(z(5, 64), z(64), n),
              lambda n: fq.rms_norm_quantize(fq.MXFP8, z(5, 64), z(64), n),
              lambda n: fq.route(z(4, 8), n),
              lambda n: fq.kv_read(*cache_args(), n, 64)):
        n = Number(2, apart)
        with pytest.raises(ValueError, match=GPU):
            f(n)
        assert n.calls == 1
