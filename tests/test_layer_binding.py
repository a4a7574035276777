"""The native module of the calls between the FP4 linear layers (no GPU): each
check of its tensors is reached, with the reason given, before anything
touches a GPU."""
import pytest
import torch

import fp4_w4a4_quantized_amd as fq
from fp4_w4a4_quantized_amd import binding

z = torch.zeros
I32, BF = dict(dtype=torch.int32), dict(dtype=torch.bfloat16)


def cache_args(rows=5):
    cache = z(4, 2, fq.kv_page_bytes(1, 16, 64), dtype=torch.uint8)
    return [1, cache, 16, z(3, **I32), z(2, 3, **I32), z(2, **I32)]


def test_host_tensors_are_refused_after_the_other_checks():
    k = z(5, 2, 64, **BF)
    gpu = "a tensor on the GPU is needed"
    with pytest.raises(ValueError, match=gpu):
        fq.kv_append(*cache_args(), k, k)
    with pytest.raises(ValueError, match=gpu):
        fq.kv_read(*cache_args(), 5, 64)
    with pytest.raises(ValueError, match=gpu):
        fq.kv_attention(*cache_args(), z(5, 4, 64, **BF), 3, 20)
    with pytest.raises(ValueError, match=gpu):
        fq.route(z(4, 8), 2)
    with pytest.raises(ValueError, match=gpu):
        fq.route_backward(z(4, 8), z(4, 2, **I32), z(4, 2))
    with pytest.raises(ValueError, match=gpu):
        fq.combine(z(8, 4), z(2, 2, **I32), z(2, 2))
    with pytest.raises(ValueError, match=gpu):
        fq.combine_backward(z(8, 4), z(2, 2, **I32), z(2, 2), z(2, 4))


@pytest.mark.parametrize("i,bad,why", [
    (1, z(4, 2, 100, dtype=torch.uint8), "cache: its page bytes"),
    (1, z(4, 2, 16 * 68, dtype=torch.int8), "cache: contiguous u8"),
    (3, z(4, **I32), "offsets: another number"), (3, z(3), "offsets: contiguous int32"),
    (4, z(6, **I32), "page_table: int32"), (4, z(2, 6, **I32)[:, ::2], "page_table: int32"),
    (5, z(3, **I32), "lens: another number"),
    (6, z(5, 2, 64), "k: bf16"), (6, z(5, 128, **BF), "k: .rows, heads, dim."),
    (6, z(5, 4, 64, **BF), "v: k's shape"), (7, z(6, 2, 64, **BF), "v: k's shape"),
    (8, z(3), "k_scale: another number"), (9, z(2, **BF), "v_scale: contiguous f32"),
    (6, None, "k: a tensor"), (4, [[0]], "page_table: a tensor")])
def test_cache_tensors(i, bad, why):
    k = z(5, 2, 64, **BF)
    args = cache_args() + [k, k, None, None]
    args[i] = bad
    with pytest.raises(ValueError, match=why):
        fq.kv_append(*args)


def test_attention_tensors():
    q = z(5, 4, 64, **BF)
    for y, why in ((z(5, 4, 64, dtype=torch.float16), "y: bf16 or f32"), (z(5, 3, 64), "y: q's shape"),
                   (z(5, 64, 4).transpose(1, 2), "y: .rows")):
        with pytest.raises(ValueError, match=why):
            fq.kv_attention_into(*cache_args(), q, 3, 20, None, None, 0, 0.1, y, None)
    with pytest.raises(ValueError, match="window: out of range"):
        fq.kv_attention(*cache_args(), q, 3, 20, window=1 << 40)
    with pytest.raises(TypeError):
        fq.kv_attention(*cache_args(), q, "3", 20)


def test_router_and_combination_tensors():
    x = z(4, 8)
    out = [z(4, 2, **I32), z(4, 2), z(9, **I32), z(8, **I32), z(4, 2, **I32)]

    def into(i, bad, why):
        t = list(out)
        t[i] = bad
        with pytest.raises(ValueError, match=why):
            fq.route_into(x, 2, 0, None, 1, 1, True, *t, None)

    into(0, z(4, 1, **I32), "experts: another number")
    into(1, z(4, 3), "weights: another number")
    into(2, z(8, **I32), "offsets: another number")
    into(3, z(7, **I32), "row_src: another number")
    into(4, z(4, 2), "row_of: contiguous int32")
    for d, why in ((z(4, 7), "d_logits: the logits"), (z(4, 8, **BF), "d_logits: the logits")):
        with pytest.raises(ValueError, match=why):
            fq.route_backward_into(x, out[0], out[1], 0, True, d)
    with pytest.raises(ValueError, match="experts: one row"):
        fq.route_backward(x, z(3, 2, **I32), z(3, 2))
    y, r, w = z(8, 4), z(2, 2, **I32), z(2, 2)
    with pytest.raises(ValueError, match="out: .tokens, cols."):
        fq.combine_into(y, r, w, z(3, 4))
    with pytest.raises(ValueError, match="d_out: .tokens, cols."):
        fq.combine_backward(y, r, w, z(2, 4, **BF))
    with pytest.raises(ValueError, match="d_y: y's shape"):
        fq.combine_backward_into(y, r, w, z(2, 4), z(7, 4), w)
    with pytest.raises(ValueError, match="row_of: .tokens, k."):
        fq.combine(y, z(4, **I32), w)


def test_the_module_names_its_argument_counts():
    with pytest.raises(TypeError, match="11 arguments"):
        binding._layer().append(None)


def test_sizes_past_a_launch_are_refused():
    L, A = binding.lib(), 0x10000
    kv = [0, A, 4, 16, 1 << 10, 128, A, 1 << 12, A, 3, 3, A, 5]
    call = lambda heads: L.fp4q_kv_attention(*kv, A, 1 << 20, heads, 1, 40, 0, 0.1, A, A, A, 1, 1 << 20,
                                             A, 1 << 30, None)
    assert call(1 << 10) == -2
    assert L.fp4q_route(A, 0, 1 << 26, 8, 8, 2, 0, None, 1, 1, 1, A, A, A, A, A, A, 1 << 40, None) == -2
    assert L.fp4q_route_backward(A, 0, 1 << 26, 8, 8, 2, 0, 1, A, A, A, 8, None) == -2
