"""GPU: calls around the products that the documentation allows beside the ones of the
operators' own tests: results over inputs in several turns of rows, queries turned
where they stand in a packed projection, F32 values beside an operand, streams."""
import numpy as np
import pytest
import torch

import fp4_w4a4_quantized_amd as fq
from gpu_helpers import need_gpu, say
from oracle import layer
from test_gpu_kv_attention import make
from test_gpu_kv_rotated import args_of, bf16, bits, freqs_of, inputs
from test_gpu_kv_rotated import dev as dev_np
from test_gpu_rms_norm import case, dev, host, same_operand, strided

pytestmark = pytest.mark.gpu

B = torch.bfloat16


@pytest.mark.parametrize("fmt", [fq.NVFP4, fq.MXFP4, fq.MXFP8])
@pytest.mark.parametrize("rows,cols", [(8201, 128), (2100, 1152), (1100, 4224)])
def test_h_over_its_inputs(fmt, rows, cols):
    """h over x or over the residual, rows of their own strides: the operand and h as
    without; y beside it in F32."""
    need_gpu()
    say(f"h in place fmt {fmt} {rows} x {cols}")
    x, res, w = case(rows, cols, B, True)
    h, _, y = layer.rms_norm(x, w, 1e-6, res)
    want = fq.rms_norm_quantize(fmt, dev(x, B), dev(w), 1e-6, dev(res, B))
    for over in (0, 1):
        tx, tr = strided(x, B, 8), strided(res, B, 3)
        a = fq.rms_norm_quantize(fmt, tx, dev(w), 1e-6, tr, h=tr if over else tx, y_dtype=fq.OUT_F32)
        assert np.array_equal(host(tr if over else tx), h) and a["h"] is (tr if over else tx)
        assert torch.equal(a["q"], want["q"]) and torch.equal(a["scales"], want["scales"])
        assert fmt != fq.NVFP4 or torch.equal(a["tscale"], want["tscale"])
        assert a["y"].dtype == torch.float32
        assert np.all(np.abs(host(a["y"]) - y) <= (2.0 ** -24 + 2.0 ** -48) * np.abs(y) + 2.0 ** -149)
        # and the plain norm, its y over the other input
        tx, tr = dev(x, B), dev(res, B)
        fq.rms_norm_into(tx, dev(w), 1e-6, tr, tr if over else tx, tx if over else tr, torch.empty(rows, device="cuda"))
        assert np.array_equal(host(tr if over else tx), h)
        assert np.array_equal(host(tx if over else tr), layer.bf16_round(y))


def test_gradient_over_its_inputs():
    need_gpu()
    for rows, cols in ((5000, 130), (1500, 4300)):
        x, res, w = case(rows, cols, B, True)
        dy, dh, _ = case(rows, cols, B, True, seed=7)
        f = fq.rms_norm(dev(x, B), dev(w), 1e-5, dev(res, B))
        args = f["h"], dev(w), f["rstd"]
        dx, dw = fq.rms_norm_backward(*args, dev(dy, B), dev(dh, B))
        for over in (0, 1):
            tdy, tdh, out = strided(dy, B, 5), strided(dh, B, 2), torch.empty(cols, device="cuda")
            fq.rms_norm_backward_into(*args, tdy, tdh, tdy if over else tdh, out)
            assert torch.equal(tdy if over else tdh, dx) and torch.equal(out, dw)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("n", [[2, 0, 7], [1700, 3]])
@pytest.mark.parametrize("inter", [False, True])
def test_queries_turned_where_they_stand(fmt, n, inter):
    """q_out is q, a part of one packed tensor with k and v: those stay, and the cache
    and the queries are as with a q_out of its own."""
    need_gpu()
    say(f"rotated append in place fmt {fmt} n {n} interleaved {inter}")
    c = make(fmt, n, [a + 9 for a in n], H=2, D=128, page=16, seed=3)
    q, k, v = inputs(c, 12, 5, extra=2)
    t = None if c["t"] is None else dev_np(c["t"])
    f = dev_np(freqs_of(64))
    qkv = bf16(np.concatenate([q, k, v], 1))
    one, two = dev_np(c["cache"]), dev_np(c["cache"])
    want = fq.kv_append_rotated(fmt, *args_of(c, one), qkv[:, :12].contiguous(), qkv[:, 12:14], qkv[:, 14:], f, t, t,
                                interleaved=inter)
    before = qkv.clone()
    fq.kv_append_rotated_into(fmt, *args_of(c, two), qkv[:, :12], qkv[:, 12:14], qkv[:, 14:], f, t, t, qkv[:, :12],
                              interleaved=inter)
    assert np.array_equal(bits(qkv[:, :12]), bits(want)) and torch.equal(one, two)
    assert np.array_equal(bits(qkv[:, 12:]), bits(before[:, 12:]))


def test_on_a_stream_beside_other_work():
    """The calls on a stream of their own while the current one is busy, results read
    there afterwards; two sets of inputs at once give what each gives alone."""
    need_gpu()
    c = make(0, [1, 40], [900, 300], G=4, H=2, D=128, page=16, seed=2)
    t = dev_np(c["t"])
    where = args_of(c, dev_np(c["cache"]))
    q = bf16(c["q"])
    x, res, w = case(300, 2048, B, True)
    tx, tr, tw = dev(x, B), dev(res, B), dev(w)

    def calls(stream):
        a = fq.rms_norm_quantize(0, tx, tw, 1e-6, tr, rstd=True, stream=stream)
        o = fq.kv_attention(0, *where, q, 40, 1000, t, t, window=200, sinks=5, stream=stream)
        return a["q"], a["scales"], a["tscale"], a["rstd"], o

    want = [u.clone() for u in calls(None)]
    busy = torch.randn(2048, 2048, device="cuda")
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        got = [calls(s) for s in streams for _ in range(4)]
        for _ in range(4):
            busy = busy @ busy * 1e-3
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        for g in got:
            for a, b in zip(g, want):
                assert torch.equal(a, b)
