"""GPU: the rotated append, the attention with a window and first tokens, the norms
into operands and the adapters together, as the example runs them
(examples/rollout_layer.py): each one's result against its plain 64-bit form on
what the layer handed to it."""
import os
import sys

import numpy as np
import pytest
import torch

import fp4_w4a4_quantized_amd as fq
from gpu_helpers import need_gpu, say
from oracle import layer as plain
from test_gpu_lora import check as check_adapters
from test_gpu_route_combine import host

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def same_codes(a, b):
    return torch.equal(a["q"], b["q"]) and torch.equal(a["scales"], b["scales"]) and \
        (a["tscale"] is None or torch.equal(a["tscale"], b["tscale"]))


@pytest.mark.parametrize("fmt", [0, 1])
def test_prompt_then_decode(fmt):
    need_gpu()
    import rollout_layer as ex
    window, sinks = 24, 3
    layer = ex.Layer(fmt, hidden=256, heads=6, kv_heads=2, dim=64, experts=8, top=3, expert_hidden=128,
                     window=window, sinks=sinks, adapters=2)
    prompts, adapters = [40, 1, 17, 70], [1, -1, 0, 1]
    seqs = ex.Sequences(layer, prompts, room=3, adapters=adapters)
    cache = seqs.cache.cpu().numpy()
    x = torch.randn(sum(prompts), 256, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    off, counts = seqs.new(prompts), prompts
    t = None if layer.kv_scale is None else layer.kv_scale.cpu().numpy()
    u, uo = (2.0 ** -11 if fmt == 0 else 2.0 ** -8), 2.0 ** -8
    for step in range(4):
        say(f"layer fmt {fmt} pass {step}")
        keep = {}
        y = ex.forward(layer, seqs, x, off, max(counts), keep)
        assert torch.isfinite(y).all() and y.shape == x.shape
        offs, table, lens = off.cpu().numpy(), seqs.table.cpu().numpy(), seqs.lens.cpu().numpy()
        rows = int(offs[-1])
        # the norms and their operands
        for a, w, h, res in ((keep["a1"], layer.norm1, x, None), (keep["a2"], layer.norm2, keep["out"], x)):
            hh, _, yy = plain.rms_norm(host(h), host(w), 1e-6, None if res is None else host(res))
            assert np.array_equal(host(a["h"]), hh) and np.array_equal(host(a["y"]), plain.bf16_round(yy))
            assert same_codes(a, fq.quantize(fmt, a["y"]))
        # the adapters
        A, B, scale = layer.adapters
        check_adapters(dict(x=host(keep["a1"]["y"]), a=host(A), b=host(B), off=offs, ad=adapters, scale=host(scale),
                            y=host(keep["shared"]), K=256, N=B.shape[1], rank=A.shape[1], dt=torch.bfloat16),
                       keep["qkv"].reshape(rows, -1))
        # rotation and append
        qkv, pos = host(keep["qkv"]), plain.token_positions(offs, lens, rows)
        turned = plain.rotate(qkv[:, :8], pos, host(layer.freqs))
        assert np.array_equal(host(keep["q"]), turned[:, :6]) and np.array_equal(host(keep["k"]), turned[:, 6:])
        plain.kv_append(fmt, cache, seqs.page, offs, table, lens, turned[:, 6:], qkv[:, 8:], t, t)
        got = seqs.cache.cpu().numpy()
        for b in range(len(prompts)):
            at = np.arange(lens[b])
            kb, _, vb, _, ks, vs = plain.kv_places(fmt, seqs.page, layer.dim)
            pid, slot = table[b][at // seqs.page], at % seqs.page
            for place in (kb, vb, ks, vs):
                assert np.array_equal(got[pid[:, None], :, place[slot]], cache[pid[:, None], :, place[slot]])
        # attention, its tolerance as in test_gpu_kv_attention.py
        o, w, s = plain.attention(fmt, cache, seqs.page, offs, table, lens, host(keep["q"]), t, t, window, None, sinks)
        d = (80 * 2.0 ** -24 + 2.0 ** -23 + (2.0 ** -25 if fmt == 0 else 0.0)) * s
        tol = (u + 2 * d + 2.0 ** -20) * w
        assert np.all(np.abs(host(keep["att"]) - o) <= tol + uo * (np.abs(o) + tol))
        # the next token of each sequence
        last = torch.tensor(offs[1:].astype(np.int64) - 1).cuda()
        x, counts = ex.norm(y[last]), [1] * len(prompts)
        off = seqs.new(counts)
        seqs.lens += 1
        seqs.bound += 1


def test_a_decode_step_captured():
    """The whole attention part of a decode step in one graph: each replay, with
    lengths that grow, against the eager calls on a copy of the cache."""
    need_gpu()
    import rollout_layer as ex
    layer = ex.Layer(0, hidden=256, heads=6, kv_heads=2, dim=64, experts=8, top=3, expert_hidden=128, window=16,
                     sinks=2, adapters=2)
    seqs = ex.Sequences(layer, [30, 9, 21], room=8, adapters=[0, 1, -1])
    seqs.cache.zero_()
    x = torch.randn(3, 256, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    off, t = seqs.new([1, 1, 1]), layer.kv_scale

    def step():
        a = fq.rms_norm_quantize(0, x, layer.norm1, y_dtype=fq.OUT_BF16)
        qkv = fq.gemm(0, a, layer.qkv, y_dtype=fq.OUT_BF16)
        fq.lora_into(a["y"], *layer.adapters[:2], off, seqs.adapters, layer.adapters[2], qkv, qkv)
        qkv = qkv.view(3, 10, 64)
        where = (seqs.cache, seqs.page, off, seqs.table, seqs.lens)
        q = fq.kv_append_rotated(0, *where, qkv[:, :6], qkv[:, 6:8], qkv[:, 8:], layer.freqs, t, t)
        att = fq.kv_attention(0, *where, q, 1, 64, t, t, window=16, sinks=2)
        return fq.rms_norm_quantize(0, att.view(3, 384), torch.ones(384, device="cuda"), y_dtype=fq.OUT_BF16)["y"]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    seqs.cache.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for i in range(4):
        seqs.lens += 1
        x.mul_(-0.9)
        before = seqs.cache.clone()
        want = step().clone()
        after = seqs.cache.clone()
        seqs.cache.copy_(before)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(seqs.cache, after)
