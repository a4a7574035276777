"""GPU: the operators between the FP4 linear layers together, as the example
runs them (examples/rollout_layer.py): each one's result against its plain
64-bit form on what the layer handed to it."""
import os
import sys

import numpy as np
import pytest
import torch

import fp4_w4a4_quantized_amd as fq
from gpu_helpers import need_gpu, say
from oracle import layer as plain
from test_gpu_kv_attention import check_close
from test_gpu_route_combine import U, host

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [0, 1])
def test_prompt_then_decode(fmt):
    need_gpu()
    import rollout_layer as ex
    layer = ex.Layer(fmt, hidden=256, heads=6, kv_heads=2, dim=64, experts=8, top=3, expert_hidden=128)
    prompts = [40, 1, 17, 70]
    seqs = ex.Sequences(layer, prompts, room=3)
    cache = seqs.cache.cpu().numpy()               # what no token owns yet: anything
    x = torch.randn(sum(prompts), 256, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    off, counts = seqs.new(prompts), prompts
    t = None if layer.kv_scale is None else layer.kv_scale.cpu().numpy()
    for step in range(4):
        say(f"layer fmt {fmt} pass {step}")
        keep = {}
        y = ex.forward(layer, seqs, x, off, max(counts), keep)
        assert torch.isfinite(y).all() and y.shape == x.shape
        offs, table, lens = off.cpu().numpy(), seqs.table.cpu().numpy(), seqs.lens.cpu().numpy()
        plain.kv_append(fmt, cache, seqs.page, offs, table, lens, host(keep["k"]), host(keep["v"]), t, t)
        got = seqs.cache.cpu().numpy()
        for b in range(len(prompts)):              # the pages' stored tokens, byte for byte
            pos = np.arange(lens[b])
            kb, _, vb, _, ks, vs = plain.kv_places(fmt, seqs.page, layer.dim)
            pid, slot = table[b][pos // seqs.page], pos % seqs.page
            for at in (kb, vb, ks, vs):
                assert np.array_equal(got[pid[:, None], :, at[slot]], cache[pid[:, None], :, at[slot]])
        check_close(dict(fmt=fmt, cache=cache, page=seqs.page, off=offs, table=table, lens=lens,
                         q=host(keep["q"]), t=t, D=layer.dim), keep["att"])
        want = plain.route(host(keep["logits"]), layer.top)
        for key in ("experts", "offsets", "row_src", "row_of"):
            assert np.array_equal(keep["route"][key].cpu().numpy(), want[key]), key
        out, mag = plain.combine(host(keep["y"]), want["row_of"], host(keep["route"]["weights"]))
        tol = (layer.top + 1) * 2.0 ** -24 * mag
        assert np.all(np.abs(host(keep["moe"]) - out) <= tol + U[torch.bfloat16] * (np.abs(out) + tol))
        # the next token of each sequence
        last = torch.tensor(offs[1:].astype(np.int64) - 1).cuda()
        x, counts = ex.norm(y[last]), [1] * len(prompts)
        off = seqs.new(counts)
        seqs.lens += 1
        seqs.bound += 1


def test_example_runs(capsys):
    need_gpu()
    import rollout_layer as ex
    argv, sys.argv = sys.argv, ["rollout_layer.py", "--steps", "3"]
    try:
        ex.main()
    finally:
        sys.argv = argv
    assert "decode: 3 steps" in capsys.readouterr().out
