"""One decoder layer of a rollout, W4A4 with an FP4 key/value cache and an
expert layer, as its caller would run it: a prompt pass of a ragged batch,
then decode steps of one token a sequence.

    python examples/rollout_layer.py [--fmt nvfp4|mxfp4] [--steps N]

Every product runs in FP4 (fp4q_gemm, fp4q_grouped_gemm) on operands that the
norms before them write, with the adapters of each sequence's request beside the
first one.  Keys are turned by their positions on the way into FP4 pages, which the
attention reads there (a sliding window and the first tokens, in the run below),
the router's order feeds the quantize-before-permute grouped products, and the
combination brings the experts' outputs back.  Weights are random; torch supplies the router's projection,
the activation and the addition of the experts' outputs to the residual stream.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fp4_w4a4_quantized_amd as fq  # noqa: E402


class Layer:
    """The layer's weights, quantized once."""

    def __init__(self, fmt, hidden=1024, heads=16, kv_heads=4, dim=64, experts=16, top=4,
                 expert_hidden=512, seed=0, window=0, sinks=0, adapters=0, rank=8):
        self.fmt, self.heads, self.kv_heads, self.dim = fmt, heads, kv_heads, dim
        self.experts, self.top, self.window, self.sinks = experts, top, window, sinks
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(n, k):
            w = torch.randn(n, k, generator=g, device="cuda") * k ** -0.5
            return fq.quantize(fmt, w.to(torch.bfloat16))

        def expert_weights(n, k):
            parts = [weight(n, k) for _ in range(experts)]
            ts = torch.cat([p["tscale"] for p in parts]) if fmt == fq.NVFP4 else None
            return (torch.stack([p["q"] for p in parts]), torch.stack([p["scales"] for p in parts]),
                    ts)

        self.qkv = weight((heads + 2 * kv_heads) * dim, hidden)
        self.out = weight(hidden, heads * dim)
        self.up = expert_weights(expert_hidden, hidden)
        self.down = expert_weights(hidden, expert_hidden)
        self.router = torch.randn(hidden, experts, generator=g, device="cuda") * hidden ** -0.5
        self.norm1 = 1.0 + 0.1 * torch.randn(hidden, generator=g, device="cuda")
        self.norm2 = 1.0 + 0.1 * torch.randn(hidden, generator=g, device="cuda")
        self.freqs = 10000.0 ** (-torch.arange(dim // 2, device="cuda") / (dim // 2))
        qkv = (heads + 2 * kv_heads) * dim
        # the requests' adapters beside the projection to queries, keys and values
        self.adapters = None if adapters == 0 else (
            (torch.randn(adapters, rank, hidden, generator=g, device="cuda") * hidden ** -0.5).to(torch.bfloat16),
            (0.3 * torch.randn(adapters, qkv, rank, generator=g, device="cuda")).to(torch.bfloat16),
            torch.full((adapters,), 0.5, device="cuda"))
        # tensor scales of keys and values, as a calibration would leave them
        self.kv_scale = (torch.full((kv_heads,), 8.0 / 2688.0, device="cuda")
                         if fmt == fq.NVFP4 else None)


class Sequences:
    """Pages, lengths and new tokens of a batch of sequences."""

    def __init__(self, layer, lengths, room, page=16, seed=1, adapters=None):
        self.page, self.lengths = page, list(lengths)
        # the adapter of each sequence (-1: none)
        self.adapters = None if adapters is None else torch.tensor(adapters, dtype=torch.int32, device="cuda")
        need = [-(-(n + room) // page) for n in lengths]
        self.cache = fq.kv_cache(layer.fmt, sum(need), page, layer.kv_heads, layer.dim)
        ids = torch.randperm(sum(need), generator=torch.Generator().manual_seed(seed)).int()
        table = torch.full((len(need), max(need)), -1, dtype=torch.int32)
        for b, part in enumerate(ids.split(need)):
            table[b, :need[b]] = part
        self.table = table.cuda()
        self.lens = torch.tensor(self.lengths, dtype=torch.int32, device="cuda")
        self.bound = max(self.lengths)         # no sequence is longer

    def new(self, counts):
        """Offsets of the new tokens' rows (counts of each sequence)."""
        off = torch.zeros(len(counts) + 1, dtype=torch.int32)
        off[1:] = torch.tensor(counts).cumsum(0)
        return off.cuda()


def norm(x):
    return fq.rms_norm(x, torch.ones(x.shape[1], device=x.device))["y"]


def forward(layer, seqs, x, offsets, max_new, keep=None):
    """x [rows, hidden] bf16: the new tokens of every sequence (already counted
    in seqs.lens).  Returns the layer's output; keep: a dict for what passes
    between the operators."""
    fmt, H, KV, D = layer.fmt, layer.heads, layer.kv_heads, layer.dim
    rows = x.shape[0]
    # attention
    a1 = fq.rms_norm_quantize(fmt, x, layer.norm1, y_dtype=fq.OUT_BF16)
    shared = fq.gemm(fmt, a1, layer.qkv, y_dtype=fq.OUT_BF16)
    qkv = shared
    if layer.adapters is not None:
        a, b, scale = layer.adapters
        qkv = fq.lora(a1["y"], a, b, offsets, seqs.adapters, scale, y=shared)
    qkv = qkv.view(rows, H + 2 * KV, D)
    k, v = qkv[:, H:H + KV], qkv[:, H + KV:]
    where = (seqs.cache, seqs.page, offsets, seqs.table, seqs.lens)
    # (to show the turned keys too, they are given as queries beside these)
    turned = fq.kv_append_rotated(fmt, *where, qkv[:, :H if keep is None else H + KV], k, v, layer.freqs,
                                  layer.kv_scale, layer.kv_scale)
    q = turned[:, :H]
    att = fq.kv_attention(fmt, *where, q, max_new, seqs.bound, layer.kv_scale, layer.kv_scale,
                          window=layer.window, sinks=layer.sinks)
    out = fq.gemm(fmt, fq.quantize(fmt, att.view(rows, H * D)), layer.out, y_dtype=fq.OUT_BF16)
    # experts
    a2 = fq.rms_norm_quantize(fmt, out, layer.norm2, residual=x, y_dtype=fq.OUT_BF16)
    x, h = a2["h"], a2["y"]
    logits = h.float() @ layer.router
    r = fq.route(logits, layer.top)
    a = fq.permute_quantized(fmt, h, a2, r["row_src"], r["offsets"])
    u = fq.grouped_gemm(fmt, r["offsets"], a, *layer.up, y_dtype=fq.OUT_BF16)
    u = torch.nn.functional.silu(u)
    a = fq.quantize(fmt, u, group_offsets=r["offsets"])
    y = fq.grouped_gemm(fmt, r["offsets"], a, *layer.down, y_dtype=fq.OUT_BF16)
    moe = fq.combine(y, r["row_of"], r["weights"])
    if keep is not None:
        keep.update(a1=a1, shared=shared, qkv=qkv, q=q, k=turned[:, H:], v=v, att=att, out=out, a2=a2,
                    logits=logits, route=r, y=y, moe=moe, offsets=offsets)
    return x + moe


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--fmt", choices=["nvfp4", "mxfp4"], default="nvfp4")
    ap.add_argument("--steps", type=int, default=32)
    args = ap.parse_args()
    fmt = fq.NVFP4 if args.fmt == "nvfp4" else fq.MXFP4
    layer = Layer(fmt, window=256, sinks=4, adapters=3)
    g = torch.Generator().manual_seed(2)
    prompts = torch.randint(17, 400, (24,), generator=g).tolist()
    seqs = Sequences(layer, prompts, args.steps, adapters=[i % 4 - 1 for i in range(len(prompts))])
    x = torch.randn(sum(prompts), 1024, generator=g).to(torch.bfloat16).cuda()
    y = forward(layer, seqs, x, seqs.new(prompts), max(prompts))
    torch.cuda.synchronize()
    print(f"prompt pass: {len(prompts)} sequences, {sum(prompts)} tokens, "
          f"output rms {y.float().square().mean().sqrt().item():.3f}", flush=True)
    last = torch.tensor(prompts).cumsum(0).cuda() - 1
    tok, off = y[last], seqs.new([1] * len(prompts))
    t0 = time.perf_counter()
    for _ in range(args.steps):
        seqs.lens += 1
        seqs.bound += 1
        tok = norm(forward(layer, seqs, tok, off, 1))
    torch.cuda.synchronize()
    dt = time.perf_counter() - t0
    print(f"decode: {args.steps} steps, {dt / args.steps * 1e3:.2f} ms a step, "
          f"{len(prompts) * args.steps / dt:.0f} tokens/s through the layer", flush=True)


if __name__ == "__main__":
    main()
