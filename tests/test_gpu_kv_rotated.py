"""GPU: keys and queries turned by their positions on the way into the paged FP4
cache, bit for bit against the plain 64-bit form: with angles, sines and
products in 64 bits on both sides, the F32 value that is rounded further is the
same but for about one in 2^28, so that no element of these sizes differs."""
import numpy as np
import pytest
import torch

import fp4_w4a4_quantized_amd as fq
from gpu_helpers import need_gpu, say
from oracle import layer
from test_gpu_kv_attention import dev, make

pytestmark = pytest.mark.gpu


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy()


def bf16(a):
    return dev(np.asarray(a, np.float32)).to(torch.bfloat16)


def freqs_of(rot, base=1e4):
    return (base ** (-np.arange(rot // 2) / max(rot // 2, 1))).astype(np.float32)


def args_of(c, cache):
    return cache, c["page"], dev(c["off"]), dev(c["table"]), dev(c["lens"])


def check(c, rot, inter, q, k, v, positions=None, extra=0, far=0):
    """extra: rows behind the last sequence; far: added to positions."""
    f = freqs_of(rot)
    rows = int(c["off"][-1])
    t = None if c["t"] is None else dev(c["t"])
    want = c["cache"].copy()
    pos = layer.token_positions(c["off"], c["lens"], rows) if positions is None else positions[:rows]
    wq, wk = (layer.rotate(a[:rows], pos, f, inter) for a in (q, k))
    layer.kv_append(c["fmt"], want, c["page"], c["off"], c["table"], c["lens"], wk, v[:rows], c["t"], c["t"])
    cache = dev(c["cache"])
    # inputs as parts of one packed tensor: strides of their own
    H, heads = k.shape[1], q.shape[1]
    qkv = bf16(np.concatenate([q, k, v], 1))
    got = fq.kv_append_rotated(c["fmt"], *args_of(c, cache), qkv[:, :heads], qkv[:, heads:heads + H],
                               qkv[:, heads + H:], dev(f), t, t, interleaved=inter,
                               positions=None if positions is None else dev(positions.astype(np.int32)))
    assert np.array_equal(bits(got[:rows]), bits(bf16(wq)))
    assert np.array_equal(bits(got[rows:]), bits(qkv[rows:, :heads])), "rows of no sequence are copied"
    bad = np.argwhere(cache.cpu().numpy() != want)
    assert bad.size == 0, f"{len(bad)} bytes of the cache differ, first {bad[:4].tolist()}"
    return qkv, got, cache


def inputs(c, heads, seed, extra=0):
    rng = np.random.default_rng(seed)
    rows = int(c["off"][-1]) + extra
    H, D = c["H"], c["D"]
    q = layer.bf16_round(2 * rng.standard_normal((rows, heads, D)))
    k = layer.bf16_round(rng.standard_normal((rows, H, D))
                         * np.where(rng.random((rows, H, 1)) < 0.2, 2.0 ** rng.integers(-30, 6, (rows, H, 1)), 1))
    return q, k, layer.bf16_round(rng.standard_normal((rows, H, D)))


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("D,page,H,heads", [(64, 16, 3, 7), (128, 32, 2, 2), (256, 64, 1, 5), (128, 1024, 9, 40)])
@pytest.mark.parametrize("inter", [False, True])
def test_bit_for_bit(fmt, D, page, H, heads, inter):
    need_gpu()
    say(f"rotated append fmt {fmt} D {D} page {page} H {H} heads {heads} interleaved {inter}")
    n, lens = [1, 0, 5, 33, page + 3], [1, 7, 2 * page, page + 33, 3 * page - 1]
    c = make(fmt, n, lens, H=H, D=D, page=page, seed=page + inter)
    q, k, v = inputs(c, heads, D + heads, extra=3)
    for rot in (D, 16, D // 2, 0):
        check(c, rot, inter, q, k, v)


@pytest.mark.parametrize("fmt", [0, 1])
def test_given_and_far_positions(fmt):
    """Positions of the whole range of int32, below 0 among them; where a key is
    stored does not go by them."""
    need_gpu()
    c = make(fmt, [9, 40], [9, 100], H=2, D=128, page=16, seed=8)
    q, k, v = inputs(c, 4, 1)
    pos = np.random.default_rng(3).integers(-2 ** 31, 2 ** 31, int(c["off"][-1]))
    pos[:4] = 0, 131071, -1, 2 ** 31 - 1
    for inter in (False, True):
        check(c, 128, inter, q, k, v, positions=pos)


def test_many_sequences():
    """More sequences than a wave looks at in one step, and empty ones."""
    need_gpu()
    rng = np.random.default_rng(5)
    n = rng.integers(0, 3, 300)
    c = make(0, n, n + rng.integers(0, 40, 300), H=1, D=64, page=16, seed=3)
    check(c, 64, False, *inputs(c, 2, 2))


def test_one_part_and_several():
    """Few tokens: the heads over several workgroups; many: one."""
    need_gpu()
    for n in (3, 2100):
        c = make(1, [n], [n + 5], H=2, D=64, page=64, seed=n)
        check(c, 32, False, *inputs(c, 36, n))


@pytest.mark.parametrize("fmt", [0, 1])
def test_tokens_without_a_place(fmt):
    """Pages that are gone and more tokens than the length: nothing stored, the
    queries turn all the same."""
    need_gpu()
    c = make(fmt, [3, 2, 4], [3, 33, 2], page=16, seed=4)
    c["table"][1, :] = -1
    c["table"][0, 0] = 10 ** 6
    check(c, 128, False, *inputs(c, 4, 7))


def test_in_place_and_unusual_values():
    """q_out = q; infinities and NaN stay in their own pair, and in rows of no
    sequence and elements that do not turn they pass."""
    need_gpu()
    c = make(1, [2, 3], [20, 3], H=1, D=64, page=16, seed=6)
    q, k, v = inputs(c, 2, 9, extra=2)
    want = layer.rotate(q[:5], layer.token_positions(c["off"], c["lens"], 5), freqs_of(32))
    t = bf16(q)
    t[1, 0, 40], t[2, 1, 3], t[5, 0, 0], t[6, 1, 9] = float("nan"), float("inf"), float("nan"), float("-inf")
    before = t.clone()
    out = t.clone()
    cache = dev(c["cache"])
    fq.kv_append_rotated_into(1, *args_of(c, cache), out, bf16(k), bf16(v), dev(freqs_of(32)), None, None, out)
    assert np.array_equal(bits(out[5:]), bits(before[5:]))
    assert torch.isnan(out[1, 0, 40])
    w = bf16(want)
    w[1, 0, 40] = before[1, 0, 40]
    skip = torch.zeros_like(w, dtype=torch.bool)
    skip[2, 1, 3], skip[2, 1, 19] = True, True
    assert not torch.isfinite(out[2, 1, 3]) and not torch.isfinite(out[2, 1, 19])
    same = (out[:5].view(torch.int16) == w.view(torch.int16)) | skip | torch.isnan(w)
    assert bool(same.all())


def test_repeats_and_captured():
    """The same call twice gives the same bytes; captured and replayed with other
    inputs it gives those of the eager call."""
    need_gpu()
    c = make(0, [1] * 5, [4, 17, 33, 9, 70], H=2, D=128, page=16, seed=11)
    q, k, v = (bf16(a) for a in inputs(c, 8, 4))
    t, f = dev(c["t"]), dev(freqs_of(128))
    cache = dev(c["cache"])
    a = args_of(c, cache)

    def call():
        return fq.kv_append_rotated(0, *a, q, k, v, f, t, t)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    for seed in (1, 2, 3):
        n = inputs(c, 8, seed)
        for x, y in zip((q, k, v), n):
            x.copy_(bf16(y))
        cache.copy_(dev(c["cache"]))
        want = call().clone()
        after = cache.clone()
        cache.copy_(dev(c["cache"]))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(cache, after)
    other = fq.kv_append_rotated(0, *a, q, k, v, f, t, t, stream=s)
    s.synchronize()
    assert torch.equal(other, want)
