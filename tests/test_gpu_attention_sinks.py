"""GPU: attention over the paged FP4 cache with a sliding window and first tokens
that stay visible, against the plain 64-bit form; tolerances as derived in
test_gpu_kv_attention.py (they count a row's own keys, whichever they are)."""
import numpy as np
import pytest
import torch

import fp4_w4a4_quantized_amd as fq
from gpu_helpers import need_gpu, say
from oracle import layer
from test_gpu_kv_attention import attend, dev, make

pytestmark = pytest.mark.gpu

FMTS = [0, 1]


def check(c, window, sinks, bf16=True, **kw):
    got = attend(c, window, sinks=sinks, y_dtype=fq.OUT_BF16 if bf16 else fq.OUT_F32, **kw)
    o, w, s = layer.attention(c["fmt"], c["cache"], c["page"], c["off"], c["table"], c["lens"], c["q"], c["t"],
                              c["t"], window, None, sinks)
    u = 2.0 ** -11 if c["fmt"] == 0 else 2.0 ** -8
    d = ((c["D"] + 16) * 2.0 ** -24 + 2.0 ** -23 + (2.0 ** -25 if c["fmt"] == 0 else 0.0)) * s
    tol = (u + 2 * d + 2.0 ** -20) * w
    tol = tol + (2.0 ** -8 if bf16 else 2.0 ** -23) * (np.abs(o) + tol) + 1e-30
    err = np.abs(got.double().cpu().numpy() - o)
    bad = np.argwhere(~(err <= tol))
    assert bad.size == 0, (f"window {window} sinks {sinks}: {len(bad)} of {o.size} outputs off; worst "
                           f"{np.nanmax(err / tol):.2f} of the bound; first {bad[:3].tolist()}")
    return got


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 128])
def test_decode(fmt, D, page):
    need_gpu()
    say(f"sinks decode fmt {fmt} D {D} page {page}")
    c = make(fmt, [1] * 9, [1, 2, 15, 16, 17, 33, 100, 129, 700], D=D, page=page, seed=D + page)
    for window, sinks in ((1, 1), (16, 4), (50, 31), (50, 32), (50, 33), (64, 100), (300, 5), (10, 2000)):
        check(c, window, sinks)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("G", [1, 3, 8, 16, 24])
def test_shared_heads_and_speculative_steps(fmt, G):
    need_gpu()
    say(f"sinks heads fmt {fmt} G {G}")
    c = make(fmt, [4, 1, 3, 2], [4, 260, 61, 1030], G=G, H=1 + (G < 8), seed=G)
    for window, sinks in ((3, 1), (33, 7), (128, 65)):
        check(c, window, sinks)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,G,H", [(64, 3, 2), (128, 8, 1), (256, 2, 1)])
def test_prompts_and_chunks(fmt, D, G, H):
    need_gpu()
    say(f"sinks prompt fmt {fmt} D {D} G {G} H {H}")
    c = make(fmt, [130, 5, 64, 300, 1], [130, 300, 64, 900, 333], D=D, G=G, H=H, page=32, seed=D)
    for window, sinks in ((1, 1), (37, 4), (200, 64), (64, 70), (1000, 3)):
        check(c, window, sinks)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,lens", [([1, 1], [20000, 40]), ([300], [9000]), ([2, 0, 1], [9001, 9, 2999])])
def test_long_windows_are_split(fmt, n, lens):
    need_gpu()
    say(f"sinks split fmt {fmt} n {n} lens {lens}")
    c = make(fmt, n, lens, G=4, H=1, page=64, seed=5)
    for window, sinks in ((1000, 4), (4000, 700), (777, 3000)):
        a = check(c, window, sinks)
        assert torch.equal(a, attend(c, window, sinks=sinks)), "two runs differ"
        check(c, window, sinks, max_len=100000)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n", [1, 90])
def test_everything_visible_is_plain_attention(fmt, n):
    """Sinks up to the window, past the length, or without a window: every key
    is seen, and no key twice."""
    need_gpu()
    c = make(fmt, [n, 1], [300, 50], page=16, seed=2)
    full = attend(c)
    assert torch.equal(attend(c, 0, sinks=5), full)
    assert torch.equal(attend(c, 0, sinks=2 ** 31 - 1), full)
    check(c, 100, 2 ** 31 - 1)
    check(c, 100, 201)
    check(c, 2 ** 31 - 1, 2 ** 31 - 1)
    a, b = attend(c, 120, sinks=0), attend(c, 120)
    assert torch.equal(a, b)
    check(c, 60, 4, bf16=False)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n", [1, 70])
def test_nan_between_sinks_and_window_stays_there(fmt, n):
    """Scales of NaN (and infinite ones) in every place that no row sees, and
    pages between that are given back."""
    need_gpu()
    c = make(fmt, [n], [700], page=16, seed=9, garbage=False)
    page, window, sinks = 16, 50, 21
    ks, vs = layer.kv_places(fmt, page, c["D"])[4:]
    nan = 0x7F if fmt == 0 else 0xFF
    first = 700 - n - window + 1                   # the window's first key for any row
    for pos in list(range(sinks, first)) + list(range(700, 704)):
        pid = c["table"][0, pos // page]
        for s in (ks, vs):
            c["cache"][pid][:, s[pos % page]] = nan
    a = check(c, window, sinks)
    for col in range(-(-sinks // page), first // page):
        c["table"][0, col] = -1
    assert torch.equal(check(c, window, sinks), a)
    c["table"][0, 0] = -1                          # a page of sinks that is gone is not seen
    check(c, window, sinks)


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_that_see_nothing(fmt):
    need_gpu()
    c = make(fmt, [0, 2, 3, 1, 40], [0, 33, 40, 20, 64], page=16, seed=4)
    c["table"][1, :] = -1                          # sees nothing
    c["table"][2, 1] = 10 ** 6                     # the middle page is not in the cache
    c["lens"][3] = 0                               # a new token before position 0
    got = check(c, 20, 3, max_len=64)
    assert torch.all(got[:2] == 0) and torch.all(got[5] == 0)
    assert torch.all(attend(c, 20, sinks=3, max_len=0) == 0)      # every key is past max_len


def test_captured_with_growing_lengths():
    """A decode step captured once: lengths that pass the window afterwards, each
    replay against the eager call."""
    need_gpu()
    c = make(0, [1, 1], [300, 40], G=4, H=2, page=16, seed=1)
    t = dev(c["t"])
    cache, off, table = dev(c["cache"]), dev(c["off"]), dev(c["table"])
    lens, q = dev(c["lens"]), dev(c["q"], torch.bfloat16)

    def call():
        return fq.kv_attention(0, cache, 16, off, table, lens, q, 1, 4096, t, t, window=64, sinks=5)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    for new in ([300, 40], [20, 17], [250, 33], [1, 1]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        want = call()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,H,n,lens", [(64, 1, [600], [600]), (128, 2, [300, 40], [2000, 40]), (128, 8, [300] * 6, [300] * 6),
                                        (256, 1, [200], [1500])])
def test_sizes_of_tiles(fmt, D, H, n, lens):
    """Few and many workgroups of rows, one and several splits of the keys."""
    need_gpu()
    say(f"sinks tiles fmt {fmt} D {D} H {H} n {n}")
    c = make(fmt, n, lens, G=3, H=H, D=D, page=32, seed=3)
    for window, sinks in ((30, 70), (1200, 4)):
        check(c, window, sinks)
