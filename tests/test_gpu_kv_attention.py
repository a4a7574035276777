"""GPU: the paged FP4 key/value cache (append, read back) bit for bit and
attention over it against the plain 64-bit forms of oracle/layer.py.

Tolerance of attention, derived from the arithmetic: with u the rounding of
the weights (2^-11 f16, 2^-8 bf16) and d the error of a score in FP32 (D
products and sums, the factor, the exponent: (D + 16) 2^-24 of the sum of
absolute terms, and 2^-25 of it again for a q held in f16; scores also carry
2^-23 of their own size through the exponential), weights and their sum are
off by at most (u + 2 d') relative, so
  |o - o*| <= (u + 2 d') sum p |v| / z + u_out |o*|.
"""
import numpy as np
import pytest
import torch

import fp4_w4a4_quantized_amd as fq
from gpu_helpers import need_gpu, say
from oracle import layer

pytestmark = pytest.mark.gpu

FMTS = [0, 1]


def make(fmt, n, lens, H=2, G=2, D=128, page=16, seed=0, extra=2, garbage=True):
    """A cache with lens[b] tokens of each sequence, the last n[b] of them new,
    pages in a random order; what no token owns holds random bytes (NaN scales
    among them)."""
    rng = np.random.default_rng(seed)
    n, lens = np.array(n), np.array(lens)
    B = len(n)
    need = [-(-max(int(x), 0) // page) for x in lens]
    pages = sum(need) + extra
    ids = rng.permutation(pages)
    table = np.full((B, max(max(need), 1)), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += need[b]
    nb = layer.kv_page_bytes(fmt, page, D)
    cache = (rng.integers(0, 256, (pages, H, nb), dtype=np.uint8) if garbage
             else np.zeros((pages, H, nb), np.uint8))
    t = None
    if fmt == 0:
        t = (0.002 + 0.002 * rng.random(H)).astype(np.float32)
    # everything before the new tokens, stored by the oracle
    old = np.maximum(lens - n, 0)
    off_all = np.concatenate([[0], np.cumsum(np.maximum(lens, 0))])
    k = layer.bf16_round(rng.standard_normal((off_all[-1], H, D)))
    v = layer.bf16_round(rng.standard_normal((off_all[-1], H, D)))
    layer.kv_append(fmt, cache, page, off_all, table, lens, k, v, t, t)
    off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    q = layer.bf16_round(2.0 * rng.standard_normal((off[-1], H * G, D)))
    return dict(fmt=fmt, cache=cache, page=page, off=off, table=table, lens=lens.astype(np.int32),
                q=q, t=t, H=H, G=G, D=D, n=n, old=old, rng=rng)


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def attend(c, window=0, scale=None, y_dtype=fq.OUT_BF16, q=None, max_len=None, **kw):
    t = None if c["t"] is None else dev(c["t"])
    q = dev(c["q"], torch.bfloat16) if q is None else q
    return fq.kv_attention(c["fmt"], dev(c["cache"]), c["page"], dev(c["off"]), dev(c["table"]),
                           dev(c["lens"]), q, int(max(c["n"].max(), 1)),
                           int(max(c["lens"].max(), 0)) if max_len is None else max_len,
                           t, t, window=window, scale=scale, y_dtype=y_dtype, **kw)


def check(c, got, window=0, scale=None):
    got = got.float().cpu().numpy().astype(np.float64) if got.dtype == torch.bfloat16 \
        else got.cpu().numpy().astype(np.float64)
    o, w, s = layer.attention(c["fmt"], c["cache"], c["page"], c["off"], c["table"], c["lens"], c["q"],
                              c["t"], c["t"], window, scale)
    u = 2.0 ** -11 if c["fmt"] == 0 else 2.0 ** -8
    d = ((c["D"] + 16) * 2.0 ** -24 + 2.0 ** -23 + (2.0 ** -25 if c["fmt"] == 0 else 0.0)) * s
    return got, o, (u + 2 * d + 2.0 ** -20) * w


def check_close(c, got, window=0, scale=None, bf16=True):
    g, o, tol = check(c, got, window, scale)
    tol = tol + (2.0 ** -8 if bf16 else 2.0 ** -23) * (np.abs(o) + tol) + 1e-30
    err = np.abs(g - o)
    bad = np.argwhere(~(err <= tol))
    assert bad.size == 0, (f"{len(bad)} of {o.size} outputs off; worst {np.nanmax(err / tol):.2f} of "
                           f"the bound; first {bad[:3].tolist()}, {np.isnan(g).sum()} NaN")


# ---- append and read ------------------------------------------------------------

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,page,H", [(64, 16, 3), (128, 32, 2), (256, 64, 1), (128, 1024, 5)])
def test_append_and_read_bit_for_bit(fmt, D, page, H):
    need_gpu()
    say(f"append fmt {fmt} D {D} page {page} H {H}")
    rng = np.random.default_rng(D + page + H + fmt)
    n, lens = [1, 0, 5, 33, page + 3], [1, 7, 2 * page, page + 1, 3 * page - 1]
    c = make(fmt, n, np.maximum(lens, n), H=H, D=D, page=page, seed=page)
    rows = int(c["off"][-1])
    k = layer.bf16_round(rng.standard_normal((rows, H, D))
                         * np.where(rng.random((rows, H, 1)) < 0.2, 2.0 ** rng.integers(-30, 6, (rows, H, 1)), 1))
    v = layer.bf16_round(rng.standard_normal((rows, H, D)))
    k[0], v[rows - 1] = 0.0, -0.0
    k[1, :, :16] = 1e30                       # far past what the tensor scale can hold
    v[2, :, ::3] = 2.0 ** -130                # bf16 subnormals
    want = c["cache"].copy()
    layer.kv_append(fmt, want, page, c["off"], c["table"], c["lens"], k, v, c["t"], c["t"])
    t = None if c["t"] is None else dev(c["t"])
    cache = dev(c["cache"])
    args = (cache, page, dev(c["off"]), dev(c["table"]), dev(c["lens"]))
    # inputs as slices of one packed qkv tensor: row strides of their own
    qkv = torch.zeros(rows, 3 * H, D, dtype=torch.bfloat16, device="cuda")
    qkv[:, H:2 * H], qkv[:, 2 * H:] = dev(k, torch.bfloat16), dev(v, torch.bfloat16)
    fq.kv_append(fmt, *args, qkv[:, H:2 * H], qkv[:, 2 * H:], t, t)
    got = cache.cpu().numpy()
    bad = np.argwhere(got != want)
    assert bad.size == 0, f"{len(bad)} bytes differ, first {bad[:4].tolist()}"
    gk, gv = fq.kv_read(fmt, *args, rows, D, t, t)
    wk, wv = layer.kv_read(fmt, want, page, c["off"], c["table"], c["lens"], rows, D, c["t"], c["t"])
    for g, w in ((gk, wk), (gv, wv)):
        assert np.array_equal(g.float().cpu().numpy(), w.astype(np.float32))


@pytest.mark.parametrize("fmt", FMTS)
def test_append_leaves_bad_places_alone(fmt):
    """Page numbers outside the cache, positions past the table or below 0 and
    rows past the last sequence: nothing is stored, zeros are read."""
    need_gpu()
    H, D, page = 2, 64, 16
    off = np.array([0, 4, 8, 12], np.int32)
    lens = np.array([4, 40, 2], np.int32)               # fine; past the table; two below 0
    table = np.array([[-1, 0], [1, 99], [2, 2]], np.int32)
    table[0, 0] = 7
    rng = np.random.default_rng(3)
    cache = rng.integers(0, 256, (4, H, layer.kv_page_bytes(fmt, page, D)), dtype=np.uint8)
    k = layer.bf16_round(rng.standard_normal((14, H, D)))
    t = np.array([0.003, 0.004], np.float32) if fmt == 0 else None
    want = cache.copy()
    layer.kv_append(fmt, want, page, off, table, lens, k, k, t, t)
    dt = None if t is None else dev(t)
    g = dev(cache)
    args = (g, page, dev(off), dev(table), dev(lens))
    fq.kv_append(fmt, *args, dev(k, torch.bfloat16), dev(k, torch.bfloat16), dt, dt)
    assert np.array_equal(g.cpu().numpy(), want)
    gk, _ = fq.kv_read(fmt, *args, 14, D, dt, dt)
    wk, _ = layer.kv_read(fmt, want, page, off, table, lens, 14, D, t, t)
    assert np.array_equal(gk.float().cpu().numpy(), wk.astype(np.float32))
    assert np.all(gk[12:].float().cpu().numpy() == 0)


# ---- attention ------------------------------------------------------------------

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 128])
def test_decode_ragged(fmt, D, page):
    need_gpu()
    say(f"decode fmt {fmt} D {D} page {page}")
    c = make(fmt, [1] * 9, [1, 2, 15, 16, 17, 33, 100, 129, 700], D=D, page=page, seed=D + page)
    check_close(c, attend(c))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("G", [1, 3, 7, 8, 16, 24])
def test_shared_heads_and_speculative_steps(fmt, G):
    need_gpu()
    say(f"heads fmt {fmt} G {G}")
    c = make(fmt, [4, 1, 3, 2], [4, 260, 61, 1030], G=G, H=1 + (G < 8), seed=G)
    check_close(c, attend(c))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,G,H", [(64, 3, 2), (128, 8, 1), (128, 1, 3), (256, 2, 1)])
@pytest.mark.parametrize("window", [0, 1, 37, 200])
def test_prompts_and_chunks(fmt, D, G, H, window):
    need_gpu()
    say(f"prompt fmt {fmt} D {D} G {G} H {H} window {window}")
    c = make(fmt, [130, 5, 64, 97, 1], [130, 300, 64, 97 + 128, 333], D=D, G=G, H=H, page=32, seed=window)
    check_close(c, attend(c, window), window)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,lens", [([1, 1], [5000, 40]), ([300], [4000]), ([2, 0, 1], [3001, 9, 2999])])
def test_long_keys_are_split(fmt, n, lens):
    need_gpu()
    say(f"split fmt {fmt} n {n} lens {lens}")
    c = make(fmt, n, lens, G=4, H=1, page=64, seed=5)
    a = attend(c)
    check_close(c, a)
    # a larger bound on the length changes the split, not the result's correctness
    check_close(c, attend(c, max_len=60000))
    check_close(c, attend(c, window=1000), 1000)
    assert torch.equal(a, attend(c)), "two runs differ"


@pytest.mark.parametrize("fmt", FMTS)
def test_f32_output_scale_and_strided_q(fmt):
    need_gpu()
    c = make(fmt, [3, 20], [50, 20], G=2, H=2, D=64, seed=1)
    rows = int(c["off"][-1])
    qkv = torch.zeros(rows, 8, 64, dtype=torch.bfloat16, device="cuda")
    qkv[:, :4] = dev(c["q"], torch.bfloat16)
    got = attend(c, scale=0.31, y_dtype=fq.OUT_F32, q=qkv[:, :4])
    check_close(c, got, scale=0.31, bf16=False)
    y = torch.full((rows, 6, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    t = None if c["t"] is None else dev(c["t"])
    fq.kv_attention_into(fmt, dev(c["cache"]), c["page"], dev(c["off"]), dev(c["table"]), dev(c["lens"]),
                         qkv[:, :4], 20, 50, t, t, 0, 0.31, y[:, :4], None)
    check_close(c, y[:, :4], scale=0.31)
    assert torch.all(y[:, 4:] == 7.0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("mult", [2.0 ** -40, 2.0 ** 30, 0.0])
def test_small_large_and_zero_queries(fmt, mult):
    """Uniform weights for tiny and zero queries; one key takes all for huge
    ones (q of 2^30 is past f16's range, and its scores differ by far more
    than any rounding of them)."""
    need_gpu()
    c = make(fmt, [1, 6], [70, 6], G=2, H=2, D=128, seed=11)
    c["q"] = layer.bf16_round(c["q"] * mult)
    got = attend(c)
    if mult < 1.0:
        check_close(c, got)
        return
    o, _, s = layer.attention(fmt, c["cache"], c["page"], c["off"], c["table"], c["lens"], c["q"], c["t"],
                              c["t"])
    assert np.all(s > 1e6)
    g = got.float().cpu().numpy()
    assert np.all(np.abs(g - o) <= 2.0 ** -7 * np.abs(o) + 1e-6)


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_that_see_nothing(fmt):
    """Empty sequences, pages that are gone, more new tokens than the length:
    zeros, whatever the cache holds."""
    need_gpu()
    c = make(fmt, [0, 2, 3, 1, 40], [0, 33, 40, 20, 64], page=16, seed=4)
    c["table"][1, :] = -1                          # sees nothing
    c["table"][2, 1] = 10 ** 6                     # the middle page is not in the cache
    c["table"][4, 0] = -7
    c["lens"][3] = 0                               # a new token before position 0
    got = attend(c, max_len=64)
    check_close(c, got)
    assert torch.all(got[:2] == 0) and torch.all(got[5] == 0)
    c["table"][:] = -1
    assert torch.all(attend(c, max_len=64) == 0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n", [1, 70])
def test_nan_outside_the_window_stays_outside(fmt, n):
    """Scales of NaN (and infinite ones) in every place that no row sees."""
    need_gpu()
    c = make(fmt, [n], [200], page=16, seed=9, garbage=False)
    D, page = c["D"], 16
    kb, kh, vb, vh, ks, vs = layer.kv_places(fmt, page, D)
    nan = 0x7F if fmt == 0 else 0xFF
    window = 50
    first = 200 - n - window + 1                   # the first key that any row sees
    for pos in list(range(0, max(first, 0))) + list(range(200, 208)):
        pid = c["table"][0, pos // page]
        for s in (ks, vs):
            c["cache"][pid][:, s[pos % page]] = nan
    check_close(c, attend(c, window), window)


def test_streams_and_graph_replay():
    """On a stream of its own, and captured: each replay against the eager
    result, with other work between the replays."""
    need_gpu()
    c = make(0, [1, 1, 1], [2000, 3, 900], G=4, H=2, page=32, seed=2)
    t, q = dev(c["t"]), dev(c["q"], torch.bfloat16)
    cache, off, table, lens = dev(c["cache"]), dev(c["off"]), dev(c["table"]), dev(c["lens"])
    rng = np.random.default_rng(0)
    k = dev(layer.bf16_round(rng.standard_normal((3, 2, 128))), torch.bfloat16)

    def step():
        fq.kv_append(0, cache, 32, off, table, lens, k, k, t, t)
        return fq.kv_attention(0, cache, 32, off, table, lens, q, 1, 2000, t, t)

    eager = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = fq.kv_attention(0, cache, 32, off, table, lens, q, 1, 2000, t, t, stream=s)
    s.synchronize()
    assert torch.equal(other, eager)
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = step()
    for i in range(3):
        y.zero_()
        k.copy_(torch.randn(k.shape, device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, step()), f"replay {i}"
