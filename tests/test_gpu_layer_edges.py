"""GPU: values and bounds at the edges of what the calls between the FP4 linear
layers define, against the plain 64-bit forms of oracle/layer.py with the
tolerances of test_gpu_kv_attention.py and test_gpu_route_combine.py."""
import numpy as np
import pytest
import torch

import fp4_w4a4_quantized_amd as fq
from gpu_helpers import need_gpu, say
from oracle import layer
from test_gpu_kv_attention import FMTS, attend, check, check_close, dev, make
from test_gpu_route_combine import U, check_route, host, logits_of

pytestmark = pytest.mark.gpu


# ---- the router -------------------------------------------------------------

@pytest.mark.parametrize("T", [13, 210])
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("E,groups,top,k", [(8, 2, 1, 1), (16, 4, 2, 2), (96, 8, 3, 9), (384, 4, 4, 17)])
def test_groups_without_a_bias_rank_by_the_logits(T, score, E, groups, top, k):
    """Scores that are equal in 64 bits (a saturated sigmoid, a softmax that
    underflows) while the logits differ: the larger logit comes first, -inf
    last.  Integer logits, so that no sum of two scores is a near tie."""
    need_gpu()
    say(f"groups by logits T{T} E{E} {groups}/{top} k{k} score {score}")
    g = torch.Generator().manual_seed(E + T)
    near = torch.randint(30, 61, (T, E), generator=g).float()
    far = -100.0 * torch.randint(0, 21, (T, E), generator=g).float()
    far[:, ::3] = torch.where(torch.rand(far[:, ::3].shape, generator=g) < 0.5, -float("inf"), far[:, ::3])
    for x in (near, far):
        for dtype in (torch.float32, torch.bfloat16):
            check_route(x.to(dtype).cuda(), k, score, None, groups, top)
            check_route(x.to(dtype).cuda(), k, score, None, groups, top, renorm=False)


def test_a_grouped_choice_by_hand():
    need_gpu()
    x = torch.zeros(1, 8)
    x[0, 1:4] = torch.tensor([40.0, 50.0, 45.0])
    assert fq.route(x.cuda(), 1, score=fq.SIGMOID, n_groups=2)["experts"].tolist() == [[2]]
    x = torch.zeros(1, 16)
    x[0, 2], x[0, 5], x[0, 6] = 38.0, 50.0, 45.0
    r = fq.route(x.cuda(), 2, score=fq.SIGMOID, n_groups=4, top_groups=2)
    assert r["experts"].tolist() == [[5, 6]]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [14, 210])
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("E,groups,top,k", [(8, 1, 1, 2), (60, 1, 1, 20), (96, 4, 2, 7)])
def test_infinite_logits(dtype, T, score, E, groups, top, k):
    """+inf counts as the largest finite number: it shares a softmax with its
    like, and neither weights nor gradients become NaN."""
    need_gpu()
    say(f"infinite logits {dtype} T{T} E{E} {groups}/{top} k{k} score {score}")
    inf = float("inf")
    x = logits_of(T, E, torch.float32, E)
    x[0, 3] = inf
    x[1, 1:7:2] = inf
    x[2] = inf
    x[3], x[3, 5] = -inf, inf
    x[4], x[4, 6], x[4, 2] = float("nan"), inf, -inf
    x[5, ::2] = inf
    x[6, 7], x[6, 4] = inf, torch.finfo(torch.float32).max
    x[T - 1, 0] = inf
    x = x.to(dtype)
    bias = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(E)).cuda()
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(T)).cuda()
    for renorm in (True, False):
        for b in (None, bias):
            r, _ = check_route(x, k, score, b, groups, top, renorm)
            d = fq.route_backward(x, r["experts"], dw, score=score, renorm=renorm)
            want, size = layer.route_backward(host(x), r["experts"].cpu().numpy(), host(dw), score, renorm)
            u = U[dtype] + (2.0 ** -24 if dtype == torch.bfloat16 else 0.0)
            assert np.all(np.abs(host(d) - want) <= u * np.abs(want) + 2.0 ** -40 * size + 1e-38)


# ---- the cache --------------------------------------------------------------

def block_bytes(fmt, page, D, slot, blk):
    """The bytes of a page of one head that hold block blk of K and of V of the
    token at slot, and V bytes' share of them (they are half another block's)."""
    kb, _, vb, vh, ks, vs = layer.kv_places(fmt, page, D)
    n = layer.BLOCK[fmt]
    el = slice(blk * n, blk * n + n)
    return kb[slot, el], vb[slot, el], vh[slot, el], ks[slot, blk], vs[slot, blk]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_is_not_finite_stays_in_its_block(fmt, D, bad):
    """One bad element in each block of a token in turn: every other block's
    bytes are those of the clean token, and its own scale is a finite one."""
    need_gpu()
    say(f"append {bad} fmt {fmt} D {D}")
    blocks, page, H = D // layer.BLOCK[fmt], 16, 2
    off, lens = np.array([0, blocks], np.int32), np.array([blocks], np.int32)
    table = np.array([[1]], np.int32)
    rng = np.random.default_rng(D)
    k = torch.from_numpy(rng.standard_normal((blocks, H, D))).to(torch.bfloat16).cuda()
    t = dev(np.array([0.003, 0.004], np.float32)) if fmt == 0 else None
    got = []
    for spoil in (False, True):
        x = k.clone()
        if spoil:
            for b in range(blocks):
                x[b, 1, b * layer.BLOCK[fmt] + b % 7] = bad
        cache = torch.zeros(2, H, layer.kv_page_bytes(fmt, page, D), dtype=torch.uint8, device="cuda")
        fq.kv_append(fmt, cache, page, dev(off), dev(table), dev(lens), x, x, t, t)
        got.append(cache.cpu().numpy())
    clean, dirty = got
    top = 0x7E if fmt == 0 else 0xFE
    for b in range(blocks):
        kb, vb, vh, ks, vs = block_bytes(fmt, page, D, b, b)
        assert dirty[1, 1, ks] <= top and dirty[1, 1, vs] <= top
        dirty[1, 1, ks], dirty[1, 1, vs] = clean[1, 1, ks], clean[1, 1, vs]
        dirty[1, 1, kb] = clean[1, 1, kb]
        for byte, shift in zip(vb, vh):            # (both halves of a byte may be this block's)
            own = 0xF << int(shift)
            dirty[1, 1, byte] = (int(dirty[1, 1, byte]) & ~own) | (int(clean[1, 1, byte]) & own)
    bad_at = np.argwhere(clean != dirty)
    assert bad_at.size == 0, f"{len(bad_at)} bytes differ, first {bad_at[:4].tolist()}"


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n", [8, 40])
def test_a_later_token_that_is_not_finite_does_not_reach_earlier_rows(fmt, n):
    need_gpu()
    c = make(fmt, [n], [n], G=2, H=2, D=128, seed=8, garbage=False)
    t = None if c["t"] is None else dev(c["t"])
    k = torch.randn(n, 2, 128, generator=torch.Generator().manual_seed(n)).to(torch.bfloat16).cuda()
    q, got = dev(c["q"], torch.bfloat16), []
    for bad in (0.0, float("nan"), float("inf")):
        x = k.clone()
        x[n - 1, :, ::5] = bad
        cache = dev(c["cache"])
        where = (cache, c["page"], dev(c["off"]), dev(c["table"]), dev(c["lens"]))
        fq.kv_append(fmt, *where, x, x, t, t)
        got.append(fq.kv_attention(fmt, *where, q, n, n, t, t)[:n - 1])
    assert torch.isfinite(got[0]).all()
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


# ---- the combination ----------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,k,rows,N", [(3, 2, 6, 64), (3, 2, 9, 64), (0, 2, 5, 8), (1, 1, 1, 3), (5, 4, 700, 96),
                                        (200, 8, 1600, 130), (200, 8, 5000, 128), (70, 3, 100, 1)])
def test_gradient_rows_that_nothing_names_are_zero(dtype, T, k, rows, N):
    """Rows of padded expert buffers, and those that an entry outside the rows
    leaves without a name; what the freed memory held (old indices among it)
    does not matter."""
    need_gpu()
    say(f"unnamed {dtype} T{T} k{k} rows {rows} N{N}")
    g = torch.Generator().manual_seed(rows + N)
    y = torch.randn(rows, N, generator=g).to(dtype).cuda()
    do = torch.randn(T, N, generator=g).to(dtype).cuda()
    w = torch.rand(T, k, generator=g).cuda()
    row_of = torch.full((T * k,), -1, dtype=torch.int32)
    row_of[:min(rows, T * k)] = torch.randperm(rows, generator=g)[:T * k].int()
    for drop in (0, T * k // 3):
        r = row_of.clone()
        r[:drop] = torch.tensor([-1, rows, 2 ** 31 - 1])[torch.arange(drop) % 3].int()
        r = r.view(T, k).cuda()
        named = r[(r >= 0) & (r < rows)].long()
        want = torch.zeros_like(y)
        t = torch.arange(T * k, device="cuda").view(T, k)[(r >= 0) & (r < rows)] // max(k, 1)
        want[named] = (w.reshape(-1)[((r >= 0) & (r < rows)).reshape(-1)][:, None] * do[t].float()).to(dtype)
        for fill in (0xFF, 0, 1):
            junk = [torch.full((n,), fill, dtype=torch.uint8, device="cuda")
                    for n in (y.untyped_storage().nbytes(), rows * 4, T * k * 4) for _ in range(2)]
            torch.cuda.synchronize()
            del junk
            d_y, d_w = fq.combine_backward(y, r, w, do)
            assert torch.equal(d_y, want), fill
            into = torch.full_like(y, 3.0)
            fq.combine_backward_into(y, r, w, do, into, torch.empty_like(w))
            want_into = torch.full_like(y, 3.0)
            want_into[named] = want[named]
            assert torch.equal(into, want_into)


def test_unnamed_gradient_rows_keep_strides():
    """The C call on rows with a stride, from an address that is not a vector's."""
    need_gpu()
    from fp4_w4a4_quantized_amd import binding
    L, p = binding.lib(), (lambda t: t.data_ptr())
    y, do = torch.randn(300, 40, device="cuda"), torch.randn(10, 40, device="cuda")
    row_of = (29 * torch.arange(10, device="cuda")).int().view(10, 1)
    w, dw = torch.rand(10, 1, device="cuda"), torch.empty(10, 1, device="cuda")
    for c0 in (0, 1, 4):
        big = torch.full((300, 56), 7.0, device="cuda")
        d = big[:, c0:c0 + 40]
        ws = torch.full((300,), 5, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        assert L.fp4q_combine_backward_zeroed(0, p(y), 300, 40, 40, p(row_of), p(w), 10, 1, p(do), 40, p(d), 56,
                                              p(dw), p(ws), 1200, None) == 0
        torch.cuda.synchronize()
        want = torch.zeros(300, 40, device="cuda")
        want[row_of[:, 0].long()] = w * do
        assert torch.equal(d, want)
        assert torch.all(big[:, :c0] == 7.0) and torch.all(big[:, c0 + 40:] == 7.0)


# ---- attention ----------------------------------------------------------------

def attend_up_to(c, max_new, max_len, y_dtype=fq.OUT_BF16, window=0):
    t = None if c["t"] is None else dev(c["t"])
    return fq.kv_attention(c["fmt"], dev(c["cache"]), c["page"], dev(c["off"]), dev(c["table"]), dev(c["lens"]),
                           dev(c["q"], torch.bfloat16), max_new, max_len, t, t, window=window, y_dtype=y_dtype)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,lens,G,D,max_new", [([3, 1, 2], [300, 9, 70], 4, 128, 1),       # one pass, few rows
                                                ([1, 4, 3], [9000, 4, 900], 5, 64, 2),      # split keys
                                                ([9, 1, 6], [700, 1, 9], 6, 128, 5),        # 30 rows of a head
                                                ([40, 17, 2], [40, 30, 2], 3, 256, 16),     # row tiles
                                                ([300, 0, 5], [1500, 0, 7], 4, 64, 100)])   # the same, split keys
def test_rows_past_max_new_give_zero(fmt, n, lens, G, D, max_new):
    need_gpu()
    say(f"max_new fmt {fmt} n {n} lens {lens} G {G} D {D} max_new {max_new}")
    c = make(fmt, n, lens, G=G, H=2, D=D, seed=sum(n))
    within = np.concatenate([np.arange(x) < max_new for x in n])
    for y_dtype in (fq.OUT_BF16, fq.OUT_F32):
        nb = len(c["q"]) * 2 * G * D * 4
        torch.full((4 * nb,), 255, dtype=torch.uint8, device="cuda")  # what freed memory may hold
        got = attend_up_to(c, max_new, max(lens), y_dtype)
        assert torch.all(got[torch.from_numpy(~within).cuda()] == 0)
        g, o, tol = check(c, got)
        tol = tol + (2.0 ** -8 if y_dtype == fq.OUT_BF16 else 2.0 ** -23) * (np.abs(o) + tol) + 1e-30
        assert np.all((np.abs(g - o) <= tol)[within])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,lens,G,D,pages", [([1, 1], [300, 40], 4, 128, 6), ([2, 1], [5000, 900], 3, 64, 190),
                                              ([70, 9], [150, 9], 4, 64, 5), ([90, 3], [1900, 800], 2, 256, 77)])
@pytest.mark.parametrize("window", [0, 60])
def test_keys_past_max_len_are_not_seen(fmt, n, lens, G, D, pages, window):
    """Whatever the split: as if the table ended there."""
    need_gpu()
    say(f"max_len fmt {fmt} n {n} lens {lens} G {G} D {D} pages {pages} window {window}")
    c = make(fmt, n, lens, G=G, H=2, D=D, page=16, seed=pages)
    got = attend_up_to(c, max(n), 16 * pages, window=window)
    c["table"] = c["table"][:, :pages]
    check_close(c, got, window)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,D,G,window", [(1, 128, 4, 0), (1, 64, 4, 700), (6, 128, 4, 0), (40, 64, 2, 64),
                                          (30, 256, 2, 1000)])
def test_the_longest_sequence(fmt, n, D, G, window):
    """The last page of a sequence of 2^31 - 4096 tokens, the others gone: what
    the page's tokens give by themselves, wherever they stand."""
    need_gpu()
    say(f"longest fmt {fmt} n {n} D {D} G {G} window {window}")
    long, page = 2 ** 31 - 4096, 1024
    c = make(fmt, [n], [page], G=G, H=1, D=D, page=page, seed=n)
    t = None if c["t"] is None else dev(c["t"])
    table = torch.full((1, 2 ** 21 - 1), -1, dtype=torch.int32, device="cuda")
    table[0, long // page - 1] = int(c["table"][0, 0])
    got = fq.kv_attention(fmt, dev(c["cache"]), page, dev(c["off"]), table,
                          torch.tensor([long], dtype=torch.int32, device="cuda"), dev(c["q"], torch.bfloat16), n, long,
                          t, t, window=window)
    check_close(c, got, window)


def test_many_row_tiles_of_many_heads():
    """16 row tiles of 4096 kv heads (their product is past 65535); rows of the
    first and last heads and tiles against the plain form."""
    need_gpu()
    H, D, page, n, window = 4096, 64, 16, 4081, 20
    say("row tiles of many heads")
    g = torch.Generator(device="cuda").manual_seed(1)
    pages = -(-n // page)
    k = torch.randn(n, 1, D, generator=g, device="cuda").to(torch.bfloat16).expand(n, H, D)
    k = k * (1 + torch.arange(H, device="cuda") % 3)[None, :, None].to(torch.bfloat16)
    cache = fq.kv_cache(1, pages, page, H, D)
    off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    lens = off[1:].clone()
    table = torch.randperm(pages, generator=g, device="cuda").int().view(1, pages)
    fq.kv_append(1, cache, page, off, table, lens, k, k)
    q = torch.randn(n, H, D, generator=g, device="cuda").to(torch.bfloat16)
    got = fq.kv_attention(1, cache, page, off, table, lens, q, n, n, window=window)
    for h in (0, 1, 2047, 4094, 4095):
        c = dict(fmt=1, cache=cache[:, h:h + 1].cpu().numpy(), page=page, off=np.array([0, n]), D=D, t=None,
                 table=table.cpu().numpy(), lens=np.array([n]), q=q[:, h:h + 1].double().cpu().numpy())
        check_close(c, got[:, h:h + 1], window)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,lens,G,D", [([9, 1], [3, 5], 2, 128), ([7, 5], [2, 0], 4, 64), ([90, 40], [33, 50], 3, 64),
                                        ([40, 30], [4, 1], 2, 256), ([50, 3], [700, 1], 4, 128)])
def test_windows_wider_than_any_length(fmt, n, lens, G, D):
    """Windows up to 2^31 - 1 are no window, for rows before position 0 too."""
    need_gpu()
    say(f"wide window fmt {fmt} n {n} lens {lens} G {G} D {D}")
    c = make(fmt, n, lens, G=G, H=2, D=D, page=16, seed=sum(n))
    want = attend(c)
    check_close(c, want)
    for window in (max(lens), max(lens) + 1, 2 ** 31 - 2, 2 ** 31 - 1):
        got = attend(c, window)
        check_close(c, got, window)
        assert torch.equal(got, want), window


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,G,D", [([1, 2], 4, 128), ([5, 1], 4, 64), ([70, 3], 4, 64), ([33, 40], 2, 256)])
@pytest.mark.parametrize("window", [0, 7, 2 ** 31 - 1])
def test_lengths_past_the_table(fmt, n, G, D, window):
    """Lengths up to the largest 32-bit number over a table of a few pages: what
    the table holds is seen, unless the window has left it."""
    need_gpu()
    say(f"past the table fmt {fmt} n {n} G {G} D {D} window {window}")
    c = make(fmt, n, [96, 95], G=G, H=2, D=D, page=16, seed=sum(n))
    for long in (97, 5000, 2 ** 31 - 40, 2 ** 31 - 1):
        c["lens"] = np.array([long, 95], np.int32)
        got = attend(c, window, max_len=5000)
        check_close(c, got, window)
        if window == 7 and long > 96 + n[0] + 7:
            assert torch.all(got[:n[0]] == 0)


MAGNITUDES = [6, 20, 22, 24, 46, 90, 200, 752, 1504, 3008, 5696, 11904, 23680, 46592, 87040, 159744]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,length", [(1, 700), (1, 3000), (2, 3000), (40, 700), (9, 4000)])
@pytest.mark.parametrize("rise", [False, True])
def test_large_scores_that_differ_little(fmt, D, n, length, rise):
    """Scores up to 2^21 in log2 units, exact in 32 bits, whose differences are
    all that counts: of two groups of keys (in different steps, waves and splits)
    that weigh about the same.  rise: the second group is a few keys late in the
    sequence, 2^9.4 times as heavy each, so that the running maximum moves.

    Tolerance: a weight's rounding u, and 2 keys 2^-24 for the sums (products
    and scores are exact, so no other term grows with the scores); 2^-14 for
    what the kernels round in between."""
    need_gpu()
    say(f"large scores fmt {fmt} D {D} n {n} length {length} rise {rise}")
    heads, scale = len(MAGNITUDES), float(np.float32(1.3))
    c = make(fmt, [n], [length], G=heads, H=1, D=D, page=16, seed=length + n)
    c["t"] = None if fmt == 1 else np.ones(1, np.float32)
    k, v = np.zeros((2, length, 1, D))
    k[:, 0, 0], k[:, 0, 41] = 6.0, 6.0          # (6 in a block: its scale is 1)
    second = np.zeros(length, bool)
    if rise:
        second[length - n - 1 - 97 * np.arange(max(length // 700, 1))] = True
        k[second, 0, 40], k[~second, 0, 40] = 4.0, -1.0
    else:
        second[(np.arange(length) // 32) % 3 == 1] = True
        second[length // 2:] ^= True
        k[second, 0, 40] = c["rng"].choice([0.5, 1.0, 1.5], second.sum())
    v[:, 0] = np.where(second, -6.0, 6.0)[:, None]
    v[:, 0, ::3] *= 0.5
    layer.kv_append(fmt, c["cache"], c["page"], np.array([0, length]), c["table"], c["lens"], k, v, c["t"], c["t"])
    c["q"] = np.zeros((n, heads, D))
    c["q"][:, :, 0], c["q"][:, :, 40] = MAGNITUDES, 1.0
    got = attend(c, scale=scale, y_dtype=fq.OUT_F32).double().cpu().numpy()
    o, w, _ = layer.attention(fmt, c["cache"], c["page"], c["off"], c["table"], c["lens"], c["q"], c["t"], c["t"], 0,
                              scale)
    tol = ((2.0 ** -11 if fmt == 0 else 2.0 ** -8) + 2.0 ** -14 + 2 * length * 2.0 ** -24) * w
    bad = np.argwhere(~(np.abs(got - o) <= tol))
    assert bad.size == 0, f"{len(bad)} off, worst {np.max(np.abs(got - o) / tol):.2f} of the bound, first {bad[:3].tolist()}"


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n", [1, 20])
@pytest.mark.parametrize("top", [1.0, 1.75])
@pytest.mark.parametrize("power", [-131, -127, -126, -120, 120, 125, 126, 127])
def test_queries_at_the_ends_of_bf16(fmt, n, top, power):
    """Rows of the smallest (subnormal) and largest magnitudes, with a scale that
    brings their scores to a few units.  A row has one value and keys are
    small, so that no product overflows and all are exact."""
    need_gpu()
    say(f"q of {top} 2^{power} fmt {fmt} n {n}")
    scale = 2.0 ** min(-power, 126)
    c = make(fmt, [n], [100], G=4, H=1, D=64, page=16, seed=5)
    c["t"] = None if fmt == 1 else np.full(1, 2.0 ** -6, np.float32)
    k, v = np.zeros((2, 100, 1, 64))
    k[:, 0, 3] = 2.0 ** -5 * c["rng"].choice([-3.0, -1.0, 0.5, 1.0, 2.0, 3.0], 100)
    k[:, 0, 4] = 6 * 2.0 ** -5                    # (the block's scale; q is 0 there)
    v[:] = layer.bf16_round(c["rng"].standard_normal(v.shape) / 16)
    layer.kv_append(fmt, c["cache"], c["page"], np.array([0, 100]), c["table"], c["lens"], k, v, c["t"], c["t"])
    c["q"] = np.zeros((n, 4, 64))
    c["q"][:, :, 3] = top * 2.0 ** power
    assert np.array_equal(c["q"], layer.bf16_round(c["q"]))
    got = attend(c, scale=scale, y_dtype=fq.OUT_F32).double().cpu().numpy()
    o, w, _ = layer.attention(fmt, c["cache"], c["page"], c["off"], c["table"], c["lens"], c["q"], c["t"], c["t"], 0,
                              scale)
    # weights' rounding, 200 roundings of the sums, 2^-14 for the exponents
    tol = ((2.0 ** -11 if fmt == 0 else 2.0 ** -8) + 200 * 2.0 ** -24 + 2.0 ** -14) * w
    bad = np.argwhere(~(np.abs(got - o) <= tol))
    assert bad.size == 0, f"{len(bad)} off, first {bad[:3].tolist()}, got {got[0, 0, :3]} want {o[0, 0, :3]}"


# ---- refusals -------------------------------------------------------------------

def test_sizes_without_room_are_refused():
    """With the call's own error, not for lack of memory."""
    need_gpu()
    x = torch.zeros(1000, 64, device="cuda")
    for k, code in ((33, "-2"), (2 ** 31 - 1, "-1"), (65, "-1"), (0, "-1")):
        with pytest.raises(fq.Fp4qError, match=code):
            fq.route(x, k)
    c = make(1, [1], [20], D=64)
    where = (1, dev(c["cache"]), 16, dev(c["off"]), dev(c["table"]), dev(c["lens"]))
    for rows in (2 ** 31, 2 ** 40, 2 ** 62, 2 ** 29):
        with pytest.raises(fq.Fp4qError, match="-2"):
            fq.kv_read(*where, rows, 64)
    for max_new, max_len in ((1, 2 ** 62), (2 ** 62, 20), (2 ** 40, 2 ** 40)):
        with pytest.raises(fq.Fp4qError, match="-2"):
            fq.kv_attention(*where, dev(c["q"], torch.bfloat16), max_new, max_len)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,G", [(1, 4), (30, 3)])
def test_the_largest_max_len_over_short_sequences(fmt, n, G):
    need_gpu()
    c = make(fmt, [n, 1], [300, 77], G=G, H=2, D=128, page=16, seed=n)
    for max_len in (2 ** 31 - 4096, 2 ** 31 - 1):
        check_close(c, attend(c, max_len=max_len))
        check_close(c, attend(c, 100, max_len=max_len), 100)
