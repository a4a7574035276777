"""GPU: the paths that attention and the router take by size (row tiles,
splits of the keys, tokens of a workgroup), at the borders of their rules,
against the plain 64-bit forms with the tolerances of
test_gpu_kv_attention.py and test_gpu_route_combine.py."""
import numpy as np
import pytest
import torch

import fp4_w4a4_quantized_amd as fq
from gpu_helpers import need_gpu, say
from oracle import layer
from test_gpu_kv_attention import FMTS, attend, check_close, dev, make
from test_gpu_route_combine import check_route, host, logits_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [16, 17, 32, 33, 63, 64, 65, 128, 129, 257])
def test_rows_around_the_tiles(fmt, D, n):
    """One head a kv head: n rows, the first that see the fewest keys included."""
    need_gpu()
    say(f"rows fmt {fmt} D {D} n {n}")
    c = make(fmt, [n, 1], [n, n + 3], G=1, H=1, D=D, seed=n)
    check_close(c, attend(c))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("page", [16, 32, 64, 1024])
@pytest.mark.parametrize("window", [0, 63, 500])
def test_prompt_chunks_over_split_keys(fmt, page, window):
    """Many rows over keys that are split, in pages smaller and larger than a
    step of 64 keys."""
    need_gpu()
    say(f"chunk fmt {fmt} page {page} window {window}")
    c = make(fmt, [70, 40], [1500, 2101], G=4, H=1, D=64, page=page, seed=page + window)
    a = attend(c, window)
    check_close(c, a, window)
    assert torch.equal(a, attend(c, window)), "two runs differ"
    check_close(c, attend(c, window, max_len=30000), window)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
def test_prompts_with_pages_gone(fmt, D):
    need_gpu()
    c = make(fmt, [60, 90, 50], [200, 90, 333], G=3, H=2, D=D, page=16, seed=D)
    c["table"][0, 2] = -1
    c["table"][0, 12] = 10 ** 6                    # of the newest tokens
    c["table"][1, :] = -1
    c["table"][2, 0:20:2] = -2147483648
    got = attend(c, max_len=333)
    check_close(c, got)
    assert torch.all(got[60:150] == 0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("mult", [2.0 ** 14, 2.0 ** 30])
def test_prompt_with_huge_scores(fmt, mult):
    """Scores far past 2^20, where their differences decide alone: the largest
    takes all."""
    need_gpu()
    c = make(fmt, [50], [90], G=2, H=2, D=128, seed=3)
    c["q"] = layer.bf16_round(c["q"] * mult)
    o, _, s = layer.attention(fmt, c["cache"], c["page"], c["off"], c["table"], c["lens"], c["q"], c["t"],
                              c["t"])
    g = attend(c).float().cpu().numpy()
    # rows whose two largest scores are further apart than 64 + the scores' own
    # rounding have one weight of 1 in both
    k, _ = zip(*[layer.kv_values(fmt, c["cache"], 16, 128, c["table"][0, np.arange(90) // 16].astype(np.int64),
                                 np.arange(90) % 16, h, c["t"], c["t"]) for h in range(2)])
    checked = 0
    for i in range(50):
        for j in range(4):
            x = np.sort((k[j // 2][:41 + i] @ c["q"][i, j]) * 128 ** -0.5)
            if x[-1] - x[-2] > 64 + 2 * 144 * 2.0 ** -24 * s[i, j, 0]:
                checked += 1
                assert np.all(np.abs(g[i, j] - o[i, j]) <= 2.0 ** -7 * np.abs(o[i, j]) + 1e-6), (i, j)
    assert checked > 100


def test_infinite_values_of_later_tokens_stay_there():
    """MXFP4: a later token's largest possible values do not reach the rows
    before it."""
    need_gpu()
    c = make(1, [64], [64], G=1, H=1, D=64, page=16, seed=6, garbage=False)
    kb, kh, vb, vh, ks, vs = layer.kv_places(1, 16, 64)
    clean = attend(c)
    c["cache"][c["table"][0, 3]][:, vs[15]] = 254   # the last token's V scales
    got = attend(c)
    assert torch.equal(got[:63], clean[:63])


@pytest.mark.parametrize("T", [15, 16, 17, 4095, 4096, 4097, 9000])
def test_router_blocks(T):
    need_gpu()
    say(f"route T {T}")
    x = logits_of(T, 40, torch.float32, T)
    check_route(x, 3)
    check_route(x, 5, 1, torch.linspace(-0.1, 0.1, 40).cuda(), 4, 2)


@pytest.mark.parametrize("T", [64 * 511, 64 * 511 + 1, 64 * 1024 * 16 + 1])
def test_router_orders_many_blocks(T):
    """Around the number of workgroups from which their counts are summed up
    apart, and past what one pass of that takes: the order follows from the
    choice (checked by itself above)."""
    need_gpu()
    say(f"route order T {T}")
    x = torch.randn(T, 6, device="cuda")
    r = fq.route(x, 2)
    e = r["experts"].long()
    assert torch.equal(e, x.sort(dim=1, descending=True, stable=True).indices[:, :2])
    flat = e.reshape(-1)
    order = flat.sort(stable=True).indices
    assert torch.equal(r["row_src"].long(), order // 2)
    assert torch.equal(r["row_of"].reshape(-1)[order].long(), torch.arange(2 * T, device="cuda"))
    assert torch.equal(r["offsets"][1:].long(), torch.bincount(flat, minlength=6).cumsum(0))
    assert int(r["offsets"][0]) == 0


def test_router_nan_logits_count_as_minus_infinity():
    need_gpu()
    x = logits_of(50, 70, torch.float32, 2)
    x[3, 5:60] = float("nan")
    x[4, :] = float("nan")
    x[7, 69] = float("nan")
    y = torch.where(torch.isnan(x), torch.full_like(x, -float("inf")), x)
    dw = torch.ones(50, 4, device="cuda")
    for score in (0, 1):
        for renorm in (False, True):
            a, b = (fq.route(v, 4, score=score, renorm=renorm) for v in (x, y))
            for key in a:
                assert torch.equal(a[key], b[key]), key
            da, db = (fq.route_backward(v, a["experts"], dw, score=score, renorm=renorm) for v in (x, y))
            assert torch.equal(da, db) and torch.isfinite(da).all()
            check_route(y, 4, score, renorm=renorm)


def test_combine_in_two_rows_of_workgroups():
    """More workgroups than one row of the grid holds (single columns)."""
    need_gpu()
    T, N = 1 << 16, 4099                           # 2^28 outputs of one value each
    y = torch.randn(4, N, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    row_of = (torch.arange(T, device="cuda") % 5 - 1).int().view(T, 1)
    w = torch.full((T, 1), 0.5, device="cuda")
    out = fq.combine(y, row_of, w)
    for t in (0, 1, 2, 4, T // 2, T - 5, T - 1):
        r = t % 5 - 1
        want = torch.zeros(N) if r < 0 else 0.5 * host(y[r])
        assert np.array_equal(host(out[t]), np.asarray(want, dtype=np.float64)), t
    assert torch.equal(out[:5].repeat(100, 1), out[T // 5 * 5 - 500:T // 5 * 5])


def test_combine_without_rows():
    need_gpu()
    row_of = torch.zeros(5, 2, dtype=torch.int32, device="cuda")
    w = torch.ones(5, 2, device="cuda")
    out = fq.combine(torch.empty(0, 64, device="cuda"), row_of, w)
    assert torch.all(out == 0)
    big = torch.full((3, 64), float("nan"), device="cuda")
    row_of[:] = -1
    row_of[0, 1] = 2
    big[2] = 1.0
    got = host(fq.combine(big, row_of, w))
    assert np.all(got[0] == 1.0) and np.all(got[1:] == 0.0)


def test_results_on_another_stream_are_of_its_own_memory():
    """Memory freed on the current stream while its work there is pending is
    not what a call on another stream writes to."""
    need_gpu()
    say("results on another stream")
    T, k, E, N = 2048, 4, 64, 512
    x = logits_of(T, E, torch.float32, 3)
    y = torch.randn(T * k, N, device="cuda")
    do = torch.randn(T, N, device="cuda")
    r = fq.route(x, k)
    dw = torch.randn(T, k, device="cuda")
    c = make(0, [1] * 16, [800] * 16, G=4, H=2, seed=5)
    kv = [0, dev(c["cache"]), c["page"], dev(c["off"]), dev(c["table"]), dev(c["lens"])]
    t, q = dev(c["t"]), dev(c["q"], torch.bfloat16)
    calls = [
        lambda s: list(fq.route(x, k, stream=s).values()),
        lambda s: [fq.route_backward(x, r["experts"], dw, stream=s)],
        lambda s: [fq.combine(y, r["row_of"], r["weights"], stream=s)],
        lambda s: list(fq.combine_backward(y, r["row_of"], r["weights"], do, stream=s)),
        lambda s: [fq.kv_attention(*kv, q, 1, 800, t, t, stream=s)],
        lambda s: list(fq.kv_read(*kv, 16, 128, t, t, stream=s)),
    ]
    s = torch.cuda.Stream()
    for i, call in enumerate(calls):
        want = [v.clone() for v in call(None)]
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        left = [torch.empty(v.untyped_storage().nbytes(), dtype=torch.uint8, device="cuda")
                for v in want for _ in range(2)]
        for b in left:
            b.fill_(255)
        del left, b
        got = call(s)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,lens,G,D", [([1, 0, 1], [300, 0, 70], 4, 128),       # one pass, few rows
                                        ([1, 1, 1], [9000, 4, 900], 5, 64),      # split keys
                                        ([5, 1, 0], [700, 1, 9], 6, 128),        # 30 rows of a head
                                        ([40, 3, 2], [40, 3, 2], 3, 256),        # row tiles
                                        ([70, 0, 0], [1500, 0, 0], 4, 64),       # the same, split keys
                                        ([0, 0, 0], [5, 0, 2], 2, 128)])         # no new tokens at all
def test_rows_past_the_offsets(fmt, n, lens, G, D):
    """Padding rows give 0; rows that the offsets name and the tensors do not
    have are left out."""
    need_gpu()
    say(f"padding fmt {fmt} n {n} lens {lens} G {G} D {D}")
    c = make(fmt, n, lens, G=G, H=2, D=D, seed=sum(n))
    rows = len(c["q"])
    c["q"] = np.concatenate([c["q"], np.full((37, 2 * G, D), np.nan)])
    for y_dtype in (fq.OUT_BF16, fq.OUT_F32):
        nb = 37 * 2 * G * D * 4
        torch.full((4 * nb,), 255, dtype=torch.uint8, device="cuda")  # what freed memory may hold
        got = attend(c, y_dtype=y_dtype)
        assert torch.all(got[rows:] == 0)
        check_close(c, got, bf16=y_dtype == fq.OUT_BF16)
    c["q"] = c["q"][:rows]
    if rows > 2:
        q = dev(c["q"][:rows - 2], torch.bfloat16)
        got = torch.cat([attend(c, q=q), attend(c)[rows - 2:]])
        check_close(c, got)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k", [(1, 1), (8, 8), (17, 16), (60, 4), (64, 16), (65, 17), (128, 8), (200, 16),
                                 (512, 3), (384, 32)])
def test_route_of_many_tokens(dtype, E, k):
    """More than 4096 tokens, the last workgroup partly filled; ties, NaN and
    infinities among the logits."""
    need_gpu()
    say(f"route many {dtype} E{E} k{k}")
    for score in (0, 1):
        x = logits_of(4099, E, dtype, E + k)
        x[1] = 0.5
        x[2, ::2] = -float("inf")
        x[3] = torch.finfo(dtype).min
        x[4098] = -float("inf")
        x[5, E // 2] = torch.finfo(dtype).max
        check_route(x, k, score, renorm=True)
        check_route(x, k, score, renorm=False)
        y = x.clone()
        y[2, ::2] = float("nan")
        a, b = fq.route(x, k, score=score), fq.route(y, k, score=score)
        for key in a:
            assert torch.equal(a[key], b[key]), key


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(1, 8, 8), (15, 17, 16), (33, 64, 17), (18, 128, 5), (9, 256, 32), (7, 300, 2)])
def test_route_gradient_of_given_experts(dtype, T, E, k):
    """Any experts, not the best: of far smaller scores, named twice, outside
    the experts (no gradient)."""
    need_gpu()
    say(f"route gradient {dtype} T{T} E{E} k{k}")
    g = torch.Generator().manual_seed(T + E)
    x = logits_of(T, E, dtype, T)
    x[0, 0] = 900.0                                # the others' scores underflow
    e = torch.randint(0, E, (T, k), generator=g).int()
    e[0] = 1
    dw = torch.randn(T, k, generator=g)
    far = e.clone()
    far[-1, 0], far[-1, -1] = -1, E
    far[0, k // 2] = 2 ** 31 - 1
    for score in (0, 1):
        for renorm in (False, True):
            got = fq.route_backward(x, e.cuda(), dw.cuda(), score=score, renorm=renorm)
            want, size = layer.route_backward(host(x), e.numpy(), dw.numpy(), score, renorm)
            u = (2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8) + 2.0 ** -24
            # an expert named k times: that many roundings of the sum
            tol = u * np.abs(want) + (2.0 ** -40 + k * 2.0 ** -24) * size + 1e-38
            assert np.all(np.abs(host(got) - want) <= tol), (score, renorm)
            # left out like weights of 0 without a gradient, where nothing divides by them
            if not renorm:
                a = fq.route_backward(x, far.cuda(), dw.cuda(), score=score, renorm=renorm)
                b = fq.route_backward(x, e.cuda(), torch.where(far == e, dw, 0.0).cuda(), score=score,
                                      renorm=renorm)
                assert torch.equal(a, b), score
            assert torch.isfinite(fq.route_backward(x, far.cuda(), dw.cuda(), score=score,
                                                    renorm=renorm)).all()


@pytest.mark.parametrize("T", [8192, 8197])
def test_route_of_full_workgroups(T):
    need_gpu()
    say(f"route full workgroups T {T}")
    x = logits_of(T, 40, torch.bfloat16, T)
    check_route(x, 5)
    check_route(x, 17)
    check_route(x.float(), 5, 1, torch.linspace(-0.1, 0.1, 40).cuda(), 4, 2)


def test_router_keys_that_differ_in_their_last_bits():
    """Scores in 64 bits that agree in their upper halves, and equal ones."""
    need_gpu()
    g = torch.Generator().manual_seed(1)
    x = 1e-7 * torch.randn(300, 96, generator=g)   # sigmoids within 2^-24 of 1/2
    x[:, ::7] = 0.0
    x[:, 1::7] = -0.0
    x = x.cuda()
    b = torch.zeros(96).cuda()
    for score in (0, 1):
        check_route(x, 9, score, b)
        check_route(x, 9, score, b - 1.0)          # keys below 0
        check_route(x, 9, score, b, 8, 3)
        check_route(x, 9, score, b - 1.0, 3, 2, renorm=False)
