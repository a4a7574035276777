"""GPU: low-rank adapters of many requests against the plain 64-bit form.

Tolerance, in units of what the products take in: x A^T is F32 sums of exact
products, K of them in some order, each addition off by at most 2^-23 (so that a
matrix instruction may round its sums towards zero); its two (three) BF16 terms
leave 2^-16 (2^-24) of it, the second product adds `rank` times as many terms, and
the addition of y and the result one rounding each."""
import numpy as np
import pytest
import torch

import fp4_w4a4_quantized_amd as fq
from gpu_helpers import need_gpu, say
from oracle import layer

pytestmark = pytest.mark.gpu

B = torch.bfloat16


def dev(a, dt=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(dt)


def ints(a):
    return torch.tensor(list(a), dtype=torch.int32, device="cuda")


def case(sizes, adapters, rank, K, N, dt, n=4, seed=0, extra=0):
    rng = np.random.default_rng(seed + rank + K + N)
    rows = sum(sizes) + extra
    r = layer.bf16_round
    y = rng.standard_normal((rows, N))
    return dict(x=r(rng.standard_normal((rows, K))), a=r(rng.standard_normal((n, rank, K)) * K ** -0.5),
                b=r(rng.standard_normal((n, N, rank))), off=np.concatenate([[0], np.cumsum(sizes)]),
                ad=list(adapters), scale=(0.5 + rng.random(n)).astype(np.float32), rank=rank, K=K, N=N, dt=dt,
                y=r(y) if dt == B else y.astype(np.float32).astype(np.float64))


def check(c, got, y=True, scale=True):
    want, inner, outer = layer.lora(c["x"], c["a"], c["b"], c["off"], c["ad"], c["scale"] if scale else None,
                                    c["y"] if y else None)
    bf = c["dt"] == B
    terms = 2 if bf else 3
    tol = ((c["K"] + 64) * 2.0 ** -23 * inner + (2.0 ** (-16 if bf else -24) + (terms * c["rank"] + 8) * 2.0 ** -23) * outer
           + 2.0 ** -24 * np.abs(want))
    tol = tol + (2.0 ** -8 if bf else 0.0) * (np.abs(want) + tol)
    err = np.abs(got.double().cpu().numpy() - want)
    bad = np.argwhere(~(err <= tol))
    assert bad.size == 0, (f"{len(bad)} of {want.size} off, worst {np.nanmax(err / np.maximum(tol, 1e-300)):.2f} of the "
                           f"bound, first {bad[:3].tolist()}")
    none = np.ones(len(want), bool)
    for g, j in enumerate(c["ad"]):
        if 0 <= j < len(c["a"]):
            none[c["off"][g]:c["off"][g + 1]] = False
    assert np.array_equal(got.double().cpu().numpy()[none], (c["y"] if y else 0 * c["y"])[none])


def call(c, y=True, scale=True, **kw):
    return fq.lora(dev(c["x"], B), dev(c["a"], B), dev(c["b"], B), ints(c["off"]), ints(c["ad"]),
                   dev(c["scale"]) if scale else None, dev(c["y"], c["dt"]) if y else None,
                   **({} if y else {"y_dtype": fq.OUT_BF16 if c["dt"] == B else fq.OUT_F32}), **kw)


@pytest.mark.parametrize("dt", [B, torch.float32])
@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 64, 72, 128])
def test_ranks(dt, rank):
    need_gpu()
    say(f"lora rank {rank} {dt}")
    for sizes, ad in (([1, 3, 0, 17, 1], [2, 0, 1, 3, 2]), ([70, 200], [1, 0])):
        c = case(sizes, ad, rank, 264, 300, dt)
        check(c, call(c))


@pytest.mark.parametrize("dt", [B, torch.float32])
@pytest.mark.parametrize("K,N", [(8, 1), (40, 15), (128, 17), (1000, 64), (4104, 257), (9000, 1023)])
def test_odd_sizes(dt, K, N):
    need_gpu()
    say(f"lora K {K} N {N} {dt}")
    for sizes, ad in (([1], [1]), ([2, 1, 40], [0, -1, 3]), ([90, 33], [3, 3])):
        c = case(sizes, ad, 16, K, N, dt)
        check(c, call(c))


def test_requests_without_adapter_and_rows_behind():
    """-1 and numbers past the adapters: y's rows, as the rows behind the last
    request; signed zeros and NaN among them pass."""
    need_gpu()
    for sizes, ad in (([2, 5, 1, 3], [-1, 1, 9, 0]), ([100, 64, 40], [0, -1, 2])):
        c = case(sizes, ad, 16, 64, 100, B, extra=21)
        c["y"][:2] = -0.0
        got = call(c)
        check(c, got)
        assert torch.equal(got[c["off"][-1]:].view(torch.int16), dev(c["y"], B)[c["off"][-1]:].view(torch.int16))
        if ad[0] == -1:
            assert torch.all(torch.signbit(got[:2]))
        check(c, call(c, y=False), y=False)
        # in place: those rows keep whatever they hold
        y = dev(c["y"], B)
        y[c["off"][-1]:] = float("nan")
        fq.lora_into(dev(c["x"], B), dev(c["a"], B), dev(c["b"], B), ints(c["off"]), ints(c["ad"]), dev(c["scale"]), y, y)
        assert torch.all(torch.isnan(y[c["off"][-1]:])) and torch.equal(y[:c["off"][-1]], got[:c["off"][-1]])


def test_strided_rows():
    need_gpu()
    for dt in (B, torch.float32):
        c = case([3, 50, 2], [0, 1, 2], 32, 96, 77, dt)
        rows = len(c["x"])
        x = torch.zeros(rows, 104, device="cuda", dtype=B)
        x[:, :96] = dev(c["x"], B)
        y = torch.full((rows, 80), 5.0, device="cuda", dtype=dt)
        y[:, 1:78] = dev(c["y"], dt)
        out = torch.full((rows, 83), 7.0, device="cuda", dtype=dt)
        fq.lora_into(x[:, :96], dev(c["a"], B), dev(c["b"], B), ints(c["off"]), ints(c["ad"]), dev(c["scale"]),
                     y[:, 1:78], out[:, 3:80])
        check(c, out[:, 3:80])
        assert torch.all(out[:, :3] == 7.0) and torch.all(out[:, 80:] == 7.0)
        check(c, call(c, scale=False), scale=False)


def test_many_requests_and_long_sums():
    need_gpu()
    rng = np.random.default_rng(0)
    sizes = rng.integers(0, 4, 200)
    c = case(sizes, rng.integers(-1, 6, 200), 16, 512, 200, B, n=6)
    check(c, call(c))
    c = case([1, 2], [0, 1], 64, 12288, 640, torch.float32)
    a = call(c)
    check(c, a)
    assert torch.equal(a, call(c)), "two runs differ"


@pytest.mark.parametrize("rank", [16, 32, 64, 128])
def test_tiles_of_many_rows(rank):
    """Rows enough for the larger tiles, requests that end inside them."""
    need_gpu()
    for dt in (B, torch.float32):
        c = case([1000, 3, 0, 130, 77], [2, 1, 0, -1, 3], rank, 136, 200, dt, extra=9)
        check(c, call(c))


def test_empty():
    need_gpu()
    c = case([0, 0], [0, 1], 16, 64, 32, B)
    assert call(c).shape == (0, 32)


def test_captured_and_on_a_stream():
    """Two captured calls of different sizes, replayed with other adapters and
    inputs; the workspaces are their own."""
    need_gpu()
    c1, c2 = case([1] * 20, np.arange(20) % 4, 16, 1024, 512, B), case([60, 70], [1, 2], 32, 256, 300, torch.float32)

    def tensors(c):
        return [dev(c["x"], B), dev(c["a"], B), dev(c["b"], B), ints(c["off"]), ints(c["ad"]), dev(c["scale"]),
                dev(c["y"], c["dt"])]

    t1, t2 = tensors(c1), tensors(c2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fq.lora(*t1)
        fq.lora(*t2)
    torch.cuda.current_stream().wait_stream(s)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        o1 = fq.lora(*t1)
    with torch.cuda.graph(g2):
        o2 = fq.lora(*t2)
    for k in (1, 2, 3):
        t1[4].copy_(torch.roll(t1[4], k))
        t2[0].mul_(-1)
        w1, w2 = fq.lora(*t1), fq.lora(*t2)
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(o1, w1) and torch.equal(o2, w2)
    s.wait_stream(torch.cuda.current_stream())
    o = fq.lora(*t1, stream=s)
    s.synchronize()
    assert torch.equal(o, w1)


@pytest.mark.parametrize("dt", [B, torch.float32])
@pytest.mark.parametrize("rank,K,sizes", [(8, 40, [3, 2, 4]), (40, 264, [5, 1, 2]), (32, 1032, [700, 100, 400])])
def test_infinities(dt, rank, K, sizes):
    """An infinite weight (in the columns that a step past the end reads again), an
    infinite and a NaN input: each row as the formula has it, its neighbours as
    without them."""
    need_gpu()
    say(f"lora infinities rank {rank} K {K} {dt}")
    c = case(sizes, [0, 1, 2], rank, K, 72, dt)
    c["a"][1, rank - 3, 2] = np.inf
    row = sizes[0] + sizes[1]
    c["a"][2, :, 5] = 0.5
    c["x"][row, 5], c["x"][row + 1, 0] = -np.inf, np.nan
    c["b"][2] = np.abs(c["b"][2])          # infinities of one sign
    with np.errstate(invalid="ignore"):
        want = layer.lora(c["x"], c["a"], c["b"], c["off"], c["ad"], c["scale"], c["y"])[0]
    got = call(c).double().cpu().numpy()
    finite = np.isfinite(want)
    assert not finite[sizes[0]:row + 2].any() and finite[:sizes[0]].all() and finite[row + 2:].all()
    assert np.isinf(want[sizes[0]:row + 1]).any() and np.isnan(want[row + 1]).all()
    assert np.array_equal(got[~finite], want[~finite], equal_nan=True)
    keep = [r for r in range(len(want)) if finite[r].all()]
    clean = dict(c, a=np.where(np.isfinite(c["a"]), c["a"], 0.0), x=np.where(np.isfinite(c["x"]), c["x"], 0.0))
    assert np.array_equal(got[keep], call(clean).double().cpu().numpy()[keep])


@pytest.mark.parametrize("dt", [B, torch.float32])
def test_no_rows_without_y(dt):
    """An empty batch's adapters alone, and into an empty result."""
    need_gpu()
    c = case([0, 0], [0, 1], 16, 64, 32, dt)
    got = call(c, y=False)
    assert got.shape == (0, 32) and got.dtype == dt
    out = torch.empty(0, 32, device="cuda", dtype=dt)
    fq.lora_into(dev(c["x"], B), dev(c["a"], B), dev(c["b"], B), ints(c["off"]), ints(c["ad"]), None, None, out)


def exact_u(c, row, k):
    """Row `row` takes x's column k alone, of A's elements 1, -2, 0.5 ..: x A^T is exact
    in BF16, its lower terms are 0."""
    c["x"][row] = 0.0
    c["x"][row, k] = 1.0
    c["a"][:, :, k] = np.resize([1.0, -2.0, 0.5, 4.0], c["a"].shape[:2])


@pytest.mark.parametrize("dt", [B, torch.float32])
@pytest.mark.parametrize("rank,sizes", [(8, [3, 2, 4]), (40, [20, 1, 2]), (128, [5, 3, 2]), (32, [700, 100, 400]),
                                        (72, [700, 100, 400])])
def test_infinite_and_nan_weights_of_the_second_product(dt, rank, sizes):
    """Infinities and a NaN in B, in whole steps of columns and behind the last one,
    against x A^T that is exact in BF16 and that has lower terms of both signs: the
    formula's value; the columns beside them as without them."""
    need_gpu()
    say(f"lora infinite b rank {rank} rows {sum(sizes)} {dt}")
    c = case(sizes, [0, 1, 2], rank, 264, 330, dt)
    c["scale"][:] = 0.5
    for row in (0, sizes[0]):
        exact_u(c, row, 9)
    bad = [3, 64, 200, 329]
    c["b"][1, bad[0], rank - 1], c["b"][1, bad[1], 0] = np.inf, -np.inf
    c["b"][0, bad[2], 1], c["b"][0, bad[2], 5] = np.inf, np.inf
    c["b"][0, bad[3], 2], c["b"][2, bad[3], 0] = np.nan, -np.inf
    with np.errstate(invalid="ignore"):
        want = layer.lora(c["x"], c["a"], c["b"], c["off"], c["ad"], c["scale"], c["y"])[0]
    got = call(c).double().cpu().numpy()
    finite = np.isfinite(want)
    assert np.isinf(want[:, bad]).sum() >= sizes[1] and np.isnan(want[:, bad]).sum() >= sizes[0]
    assert np.array_equal(got[~finite], want[~finite], equal_nan=True)
    keep = np.ones(330, bool)
    keep[bad] = False
    clean = dict(c, b=np.where(np.isfinite(c["b"]), c["b"], 0.0))
    assert finite[:, keep].all() and np.array_equal(got[:, keep], call(clean).double().cpu().numpy()[:, keep])
    # a zero in x A^T times an infinity is NaN, and stays in its row
    c["x"][sum(sizes[:2])] = 0.0
    assert torch.all(torch.isnan(call(c)[sum(sizes[:2]), bad[3]]))


@pytest.mark.parametrize("dt", [B, torch.float32])
def test_inner_sums_past_the_largest_bf16(dt):
    """x A^T between the largest BF16 and the largest F32: its first term is the former,
    not infinity."""
    need_gpu()
    c = case([3, 2], [0, 1], 8, 16, 70, dt)
    top = layer.bf16_round(1.9921875)
    c["x"][:], c["a"][:], c["scale"][:] = 0.0, 0.0, 1.0
    c["x"][:, 0], c["x"][:, 1] = 2.0 ** 64, 2.0 ** 60
    c["a"][:, ::2, 0], c["a"][:, ::2, 1] = top * 2.0 ** 63, 1.5 * 2.0 ** 59
    c["a"][:, 1::2, 0], c["a"][:, 1::2, 1] = -top * 2.0 ** 63, -1.75 * 2.0 ** 59
    u = c["x"][0] @ c["a"][0].T
    assert np.all(np.abs(u) > top * 2.0 ** 127) and np.all(np.abs(u) < 2.0 ** 128)
    assert np.all(np.isinf(dev(u, B).float().cpu().numpy()))
    c["b"] = c["b"] * 2.0 ** -100
    check(c, call(c))


def test_nan_and_infinite_y_are_copied():
    """Rows of none and of requests without adapter, into an out of its own."""
    need_gpu()
    for dt in (B, torch.float32):
        c = case([4, 3], [-1, 1], 16, 64, 101, dt, extra=5)
        c["y"][:4, ::3], c["y"][7:, 1::2], c["y"][5, 50], c["y"][9, 0] = np.nan, np.inf, np.nan, -np.inf
        got = call(c).double().cpu().numpy()
        rest = np.r_[0:4, 7:12]
        assert np.array_equal(got[rest], c["y"][rest], equal_nan=True)
        assert np.isnan(got[5, 50]) and np.isfinite(np.delete(got[4:7], 50, 1)).all()


def test_no_requests():
    need_gpu()
    c = case([0], [0], 16, 64, 32, B)
    c.update(off=[0], ad=[])
    assert call(c).shape == call(c, y=False).shape == (0, 32)
