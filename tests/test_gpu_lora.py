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
