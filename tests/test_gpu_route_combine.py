"""GPU: the router (choice, weights, expert order, gradient) and the
combination of the experts' outputs (and its gradients) against the plain
64-bit forms of oracle/layer.py.

Tolerances: choices and orders are equal.  Weights and the logits' gradient
are computed in 64 bits and rounded once: half a step of the output's type
(2^-24 f32, 2^-8 bf16), and 2^-40 of the terms' size for the 64-bit
functions.  A combination adds k products in FP32: (k + 1) 2^-24 of the sum
of magnitudes, then the output's rounding; d_weights adds N products:
N 2^-24 of theirs.
"""
import numpy as np
import pytest
import torch

import fp4_w4a4_quantized_amd as fq
from gpu_helpers import need_gpu, say
from oracle import layer

pytestmark = pytest.mark.gpu

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def host(t):
    return t.detach().double().cpu().numpy()


def logits_of(T, E, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = 1.5 * torch.randn(T, E, generator=g) + torch.randn(E, generator=g)
    return x.to(dtype).cuda()


def check_route(x, k, score=0, bias=None, groups=1, top=1, renorm=True):
    r = fq.route(x, k, score=score, bias=bias, n_groups=groups, top_groups=top, renorm=renorm)
    want = layer.route(host(x), k, score, None if bias is None else host(bias), groups, top, renorm)
    for key in ("experts", "offsets", "row_src", "row_of"):
        g = r[key].cpu().numpy()
        bad = np.argwhere(g != want[key])
        assert bad.size == 0, f"{key}: {len(bad)} differ, first {bad[:3].tolist()}"
    w = host(r["weights"])
    assert np.all(np.abs(w - want["weights"]) <= (2.0 ** -24 + 2.0 ** -40) * want["weights"] + 1e-45)
    return r, want


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(1, 128, 8), (5, 8, 1), (63, 60, 4), (64, 64, 6), (65, 96, 10),
                                   (200, 160, 5), (129, 256, 8), (300, 384, 7), (70, 512, 32), (3, 1, 1),
                                   (2, 10, 10)])
@pytest.mark.parametrize("score", [0, 1])
def test_route(dtype, T, E, k, score):
    need_gpu()
    say(f"route {dtype} T{T} E{E} k{k} score {score}")
    x = logits_of(T, E, dtype, T + E)
    check_route(x, k, score)
    check_route(x, k, score, renorm=False)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("E,groups,top,k", [(256, 8, 4, 8), (60, 4, 2, 5), (96, 2, 1, 10), (512, 8, 8, 10),
                                            (64, 64, 5, 4), (384, 3, 2, 6), (15, 5, 2, 6), (128, 1, 1, 8)])
def test_route_bias_and_groups(score, E, groups, top, k):
    need_gpu()
    say(f"groups E{E} {groups}/{top} k{k} score {score}")
    for T, dtype in ((77, torch.float32), (130, torch.bfloat16)):
        x = logits_of(T, E, dtype, E + groups)
        b = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(E)).cuda()
        check_route(x, k, score, b, groups, top)
        check_route(x, k, score, None, groups, top, renorm=False)


def test_route_ties_and_masked_experts():
    """Equal logits go to the lower index; -inf takes an expert out of the
    running while others are left; a row of nothing but -inf has weights 0."""
    need_gpu()
    x = torch.zeros(5, 70, device="cuda")
    x[1, 3:60] = -0.0
    x[2, :] = -float("inf")
    x[2, 65], x[2, 9] = 1.0, 1.0
    x[3, :] = -float("inf")
    for score in (0, 1):
        r, _ = check_route(x, 4, score)
        assert r["experts"].cpu().tolist() == [[0, 1, 2, 3], [0, 1, 2, 3], [9, 65, 0, 1], [0, 1, 2, 3],
                                               [0, 1, 2, 3]]
        assert torch.all(r["weights"][3] == 0)
        d = fq.route_backward(x, r["experts"], torch.ones(5, 4, device="cuda"), score=score)
        assert torch.isfinite(d).all() and torch.all(d[3] == 0)
    # coarse logits: many ties at the border of the choice, and between groups
    g = torch.Generator().manual_seed(1)
    x = (torch.randn(200, 64, generator=g).round() / 2).cuda()
    check_route(x, 8)
    check_route(x, 6, 1, torch.zeros(64).cuda(), 8, 3)


def test_route_strided_logits():
    need_gpu()
    big = logits_of(100, 200, torch.float32, 3)
    x = big[:, 17:17 + 128]
    r, _ = check_route(x, 8)
    out = torch.full((100, 150), 9.0, device="cuda")
    fq.route_backward_into(x, r["experts"], torch.ones(100, 8, device="cuda"), 0, False, out[:, 5:133])
    want, size = layer.route_backward(host(x), r["experts"].cpu().numpy(), np.ones((100, 8)), 0, False)
    assert np.all(np.abs(host(out[:, 5:133]) - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -40 * size)
    assert torch.all(out[:, :5] == 9.0) and torch.all(out[:, 133:] == 9.0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 16, 2), (77, 60, 4), (130, 384, 10), (40, 512, 32)])
def test_route_backward(dtype, score, renorm, T, E, k):
    need_gpu()
    say(f"route_backward {dtype} T{T} E{E} k{k} score {score} renorm {renorm}")
    x = logits_of(T, E, dtype, T)
    r = fq.route(x, k, score=score, renorm=renorm)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(5)).cuda()
    d = fq.route_backward(x, r["experts"], dw, score=score, renorm=renorm)
    assert d.dtype == dtype
    want, size = layer.route_backward(host(x), r["experts"].cpu().numpy(), host(dw), score, renorm)
    u = U[dtype] + (2.0 ** -24 if dtype == torch.bfloat16 else 0.0)
    assert np.all(np.abs(host(d) - want) <= u * np.abs(want) + 2.0 ** -40 * size + 1e-38)


def test_route_gradient_against_differences():
    """The gradient against differences of the GPU's own weights."""
    need_gpu()
    x = logits_of(6, 24, torch.float32, 2)
    dw = torch.randn(6, 3, generator=torch.Generator().manual_seed(6)).cuda()
    for score in (0, 1):
        for renorm in (False, True):
            r = fq.route(x, 3, score=score, renorm=renorm)
            d = host(fq.route_backward(x, r["experts"], dw, score=score, renorm=renorm))
            h = 2.0 ** -9
            for e in range(24):
                up, dn = x.clone(), x.clone()
                up[:, e] += h
                dn[:, e] -= h
                # the weights at the fixed choice (a step may change the choice itself)
                ru, rd = (fq.route(v, 3, score=score, renorm=renorm) for v in (up, dn))
                same = ((ru["experts"] == r["experts"]).all(1) & (rd["experts"] == r["experts"]).all(1))
                # the steps as the logits hold them
                step = host(up[:, e]) - host(dn[:, e])
                diff = (host((ru["weights"] - rd["weights"])) * host(dw)).sum(1) / step
                # f32 weights: 2 * 2^-24 |dw| / step each; the difference's own error ~ h^2
                tol = 3 * 2.0 ** -23 * 4.0 / (2 * h) + 8.0 * h * h
                assert np.all(np.abs(diff - d[:, e])[same.cpu().numpy()] <= tol)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,k,N", [(1, 1, 128), (3, 8, 2048), (65, 4, 136), (33, 3, 100), (7, 2, 1),
                                   (20, 6, 4096), (2, 40, 72)])
def test_combine(dtype, T, k, N):
    need_gpu()
    say(f"combine {dtype} T{T} k{k} N{N}")
    g = torch.Generator().manual_seed(T * k + N)
    y = torch.randn(T * k, N, generator=g).to(dtype).cuda()
    row_of = torch.randperm(T * k, generator=g).int().view(T, k).cuda()
    w = torch.softmax(torch.randn(T, k, generator=g), 1).cuda()
    do = torch.randn(T, N, generator=g).to(dtype).cuda()
    u = U[dtype]
    out = fq.combine(y, row_of, w)
    want, mag = layer.combine(host(y), row_of.cpu().numpy(), host(w))
    tol = (k + 1) * 2.0 ** -24 * mag
    assert np.all(np.abs(host(out) - want) <= tol + u * (np.abs(want) + tol))
    d_y, d_w = fq.combine_backward(y, row_of, w, do)
    wy, ww, mag = layer.combine_backward(host(y), row_of.cpu().numpy(), host(w), host(do))
    assert np.all(np.abs(host(d_y) - wy) <= (u + 2.0 ** -24 * (1 + u)) * np.abs(wy) + 1e-38)
    assert np.all(np.abs(host(d_w) - ww) <= (N + 1) * 2.0 ** -24 * mag + 1e-38)


def test_combine_strides_and_left_out_rows():
    """Row strides, an odd base address, entries outside the rows, and rows
    that no entry names (their gradient is left as it is)."""
    need_gpu()
    g = torch.Generator().manual_seed(8)
    for dtype in (torch.float32, torch.bfloat16):
        for c0 in (0, 1, 8):
            y = torch.randn(20, 96, generator=g).to(dtype).cuda()[:, c0:c0 + 64]
            row_of = torch.tensor([[3, -1, 19], [20, 0, 5], [-2147483648, 2147483647, 7]],
                                  dtype=torch.int32).cuda()
            w = torch.rand(3, 3, generator=g).cuda()
            out = torch.full((3, 96), 5.0, dtype=dtype, device="cuda")
            fq.combine_into(y, row_of, w, out[:, c0:c0 + 64])
            want, mag = layer.combine(host(y), row_of.cpu().numpy(), host(w))
            got = host(out[:, c0:c0 + 64])
            assert np.all(np.abs(got - want) <= 4 * 2.0 ** -24 * mag + U[dtype] * 1.01 * np.abs(want) + 1e-30)
            assert torch.all(out[:, c0 + 64:] == 5.0)
            do = torch.randn(3, 64, generator=g).to(dtype).cuda()
            d_y = torch.full((20, 64), 3.0, dtype=dtype, device="cuda")
            d_w = torch.full((3, 3), 3.0, device="cuda")
            fq.combine_backward_into(y, row_of, w, do, d_y, d_w)
            wy, ww, mag = layer.combine_backward(host(y), row_of.cpu().numpy(), host(w), host(do))
            named = [3, 19, 0, 5, 7]
            assert np.all(np.abs(host(d_y)[named] - wy[named]) <= 1.01 * (U[dtype] + 2.0 ** -24) * np.abs(wy[named]) + 1e-30)
            rest = [i for i in range(20) if i not in named]
            assert torch.all(d_y[rest] == 3.0)
            assert np.all(np.abs(host(d_w) - ww) <= 65 * 2.0 ** -24 * mag)


def test_empty():
    need_gpu()
    r = fq.route(torch.empty(0, 16, device="cuda"), 2)
    assert r["offsets"].cpu().tolist() == [0] * 17 and r["experts"].shape == (0, 2)
    assert fq.route_backward(torch.empty(0, 16, device="cuda"), r["experts"],
                             torch.empty(0, 2, device="cuda")).shape == (0, 16)
    assert fq.combine(torch.empty(0, 8, device="cuda"), r["row_of"],
                      torch.empty(0, 2, device="cuda")).shape == (0, 8)


def test_graph_replays():
    """Router, order, combination and gradients captured: each replay against
    the eager calls on that replay's inputs."""
    need_gpu()
    x = logits_of(200, 64, torch.float32, 1)
    y = torch.randn(200 * 4, 128, device="cuda")
    do = torch.randn(200, 128, device="cuda")

    def step():
        r = fq.route(x, 4, score=1, bias=None, n_groups=4, top_groups=2)
        out = fq.combine(y, r["row_of"], r["weights"])
        d_y, d_w = fq.combine_backward(y, r["row_of"], r["weights"], do)
        dx = fq.route_backward(x, r["experts"], d_w, score=1)
        return [r["experts"], r["weights"], r["offsets"], r["row_src"], r["row_of"], out, d_y, d_w, dx]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for i in range(3):
        x.copy_(torch.randn(200, 64, generator=torch.Generator().manual_seed(i)))
        y.copy_(torch.randn(800, 128, generator=torch.Generator().manual_seed(i)))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip([o.clone() for o in outs], step()):
            assert torch.equal(a, b), f"replay {i}"
