"""GPU: low-rank adapters at the edges: empty batches, infinite and NaN weights of the
second product, inner sums past the largest BF16, what is copied.  Tolerances as
test_gpu_lora.py derives them."""
import numpy as np
import pytest
import torch

import fp4_w4a4_quantized_amd as fq
from gpu_helpers import need_gpu, say
from oracle import layer
from test_gpu_lora import B, call, case, check, dev, ints

pytestmark = pytest.mark.gpu


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
