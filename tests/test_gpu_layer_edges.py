"""GPU: values and bounds at the edges of what the calls between the FP4 linear
layers define, against the plain 64-bit forms of oracle/layer.py with the
tolerances of test_gpu_kv_attention.py and test_gpu_route_combine.py."""
import numpy as np
import pytest
import torch

import fp4_w4a4_quantized_amd as fq
from gpu_helpers import need_gpu, say
from test_gpu_route_combine import check_route

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
