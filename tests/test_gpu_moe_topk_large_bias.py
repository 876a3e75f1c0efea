"""Routing under biases as large as FP32 has them, such as masks of the type's lowest value:
the sum of a group's two best choices then leaves FP32's range, and groups still order by the
64-bit sums."""
import numpy as np
import pytest
import torch

from test_gpu_moe_topk import _check

pytestmark = pytest.mark.gpu

LOW = torch.finfo(torch.float32).min
INF = float("inf")


def _bias(kind, E, groups, g):
    per = E // groups
    b = 0.1 * torch.randn(E, generator=g)
    v = b.view(groups, per)
    if kind == "lowest behind -inf":        # nothing left in group 0; group 1 masked by LOW
        v[0], v[1], v[2] = -INF, LOW, LOW
    elif kind == "all lowest":
        b[:] = LOW
        v[2] = -INF
        v[0, 1:] = -INF                     # one finite choice: a sum of -inf
    elif kind == "large":                   # 4.5e38, 6e38, 6.4e38 and ordinary ones
        v[0, :2] = torch.tensor([2e38, 2.5e38])
        v[1, :2] = torch.tensor([3e38, 3e38])
        v[3, :2] = torch.tensor([3.2e38, 3.2e38])
    else:                                   # both signs, one infinite
        v[0, :2] = torch.tensor([3e38, -3e38])
        v[1] = -2e38
        v[2] = -3e38
        v[3, :2] = torch.tensor([INF, 1.0])
    return b


@pytest.mark.parametrize("E,groups", [(32, 4), (24, 4), (256, 8), (128, 4)])
@pytest.mark.parametrize("kind", ["lowest behind -inf", "all lowest", "large", "mixed"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_under_large_biases(E, groups, kind, score):
    g = torch.Generator().manual_seed(E + groups)
    logits = 2 * torch.randn(64, E, generator=g)
    bias = _bias(kind, E, groups, g)
    per = E // groups
    for top_groups in range(1, groups + 1):
        for k in {1, min(4, per), min(32, top_groups * per)}:
            _check(logits, k, bias=bias, score=score, groups=groups, top_groups=top_groups)
            _check(logits.to(torch.bfloat16), k, bias=bias, score=score, groups=groups,
                   top_groups=top_groups, group_top=1)
