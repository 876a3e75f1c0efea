"""Softmax weights that are not renormalised: a 64-bit exponential of the chosen logit over the
64-bit sum of all experts' FP32 exponentials, rounded once to FP32.

Tolerance, in units of 2^-24: an FP32 exponential exp(-d), d = max - x, is off by one step
(2 units) and by its argument's rounding (d units).  In the sum these weigh in by their terms:
2 + <d>, with <d> <= ln E by the entropy of the scores.  The weight's rounding adds 1:
3 + ln E in all, whatever the logits."""
import math

import numpy as np
import pytest
import torch

from test_gpu_moe_topk import _oracle
import block_scaled_precision_nvfp4_b200 as nv

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -24


def _off(logits, k, **kw):
    ids, w = nv.moe_topk(logits.cuda(), k, renormalize=False, **kw)
    bias = kw.pop("bias", None)
    ri, rw = _oracle(logits.float().numpy(), k, renormalize=False,
                     bias=None if bias is None else bias.cpu().numpy(), **kw)
    assert np.array_equal(ids.cpu().numpy(), ri)
    big = rw > 2.0 ** -100
    return (np.abs(w.cpu().numpy().astype(np.float64) - rw)[big] / rw[big]).max() / UNIT


@pytest.mark.parametrize("E,k", [(8, 8), (60, 32), (64, 6), (100, 32), (128, 8), (255, 8), (256, 32)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [0.1, 2.0, 20.0])
def test_within_the_sums_bound(E, k, dtype, size):
    g = torch.Generator().manual_seed(E + k)
    logits = (size * torch.randn(500, E, generator=g)).to(dtype)
    assert _off(logits, k) <= 3 + math.log(E)
    assert _off(logits, k, bias=torch.zeros(E, device="cuda")) <= 3 + math.log(E)   # every choice near a tie or not


@pytest.mark.parametrize("E", [64, 128, 200, 256])
def test_many_small_terms_beside_a_large_one(E):
    """One score near 1 and E - 1 of 2^-25: the large term is exact and the small ones' errors
    weigh less than 2^-13, so that all but 2^-13 units is the rounding of the weight.  A sum
    held in 32 bits would lose small terms one by one."""
    x = torch.full((E, E), -25 * math.log(2.0))
    x.fill_diagonal_(0.0)
    assert _off(x, 1) <= 1 + 2.0 ** -13
