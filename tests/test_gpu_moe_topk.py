"""Routing to experts on the GPU against the formulas in 64 bits.

ids must be equal.  Weights are FP32: computed in 64 bits and rounded once (2^-24, the
tests allow 2^-23), except that the softmax sum over all experts may be an FP32 sum
(each term's exponential 2 steps and its argument's rounding, 16 additions: below 2^-19)."""
import numpy as np
import pytest
import torch

from oracle import moe as om
import block_scaled_precision_nvfp4_b200 as nv

pytestmark = pytest.mark.gpu


def _oracle(x, k, score="softmax", bias=None, groups=1, top_groups=1, group_top=2,
            renormalize=True, scale=1.0):
    T, E = x.shape
    x = np.where(np.isnan(x), -np.inf, np.minimum(x.astype(np.float64), np.finfo(np.float32).max))
    with np.errstate(invalid="ignore", over="ignore"):
        if score == "softmax":
            m = x.max(axis=1, keepdims=True)
            e = np.where(x > -np.inf, np.exp(x - np.where(m > -np.inf, m, 0.0)), 0.0)
            tot = e.sum(axis=1, keepdims=True)
            s = np.divide(e, tot, out=np.zeros_like(e), where=tot > 0)
        else:
            s = 1.0 / (1.0 + np.exp(-x))
        c = s if bias is None else s + bias.astype(np.float64)
        c = np.where(np.isnan(c), -np.inf, c)
        inside = np.ones((T, E), bool)
        if groups > 1:
            per = E // groups
            top = -np.sort(-c.reshape(T, groups, per), axis=2)[:, :, :group_top]
            gs = top.sum(axis=2)
            gs = np.where(np.isnan(gs), -np.inf, gs)
            order = np.argsort(-gs, axis=1, kind="stable")[:, :top_groups]
            keep = np.zeros((T, groups), bool)
            np.put_along_axis(keep, order, True, axis=1)
            inside = np.repeat(keep, per, axis=1)
    key = c if bias is not None else x
    ids = np.empty((T, k), np.int32)
    for t in range(T):
        idx = np.flatnonzero(inside[t])
        ids[t] = idx[np.argsort(-key[t, idx], kind="stable")[:k]]
    w = np.take_along_axis(s, ids.astype(np.int64), axis=1)
    if renormalize:
        tot = w.sum(axis=1, keepdims=True)
        w = np.divide(w, tot, out=np.zeros_like(w), where=tot > 0)
    return ids, w * scale


def _check(logits, k, bias=None, **kw):
    ids, w = nv.moe_topk(logits.cuda(), k, bias=None if bias is None else bias.cuda(), **kw)
    ri, rw = _oracle(logits.float().numpy(), k, bias=None if bias is None else bias.numpy(), **kw)
    assert ids.dtype == torch.int32 and w.dtype == torch.float32
    assert np.array_equal(ids.cpu().numpy(), ri), \
        f"{(ids.cpu().numpy() != ri).any(axis=1).sum()} rows differ"
    tol = 2.0 ** -19 if kw.get("score", "softmax") == "softmax" and not kw.get("renormalize", True) \
        else 2.0 ** -23
    got = w.cpu().numpy().astype(np.float64)
    # below the smallest normal FP32 the step is absolute
    assert (np.abs(got - rw) <= tol * np.abs(rw) + 2.0 ** -149).all()


CASES = [  # T, E, k, groups, top_groups, group_top
    (1, 1, 1, 1, 1, 2), (1, 8, 2, 1, 1, 2), (7, 5, 5, 1, 1, 2), (100, 16, 4, 1, 1, 2),
    (1000, 60, 6, 1, 1, 2), (333, 64, 8, 1, 1, 2), (129, 100, 3, 1, 1, 2), (64, 128, 8, 1, 1, 2),
    (50, 255, 8, 1, 1, 2), (2000, 256, 8, 1, 1, 2), (40, 256, 32, 1, 1, 2), (33, 32, 32, 1, 1, 2),
    (100, 256, 8, 8, 4, 2), (100, 256, 8, 8, 4, 1), (90, 160, 6, 8, 3, 1), (77, 255, 5, 5, 2, 2),
    (77, 255, 12, 3, 1, 2), (64, 32, 4, 32, 9, 2), (64, 64, 2, 32, 1, 1), (30, 24, 6, 3, 3, 2),
    (30, 6, 2, 2, 1, 2), (31, 256, 16, 16, 1, 2), (31, 28, 4, 7, 2, 2)]


@pytest.mark.parametrize("T,E,k,groups,top_groups,group_top", CASES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("with_bias", [False, True])
def test_topk(T, E, k, groups, top_groups, group_top, score, dtype, with_bias):
    g = torch.Generator().manual_seed(T * 1000 + E * 10 + k)
    logits = (2 * torch.randn(T, E, generator=g)).to(dtype)
    bias = 0.2 * torch.randn(E, generator=g) if with_bias else None
    for renorm, scale in ((True, 1.0), (False, 2.5)):
        _check(logits, k, bias=bias, score=score, groups=groups, top_groups=top_groups,
               group_top=group_top, renormalize=renorm, scale=scale)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top_groups", [(1, 1), (4, 2)])
def test_ties_go_to_the_lowest_index(score, groups, top_groups):
    """Logits on a coarse grid, so that most rows have equal scores at the border; a bias
    of equal values keeps the ties, one of two values makes some."""
    g = torch.Generator().manual_seed(4)
    logits = torch.randint(-2, 3, (500, 64), generator=g).float()
    for bias in (None, torch.zeros(64), torch.randint(0, 2, (64,), generator=g).float()):
        _check(logits, 6, bias=bias, score=score, groups=groups, top_groups=top_groups)
    _check(torch.zeros(5, 64), 16, score=score, groups=groups, top_groups=top_groups)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_choices_closer_than_fp32_steps(score):
    """Biases that bring the choices of a row to within 1e-9 of each other, where sums in
    FP32 are equal: the order is that of the 64-bit values."""
    rng = np.random.default_rng(8)
    E = 48
    x = rng.normal(size=E).astype(np.float32)
    x64 = x.astype(np.float64)
    s = np.exp(x64) / np.exp(x64).sum() if score == "softmax" else 1 / (1 + np.exp(-x64))
    bias = (1.0 - s).astype(np.float32)            # s + bias = 1 + (rounding of the bias)
    logits = torch.from_numpy(np.tile(x, (20, 1)))
    c = s + bias.astype(np.float64)
    assert np.ptp(c) < 1e-7 and len(np.unique(c)) == E
    _check(logits, 8, bias=torch.from_numpy(bias), score=score)
    _check(logits, 4, bias=torch.from_numpy(bias), score=score, groups=6, top_groups=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top_groups", [(1, 1), (4, 1), (4, 3)])
@pytest.mark.parametrize("with_bias", [False, True])
def test_masked_infinite_and_nan_logits(score, groups, top_groups, with_bias):
    inf = float("inf")
    g = torch.Generator().manual_seed(5)
    x = torch.randn(12, 32, generator=g)
    x[0] = -inf                                     # nothing left
    x[1] = -inf
    x[1, 17] = 0.3                                  # one left
    x[2, ::2] = float("nan")
    x[3] = float("nan")
    x[4, 9] = inf
    x[5, 3], x[5, 20], x[5, 30] = inf, inf, 3.4e38
    x[6] = torch.finfo(torch.float32).min           # masks of the type's lowest value
    x[7] = torch.finfo(torch.float32).min
    x[7, 5], x[7, 8] = 1.0, -2.0
    x[8] = -inf
    x[8, :3] = torch.tensor([-1e30, 2e30, -3e30])
    x[9] = 100 * torch.randn(32, generator=g)       # scores that vanish
    x[10] = 200.0 + x[10]
    x[11] = -0.0
    x[11, 1::2] = 0.0
    bias = None
    if with_bias:
        bias = 0.1 * torch.randn(32, generator=g)
        bias[4], bias[12], bias[21] = -inf, -inf, float("nan")
    _check(x, 6, bias=bias, score=score, groups=groups, top_groups=top_groups)
    _check(x, 6, bias=bias, score=score, groups=groups, top_groups=top_groups, renormalize=False)


def test_long_and_one_token():
    g = torch.Generator().manual_seed(6)
    for T in (1, 20011):
        logits = torch.randn(T, 256, generator=g)
        bias = 0.05 * torch.randn(256, generator=g)
        _check(logits, 8, bias=bias, score="sigmoid", groups=8, top_groups=4, scale=2.5)


def test_empty_captured_and_side_stream():
    ids, w = nv.moe_topk(torch.empty(0, 8, device="cuda"), 2)
    assert tuple(ids.shape) == (0, 2) and tuple(w.shape) == (0, 2)
    x = torch.randn(64, 60, device="cuda")
    out = nv.moe_topk(x, 4)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nv.moe_topk(x, 4, out=out)
    x.copy_(torch.randn(64, 60, device="cuda"))
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(out[0].cpu().numpy(), _oracle(x.cpu().numpy(), 4)[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ids, _ = nv.moe_topk(x, 4, stream=side)
    side.synchronize()
    assert torch.equal(ids, out[0])


def test_refusals():
    x = torch.zeros(4, 12, device="cuda")
    for kw in (dict(k=0), dict(k=13), dict(k=33), dict(k=2, groups=5), dict(k=2, groups=0),
               dict(k=2, groups=3, top_groups=4), dict(k=2, groups=3, top_groups=0),
               dict(k=5, groups=3, top_groups=1), dict(k=2, groups=3, group_top=3)):
        with pytest.raises(nv.NvFp4Error) as e:
            nv.moe_topk(x, **kw)
        assert e.value.status == nv.Status.INVALID_ARG, kw
    with pytest.raises(nv.NvFp4Error):
        nv.moe_topk(torch.zeros(4, 257, device="cuda"), 2)
    with pytest.raises(ValueError):
        nv.moe_topk(x, 2, score="tanh")
    with pytest.raises(TypeError):
        nv.moe_topk(x.half(), 2)
    with pytest.raises(TypeError):
        nv.moe_topk(x[0], 2)
    with pytest.raises(ValueError):
        nv.moe_topk(x.t(), 2)
    with pytest.raises(ValueError):
        nv.moe_topk(x, 2, bias=torch.zeros(11, device="cuda"))
    with pytest.raises(ValueError):
        nv.moe_topk(x.cpu(), 2)
    with pytest.raises(nv.NvFp4Error) as e:
        nv.moe_topk(torch.zeros(49, device="cuda")[1:].view(4, 12), 2)
    assert e.value.status == nv.Status.MISALIGNED


@pytest.mark.parametrize("T,k,E,N,K,kw", [
    (1, 2, 8, 264, 1040, {}),
    (77, 2, 8, 512, 512, {}),
    (300, 8, 64, 256, 400, dict(score="sigmoid", groups=8, top_groups=3, scale=2.5)),
    (1200, 1, 4, 520, 768, dict(renormalize=False))])
def test_int8_expert_layer(T, k, E, N, K, kw):
    """A whole layer from the router's logits: top-k, route, quantise into the experts'
    order, the experts' INT8 products, the weighted combine -- against the oracle's route
    and combine of exact integer products of the same codes."""
    rng = np.random.default_rng(T + N)
    x = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).to(torch.bfloat16).cuda()
    w = torch.from_numpy(0.02 * rng.standard_normal((E * N, K)).astype(np.float32)).to(torch.bfloat16)
    W, sW = nv.int8_quantize_bf16(w.cuda())
    W, sW = W.view(E, N, K), sW.view(E, N)
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
    bias = torch.from_numpy(0.1 * rng.standard_normal(E).astype(np.float32)).cuda()

    def layer():
        ids, weights = nv.moe_topk(logits, k, bias=bias, **kw)
        off, dest, src = nv.moe_route(ids, E)
        codes, scales = nv.int8_quantize_bf16_routed(x, dest, k)
        Yg = nv.gemm_int8_w8a8_grouped(codes, scales, W, sW, off)
        return ids, weights, codes, scales, off, Yg, nv.moe_combine(Yg, dest, weights, T, k)

    ids, weights, codes, scales, off, Yg, Y = layer()
    torch.cuda.synchronize()
    nv.nvfp4_check_device_error()
    ri, rw = _oracle(logits.cpu().numpy(), k, bias=bias.cpu().numpy(), **kw)
    assert np.array_equal(ids.cpu().numpy(), ri)
    ro, rd, rs = om.route(ri, E)
    assert np.array_equal(off.cpu().numpy(), ro)
    plain, ps = nv.int8_quantize_bf16(x)
    c64, s64 = plain.double().cpu().numpy()[rs // k], ps.double().cpu().numpy()[rs // k]
    ref = np.empty((T * k, N))
    for e in range(E):
        r = slice(ro[e], ro[e + 1])
        ref[r] = (c64[r] @ W[e].double().cpu().numpy().T) * s64[r, None] * sW[e].double().cpu().numpy()
    got = Yg.double().cpu().numpy()
    assert (np.abs(got - ref) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(ref)).all()
    # the combine of those rows: k FP32 products and sums, one rounding to BF16
    y64 = om.combine(got, rd, weights.cpu().numpy(), T, k)
    size = om.combine(np.abs(got), rd, np.abs(weights.cpu().numpy()), T, k)
    assert (np.abs(Y.double().cpu().numpy() - y64) <= 2.0 ** -8 * np.abs(y64) + 2 * k * 2.0 ** -24 * size
            * (1 + 2.0 ** -8)).all()

    # the same layer captured once and replayed on other tokens
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = layer()
    logits.copy_(torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)))
    x.copy_(torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)))
    g.replay()
    torch.cuda.synchronize()
    nv.nvfp4_check_device_error()
    again = layer()
    torch.cuda.synchronize()
    for a, b in zip(captured, again):
        assert torch.equal(a, b)


def test_nvfp4_expert_layer_from_the_routers_logits():
    """The same routing ahead of the NVFP4 experts: planned, packed and multiplied from device
    offsets, combined with the router's weights -- bit for bit the layer that gets the
    formula's ids and weights from the host."""
    from block_scaled_precision_nvfp4_b200 import workloads as wl
    rng = np.random.default_rng(31)
    T, k, E, N, K = 333, 2, 8, 512, 512
    x = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).to(torch.bfloat16).cuda()
    experts = [wl.quantize_nvfp4(rng.standard_normal((N, K), dtype=np.float32) * np.float32(0.02))
               for _ in range(E)]
    W = torch.from_numpy(np.stack([e.codes for e in experts])).cuda()
    sW = torch.from_numpy(np.stack([e.scales for e in experts])).cuda()
    sw_p = nv.nvfp4_pack_scales_grouped(sW.view(E * N, K // 16), [i * N for i in range(E + 1)], K)
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
    bias = torch.from_numpy(0.1 * rng.standard_normal(E).astype(np.float32)).cuda()

    def layer(ids, weights):
        off, dest, src = nv.moe_route(ids, E)
        codes, scales, g = nv.nvfp4_quantize_bf16_routed(x, dest, k)
        sched = nv.GroupedSchedule(off, E, T * k, N, K, [e.g for e in experts], gA=g)
        y = sched.gemm(codes, sched.pack(scales), W, sw_p)
        return nv.moe_combine(y, dest, weights, T, k)
    ids, weights = nv.moe_topk(logits, k, score="sigmoid", bias=bias)
    Y = layer(ids, weights)
    ri, rw = _oracle(logits.cpu().numpy(), k, score="sigmoid", bias=bias.cpu().numpy())
    assert np.array_equal(ids.cpu().numpy(), ri)
    assert (np.abs(weights.cpu().numpy() - rw) <= 2.0 ** -23 * rw).all()
    ref = layer(torch.from_numpy(ri).cuda(), weights)
    torch.cuda.synchronize()
    nv.nvfp4_check_device_error()
    assert torch.equal(Y.view(torch.int16), ref.view(torch.int16)) and Y.float().abs().max() > 0
