"""The two ways the INT8 path's calls take to the library -- the CPython module for the plain
case, Python for the rest -- give the same results and raise the same errors."""
import numpy as np
import pytest
import torch

import block_scaled_precision_nvfp4_b200 as nv

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["module", "python"])
def way(request, monkeypatch):
    h = nv._host()
    if request.param == "module":
        assert h.fast_gemm is not nv._no_fast_call, "the module is not built"
    else:
        for name in ("fast_gemm", "fast_grouped", "fast_quantize", "fast_topk"):
            monkeypatch.setattr(h, name, nv._no_fast_call)
    return request.param


def _inputs():
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(40, 256, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(2, 96, 256, generator=g, device="cuda").to(torch.bfloat16)
    logits = torch.randn(40, 16, generator=g, device="cuda")
    bias = 0.1 * torch.randn(16, generator=g, device="cuda")
    return x, w, logits, bias


def test_results(way):
    x, w, logits, bias = _inputs()
    a, sa = nv.int8_quantize_bf16(x)
    b, sb = nv.int8_quantize_bf16(w.view(-1, 256))
    dest = torch.randperm(80, generator=torch.Generator().manual_seed(0)).to(torch.int32).cuda()
    ra, rs = nv.int8_quantize_bf16_routed(x, dest, 2)
    off = torch.tensor([0, 33, 80], dtype=torch.int32, device="cuda")
    W, sW = b.view(2, 96, 256), sb.view(2, 96)
    y = nv.gemm_int8_w8a8(a, sa, W[0], sW[0])
    yg = nv.gemm_int8_w8a8_grouped(ra, rs, W, sW, off)
    ids, wt = nv.moe_topk(logits, 3, score="sigmoid", bias=bias, groups=4, top_groups=2, scale=2.5)
    for t, shape, dtype in ((a, (40, 256), torch.int8), (sa, (40,), torch.float32), (y, (40, 96), torch.bfloat16),
                            (ra, (80, 256), torch.int8), (yg, (80, 96), torch.bfloat16),
                            (ids, (40, 3), torch.int32), (wt, (40, 3), torch.float32)):
        assert tuple(t.shape) == shape and t.dtype == dtype and t.is_contiguous() and t.is_cuda
    # against the same calls into given outputs, which always go through Python
    for got, into in (
            ((a, sa), nv.int8_quantize_bf16(x, out=(torch.empty_like(a), torch.empty_like(sa)))),
            ((ra, rs), nv.int8_quantize_bf16_routed(x, dest, 2, out=(torch.empty_like(ra), torch.empty_like(rs)))),
            ((y,), (nv.gemm_int8_w8a8(a, sa, W[0], sW[0], out=torch.empty_like(y)),)),
            ((yg,), (nv.gemm_int8_w8a8_grouped(ra, rs, W, sW, off, out=torch.empty_like(yg)),)),
            ((ids, wt), nv.moe_topk(logits, 3, score="sigmoid", bias=bias, groups=4, top_groups=2,
                                    scale=2.5, out=(torch.empty_like(ids), torch.empty_like(wt))))):
        for p, q in zip(got, into):
            assert torch.equal(p, q)


def test_runs_on_the_current_stream(way):
    x, *_ = _inputs()
    ref = nv.int8_quantize_bf16(x)
    torch.cuda.synchronize()
    late = torch.zeros_like(x)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)     # the copy below comes some 10 ms from now
        late.copy_(x)
        got = nv.int8_quantize_bf16(late)
    side.synchronize()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_errors(way):
    x, w, logits, bias = _inputs()
    a, sa = nv.int8_quantize_bf16(x)
    b, sb = nv.int8_quantize_bf16(w.view(-1, 256))
    W, sW = b.view(2, 96, 256), sb.view(2, 96)
    off = torch.tensor([0, 33, 40], dtype=torch.int32, device="cuda")
    dest = torch.arange(80, dtype=torch.int32, device="cuda")
    z8 = torch.zeros(40, 24, dtype=torch.int8, device="cuda")
    for err, call in (
            (TypeError, lambda: nv.gemm_int8_w8a8(None, sa, b, sb)),
            (TypeError, lambda: nv.gemm_int8_w8a8(a, sa, x, sb)),
            (TypeError, lambda: nv.gemm_int8_w8a8(a, None, b, sb)),
            (TypeError, lambda: nv.gemm_int8_w8a8(a, sa.double(), b, sb)),
            (ValueError, lambda: nv.gemm_int8_w8a8(a, sa[1:], b, sb)),
            (ValueError, lambda: nv.gemm_int8_w8a8(a.cpu(), sa, b, sb)),
            (ValueError, lambda: nv.gemm_int8_w8a8(a, sa.cpu(), b, sb)),
            (ValueError, lambda: nv.gemm_int8_w8a8(a.t().contiguous().t(), sa, b, sb)),
            (nv.NvFp4Error, lambda: nv.gemm_int8_w8a8(z8, sa, z8, sa)),
            (TypeError, lambda: nv.gemm_int8_w8a8_grouped(a, sa, W, sW, off.long())),
            (ValueError, lambda: nv.gemm_int8_w8a8_grouped(a, sa, W, sW, off[:2])),
            (TypeError, lambda: nv.gemm_int8_w8a8_grouped(a, sa, b, sb, off)),
            (TypeError, lambda: nv.int8_quantize_bf16(x.float())),
            (ValueError, lambda: nv.int8_quantize_bf16(x[:, ::2])),
            (nv.NvFp4Error, lambda: nv.int8_quantize_bf16(x[:, :24].contiguous())),
            (ValueError, lambda: nv.int8_quantize_bf16_routed(x, dest, 3)),
            (ValueError, lambda: nv.int8_quantize_bf16_routed(x, dest, 0)),
            (nv.NvFp4Error, lambda: nv.int8_quantize_bf16_routed(x[:2].contiguous(), dest[:66], 33)),
            (ValueError, lambda: nv.moe_topk(logits, 2, score="tanh")),
            (ValueError, lambda: nv.moe_topk(logits, 2, bias=bias[1:])),
            (TypeError, lambda: nv.moe_topk(logits.half(), 2)),
            (nv.NvFp4Error, lambda: nv.moe_topk(logits, 17)),
            (nv.NvFp4Error, lambda: nv.moe_topk(logits, 0)),
            (nv.NvFp4Error, lambda: nv.moe_topk(logits, 2, groups=3))):
        with pytest.raises(err):
            call()
    with pytest.raises(nv.NvFp4Error) as e:
        nv.moe_topk(logits, 2, groups=3)
    assert e.value.status == nv.Status.INVALID_ARG and "groups" in str(e.value)
    # an int for the scale and numpy integers are fine on either way
    p, q = nv.moe_topk(logits, np.int64(2), scale=2), nv.moe_topk(logits, 2, scale=2.0)
    assert torch.equal(p[0], q[0]) and torch.equal(p[1], q[1])
