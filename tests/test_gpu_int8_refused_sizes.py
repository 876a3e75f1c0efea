"""Counts that no call takes are refused as such, before anything of their size is allocated and
without being cut to a C int on the way."""
import pytest
import torch

import block_scaled_precision_nvfp4_b200 as nv

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["module", "python"])
def way(request, monkeypatch):
    h = nv._host()
    if request.param == "python":
        for name in ("fast_gemm", "fast_grouped", "fast_quantize", "fast_topk"):
            monkeypatch.setattr(h, name, nv._no_fast_call)
    return request.param


def _refused(call):
    with pytest.raises(nv.NvFp4Error) as e:
        call()
    assert e.value.status == nv.Status.INVALID_ARG


@pytest.mark.parametrize("T,E", [(1, 8), (8192, 256)])
@pytest.mark.parametrize("k", [257, 2 ** 31 - 1, 2 ** 31, 2 ** 32 + 2, 2 ** 63, -2 ** 32 + 2, -1])
def test_router_k(way, T, E, k):
    x = torch.zeros(T, E, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    _refused(lambda: nv.moe_topk(x, k))
    assert torch.cuda.max_memory_allocated() - before <= 8 * T * E + 2048


@pytest.mark.parametrize("kw", [dict(groups=2 ** 32 + 1), dict(groups=2, top_groups=2 ** 32 + 1),
                                dict(groups=2, top_groups=-2 ** 32 + 1), dict(groups=2, group_top=2 ** 32 + 2)])
def test_router_groups(way, kw):
    x = torch.zeros(4, 8, device="cuda")
    _refused(lambda: nv.moe_topk(x, 2, **kw))


def test_more_rows_than_a_c_int(way):
    T = 2 ** 32 + 2
    x = torch.empty(T, 1, dtype=torch.bfloat16, device="cuda")
    ids = torch.empty(T, 1, dtype=torch.int32, device="cuda")
    w = torch.empty(T, 1, dtype=torch.float32, device="cuda")
    _refused(lambda: nv.moe_topk(x, 1, out=(ids, w)))
    del x, ids
    K = 16
    A = torch.empty(T, K, dtype=torch.int8, device="cuda")
    y = torch.empty(T, 1, dtype=torch.bfloat16, device="cuda")
    one = torch.ones(1, device="cuda")
    _refused(lambda: nv.gemm_int8_w8a8(A, w.view(-1), A[:1], one, out=y))
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    _refused(lambda: nv.gemm_int8_w8a8_grouped(A, w.view(-1), A[:1].view(1, 1, K), one.view(1, 1), off, out=y))
