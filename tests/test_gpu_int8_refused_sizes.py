"""Counts that no call takes are refused as such, before anything of their size is allocated and
without being cut to a C int on the way."""
import gc

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


def _rows_beyond_a_c_int(monkeypatch):
    T = 2 ** 32 + 2
    x = torch.empty(T, 1, dtype=torch.bfloat16, device="cuda")
    ids = torch.empty(T, 1, dtype=torch.int32, device="cuda")
    w = torch.empty(T, 1, dtype=torch.float32, device="cuda")
    _refused(lambda: nv.moe_topk(x, 1, out=(ids, w)))
    # the products' row count, as it reaches the library (K = 1 keeps the codes small; no call)
    seen = []
    monkeypatch.setattr(nv._host(), "gemm", lambda *a: seen.append(a[5]) or 0)
    monkeypatch.setattr(nv._host(), "grouped", lambda *a: seen.append(a[6]) or 0)
    A, y, one = ids.view(torch.int8)[:, :1].contiguous(), x, torch.ones(1, device="cuda")
    nv.gemm_int8_w8a8(A, w.view(-1), A[:1], one, out=y)
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    nv.gemm_int8_w8a8_grouped(A, w.view(-1), A[:1].view(1, 1, 1), one.view(1, 1), off, out=y)
    assert seen == [2 ** 31 - 1] * 2          # more rows than any call takes


def test_more_rows_than_a_c_int(monkeypatch):
    try:
        _rows_beyond_a_c_int(monkeypatch)
    finally:
        gc.collect()                          # some 50 GB
        torch.cuda.empty_cache()
