"""INT8 entry points without a device: argument checks, the planner's answers, names."""
import pytest

import block_scaled_precision_nvfp4_b200 as nv

S = nv.Status


def test_argument_errors_need_no_device():
    lib = nv.load_library()

    def call(A=16, sA=4, W=16, sW=4, Y=16, M=4, N=4, K=64):
        return lib.gemm_int8_w8a8(A, sA, W, sW, Y, M, N, K, None)
    for kw in (dict(M=-1), dict(N=-1), dict(K=0), dict(K=8), dict(K=40), dict(K=-16),
               dict(K=131072), dict(M=2 ** 31 - 1), dict(N=2 ** 31 - 1000), dict(A=0), dict(sA=0), dict(W=0), dict(sW=0), dict(Y=0)):
        assert call(**kw) == S.INVALID_ARG, kw
    for kw in (dict(A=24), dict(W=17), dict(Y=8), dict(sA=2), dict(sW=7)):
        assert call(**kw) == S.MISALIGNED, kw


def test_grouped_argument_errors_need_no_device():
    lib = nv.load_library()

    def call(A=16, off=4, E=2, M=4, N=4, K=64):
        return lib.gemm_int8_w8a8_grouped(A, 4, 16, 4, off, E, M, 16, N, K, None)
    for kw in (dict(E=0), dict(E=257), dict(E=-1), dict(off=0), dict(M=-1), dict(N=-2), dict(K=72),
               dict(A=0), dict(E=256, N=2 ** 23), dict(M=2 ** 31 - 1024)):
        assert call(**kw) == S.INVALID_ARG, kw
    assert call(off=6) == S.MISALIGNED
    assert call(A=40) == S.MISALIGNED


def test_planner_knows_the_int8_pair():
    F, E = nv.Fmt, nv.Exec
    assert nv.nvfp4_kind_of(F.INT8) == nv.Kind.INT8_MMA
    assert nv.nvfp4_exec_of_arch(100, F.INT8, F.INT8) == E.INT8_MMA
    assert nv.nvfp4_exec_of_arch(100, F.INT8, F.INT8, fp4_kernel_disabled=True) == E.INT8_MMA
    for arch in (80, 89, 90, 103, 120):
        assert nv.nvfp4_exec_of_arch(arch, F.INT8, F.INT8) == E.NO_PATH
    for f in (F.BF16, F.FP8_E4M3, F.NVFP4):   # integer codes never meet floating-point ones
        assert nv.nvfp4_exec_of_arch(100, F.INT8, f) == E.NO_PATH
        assert nv.nvfp4_exec_of_arch(100, f, F.INT8) == E.NO_PATH
    assert nv.nvfp4_node_exec(100, [(F.INT8, F.INT8), (F.NVFP4, F.INT8)]) == [E.INT8_MMA, E.NO_PATH]


def test_names():
    F = nv.Fmt
    assert nv.nvfp4_pair_name(F.INT8, F.INT8) == "W8IA8I"
    assert nv.nvfp4_pair_name(F.NVFP4, F.INT8) == "W4A8I"
    assert nv.nvfp4_pair_name(F.FP8_E4M3, F.FP8_E4M3) == "W8A8"
    assert nv.nvfp4_exec_name(nv.Exec.INT8_MMA) == "INT8_MMA"
    assert len({nv.nvfp4_pair_name(a, b) for a in F for b in F}) == len(F) ** 2


@pytest.mark.parametrize("op", [nv.Op.INT8, nv.Op.INT8_GROUPED])
def test_no_workspace(op):
    assert nv.nvfp4_workspace_size(op, 4096, 5376, 14336, 8) == 0


def test_cpu_tensors_are_refused():
    import torch
    z = lambda *s: torch.zeros(s, dtype=torch.int8)
    with pytest.raises(ValueError):
        nv.gemm_int8_w8a8(z(2, 32), torch.zeros(2), z(4, 32), torch.zeros(4))


def test_quantiser_argument_errors_need_no_device():
    lib = nv.load_library()

    def call(X=16, rows=4, K=64, c=16, s=4):
        return lib.int8_quantize_bf16(X, rows, K, c, s, None)
    for kw in (dict(rows=-1), dict(rows=2 ** 31 - 1), dict(K=0), dict(K=8), dict(K=24), dict(X=0), dict(c=0), dict(s=0)):
        assert call(**kw) == S.INVALID_ARG, kw
    for kw in (dict(X=18), dict(c=24), dict(s=6)):
        assert call(**kw) == S.MISALIGNED, kw

    def routed(dest=4, k=2, rows=4, K=64):
        return lib.int8_quantize_bf16_routed(16, rows, K, dest, k, 16, 4, None)
    for kw in (dict(k=0), dict(k=33), dict(dest=0), dict(rows=2 ** 30, k=2), dict(K=40)):
        assert routed(**kw) == S.INVALID_ARG, kw
    assert routed(dest=2) == S.MISALIGNED


def test_router_argument_errors_need_no_device():
    lib = nv.load_library()

    def call(x=16, bf16=0, T=4, E=16, k=2, score=0, bias=4, groups=4, top=2, gt=2, ids=4, w=4):
        return lib.nvfp4_moe_topk(x, bf16, T, E, k, score, bias, groups, top, gt, 1, 1.0, ids, w, None)
    for kw in (dict(T=-1), dict(T=2 ** 31 - 1), dict(E=0), dict(E=257), dict(k=0), dict(k=9), dict(k=33, E=256, groups=1, top=1),
               dict(score=2), dict(score=-1), dict(groups=3), dict(groups=0), dict(groups=64, E=128),
               dict(top=0), dict(top=5), dict(gt=0), dict(gt=3), dict(x=0), dict(ids=0), dict(w=0)):
        assert call(**kw) == S.INVALID_ARG, kw
    for kw in (dict(x=8), dict(bias=5), dict(ids=2), dict(w=1)):
        assert call(**kw) == S.MISALIGNED, kw


@pytest.mark.parametrize("op", [nv.Op.INT8_QUANTIZE, nv.Op.MOE_TOPK])
def test_router_and_quantiser_need_no_workspace(op):
    assert nv.nvfp4_workspace_size(op, 4096, 256, 14336, 8) == 0
