"""A wait of the INT8 kernel's epilogue that expires in one warp only, on the GPU, without a
fault: in the test-only build of the same sources one of the four warps that share a half of
each tile gives up on its first tile, while the others saw the accumulator in time.  Its
cluster's tiles differ in rows (up to 32: the second half has nothing to store; and more), so
the warps must agree on every tile.  The call must end, report DEVICE_TIMEOUT once, and
leave the next call right."""
import ctypes

import numpy as np
import pytest
import torch

import block_scaled_precision_nvfp4_b200 as nv
from block_scaled_precision_nvfp4_b200 import _build

pytestmark = pytest.mark.gpu


def _lib():
    lib = ctypes.CDLL(_build.build_wait_test())
    P, I = ctypes.c_void_p, ctypes.c_int
    lib.gemm_int8_w8a8_grouped.argtypes = [P, P, P, P, P, I, I, P, I, I, P]
    lib.nvfp4_check_device_error.argtypes = [P]
    lib.nvfp4_test_set_wait.argtypes = [ctypes.c_uint64, I]
    return lib


@pytest.mark.parametrize("counts,N,K", [
    ([20, 100] * 32, 2048, 512),            # tiles of 20 rows and of 64 or more, in turn
    ([5, 70, 32, 33, 1, 200] * 11, 2056, 272)])
def test_one_warp_gives_up(counts, N, K):
    lib = _lib()
    E, M = len(counts), sum(counts)
    plan, clusters = (ctypes.c_int * 6)(), (ctypes.c_int * 5)()
    assert lib.nvfp4_test_int8_plan(M, N, K, E, 1, clusters, plan) == nv.Status.OK
    bt, split, tiles, ctas = plan[0], plan[1], plan[4], plan[5]
    assert bt >= 64 and split == 1 and tiles > 4 * ctas // 2, list(plan)
    rng = np.random.default_rng(M)
    A = torch.from_numpy(rng.integers(-127, 128, (M, K), dtype=np.int8)).cuda()
    W = torch.from_numpy(rng.integers(-127, 128, (E, N, K), dtype=np.int8)).cuda()
    sA, sW = torch.rand(M, device="cuda"), torch.rand(E, N, device="cuda")
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
    stream = torch.cuda.current_stream().cuda_stream

    def call(y):
        return lib.gemm_int8_w8a8_grouped(A.data_ptr(), sA.data_ptr(), W.data_ptr(), sW.data_ptr(),
                                          off.data_ptr(), E, M, y.data_ptr(), N, K, stream)
    y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    assert lib.nvfp4_check_device_error(stream) == nv.Status.OK
    try:
        assert lib.nvfp4_test_set_wait(2_000_000, 2) == nv.Status.OK
        assert call(y) == nv.Status.OK
        assert lib.nvfp4_check_device_error(stream) == nv.Status.DEVICE_TIMEOUT
        assert lib.nvfp4_check_device_error(stream) == nv.Status.OK
    finally:
        assert lib.nvfp4_test_set_wait(2_000_000_000, 0) == nv.Status.OK
    assert call(y) == nv.Status.OK
    assert lib.nvfp4_check_device_error(stream) == nv.Status.OK
    ref = nv.gemm_int8_w8a8_grouped(A, sA, W, sW, off)
    torch.cuda.synchronize()
    nv.nvfp4_check_device_error()
    assert torch.equal(y.view(torch.int16), ref.view(torch.int16))
