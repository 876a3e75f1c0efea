"""Split tiles of the INT8 kernel whose owners give up waiting for the other pairs' partial
sums, on the GPU, without a fault: in the test-only build of the same sources the owners'
waits count as expired.  The sums arrive all the same, and pairs that own no column leave
right behind their sends, so an owner must not leave before them.  The call must report
DEVICE_TIMEOUT once and write nothing, and the next call must be right."""
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
    lib.gemm_int8_w8a8.argtypes = [P, P, P, P, P, I, I, I, P]
    lib.nvfp4_check_device_error.argtypes = [P]
    lib.nvfp4_test_set_wait.argtypes = [ctypes.c_uint64, I]
    return lib


@pytest.mark.parametrize("M,N,K", [(1, 2048, 8192), (3, 5376, 4096), (64, 5376, 14336)])
def test_owners_give_up(M, N, K):
    lib = _lib()
    plan, clusters = (ctypes.c_int * 6)(), (ctypes.c_int * 5)()
    assert lib.nvfp4_test_int8_plan(M, N, K, 1, 1, clusters, plan) == nv.Status.OK
    assert plan[1] > 1, list(plan)
    rng = np.random.default_rng(M)
    A = torch.from_numpy(rng.integers(-127, 128, (M, K), dtype=np.int8)).cuda()
    W = torch.from_numpy(rng.integers(-127, 128, (N, K), dtype=np.int8)).cuda()
    sA, sW = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream

    def call(y):
        return lib.gemm_int8_w8a8(A.data_ptr(), sA.data_ptr(), W.data_ptr(), sW.data_ptr(),
                                  y.data_ptr(), M, N, K, stream)
    assert lib.nvfp4_check_device_error(stream) == nv.Status.OK
    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    try:
        assert lib.nvfp4_test_set_wait(2_000_000, 3) == nv.Status.OK
        for _ in range(20):
            assert call(y) == nv.Status.OK
        assert lib.nvfp4_check_device_error(stream) == nv.Status.DEVICE_TIMEOUT
        assert lib.nvfp4_check_device_error(stream) == nv.Status.OK
        assert bool((y.float() == 7.0).all())
    finally:
        assert lib.nvfp4_test_set_wait(2_000_000_000, 0) == nv.Status.OK
    assert call(y) == nv.Status.OK
    assert lib.nvfp4_check_device_error(stream) == nv.Status.OK
    ref = nv.gemm_int8_w8a8(A, sA, W, sW)
    torch.cuda.synchronize()
    nv.nvfp4_check_device_error()
    assert torch.equal(y.view(torch.int16), ref.view(torch.int16))
