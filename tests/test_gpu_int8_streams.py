"""The INT8 path's calls among others: first calls under capture, kernels that start early
behind and before the NVFP4 ones, graphs replayed at once, tensors beyond 2^31 elements."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import block_scaled_precision_nvfp4_b200 as nv
from block_scaled_precision_nvfp4_b200 import workloads as wl

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FIRST_CALL = """
import torch
import block_scaled_precision_nvfp4_b200 as nv
g = torch.Generator(device="cuda").manual_seed(0)
x = torch.randn(200, 512, generator=g, device="cuda").to(torch.bfloat16)
w = torch.randn(300, 512, generator=g, device="cuda").to(torch.bfloat16)
logits = torch.randn(200, 16, generator=g, device="cuda")
def calls():
    a, sa = nv.int8_quantize_bf16(x)
    b, sb = nv.int8_quantize_bf16(w)
    return nv.moe_topk(logits, 2) + (a, sa, nv.gemm_int8_w8a8(a, sa, b, sb))
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = calls()
graph.replay()
torch.cuda.synchronize()
for p, q in zip(out, calls()):
    assert torch.equal(p, q)
nv.nvfp4_check_device_error()
print("captured first")
"""


def test_the_first_call_of_a_process_can_be_captured():
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


def _int8(rng, M, N, K):
    A = torch.from_numpy(rng.integers(-127, 128, (M, K), dtype=np.int8)).cuda()
    W = torch.from_numpy(rng.integers(-127, 128, (N, K), dtype=np.int8)).cuda()
    return (A, torch.rand(M, device="cuda"), W, torch.rand(N, device="cuda"))


def test_between_nvfp4_kernels_on_one_stream():
    """INT8 and NVFP4 kernels launched behind one another, each reading what the one before
    wrote: a kernel that starts its set-up early must not start its work early."""
    rng = np.random.default_rng(2)
    M, N, K = 256, 512, 512
    W4 = wl.quantize_nvfp4(rng.standard_normal((K, N), dtype=np.float32) * np.float32(0.05))
    W8 = torch.from_numpy(rng.standard_normal((N, K)).astype(np.float32) * 0.05).to(torch.bfloat16).cuda()
    w8, s8 = nv.int8_quantize_bf16(W8)
    w4, s4 = torch.from_numpy(W4.codes).cuda(), torch.from_numpy(W4.scales).cuda()
    s4p = nv.nvfp4_pack_scales(s4, N)

    def chain(x):
        for _ in range(4):
            a, sa = nv.int8_quantize_bf16(x)                 # [M, K]
            y = nv.gemm_int8_w8a8(a, sa, w8, s8)             # [M, N]
            codes, _, sp, g = nv.nvfp4_quantize_bf16(y, plain=False)
            x = nv.gemm_nvfp4_w4a4_packed(codes, sp, 1e-3, w4, s4p, W4.g)   # [M, K]
        return x

    def stepwise(x):
        for _ in range(4):
            a, sa = nv.int8_quantize_bf16(x)
            torch.cuda.synchronize()
            y = nv.gemm_int8_w8a8(a, sa, w8, s8)
            torch.cuda.synchronize()
            codes, _, sp, g = nv.nvfp4_quantize_bf16(y, plain=False)
            torch.cuda.synchronize()
            x = nv.gemm_nvfp4_w4a4_packed(codes, sp, 1e-3, w4, s4p, W4.g)
            torch.cuda.synchronize()
        return x

    for seed in range(5):
        x = torch.from_numpy(np.random.default_rng(seed).standard_normal((M, K)).astype(np.float32)) \
            .to(torch.bfloat16).cuda()
        ref = stepwise(x)
        assert torch.isfinite(ref.float()).all() and ref.float().abs().max() > 0
        for _ in range(10):
            assert torch.equal(chain(x).view(torch.int16), ref.view(torch.int16))
    nv.nvfp4_check_device_error()


def test_two_graphs_replayed_at_once():
    """Two captured products (one of them split over K) in flight together."""
    rng = np.random.default_rng(6)
    sides, graphs, outs, refs = [], [], [], []
    for M, N, K in [(3, 2816, 8192), (300, 1280, 2048)]:
        args = _int8(rng, M, N, K)
        refs.append(nv.gemm_int8_w8a8(*args))
        torch.cuda.synchronize()
        out = torch.empty_like(refs[-1])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(5):
                nv.gemm_int8_w8a8(*args, out=out)
        sides.append(torch.cuda.Stream())
        graphs.append((g, args))
        outs.append(out)
    for _ in range(20):
        for s, (g, _) in zip(sides, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    nv.nvfp4_check_device_error()
    for out, ref in zip(outs, refs):
        assert torch.equal(out.view(torch.int16), ref.view(torch.int16))


def test_more_than_2_31_elements_quantised():
    rows, K = 150016, 14336
    x = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda")
    x.copy_(torch.randn(1, K, device="cuda").expand(rows, K))
    x *= (torch.arange(rows, device="cuda") % 97 + 1).to(torch.bfloat16)[:, None]
    codes, scales = nv.int8_quantize_bf16(x)
    torch.cuda.synchronize()
    for r in (0, 1, 149795, rows - 97, rows - 1):
        c, s = nv.int8_quantize_bf16(x[r:r + 1].clone())
        assert torch.equal(codes[r:r + 1], c) and torch.equal(scales[r:r + 1], s)


def test_more_than_2_31_elements_of_output_and_2_32_of_weights():
    rng = np.random.default_rng(8)
    M, N, K = 270000, 8192, 16                    # Y: 2.2e9 elements
    A, sA, W, sW = _int8(rng, 1000, N, K)
    A, sA = A.repeat(270, 1), sA.repeat(270)
    Y = nv.gemm_int8_w8a8(A, sA, W, sW)
    for r in (0, 131000, M - 1000):
        part = nv.gemm_int8_w8a8(A[r:r + 1000], sA[r:r + 1000], W, sW)
        assert torch.equal(Y[r:r + 1000].view(torch.int16), part.view(torch.int16))
    del Y, A, W
    E, N, K = 80, 4096, 16384                     # W: 5.4e9 elements
    W = torch.randint(-127, 128, (E, N, K), dtype=torch.int8, device="cuda")
    sW = torch.rand(E, N, device="cuda")
    A = torch.randint(-127, 128, (E, K), dtype=torch.int8, device="cuda")
    sA = torch.rand(E, device="cuda")
    off = torch.arange(E + 1, dtype=torch.int32, device="cuda")
    Y = nv.gemm_int8_w8a8_grouped(A, sA, W, sW, off)
    for e in (0, 31, 63, 64, 79):
        one = nv.gemm_int8_w8a8(A[e:e + 1], sA[e:e + 1].clone(), W[e], sW[e])
        assert torch.equal(Y[e:e + 1].view(torch.int16), one.view(torch.int16))
    torch.cuda.synchronize()
    nv.nvfp4_check_device_error()
