"""INT8 products by the plan they run on: every width of a tile, with whole tiles and with tiles
split over 2 to 4 pairs, one and two chunks a stage, many steps of K, ragged last tiles, rows on
and off 16 bytes -- against exact integer sums scaled in FP64.

The plans are those of a B200, which runs 74, 33, 22 and 15 clusters of 1 to 4 pairs at once;
the first test holds the lists to them without a device, so that a change of the plan's costs
cannot drop one unseen.

Tolerance: two FP32 products and the sum's conversion (2^-24 each), one rounding to BF16
(2^-8)."""
import ctypes

import numpy as np
import pytest
import torch

import block_scaled_precision_nvfp4_b200 as nv
from block_scaled_precision_nvfp4_b200 import _build

REL = 2.0 ** -8 + 4 * 2.0 ** -24
CLUSTERS = (0, 74, 33, 22, 15)

DENSE = [  # M, N, K, token columns, pairs per tile
    (2, 129, 464, 32, 2), (29, 1001, 3200, 32, 4), (36, 3698, 3024, 64, 2), (64, 5376, 14336, 64, 3),
    (33, 576, 1984, 64, 4), (2173, 87, 9680, 96, 2), (66, 3043, 5136, 96, 3), (1424, 87, 7472, 96, 4),
    (2215, 82, 9504, 128, 3),
    (513, 1025, 400, 64, 1), (2580, 277, 80, 96, 1), (333, 5376, 14336, 128, 1), (512, 9000, 272, 128, 1),
    (130, 9620, 1040, 160, 1), (300, 14336, 4096, 160, 1), (700, 9001, 784, 192, 1),
    (1900, 4096, 2048, 224, 1), (1895, 4093, 2064, 224, 1), (2001, 4102, 2000, 256, 1),
    (4096, 5376, 14336, 256, 1)]


def _counts(rng, E, M):
    """Ragged counts, some experts without a row."""
    p = rng.random(E) ** 2
    p[rng.integers(E)] = 0.0
    return rng.multinomial(M, p / p.sum())


GROUPED = [  # E, M, N, K, token columns, pairs per tile
    (16, 8, 469, 656, 32, 2), (3, 32, 1226, 2784, 64, 2), (8, 32, 344, 3904, 64, 3), (3, 32, 69, 1904, 64, 4),
    (64, 3840, 2048, 512, 64, 1), (64, 4064, 80, 144, 96, 1), (20, 4000, 4096, 512, 128, 1),
    (3, 9404, 76, 272, 160, 1), (64, 8313, 290, 144, 192, 1), (8, 5000, 4097, 1040, 224, 1),
    (3, 4000, 3000, 4096, 224, 1), (8, 8091, 770, 400, 256, 1)]


def _plan(M, N, K, E=1):
    lib = ctypes.CDLL(_build.build_wait_test())
    out = (ctypes.c_int * 6)()
    assert lib.nvfp4_test_int8_plan(M, N, K, E, 0, (ctypes.c_int * 5)(*CLUSTERS), out) == 0
    return tuple(out)  # token columns, pairs per tile, chunks, stages, tiles, CTAs


def test_the_lists_reach_every_plan():
    dense = {c[:3]: _plan(*c[:3]) for c in DENSE}
    grouped = {c[:4]: _plan(*c[1:4], E=c[0]) for c in GROUPED}
    for c in DENSE:
        assert dense[c[:3]][:2] == c[3:], (c, dense[c[:3]])
    for c in GROUPED:
        assert grouped[c[:4]][:2] == c[4:], (c, grouped[c[:4]])
    widths = set(range(64, 257, 32))
    for plans, split in ((dense, {(32, 2), (32, 4), (64, 2), (64, 3), (64, 4), (96, 2), (96, 3), (96, 4), (128, 3)}),
                         (grouped, {(32, 2), (64, 2), (64, 3), (64, 4)})):
        assert {p[0] for p in plans.values() if p[1] == 1} >= widths
        assert {p[:2] for p in plans.values() if p[1] > 1} >= split
        assert {p[2] for p in plans.values()} == {1, 2}
    # of the unsplit ones: many tiles per cluster, ragged ends, K off 128 and N off 8
    whole = [(c, dense[c]) for c in dense if dense[c][1] == 1]
    assert any(c[0] % p[0] and c[1] % 8 and c[2] % 128 and p[2] == 1 for c, p in whole)
    assert any(c[0] % p[0] and c[1] % 8 and c[2] % 128 and p[2] == 2 for c, p in whole)
    assert any(p[4] > 2 * p[5] // 2 and p[2] == 1 and c[2] > 4096 for c, p in whole)


def _operands(seed, M, N, K, E=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    code = lambda *s: torch.randint(-128, 128, s, generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
    scale = lambda *s: 0.01 * torch.exp(torch.randn(*s, generator=g, device="cuda"))
    lead = () if E is None else (E,)
    return code(M, K), scale(M), code(*lead, N, K), scale(*lead, N)


def _close(y, A, sA, W, sW):
    ref = (A.double() @ W.double().t()) * sA.double()[:, None] * sW.double()[None, :]  # sums below 2^53
    off = (y.double() - ref).abs() > REL * ref.abs()
    assert not bool(off.any()), f"{int(off.sum())} of {off.numel()} off, first at {off.nonzero()[0].tolist()}"


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [c[:3] for c in DENSE])
def test_dense(M, N, K):
    A, sA, W, sW = _operands(M + N + K, M, N, K)
    y = nv.gemm_int8_w8a8(A, sA, W, sW)
    torch.cuda.synchronize()
    nv.nvfp4_check_device_error()
    _close(y, A, sA, W, sW)


@pytest.mark.gpu
@pytest.mark.parametrize("E,M,N,K", [c[:4] for c in GROUPED])
def test_grouped(E, M, N, K):
    counts = _counts(np.random.default_rng(M + N), E, M - M // 20)  # some rows behind the last
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    A, sA, W, sW = _operands(M + N + K, M, N, K, E)
    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    nv.gemm_int8_w8a8_grouped(A, sA, W, sW, torch.from_numpy(off).cuda(), out=y)
    torch.cuda.synchronize()
    nv.nvfp4_check_device_error()
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        if counts[e]:
            _close(y[r], A[r], sA[r], W[e], sW[e])
    assert bool((y[int(off[-1]):] == 7.0).all())


@pytest.mark.gpu
def test_rows_beyond_2_31_outputs():
    M, N, K = 270000, 8192, 16                      # Y: 2.2e9 elements, tiles of 256 tokens
    A, sA, W, sW = _operands(1, M, N, K)
    y = nv.gemm_int8_w8a8(A, sA, W, sW)
    for r in (slice(0, 300), slice(131000, 131300), slice(262000, 262400), slice(M - 300, M)):
        _close(y[r], A[r], sA[r], W, sW)
