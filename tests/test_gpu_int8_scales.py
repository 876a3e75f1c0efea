"""INT8 products under scales of every size, against exact integer sums scaled in FP64.

Scales are powers of two times a mantissa: sA from the smallest subnormal FP32 to the largest
finite value, sW over 2^-126 .. 2^96.  Their product alone may leave FP32's range while the
result does not.  Scales sW outside are held to the documented FP32 products, bit for bit.

Tolerance: three FP32 roundings (the sum's conversion and two products, 2^-24 each) and one
to BF16 (2^-8); below BF16's normal range half a subnormal step instead, 2^-134, and the
FP32 ones 2^-150 each.  From 2^128 (1 - 2^-9) on, BF16 rounds to infinity; within the FP32
roundings of that border either is right."""
import numpy as np
import pytest
import torch

import block_scaled_precision_nvfp4_b200 as nv

pytestmark = pytest.mark.gpu

REL = 2.0 ** -8 + 4 * 2.0 ** -24
ABS = 2.0 ** -134 + 3 * 2.0 ** -150
TOP = 2.0 ** 128 * (1 - 2.0 ** -9)
FP32 = 4 * 2.0 ** -24
EXPONENTS = [-149, -140, -127, -126, -125, -100, -64, -33, -1, 0, 31, 64, 95, 96, 97, 110, 127]
INSIDE = [e for e in EXPONENTS if -126 <= e < 96]


def _scales(rng, n, exponents=EXPONENTS):
    e = np.array(exponents)[np.arange(n) % len(exponents)]
    m = 1.0 + rng.integers(0, 2 ** 20, n) / 2.0 ** 20
    s = np.ldexp(m, e).astype(np.float32)            # subnormals round
    assert np.isfinite(s).all() and (s > 0).all()
    return s


def _d(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _check(y, A, sA, W, sW):
    y = y.float().cpu().numpy().astype(np.float64)
    acc = A.astype(np.float64) @ W.astype(np.float64).T          # exact
    ref = acc * sA.astype(np.float64)[:, None] * sW.astype(np.float64)[None, :]
    size = np.abs(ref)
    over, inside = size >= TOP * (1 + FP32), size <= TOP * (1 - FP32)
    assert np.isinf(y[over]).all() and (np.sign(y[over]) == np.sign(ref[over])).all()
    border = ~over & ~inside
    assert (np.isinf(y[border]) | (np.abs(y[border]) >= TOP * (1 - 2.0 ** -8))).all()
    bad = inside & ~(np.abs(y - ref) <= REL * size + ABS)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, first {y[bad][0]} for {ref[bad][0]} " \
                          f"(scales {sA[np.argwhere(bad)[0][0]]}, {sW[np.argwhere(bad)[0][1]]})"


def _operands(rng, M, N, K, exponents=INSIDE):
    A = rng.integers(-127, 128, (M, K), dtype=np.int8)
    W = rng.integers(-127, 128, (N, K), dtype=np.int8)
    W[::7] = 0                                       # sums of 0 under every scale
    A[1::9] = 0
    A[2::9, 1:], W[2::7, 1:] = 0, 0                  # small sums
    return A, W, _scales(rng, M), _scales(rng, N, exponents)


SHAPES = [(34, 289, 64), (300, 131, 256), (170, 1360, 512),      # whole tiles, rows on and off 16 bytes
          (34, 512, 8192), (3, 340, 4096)]                       # split over K


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_scales_of_every_size(M, N, K):
    rng = np.random.default_rng(M + N + K)
    A, W, sA, sW = _operands(rng, M, N, K)
    _check(nv.gemm_int8_w8a8(_d(A), _d(sA), _d(W), _d(sW)), A, sA, W, sW)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_the_documented_products_bit_for_bit(M, N, K):
    rng = np.random.default_rng(M + N + K + 1)
    A, W, sA, sW = _operands(rng, M, N, K, EXPONENTS)
    acc = (A.astype(np.float64) @ W.astype(np.float64).T).astype(np.float32)   # one rounding
    with np.errstate(over="ignore", invalid="ignore", under="ignore"):
        v = acc * sW[None, :] * sA[:, None]
    assert v.dtype == np.float32 and not np.isnan(v).any()
    y = nv.gemm_int8_w8a8(_d(A), _d(sA), _d(W), _d(sW)).cpu()
    assert torch.equal(y.view(torch.int16), torch.from_numpy(v).to(torch.bfloat16).view(torch.int16))


def test_experts_scales_of_every_size():
    rng = np.random.default_rng(4)
    counts, N, K = [40, 0, 3, 90], 340, 256
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    ops = [_operands(rng, c, N, K) for c in counts]
    sW = np.stack([np.roll(o[3], 5 * i) for i, o in enumerate(ops)])
    A, sA = np.concatenate([o[0] for o in ops]), np.concatenate([o[2] for o in ops])
    W = np.stack([o[1] for o in ops])
    y = nv.gemm_int8_w8a8_grouped(_d(A), _d(sA), _d(W), _d(sW), _d(off))
    for e, c in enumerate(counts):
        r = slice(off[e], off[e + 1])
        if c:
            _check(y[r], A[r], sA[r], W[e], sW[e])


@pytest.mark.parametrize("M", [5, 300])
def test_special_scales_follow_the_formula(M):
    """0, infinite and NaN scales: what (sum * sW) * sA gives."""
    rng = np.random.default_rng(M)
    A, W, sA, sW = _operands(rng, M, 150, 64)
    sA[0], sA[3], sA[4] = 0.0, np.inf, np.nan
    sA[1:3] = 1.0
    sW[:] = 1.0
    sW[0:6] = [0.0, np.inf, np.nan, 2.0 ** -140, 2.0 ** 120, -1.0]
    y = nv.gemm_int8_w8a8(_d(A), _d(sA), _d(W), _d(sW)).float().cpu().numpy()
    acc = (A.astype(np.float64) @ W.astype(np.float64).T).astype(np.float32)
    # The documented order, in FP32: sum * 2^120 is infinite for sums from 2^8 on, and NaN
    # under sA = 0.  Without that column FP64 has the same NaNs in any order.
    with np.errstate(invalid="ignore", over="ignore"):
        v = acc * sW[None, :] * sA[:, None]
        ref = acc.astype(np.float64) * (sA.astype(np.float64)[:, None] * sW.astype(np.float64)[None, :])
    want = torch.from_numpy(v).to(torch.bfloat16).float().numpy()
    assert np.array_equal(y, want, equal_nan=True)
    cols = np.arange(150) != 4
    assert np.array_equal(np.isnan(y[:, cols]), np.isnan(ref[:, cols]))
    assert (y[0, [3, 5]] == 0).all() and (y[0, 6:] == 0).all()
