"""The INT8 row quantiser on the GPU: codes and scales bit for bit against 64-bit values.

127 * x is exact in 64 bits and a quotient of two BF16 values that is no half-integer is
at least 2^-16 (relative) away from one, so numpy's rounded division decides every code."""
import numpy as np
import pytest
import torch

import block_scaled_precision_nvfp4_b200 as nv

pytestmark = pytest.mark.gpu


def _oracle(x):
    """x float64 [rows, K] -> codes int8, scales float32."""
    amax = np.max(np.abs(x), axis=1) if x.shape[1] else np.zeros(len(x))
    finite = np.isfinite(x).all(axis=1)
    codes = np.zeros(x.shape, np.int8)
    scales = np.full(len(x), np.nan, np.float32)
    for r in np.flatnonzero(finite):
        scales[r] = np.float32(amax[r] / 127.0) if amax[r] > 0 else 1.0
        if amax[r] > 0:
            codes[r] = np.rint(127.0 * x[r] / amax[r]).astype(np.int8)
    return codes, scales


def _f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def _check(x, got):
    codes, scales = _oracle(_f64(x))
    assert got[0].dtype == torch.int8 and got[1].dtype == torch.float32
    assert np.array_equal(got[0].cpu().numpy(), codes)
    assert np.array_equal(got[1].cpu().numpy(), scales, equal_nan=True)


@pytest.mark.parametrize("rows,K", [(1, 16), (3, 48), (1, 1024), (17, 1040), (5, 2048), (9, 2064),
                                    (33, 4096), (2, 4112), (300, 8192), (7, 8208), (64, 14336),
                                    (3, 16384), (2, 16400), (5, 40000), (8191, 128)])
def test_rows(rows, K):
    g = torch.Generator(device="cuda").manual_seed(rows + K)
    x = torch.randn(rows, K, generator=g, device="cuda")
    x = (x * torch.exp(3 * torch.randn(rows, 1, generator=g, device="cuda"))).to(torch.bfloat16)
    _check(x, nv.int8_quantize_bf16(x))


def test_every_pair_of_mantissas():
    """All 128 mantissas of amax against all mantissas of x over ten binades: every exact
    half-integer and every nearest miss that BF16 can express."""
    frac = torch.arange(128, 256, dtype=torch.float64)
    vals = torch.cat([frac * 2.0 ** j for j in range(-9, 1)])
    for e in (-130, -128, -110, -60, 0, 60, 119):
        x = torch.zeros(128, 2 * len(vals) + 16, dtype=torch.float64)
        x[:, :len(vals)] = vals
        x[:, len(vals):2 * len(vals)] = -vals
        x = torch.where(x.abs() <= frac[:, None], x, torch.zeros_like(x))
        x[:, -1] = frac
        x = (x * 2.0 ** e).to(torch.bfloat16)
        if e > -120:
            assert torch.equal(x.double(), x.double().to(torch.bfloat16).double())
        _check(x, nv.int8_quantize_bf16(x.cuda()))


def test_zero_subnormal_and_nonfinite_rows():
    x = torch.zeros(8, 64, dtype=torch.float32)
    x[1, 3], x[1, 4] = 2.0 ** -133, -(2.0 ** -132)         # BF16 subnormals
    x[2] = 1.0
    x[2, 5] = float("nan")
    x[3, 0] = float("inf")
    x[4, 63] = -float("inf")
    x[5] = torch.linspace(-3e38, 3e38, 64)
    x[6, 7] = -0.0
    x[7, 0], x[7, 1] = 127.0, 0.5                            # scale 1: ties to even
    x[7, 2], x[7, 3], x[7, 4] = 1.5, -2.5, 63.5
    x = x.to(torch.bfloat16)
    codes, scales = nv.int8_quantize_bf16(x.cuda())
    _check(x, (codes, scales))
    assert scales[0] == 1 and scales[6] == 1 and torch.isnan(scales[2:5]).all()
    assert codes[7, :5].tolist() == [127, 0, 2, -2, 64]


@pytest.mark.parametrize("T,K,k,E", [(1, 16, 1, 1), (50, 4096, 2, 8), (333, 1040, 8, 64),
                                     (64, 14336, 4, 16), (20, 20000, 3, 5)])
def test_routed_is_quantise_then_permute(T, K, k, E):
    rng = np.random.default_rng(T + K)
    x = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).to(torch.bfloat16).cuda()
    ids = torch.from_numpy(rng.integers(0, E, (T, k)).astype(np.int32)).cuda()
    off, dest, src = nv.moe_route(ids, E)
    codes, scales = nv.int8_quantize_bf16(x)
    gc, gs = nv.int8_quantize_bf16_routed(x, dest, k)
    tok = torch.div(src.long(), k, rounding_mode="floor")
    assert torch.equal(gc, codes[tok]) and torch.equal(gs, scales[tok])


def test_routed_leaves_out_what_is_sent_nowhere():
    x = torch.randn(4, 64, device="cuda").to(torch.bfloat16)
    dest = torch.tensor([0, -1, 8, 5, -7, 3, 2, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    out = (torch.full((8, 64), 99, dtype=torch.int8, device="cuda"),
           torch.full((8,), 5.0, device="cuda"))
    nv.int8_quantize_bf16_routed(x, dest, 2, out=out)
    codes, scales = nv.int8_quantize_bf16(x)
    for p, d in enumerate(dest.tolist()):
        if 0 <= d < 8:
            assert torch.equal(out[0][d], codes[p // 2]) and out[1][d] == scales[p // 2]
    for r in (1, 4, 6, 7):
        assert (out[0][r] == 99).all() and out[1][r] == 5.0


def test_empty_and_captured_and_side_stream():
    c, s = nv.int8_quantize_bf16(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"))
    assert tuple(c.shape) == (0, 64) and tuple(s.shape) == (0,)
    x = torch.randn(40, 4096, device="cuda").to(torch.bfloat16)
    out = nv.int8_quantize_bf16(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nv.int8_quantize_bf16(x, out=out)
    x.copy_(torch.randn(40, 4096, device="cuda") * 3)
    g.replay()
    torch.cuda.synchronize()
    _check(x, out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = nv.int8_quantize_bf16(x, stream=side)
    side.synchronize()
    _check(x, got)


def test_int8_weights_and_activations_through_the_product():
    """Quantised activations and weights (a weight's rows are its output channels), then the
    product: within the quantisation's own error of the BF16 operands' product."""
    g = torch.Generator(device="cuda").manual_seed(1)
    M, N, K = 70, 260, 1040
    x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    w = (0.02 * torch.randn(N, K, generator=g, device="cuda")).to(torch.bfloat16)
    a, sa = nv.int8_quantize_bf16(x)
    b, sb = nv.int8_quantize_bf16(w)
    y = nv.gemm_int8_w8a8(a, sa, b, sb).double()
    xd, wd = x.double(), w.double()
    ref = xd @ wd.t()
    # |a s - x| <= s/2 and |b s' - w| <= s'/2 for every element (scales add 2^-24)
    bound = (sa.double()[:, None] / 2 * wd.abs().sum(1)[None, :]
             + sb.double()[None, :] / 2 * xd.abs().sum(1)[:, None]
             + K * sa.double()[:, None] * sb.double()[None, :] / 4)
    assert ((y - ref).abs() <= bound * 1.001 + 2.0 ** -8 * (ref.abs() + bound)).all()


def test_refusals():
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        nv.int8_quantize_bf16(b(4, 16).float())
    with pytest.raises(TypeError):
        nv.int8_quantize_bf16(b(4, 4, 16))
    with pytest.raises(ValueError):
        nv.int8_quantize_bf16(b(4, 32)[:, ::2])
    with pytest.raises(ValueError):
        nv.int8_quantize_bf16_routed(b(4, 16), i(7), 2)
    with pytest.raises(TypeError):
        nv.int8_quantize_bf16_routed(b(4, 16), i(8).long(), 2)
    for bad in (lambda: nv.int8_quantize_bf16(b(4, 24)),
                lambda: nv.int8_quantize_bf16_routed(b(4, 16), i(132), 33),
                lambda: nv.int8_quantize_bf16_routed(b(4, 16), i(0), 0)):
        with pytest.raises((nv.NvFp4Error, ValueError)):
            bad()
    with pytest.raises(nv.NvFp4Error) as e:
        nv.int8_quantize_bf16(b(4 * 16 + 1)[1:].view(4, 16))
    assert e.value.status == nv.Status.MISALIGNED
