"""INT8 products on the GPU against exact integer sums scaled in FP64.

Tolerance, element by element: the INT32 sum is exact, so an output carries the FP32
roundings of sA*sW, of the sum's conversion and of their product (2^-24 relative each)
and one rounding to BF16 (2^-8 relative)."""
import numpy as np
import pytest
import torch

import block_scaled_precision_nvfp4_b200 as nv

pytestmark = pytest.mark.gpu

REL = 2.0 ** -8 + 4 * 2.0 ** -24


def _codes(rng, *shape):
    return rng.integers(-128, 128, size=shape, dtype=np.int8)


def _scales(rng, *shape):
    return np.exp(rng.normal(size=shape)).astype(np.float32) * np.float32(0.01)


def _ref(A, sA, W, sW):
    acc = A.astype(np.float64) @ W.astype(np.float64).T       # below 2^53: exact
    return acc * sA.astype(np.float64)[:, None] * sW.astype(np.float64)[None, :]


def _close(y, ref):
    y = y.float().cpu().numpy().astype(np.float64)
    assert y.shape == ref.shape
    bad = ~(np.abs(y - ref) <= REL * np.abs(ref))
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: " \
                          f"{y[tuple(np.argwhere(bad)[0])]} for {ref[tuple(np.argwhere(bad)[0])]}"


def _d(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _bits(y):
    return y.view(torch.int16)


SHAPES = [  # M, N, K: one token, ragged tiles and K tails, split K, single SMs, pairs of SMs
    (1, 1, 16), (1, 128, 128), (1, 1000, 4096), (2, 129, 144), (15, 257, 1040), (16, 512, 2048),
    (17, 127, 272), (33, 640, 8192), (64, 384, 3200), (65, 200, 1168), (100, 1001, 512),
    (128, 256, 4096), (129, 130, 2064), (160, 512, 6400), (200, 72, 528), (255, 384, 1024),
    (256, 640, 4112), (257, 256, 128), (300, 515, 784), (512, 512, 1024), (513, 1025, 400),
    (1000, 300, 2000), (2049, 2305, 256)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K):
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    A, W, sA, sW = _codes(rng, M, K), _codes(rng, N, K), _scales(rng, M), _scales(rng, N)
    y = nv.gemm_int8_w8a8(_d(A), _d(sA), _d(W), _d(sW))
    torch.cuda.synchronize()
    nv.nvfp4_check_device_error()
    assert y.dtype == torch.bfloat16
    _close(y, _ref(A, sA, W, sW))


@pytest.mark.parametrize("M,N,K", [(0, 64, 64), (64, 0, 64)])
def test_empty(M, N, K):
    z = lambda *s, dt=torch.int8: torch.zeros(s, dtype=dt, device="cuda")
    y = nv.gemm_int8_w8a8(z(M, K), z(M, dt=torch.float32), z(N, K), z(N, dt=torch.float32))
    assert tuple(y.shape) == (M, N)


@pytest.mark.parametrize("M", [3, 300])
def test_largest_sums_do_not_overflow(M):
    K = 131056
    A = np.full((M, K), -128, np.int8)
    W = np.full((130, K), -128, np.int8)
    W[1] = 127
    sA, sW = np.full(M, 2.0 ** -20, np.float32), np.ones(130, np.float32)
    _close(nv.gemm_int8_w8a8(_d(A), _d(sA), _d(W), _d(sW)), _ref(A, sA, W, sW))


def test_a_nan_or_inf_scale_stays_in_its_row_and_channel():
    rng = np.random.default_rng(5)
    for M in (5, 290):
        A, W, sA, sW = _codes(rng, M, 256), _codes(rng, 140, 256), _scales(rng, M), _scales(rng, 140)
        sA[2], sW[7] = np.nan, np.nan
        y = nv.gemm_int8_w8a8(_d(A), _d(sA), _d(W), _d(sW)).float().cpu().numpy()
        nan = np.isnan(y)
        assert nan[2].all() and nan[:, 7].all()
        assert nan.sum() == M + 140 - 1


def test_operands_may_be_one_buffer_and_scales_start_anywhere():
    """A . A^T, and scales that are slices (4-byte aligned)."""
    rng = np.random.default_rng(12)
    A, s = _codes(rng, 150, 400), _scales(rng, 153)
    dA, ds = _d(A), _d(s)
    for o in (1, 2, 3):
        y = nv.gemm_int8_w8a8(dA, ds[o:150 + o], dA, ds[3 - o:153 - o])
        _close(y, _ref(A, s[o:150 + o], A, s[3 - o:153 - o]))


def test_rows_do_not_depend_on_their_batch():
    """One row alone, in a small batch and in a large one: the same bits (split K, single
    SMs and pairs of SMs all sum the same integers and scale in the same order)."""
    rng = np.random.default_rng(9)
    M, N, K = 700, 640, 2304
    A, W, sA, sW = _d(_codes(rng, M, K)), _d(_codes(rng, N, K)), _d(_scales(rng, M)), _d(_scales(rng, N))
    whole = nv.gemm_int8_w8a8(A, sA, W, sW)
    for m in (1, 17, 64, 130, 256):
        part = nv.gemm_int8_w8a8(A[:m], sA[:m], W, sW)
        assert torch.equal(_bits(part), _bits(whole[:m])), m


def _offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


GROUPS = [  # counts per expert, N, K
    ([1], 128, 128), ([0, 0, 1, 0], 300, 512), ([5, 0, 3, 17, 1, 0], 256, 1040),
    ([0, 200, 0, 31, 1, 90, 0, 2], 130, 272), ([300, 1, 700, 0, 257, 256], 520, 400),
    ([1000, 0, 16, 900], 256, 2048), ([2] * 64, 136, 256), (list(range(40)) + [0] * 216, 64, 144),
    ([40] * 33, 72, 3200)]


@pytest.mark.parametrize("counts,N,K", GROUPS)
@pytest.mark.parametrize("spare", [0, 37])
def test_grouped(counts, N, K, spare):
    """Ragged and empty experts; `spare` rows behind the last expert stay as they were."""
    E, off = len(counts), _offsets(counts)
    P = int(off[-1])
    M = P + spare
    rng = np.random.default_rng(E * 11 + N + K)
    A, W, sA, sW = _codes(rng, M, K), _codes(rng, E, N, K), _scales(rng, M), _scales(rng, E, N)
    out = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    dA, dsA, dW, dsW = _d(A), _d(sA), _d(W), _d(sW)
    y = nv.gemm_int8_w8a8_grouped(dA, dsA, dW, dsW, _d(off), out=out)
    torch.cuda.synchronize()
    nv.nvfp4_check_device_error()
    assert y is out and torch.all(y[P:] == 7.0)
    for e in range(E):
        r = slice(off[e], off[e + 1])
        if counts[e]:
            _close(y[r], _ref(A[r], sA[r], W[e], sW[e]))
            one = nv.gemm_int8_w8a8(dA[r].clone(), dsA[r].clone(), dW[e], dsW[e].clone())
            assert torch.equal(_bits(one), _bits(y[r]))


@pytest.mark.parametrize("off", [[1, 3, 5], [0, 4, 3], [0, 3, 7], [0, -1, 5], [0, 9, 5]])
@pytest.mark.parametrize("scale", [1, 100])
def test_bad_offsets_write_nothing_and_are_reported(off, scale):
    off = np.array(off, np.int32) * scale
    M = 5 * scale
    z = lambda *s, dt=torch.int8: torch.zeros(s, dtype=dt, device="cuda")
    out = torch.full((M, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    nv.gemm_int8_w8a8_grouped(z(M, 128), z(M, dt=torch.float32), z(2, 64, 128),
                              z(2, 64, dt=torch.float32), _d(off), out=out)
    with pytest.raises(nv.NvFp4Error) as err:
        nv.nvfp4_check_device_error()
    assert err.value.status == nv.Status.INVALID_ARG
    nv.nvfp4_check_device_error()
    assert torch.all(out == 3.0)


def test_captured_calls_replay_on_new_inputs_and_offsets():
    rng = np.random.default_rng(3)
    E, N, K, M = 4, 384, 768, 500
    A, W, sA, sW = _codes(rng, M, K), _codes(rng, E, N, K), _scales(rng, M), _scales(rng, E, N)
    dA, dsA, dW, dsW = _d(A), _d(sA), _d(W), _d(sW)
    off = _d(_offsets([100, 0, 300, 100]))
    y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    y1 = torch.empty((9, N), dtype=torch.bfloat16, device="cuda")
    one = lambda: nv.gemm_int8_w8a8(dA[:9], dsA[:9], dW[1], dsW[1], out=y1)
    nv.gemm_int8_w8a8_grouped(dA, dsA, dW, dsW, off, out=y)
    one()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nv.gemm_int8_w8a8_grouped(dA, dsA, dW, dsW, off, out=y)
        one()
    for counts in ([0, 500, 0, 0], [1, 2, 3, 494], [125, 125, 125, 125]):
        A = _codes(rng, M, K)
        dA.copy_(_d(A))
        o = _offsets(counts)
        off.copy_(_d(o))
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        for e in range(E):
            r = slice(o[e], o[e + 1])
            if counts[e]:
                _close(y[r], _ref(A[r], sA[r], W[e], sW[e]))
        _close(y1, _ref(A[:9], sA[:9], W[1], sW[1]))


def test_two_streams_at_once():
    """Calls of every form in flight on two streams: no state is shared between them."""
    rng = np.random.default_rng(21)
    cases = []
    for M, N, K in [(4, 900, 4096), (200, 640, 1024), (600, 512, 1024)]:
        A, W, sA, sW = _codes(rng, M, K), _codes(rng, N, K), _scales(rng, M), _scales(rng, N)
        cases.append((tuple(map(_d, (A, sA, W, sW))), _ref(A, sA, W, sW)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(20):
        for s in streams:
            for args, ref in cases:
                got.append((nv.gemm_int8_w8a8(*args, stream=s), ref))
    torch.cuda.synchronize()
    nv.nvfp4_check_device_error()
    for y, ref in got[-len(cases) * 2:]:
        _close(y, ref)
    for i, (y, _) in enumerate(got):
        assert torch.equal(_bits(y), _bits(got[i % len(cases)][0]))


@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (33, 127, 64), (40, 129, 64), (300, 131, 64), (257, 250, 64),
                                   (100, 1001, 64), (64, 383, 64), (300, 515, 64), (70, 1285, 64),
                                   (520, 254, 64), (31, 6, 64), (200, 2, 64), (5, 259, 4096)])
def test_nothing_is_written_around_the_output(M, N, K):
    """Every row start modulo 16 bytes, widths around the tile's; a frame around Y stays."""
    rng = np.random.default_rng(M + N)
    A, W, sA, sW = _codes(rng, M, K), _codes(rng, N, K), _scales(rng, M), _scales(rng, N)
    frame = 4096
    buf = torch.full((2 * frame + M * N + 8,), 9.0, dtype=torch.bfloat16, device="cuda")
    out = buf[frame:frame + M * N].view(M, N)
    nv.gemm_int8_w8a8(_d(A), _d(sA), _d(W), _d(sW), out=out)
    torch.cuda.synchronize()
    _close(out, _ref(A, sA, W, sW))
    assert (buf[:frame] == 9.0).all() and (buf[frame + M * N:] == 9.0).all()


def test_python_refusals():
    z = lambda *s, dt=torch.int8: torch.zeros(s, dtype=dt, device="cuda")
    f = lambda *s: z(*s, dt=torch.float32)
    ok = dict(A=z(4, 64), sA=f(4), W=z(8, 64), sW=f(8))

    def call(**kw):
        return nv.gemm_int8_w8a8(**{**ok, **kw})
    call()
    for kw, err in [(dict(A=z(4, 64, dt=torch.uint8)), TypeError), (dict(W=f(8, 64)), TypeError),
                    (dict(sA=f(5)), ValueError), (dict(sW=f(8, 1)), ValueError),
                    (dict(sA=torch.zeros(4)), ValueError), (dict(A=z(4, 128)[:, ::2]), ValueError),
                    (dict(W=z(8, 80)), ValueError), (dict(A=z(64)), TypeError),
                    (dict(out=f(4, 8)), TypeError),
                    (dict(out=z(8, 4, dt=torch.bfloat16)), ValueError)]:
        with pytest.raises(err):
            call(**kw)
    with pytest.raises(nv.NvFp4Error) as e:
        nv.gemm_int8_w8a8(z(4, 24), f(4), z(8, 24), f(8))
    assert e.value.status == nv.Status.INVALID_ARG
    with pytest.raises(nv.NvFp4Error) as e:
        call(A=z(4 * 64 + 8)[8:].view(4, 64))
    assert e.value.status == nv.Status.MISALIGNED
    with pytest.raises(TypeError):
        nv.gemm_int8_w8a8_grouped(ok["A"], ok["sA"], ok["W"], ok["sW"], z(2, dt=torch.int32))
    with pytest.raises(ValueError):
        nv.gemm_int8_w8a8_grouped(ok["A"], ok["sA"], z(2, 8, 64), f(2, 8), z(2, dt=torch.int32))
