"""GPU tests of the 4-bit matrix operators and the table lookup with its gradient, against tests/lowbit_ref.py.

Codes, scales, values and looked-up rows are compared bit for bit.  Sums are compared with the 64-bit ones within a
bound counted from the operations: a step of an fp32 sum is off by at most half a unit of the sum's last place (2^-24 of
the sum of magnitudes so far, S), a step of a tensor-core sum, whose rounding is not specified, is given 2^-22; the
output adds half a step of its type relative to the result.
"""
from __future__ import annotations

import threading

import numpy as np
import pytest
import torch

import int8_gemm_b200 as bs
import lowbit_ref as ref
import oracle

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_device):
    bs.lib()
    yield
    assert bs.device_error() == 0, "a kernel reported a timed-out wait"


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _weights(N, K, seed, dtype=BF):
    g = _gen(seed)
    x = torch.randn(N, K, generator=g) * 0.02
    return torch.where(torch.rand(N, K, generator=g) < 0.01, x * 10, x).to(dtype)


def _matrix(N, K, group, seed, scale_dtype=F, asym=False):
    """Random codes with scales (and zero points): the host's numbers and the device's tensors."""
    rng = np.random.default_rng(seed)
    G = -(-K // group)
    codes = rng.integers(0, 16, (N, K))
    scale = torch.from_numpy((rng.random((N, G)) + 0.5).astype(np.float32) * 0.01).to(scale_dtype)
    zero = rng.integers(0, 16, (N, G)) if asym else np.full((N, G), 8)
    q = bs._empty_out((N,), (K + 1) // 2, torch.uint8, DEV)
    q.copy_(torch.from_numpy(ref.pack(codes, zero, group)))
    z = torch.from_numpy(zero.astype(np.uint8)).to(DEV) if asym else None
    return (codes, scale.float().numpy(), zero), (q, scale.to(DEV), z)


def _eps(dtype):
    return torch.finfo(dtype).eps / 2


def _bits(t):
    t = t.contiguous().cpu()
    return t.view({4: torch.int32, 2: torch.int16, 1: torch.uint8}[t.element_size()])


def same(a, b):
    return torch.equal(_bits(a), _bits(b))


# ---------------------------------------------------------------------------
# quantiser and dequantiser
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("asym", [False, True])
@pytest.mark.parametrize("scale_dtype", [F, BF])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("N,K,group", [(1, 1, 32), (3, 31, 32), (5, 33, 32), (7, 130, 64), (33, 1024, 128), (2, 4097, 128),
                                       (130, 2050, 32), (16, 512, 64), (9, 1040, 128)])
def test_quantize_bit_exact(N, K, group, dtype, scale_dtype, asym):
    x = _weights(N, K, 100 + N + K, dtype)
    if N > 4:
        x[1] = 0
        x[2] = x[2].abs()
        x[3] = -x[3].abs()
        x[4, K // 2:] = 0
    q, s, z = bs.bs_quantize_int4(x.to(DEV), group=group, scale_dtype=scale_dtype, asymmetric=asym)
    codes, scale, zero = ref.quantize_int4(x, group, scale_dtype == BF, asym)
    assert np.array_equal(s.float().cpu().numpy(), scale)
    assert np.array_equal(q.cpu().numpy(), ref.pack(codes, zero, group))
    assert (z is None) == (not asym)
    if asym:
        assert np.array_equal(z.cpu().numpy(), zero)
    for out_dtype in (BF, F):
        w = bs.bs_dequantize_int4(q, s, z, K=K, group=group, out_dtype=out_dtype)
        assert same(w, torch.from_numpy(ref.values(codes, scale, zero, group)).to(out_dtype))


@pytest.mark.parametrize("dtype,scale_dtype,asym,group", [(BF, F, False, 128), (F, BF, True, 32), (BF, BF, True, 64)])
def test_quantize_large_bit_exact(dtype, scale_dtype, asym, group):
    """More than 2^24 elements: the kernel with two passes per warp."""
    N, K = 4100, 4099
    x = _weights(N, K, 17, dtype)
    q, s, z = bs.bs_quantize_int4(x.to(DEV), group=group, scale_dtype=scale_dtype, asymmetric=asym)
    codes, scale, zero = ref.quantize_int4(x, group, scale_dtype == BF, asym)
    assert np.array_equal(s.float().cpu().numpy(), scale)
    assert np.array_equal(q.cpu().numpy(), ref.pack(codes, zero, group))
    if asym:
        assert np.array_equal(z.cpu().numpy(), zero)
    w = bs.bs_dequantize_int4(q, s, z, K=K, group=group, out_dtype=dtype)
    assert same(w, torch.from_numpy(ref.values(codes, scale, zero, group)).to(dtype))


@pytest.mark.parametrize("asym", [False, True])
def test_quantize_ranges_from_subnormal_to_huge(asym):
    """Scales that underflow to one, subnormal scales, scales on both sides of the fast quotient's range, the largest
    finite values, one-sided groups and quotients at code borders."""
    rows = []
    for e in (-149, -147, -140, -133, -126, -120, -91, -88, -87, -60, 0, 60, 120, 127):
        base = np.ldexp(1.0, e)
        rows.append(np.array([k * base / 14 for k in range(-14, 15)] + [0, -0.0, base], np.float64))
    rows.append(np.full(32, np.finfo(np.float32).max))
    rows.append(np.concatenate([np.full(16, -np.finfo(np.float32).max), np.full(16, np.finfo(np.float32).max)]))
    x = torch.from_numpy(np.stack(rows).astype(np.float32))
    for scale_dtype in (F, BF):
        q, s, z = bs.bs_quantize_int4(x.to(DEV), group=32, scale_dtype=scale_dtype, asymmetric=asym)
        codes, scale, zero = ref.quantize_int4(x, 32, scale_dtype == BF, asym)
        assert np.array_equal(s.float().cpu().numpy(), scale)
        assert np.array_equal(q.cpu().numpy(), ref.pack(codes, zero, 32))
        if asym:
            assert np.array_equal(z.cpu().numpy(), zero)


def test_quantize_views_and_untouched_bytes():
    """Unaligned rows, padded strides and buffers given by the caller; nothing outside the matrix is written."""
    N, K, group = 11, 301, 64
    big = _weights(N, K + 9, 7, BF).to(DEV)
    x = big[:, 3:3 + K]
    canvas = torch.full((N, 170), 0xAB, dtype=torch.uint8, device=DEV)
    s_canvas = torch.full((N, 9), -7.0, device=DEV)
    z_canvas = torch.full((N, 9), 77, dtype=torch.uint8, device=DEV)
    q, s, z = bs.bs_quantize_int4(x, group=group, asymmetric=True, q=canvas[:, 5:156], scale=s_canvas[:, 2:7],
                                  zero=z_canvas[:, 1:6])
    codes, scale, zero = ref.quantize_int4(x.cpu(), group, False, True)
    assert np.array_equal(q.cpu().numpy(), ref.pack(codes, zero, group))
    assert np.array_equal(s.cpu().numpy(), scale) and np.array_equal(z.cpu().numpy(), zero)
    assert torch.all(canvas[:, :5] == 0xAB) and torch.all(canvas[:, 156:] == 0xAB)
    assert torch.all(s_canvas[:, :2] == -7) and torch.all(s_canvas[:, 7:] == -7)
    assert torch.all(z_canvas[:, :1] == 77) and torch.all(z_canvas[:, 6:] == 77)
    out = torch.full((N, K + 8), 3.0, dtype=BF, device=DEV)
    bs.bs_dequantize_int4(q, s, z, K=K, group=group, out=out[:, 5:5 + K])
    assert same(out[:, 5:5 + K], torch.from_numpy(ref.values(codes, scale, zero, group)).to(BF))
    assert torch.all(out[:, :5] == 3) and torch.all(out[:, 5 + K:] == 3)


def test_quantize_non_finite_inputs_stay_inside_their_group():
    x = _weights(4, 256, 9, F)
    clean = bs.bs_quantize_int4(x.to(DEV), group=64)
    x[1, 70], x[2, 5], x[3, 200] = float("nan"), float("inf"), float("-inf")
    q, s, _ = bs.bs_quantize_int4(x.to(DEV), group=64)
    keep = torch.ones(4, 4, dtype=torch.bool)
    keep[1, 1] = keep[2, 0] = keep[3, 3] = False
    assert torch.equal(s.cpu()[keep], clean[1].cpu()[keep])
    assert torch.equal(q.cpu().view(4, 4, 32)[keep], clean[0].cpu().view(4, 4, 32)[keep])


def test_empty_matrices():
    for N, K in ((0, 64), (5, 0), (0, 0)):
        q, s, z = bs.bs_quantize_int4(torch.empty(N, K, device=DEV), asymmetric=True)
        assert q.shape == (N, K // 2) and s.shape == (N, -(-K // 128)) and z.shape == s.shape
        assert bs.bs_dequantize_int4(q, s, z).shape == (N, K)
        y = bs.bs_gemv_int4(torch.empty(3, K, device=DEV), q, s, z, out_dtype=F)
        assert y.shape == (3, N) and torch.all(y == 0)
    b = torch.arange(5.0, device=DEV)
    q, s, _ = bs.bs_quantize_int4(torch.empty(5, 0, device=DEV))
    assert torch.equal(bs.bs_gemv_int4(torch.empty(2, 0, device=DEV), q, s, bias=b, out_dtype=F), b.expand(2, 5))
    assert bs.bs_gemv_int4(torch.empty(0, 64, device=DEV), *bs.bs_quantize_int4(torch.ones(4, 64, device=DEV))[:2]).shape == (0, 4)


# ---------------------------------------------------------------------------
# product
# ---------------------------------------------------------------------------
def _product_check(x, host, dev, group, out_dtype, bias=None, x_dev=None, what=""):
    y = bs.bs_gemv_int4(x.to(DEV) if x_dev is None else x_dev, *dev, bias=None if bias is None else bias.to(DEV),
                        group=group, out_dtype=out_dtype)
    want, S = ref.product(x.double().numpy().reshape(-1, x.shape[-1]), *host, group, None if bias is None else bias.numpy())
    K = x.shape[-1]
    # steps from a term to the result: a group's MMAs (16 k each, three parts for fp32), the groups of the whole row (a
    # split of K makes them fewer), at most 16 parts of K joined, and the bias
    parts = 3 if x.dtype == F else 1
    steps = parts * -(-group // 16) + -(-K // group) + 16 + 1
    tol = steps * 2.0**-22 * S + _eps(out_dtype) * np.abs(want) + 1e-38
    got = y.double().cpu().numpy().reshape(want.shape)
    worst = np.max(np.abs(got - want) / tol)
    assert worst <= 1, f"{what}: {worst}"
    return y


@pytest.mark.parametrize("x_dtype,out_dtype", [(BF, BF), (F, F), (BF, F)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 16, 32), (2, 17, 33), (3, 5, 127), (8, 40, 128), (9, 33, 129), (1, 1024, 4096),
                                   (16, 100, 1000), (17, 64, 2050), (32, 130, 640), (31, 7, 5001), (5, 259, 8208)])
def test_product(M, N, K, group, x_dtype, out_dtype):
    host, dev = _matrix(N, K, group, M + N + K, asym=(N + group // 32) % 2 == 0, scale_dtype=BF if K % 2 else F)
    x = torch.randn(M, K, generator=_gen(M * K)).to(x_dtype)
    bias = torch.randn(N, generator=_gen(1)) if M % 2 else None
    _product_check(x, host, dev, group, out_dtype, bias, what=f"{M}x{N}x{K} group {group}")


@pytest.mark.parametrize("M", list(range(1, 33)))
def test_product_every_row_count(M):
    host, dev = _matrix(70, 768, 64, M, asym=True)
    x = torch.randn(M, 768, generator=_gen(M)).to(BF)
    y = _product_check(x, host, dev, 64, F, what=f"M={M}")
    assert same(y, bs.bs_gemv_int4(x.to(DEV), *dev, group=64, out_dtype=F))  # the same bits on every run


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("M", [1, 9, 20])
@pytest.mark.parametrize("K", [1, 100, 128, 129, 300, 600, 1024, 1100])
def test_product_many_rows_and_every_split_of_k(K, M, dtype):
    """Enough rows for the wide row tiles, with one to eight warps sharing K: the last tile ragged."""
    N, group = 5000, 64
    host, dev = _matrix(N, K, group, K, asym=K % 2 == 0)
    x = torch.randn(M, K, generator=_gen(K + M)).to(dtype)
    _product_check(x, host, dev, group, F, torch.randn(N, generator=_gen(2)), what=f"{M}x{N}x{K}")


def test_product_more_tiles_than_ctas():
    N, K, group = 40000, 256, 128  # every CTA takes several tiles
    host, dev = _matrix(N, K, group, 3)
    for M in (2, 12, 30):
        _product_check(torch.randn(M, K, generator=_gen(M)).to(BF), host, dev, group, BF)


def test_product_one_hot_rows_read_out_the_matrix():
    """x = e_k gives column k of the values: every code meets its own activation, in every position of a block."""
    N, K = 48, 288
    for group in (32, 64, 128):
        for dtype in (BF, F):
            host, dev = _matrix(N, K, group, 5, asym=True)
            want = ref.values(*host, group)
            for k0 in range(0, K, 32):
                x = torch.zeros(32, K, dtype=dtype)
                x[torch.arange(32), k0 + torch.arange(32)] = 1
                y = bs.bs_gemv_int4(x.to(DEV), *dev, group=group, out_dtype=F)
                assert np.array_equal(y.cpu().numpy(), want[:, k0:k0 + 32].T)


def test_product_fp32_activations_keep_their_bits():
    """A value of 24 significant bits times one code: the three bf16 parts add up to it."""
    host, dev = _matrix(16, 128, 128, 8)
    codes, _, _ = host
    ones = torch.ones(16, 1, device=DEV)
    for value in (1 + 2**-23, 1.9999998807907104, 3.1415927410125732, -2.7182817459106445, 2.0**-100 * (1 + 2**-23), 1e30):
        x = torch.zeros(1, 128)
        x[0, 77] = value
        y = bs.bs_gemv_int4(x.to(DEV), dev[0], ones, out_dtype=F).cpu().numpy()[0]
        want = np.float32(np.float64(np.float32(value)) * (codes[:, 77] - 8))
        # codes below 16 in magnitude: three products of 8 bits by 4, added in fp32 (two roundings)
        assert np.all(np.abs(y - want) <= 2.0**-22 * np.abs(want))


def test_product_non_finite_activations():
    host, dev = _matrix(40, 256, 64, 9, asym=True)
    codes, scale, zero = host
    for dtype in (BF, F):
        for value in (float("inf"), float("-inf"), float("nan")):
            x = torch.randn(3, 256, generator=_gen(4)).to(dtype)
            base = bs.bs_gemv_int4(x.to(DEV), *dev, group=64, out_dtype=F)
            x[1, 100] = value
            y = bs.bs_gemv_int4(x.to(DEV), *dev, group=64, out_dtype=F)
            assert same(y[0], base[0]) and same(y[2], base[2])
            w = codes[:, 100] - zero[:, 1]
            with np.errstate(invalid="ignore"):
                want = np.where(w == 0, np.nan, np.sign(w) * value)
            assert np.array_equal(y[1].cpu().numpy(), want.astype(np.float32), equal_nan=True)


def test_product_views_vectors_and_untouched_output():
    N, K, group = 37, 250, 64
    host, dev = _matrix(N, K, group, 11)
    big = torch.randn(6, K + 5, generator=_gen(2)).to(BF).to(DEV)
    x = big[1:5, 3:3 + K]  # unaligned rows
    canvas = torch.full((6, N + 4), 9.0, dtype=F, device=DEV)
    view = canvas[1:5, 3:3 + N]
    bs.bs_gemv_int4(x, *dev, group=group, out_dtype=F, out=view)
    assert same(view, _product_check(x.cpu(), host, dev, group, F))
    canvas[1:5, 3:3 + N] = 9
    assert torch.all(canvas == 9)
    one = bs.bs_gemv_int4(x[0].contiguous(), *dev, group=group, out_dtype=F)
    assert one.shape == (N,) and same(one, bs.bs_gemv_int4(x[:1], *dev, group=group, out_dtype=F)[0])
    # strided scales and zero points
    sc = torch.zeros(N, 9, device=DEV)
    sc[:, 1:5] = dev[1]
    assert same(bs.bs_gemv_int4(x, dev[0], sc[:, 1:5], group=group, out_dtype=F), bs.bs_gemv_int4(x, *dev, group=group, out_dtype=F))


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("M", [1, 2, 8, 13, 32])
@pytest.mark.parametrize("N", [70, 5000])
def test_product_activation_rows_on_every_boundary(N, M, dtype):
    """Rows that start 16, 8, 4 and 2 bytes off a boundary, together or in turn, give the bits of aligned rows, and no
    neighbour of a row is taken for one of its elements."""
    K, group = 430, 64  # whole blocks and a ragged one
    host, dev = _matrix(N, K, group, 6)
    x = torch.randn(M, K, generator=_gen(M + N)).to(dtype)
    want = _product_check(x, host, dev, group, F, x_dev=_aligned(x))
    for off, pad in ((0, 1), (1, 0), (1, 1), (0, 2), (2, 0), (2, 4), (3, 3), (4, 4), (4, 8), (8, 8), (7, 16)):
        flat = torch.full((off + M * (K + pad) + 8,), float("nan"), dtype=dtype, device=DEV)
        view = flat[off:off + M * (K + pad)].view(M, K + pad)[:, :K]
        view.copy_(x)
        assert same(want, bs.bs_gemv_int4(view, *dev, group=group, out_dtype=F)), (off, pad)


def _aligned(x):
    """x on the GPU with rows on 16-byte boundaries."""
    return bs._empty_out((x.shape[0],), x.shape[1], x.dtype, DEV).copy_(x)


def _us(call, reps=20):
    """The least time of a call among others, on the device."""
    graph = torch.cuda.CUDAGraph()
    call()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for _ in range(8):
            call()
    times = []
    for _ in range(reps):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        graph.replay()
        end.record()
        end.synchronize()
        times.append(start.elapsed_time(end))
    return min(times) * 1e3 / 8


@pytest.mark.slow
@pytest.mark.parametrize("K", [4100, 4098, 4097])
def test_product_activation_rows_off_boundaries_cost_no_multiple(K):
    """Contiguous rows of a length that is no multiple of 16 bytes: 1.2 to 1.8 times aligned rows' time (element by
    element they took four times)."""
    M, N = 32, 32768
    _, dev = _matrix(N, K, 128, 6)
    x = torch.randn(M, K, generator=_gen(1)).to(BF)
    out = torch.empty(M, N, dtype=BF, device=DEV)
    times = [_us(lambda x=x: bs.bs_gemv_int4(x, *dev, out=out)) for x in (_aligned(x), x.to(DEV))]
    assert times[1] <= 2.5 * times[0], times


def test_binding_refusals():
    host, dev = _matrix(8, 128, 64, 1)
    x = torch.randn(2, 128, device=DEV)
    bad = [
        (bs.BS_ERR_SHAPE, lambda: bs.bs_gemv_int4(torch.randn(33, 128, device=DEV), *dev, group=64)),
        (bs.BS_ERR_SHAPE, lambda: bs.bs_gemv_int4(x[:, :100], *dev, group=64)),
        (bs.BS_ERR_SHAPE, lambda: bs.bs_gemv_int4(x, *dev, group=128)),
        (bs.BS_ERR_SHAPE, lambda: bs.bs_gemv_int4(x, *dev, group=48)),
        (bs.BS_ERR_SHAPE, lambda: bs.bs_gemv_int4(x[None], *dev, group=64)),
        (bs.BS_ERR_SHAPE, lambda: bs.bs_gemv_int4(x, *dev, bias=torch.ones(7, device=DEV), group=64)),
        (bs.BS_ERR_DTYPE, lambda: bs.bs_gemv_int4(x.half(), *dev, group=64)),
        (bs.BS_ERR_DTYPE, lambda: bs.bs_gemv_int4(x, *dev, group=64, out_dtype=torch.float16)),
        (bs.BS_ERR_DTYPE, lambda: bs.bs_gemv_int4(x, dev[0].to(torch.int8), dev[1], group=64)),
        (bs.BS_ERR_DTYPE, lambda: bs.bs_gemv_int4(x, dev[0], dev[1].double(), group=64)),
        (bs.BS_ERR_LAYOUT, lambda: bs.bs_gemv_int4(x.t().contiguous().t(), *dev, group=64)),
        (bs.BS_ERR_LAYOUT, lambda: bs.bs_gemv_int4(x[:1].expand(2, 128), *dev, group=64)),
        (bs.BS_ERR_ALIGNMENT, lambda: bs.bs_gemv_int4(x[:, :88].contiguous(), dev[0][:, :44].contiguous(), dev[1], group=64)),
        (bs.BS_ERR_DEVICE, lambda: bs.bs_gemv_int4(x, dev[0].cpu(), dev[1], group=64)),
        (bs.BS_ERR_SHAPE, lambda: bs.bs_gemv_int4(x, *dev, group=64, out_dtype=F, out=torch.empty(2, 9, device=DEV))),
        (bs.BS_ERR_SHAPE, lambda: bs.bs_quantize_int4(x, zero=torch.zeros(2, 1, dtype=torch.uint8, device=DEV))),
        (bs.BS_ERR_SHAPE, lambda: bs.bs_quantize_int4(x[0])),
        (bs.BS_ERR_SHAPE, lambda: bs.bs_dequantize_int4(*dev, K=126, group=64)),
        (bs.BS_ERR_DTYPE, lambda: bs.bs_embedding(torch.zeros(2, device=DEV), x)),
        (bs.BS_ERR_DTYPE, lambda: bs.bs_embedding(torch.zeros(2, dtype=torch.int64, device=DEV), x, format="fp8")),
        (bs.BS_ERR_NULL, lambda: bs.bs_embedding(torch.zeros(2, dtype=torch.int64, device=DEV), dev[0], format="int4")),
        (bs.BS_ERR_SHAPE, lambda: bs.bs_embedding(torch.zeros(2, dtype=torch.int64, device=DEV), x, dev[1])),
        (bs.BS_ERR_SHAPE, lambda: bs.bs_embedding(torch.zeros(2, dtype=torch.int64, device=DEV), x, dim=64)),
        (bs.BS_ERR_SHAPE, lambda: bs.bs_embedding_grad(torch.zeros(3, dtype=torch.int64, device=DEV), x, 5)),
        (bs.BS_ERR_SHAPE, lambda: bs.bs_embedding_grad(torch.zeros(2, dtype=torch.int64, device=DEV), x, 5, padding_idx=5)),
        (bs.BS_ERR_NULL, lambda: bs.bs_embedding_grad(torch.zeros(2, dtype=torch.int64, device=DEV), x, 5, accumulate=True)),
        (bs.BS_ERR_LAYOUT, lambda: bs.bs_embedding_grad(torch.zeros(2, dtype=torch.int64, device=DEV), x[:1].expand(2, 128), 5)),
    ]
    for i, (status, call) in enumerate(bad):
        with pytest.raises(bs.BsgemmError) as e:
            call()
        assert e.value.status == status, (i, str(e.value))


def test_binding_refuses_missing_tensors():
    """A None in the place of a tensor that the call needs raises the library's error, in every place."""
    _, (q, scale, _) = _matrix(8, 128, 64, 1)
    x, t = torch.randn(2, 128, device=DEV), torch.zeros(2, dtype=torch.int64, device=DEV)
    null, device = bs.BS_ERR_NULL, bs.BS_ERR_DEVICE
    bad = [
        (device, lambda: bs.bs_quantize_int4(None)),
        (device, lambda: bs.bs_dequantize_int4(None, scale, group=64)),
        (null, lambda: bs.bs_dequantize_int4(q, None, group=64)),
        (device, lambda: bs.bs_gemv_int4(None, q, scale, group=64)),
        (null, lambda: bs.bs_gemv_int4(x, None, scale, group=64)),
        (null, lambda: bs.bs_gemv_int4(x, q, None, group=64)),
        (device, lambda: bs.bs_embedding(None, x)),
        (null, lambda: bs.bs_embedding(t, None)),
        (null, lambda: bs.bs_embedding(t, None, scale, format="int4", group=64)),
        (device, lambda: bs.bs_embedding_grad(None, x, 5)),
        (null, lambda: bs.bs_embedding_grad(t, None, 5)),
    ]
    for i, (status, call) in enumerate(bad):
        with pytest.raises(bs.BsgemmError) as e:
            call()
        assert e.value.status == status, (i, str(e.value))


# ---------------------------------------------------------------------------
# lookup
# ---------------------------------------------------------------------------
TOKENS = [0, 5, 5, 49, 50, -1, 7, 2**31 - 1, 3, 0]


def _table(fmt, V, D, seed, group=32):
    """(fp32 values, table, keyword arguments) of a random table."""
    rng = np.random.default_rng(seed)
    if fmt in ("bf16", "f32"):
        dtype = BF if fmt == "bf16" else F
        t = torch.from_numpy(rng.standard_normal((V, D)).astype(np.float32)).to(dtype)
        return t.float().numpy(), t.to(DEV), {}
    if fmt == "int4":
        host, (q, s, z) = _matrix(V, D, group, seed, asym=True)
        return ref.values(*host, group), q, {"scale": s, "zero": z, "format": "int4", "dim": D, "group": group}
    x = torch.from_numpy(rng.standard_normal((V, D)).astype(np.float32))
    q, s = bs.bs_quantize_fp8_1x128(x.to(DEV), "f32" if fmt == "e4m3" else "e8m0")
    sc = s.cpu().numpy() if fmt == "e4m3" else np.ldexp(1.0, s.cpu().numpy().astype(np.int64) - 127).astype(np.float32)
    v = oracle.e4m3_table()[q.cpu().numpy()].astype(np.float32) * ref.spread(sc, 128, D)
    return v, q, {"scale": s, "format": "e4m3"}


@pytest.mark.parametrize("fmt", ["bf16", "f32", "e4m3", "e8m0", "int4"])
@pytest.mark.parametrize("out_dtype", [BF, F])
@pytest.mark.parametrize("D", [1, 2, 7, 8, 31, 64, 100, 256, 1001, 5120])
def test_lookup_bit_exact(D, out_dtype, fmt):
    values, table, kw = _table(fmt, 50, D, D)
    for dtype in (torch.int64, torch.int32):
        tokens = torch.tensor(TOKENS, dtype=dtype)
        for alpha in (1.0, D ** 0.5):
            got = bs.bs_embedding(tokens.to(DEV), table, alpha=alpha, out_dtype=out_dtype, **kw)
            assert got.shape == (len(TOKENS), D)
            assert same(got, torch.from_numpy(ref.lookup(tokens.numpy(), values, alpha)).to(out_dtype))


@pytest.mark.parametrize("fmt", ["bf16", "f32", "e4m3", "e8m0", "int4"])
@pytest.mark.parametrize("out_dtype", [BF, F])
@pytest.mark.parametrize("T,D", [(1100, 5120), (2500, 1001), (40000, 72), (600000, 4)])
def test_lookup_large_bit_exact(T, D, out_dtype, fmt):
    """Outputs of more than 4 MB: several pieces per lane, whole runs and ragged ones."""
    values, table, kw = _table(fmt, 400, D, D)
    tokens = torch.randint(-5, 405, (T,), generator=_gen(T))
    got = bs.bs_embedding(tokens.to(DEV), table, alpha=1.7, out_dtype=out_dtype, **kw)
    assert same(got, torch.from_numpy(ref.lookup(tokens.numpy(), values, 1.7)).to(out_dtype))


@pytest.mark.parametrize("T", [0, 1, 2, 255, 4097])
def test_lookup_lengths_and_shapes(T):
    values, table, kw = _table("int4", 300, 96, 2)
    tokens = torch.randint(-3, 303, (T,), generator=_gen(T))
    want = torch.from_numpy(ref.lookup(tokens.numpy(), values, 3.0)).to(BF)
    assert same(bs.bs_embedding(tokens.to(DEV), table, alpha=3.0, **kw), want)
    if T == 4097:
        t2 = tokens[:4096].view(8, 512).to(DEV)
        assert same(bs.bs_embedding(t2, table, alpha=3.0, **kw), want[:4096].view(8, 512, 96))
        assert same(bs.bs_embedding(t2.t(), table, alpha=3.0, **kw), want[:4096].view(8, 512, 96).transpose(0, 1).contiguous())


def test_lookup_views_and_untouched_output():
    V, D = 40, 130
    g = _gen(6)
    for off in (0, 1, 3):  # rows that do not start on 16-byte boundaries
        big = torch.randn(V, D + 11, generator=g).to(BF).to(DEV)
        table = big[:, off:off + D]
        tokens = torch.tensor([39, 0, 17, 40, 17])
        out = torch.full((7, D + 6), 5.0, dtype=BF, device=DEV)
        view = out[1:6, off:off + D]
        bs.bs_embedding(tokens.to(DEV), table, alpha=2.0, out=view)
        assert same(view, torch.from_numpy(ref.lookup(tokens.numpy(), table.float().cpu().numpy(), 2.0)).to(BF))
        out[1:6, off:off + D] = 5
        assert torch.all(out == 5)


def test_lookup_empty_table_and_single_row():
    tokens = torch.tensor([0, -1, 1], device=DEV)
    assert torch.all(bs.bs_embedding(tokens, torch.empty(0, 16, device=DEV), out_dtype=F) == 0)
    one = torch.randn(1, 16, device=DEV)
    got = bs.bs_embedding(tokens, one, out_dtype=F)
    assert same(got[0], one[0]) and torch.all(got[1:] == 0)
    assert bs.bs_embedding(tokens, torch.empty(5, 0, device=DEV)).shape == (3, 0)


def test_lookup_e8m0_scale_bytes_at_their_ends():
    """Byte 0 is 2^-127, byte 254 2^127 and byte 255 NaN, whatever the codes it scales."""
    V, D = 4, 256
    codes = torch.randint(0, 127, (V, D), generator=_gen(12), dtype=torch.uint8)
    codes[:, ::5] = 0
    scale = torch.tensor([[0, 1], [254, 127], [255, 127], [127, 255]], dtype=torch.uint8)
    factor = torch.tensor([[2.0**-127, 2.0**-126], [2.0**127, 1], [float("nan"), 1], [1, float("nan")]])
    want = torch.from_numpy(oracle.e4m3_table()[codes.numpy()].astype(np.float32)) * factor.repeat_interleave(128, 1)
    for out_dtype in (BF, F):
        got = bs.bs_embedding(torch.arange(V, device=DEV), codes.to(DEV), scale.to(DEV), format="e4m3", out_dtype=out_dtype)
        # (compared as numbers: the bits of a NaN are not specified)
        assert np.array_equal(got.float().cpu().numpy(), want.to(out_dtype).float().numpy(), equal_nan=True)


# ---------------------------------------------------------------------------
# gradient
# ---------------------------------------------------------------------------
def _grad_check(tokens, grad, V, alpha=1.0, padding_idx=None, out_dtype=F, grad_dev=None, base=None):
    kw = {}
    if base is not None:
        kw = {"out": base.clone(), "accumulate": True}
    d = bs.bs_embedding_grad(tokens.to(DEV), grad.to(DEV) if grad_dev is None else grad_dev, V, alpha=alpha,
                             padding_idx=padding_idx, out_dtype=out_dtype, **kw)
    D = grad.shape[-1]
    want, S, n = ref.lookup_grad(tokens.reshape(-1).numpy(), grad.double().reshape(-1, D).numpy(), V, alpha, padding_idx)
    got = d.double().cpu().numpy()
    if base is not None:
        b = base.double().cpu().numpy()
        assert same(d.cpu()[n == 0], base.cpu()[n == 0])  # rows without a token stay as they are
        want, S, n = want + b, S + np.abs(b), n + 1
    else:
        assert np.all(got[n == 0] == 0)
    # n - 1 additions, the factor and (accumulating) one more addition, each half a unit of the last place
    tol = (n[:, None] + 1) * 2.0**-24 * S + _eps(out_dtype) * np.abs(want)
    bad = np.abs(got - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])
    return d


@pytest.mark.parametrize("grad_dtype,out_dtype", [(BF, F), (F, F), (BF, BF), (F, BF)])
@pytest.mark.parametrize("T,V,D", [(1, 1, 1), (31, 10, 7), (32, 10, 8), (33, 3, 64), (64, 1, 100), (65, 40, 33), (255, 7168, 101),
                                   (1000, 256, 264), (4096, 255, 16), (5000, 70000, 40), (513, 20, 2056),
                                   (512, 300, 130), (513, 300, 130), (512, 1, 20), (513, 1, 20), (1500, 511, 9),
                                   (4096, 700, 30), (4097, 700, 30), (2100, 20_000_000, 1),
                                   (1500, 512, 2050), (20000, 300000, 4)])
def test_gradient(T, V, D, grad_dtype, out_dtype):
    g = _gen(T + V + D)
    # the frequencies of text, and tokens outside the table among them
    tokens = (torch.pow(float(V), torch.rand(T, generator=g)).long() * 7) % V
    tokens[torch.rand(T, generator=g) < 0.05] = -1
    tokens[torch.rand(T, generator=g) < 0.05] = V
    grad = torch.randn(T, D, generator=g).to(grad_dtype)
    _grad_check(tokens, grad, V, 1.0, None, out_dtype)
    _grad_check(tokens.int(), grad, V, float(D) ** 0.5, V // 2, out_dtype)
    _grad_check(tokens, grad, V, 0.25, 0, out_dtype, base=torch.randn(V, D, generator=g).to(out_dtype).to(DEV))


@pytest.mark.parametrize("T", [1, 31, 32, 33, 63, 64, 65, 96, 97, 511, 512, 513, 544, 545, 2048, 2049, 4096, 4097, 20000])
def test_gradient_one_row_takes_all(T):
    """A single row named by every token, at the ends of the table and among others."""
    D, V = 24, 1000
    grad = torch.randn(T, D, generator=_gen(T))
    for row in (0, 517, 999):
        _grad_check(torch.full((T,), row), grad, V)
    tokens = torch.full((T,), 517)
    tokens[::3] = torch.arange(len(tokens[::3])) % V
    _grad_check(tokens, grad, V)


def test_gradient_no_token_counts():
    grad = torch.randn(50, 16, generator=_gen(1))
    for tokens in (torch.full((50,), -1), torch.full((50,), 9), torch.full((50,), 2**40), torch.full((50,), 4)):
        d = bs.bs_embedding_grad(tokens.to(DEV), grad.to(DEV), 9, padding_idx=4)
        assert d.shape == (9, 16) and torch.all(d == 0)
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    assert torch.all(bs.bs_embedding_grad(none, torch.empty(0, 16, device=DEV), 9) == 0)
    keep = torch.randn(9, 16, device=DEV)
    assert same(bs.bs_embedding_grad(none, torch.empty(0, 16, device=DEV), 9, out=keep.clone(), accumulate=True), keep)
    assert bs.bs_embedding_grad(none, torch.empty(0, 0, device=DEV), 9).shape == (9, 0)


def test_gradient_is_deterministic_and_ordered():
    """The same bits on every run, and the bits of adding each chunk of 32 sorted tokens in order."""
    T, V, D = 3000, 12, 72
    g = _gen(8)
    tokens = torch.randint(0, V, (T,), generator=g)
    grad = torch.randn(T, D, generator=g)
    first = bs.bs_embedding_grad(tokens.to(DEV), grad.to(DEV), V)
    for _ in range(5):
        assert same(first, bs.bs_embedding_grad(tokens.to(DEV), grad.to(DEV), V))
    order = torch.argsort(tokens, stable=True)
    want = torch.zeros(V, D)
    parts: dict = {}
    for i, t in enumerate(order.tolist()):
        key = (int(tokens[t]), i // 32)
        parts[key] = parts[key] + grad[t] if key in parts else grad[t].clone()
    for (v, _), p in sorted(parts.items()):
        want[v] = want[v] + p
    assert same(first, want)


def test_gradient_is_the_lookup_s_derivative():
    """Differences of a loss through the lookup: with small integers every number is exact."""
    V, D, T = 6, 9, 40
    rng = np.random.default_rng(1)
    tokens = torch.from_numpy(rng.integers(-1, V + 1, T)).to(DEV)
    c = torch.from_numpy(rng.integers(-4, 5, (T, D))).float().to(DEV)
    table = torch.from_numpy(rng.integers(-4, 5, (V, D))).float().to(DEV)
    d = bs.bs_embedding_grad(tokens, c, V, alpha=2.0)
    loss = lambda t: float((bs.bs_embedding(tokens, t, alpha=2.0, out_dtype=F) * c).double().sum())  # noqa: E731
    for v in range(V):
        for j in range(D):
            up, down = table.clone(), table.clone()
            up[v, j] += 1
            down[v, j] -= 1
            assert (loss(up) - loss(down)) / 2 == float(d[v, j])


def test_gradient_views_and_untouched_output():
    T, V, D = 77, 30, 45
    g = _gen(3)
    big = torch.randn(T, D + 7, generator=g).to(DEV)
    tokens = torch.randint(0, V, (7, 11), generator=g)
    grad = big[:, 2:2 + D]
    canvas = torch.full((V + 2, D + 5), 4.0, device=DEV)
    view = canvas[1:1 + V, 3:3 + D]
    d = bs.bs_embedding_grad(tokens.view(-1).to(DEV), grad, V, out=view)
    assert d.data_ptr() == view.data_ptr()
    assert same(view, _grad_check(tokens.view(-1), grad.cpu(), V))
    canvas[1:1 + V, 3:3 + D] = 4
    assert torch.all(canvas == 4)
    g3 = big[:, :D].contiguous().view(7, 11, D)
    assert same(_grad_check(tokens, g3.cpu(), V), _grad_check(tokens.view(-1), big[:, :D].cpu(), V))
    # tokens read column-wise: every other element of a wider tensor
    wide = torch.stack([tokens.view(-1), tokens.view(-1) * 0 - 1], 1).to(DEV)
    assert same(bs.bs_embedding_grad(wide[:, 0], g3.view(-1, D), V), _grad_check(tokens.view(-1), g3.cpu().view(-1, D), V))


def test_gradient_non_finite_values_stay_in_their_row():
    tokens = torch.tensor([1, 2, 1, 3, 2] * 20)
    grad = torch.randn(100, 16, generator=_gen(5))
    base = bs.bs_embedding_grad(tokens.to(DEV), grad.to(DEV), 5)
    grad[7, 3] = float("inf")  # token 1
    d = bs.bs_embedding_grad(tokens.to(DEV), grad.to(DEV), 5)
    keep = torch.ones(5, 16, dtype=torch.bool)
    keep[tokens[7], 3] = False
    assert torch.equal(d.cpu()[keep], base.cpu()[keep]) and torch.isinf(d[tokens[7], 3])
    # a token that does not count hides what its row holds
    tokens[7] = 4
    grad[7] = float("nan")
    assert not torch.isnan(bs.bs_embedding_grad(tokens.to(DEV), grad.to(DEV), 5, padding_idx=4)).any()


# ---------------------------------------------------------------------------
# far offsets, streams, graphs, threads, and the operators together
# ---------------------------------------------------------------------------
@pytest.mark.slow
def test_offsets_past_32_bits():
    V, D = 270000, 8192  # 2.2e9 elements: the last rows lie past 2^31 elements and 2^32 bytes
    table = torch.zeros(V, D, dtype=BF, device=DEV)
    table[-3:] = torch.randn(3, D, device=DEV).to(BF)
    tokens = torch.tensor([V - 1, V - 3, 0, V - 2, V - 1], device=DEV)
    out = bs.bs_embedding(tokens, table, alpha=2.0)
    assert same(out, (table[tokens].float() * 2).to(BF))
    del table
    grad = torch.randn(5, D, device=DEV)
    d = torch.full((V, D), 3.0, device=DEV)
    bs.bs_embedding_grad(tokens, grad, V, out=d)
    assert same(d[V - 1], grad[0] + grad[4]) and same(d[V - 3], grad[1]) and same(d[V - 2], grad[3]) and same(d[0], grad[2])
    assert int(torch.count_nonzero(d[1:V - 3].view(-1)[:2**30])) == 0 and int(torch.count_nonzero(d[V - 1000:V - 3])) == 0


@pytest.mark.slow
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("T", [5, 700, 9000])
def test_gradient_offsets_past_32_bits_in_every_row(T, accumulate):
    """A gradient of 2.2e9 elements by each of the three sorts, every row looked at: small integers, so that sums are exact,
    and tokens on both sides of 2^31 elements, the last rows named by more than a chunk of them."""
    V, D = 270000, 8192
    g = _gen(T)
    tokens = torch.randint(0, V, (T,), generator=g)
    near = torch.tensor([V - 1, V - 3, 0, V - 2, V - 1, 2**18 - 1, 2**18])  # row 2^18 begins at element 2^31
    tokens[::2] = near[torch.randint(0, len(near), (len(tokens[::2]),), generator=g)]
    tokens = tokens.to(DEV)
    grad = torch.randint(-8, 9, (T, D), generator=g).float().to(DEV)
    d = torch.full((V, D), 3.0, device=DEV)
    bs.bs_embedding_grad(tokens, grad, V, out=d, accumulate=accumulate)
    rows, place = torch.unique(tokens, return_inverse=True)
    sums = torch.zeros(len(rows), D, device=DEV).index_add_(0, place, grad)
    rest = 3.0 if accumulate else 0.0
    for r, want in zip(rows.tolist(), sums + rest):
        assert torch.equal(d[r], want), r
        d[r] = rest
    for lo in range(0, V, 16384):
        assert torch.all(d[lo:lo + 16384] == rest), lo


@pytest.mark.slow
def test_lookup_output_past_32_bits():
    T, V, D = 270000, 50, 8192  # 2.2e9 elements of output
    tokens = torch.randint(-1, V + 1, (T,), generator=_gen(1)).to(DEV)
    for fmt in ("bf16", "int4"):
        values, table, kw = _table(fmt, V, D, 3)
        want = torch.cat([torch.from_numpy(values).to(BF), torch.zeros(1, D, dtype=BF)]).to(DEV)
        row = torch.where((tokens >= 0) & (tokens < V), tokens, V)
        out = bs.bs_embedding(tokens, table, **kw)
        for lo in range(0, T, 16384):
            assert torch.equal(out[lo:lo + 16384], want[row[lo:lo + 16384]]), (fmt, lo)
        del out


@pytest.mark.slow
@pytest.mark.parametrize("N,M", [(2200, 32), (5000, 9)])
def test_wide_row_strides_past_32_bits(N, M):
    """Inputs and outputs whose rows lie so far apart that the last ones are past 2^32 bytes, against dense ones: the
    quantiser, the dequantiser, the lookup and the product (both sizes of its row tiles)."""
    K, group = 260, 32
    G = -(-K // group)

    def far(rows, cols, dtype, like=None):
        ld = -(-(2**32 // dtype.itemsize) // (rows - 1) // 64) * 64 + 256  # the last row begins past 2^32 bytes
        t = torch.empty(rows * ld, dtype=dtype, device=DEV).view(rows, ld)[:, 5 * 16 // dtype.itemsize:][:, :cols]
        assert (rows - 1) * ld * dtype.itemsize > 2**32
        return t if like is None else t.copy_(like)

    x = _weights(N, K, 3).to(DEV)
    near = bs.bs_quantize_int4(x, group=group, asymmetric=True)
    q, s, z = bs.bs_quantize_int4(far(N, K, BF, x), group=group, asymmetric=True, q=far(N, K // 2, torch.uint8),
                                  scale=far(N, G, F), zero=far(N, G, torch.uint8))
    for a, b in zip((q, s, z), near):
        assert same(a, b)
    dense = bs.bs_dequantize_int4(*near, group=group)
    assert same(bs.bs_dequantize_int4(q, s, z, group=group, out=far(N, K, BF)), dense)
    tokens = torch.arange(N - 1, -1, -1, device=DEV)
    assert same(bs.bs_embedding(tokens, q, s, z, format="int4", group=group, out=far(N, K, BF)), dense.flip(0))
    act = torch.randn(M, K, generator=_gen(4)).to(BF).to(DEV)
    want = bs.bs_gemv_int4(act, *near, group=group)
    assert same(bs.bs_gemv_int4(far(M, K, BF, act), q, s, z, group=group, out=far(M, N, BF)), want)


@pytest.mark.slow
@pytest.mark.parametrize("T", [300, 1000, 5000])
def test_gradient_of_a_very_long_table(T):
    """More rows than a CTA marks at a time; small integers, so that every sum is exact."""
    V, D = 90_000_001, 2
    g = _gen(T)
    tokens = torch.randint(0, V, (T,), generator=g)
    tokens[::7] = V - 1
    tokens[1::7] = 0
    grad = torch.randint(-8, 9, (T, D), generator=g).float()
    d = torch.full((V, D), 5.0, device=DEV)
    bs.bs_embedding_grad(tokens.to(DEV), grad.to(DEV), V, out=d)
    want = torch.zeros(V, D, device=DEV).index_add_(0, tokens.to(DEV), grad.to(DEV))
    assert torch.equal(d, want)


def test_other_stream_and_threads():
    host, dev = _matrix(300, 512, 64, 21)
    x = torch.randn(4, 512, generator=_gen(1)).to(DEV)
    tokens = torch.randint(0, 300, (5000,), generator=_gen(2)).to(DEV)
    grad = torch.randn(5000, 64, generator=_gen(3)).to(DEV)
    want = (bs.bs_gemv_int4(x, *dev, group=64, out_dtype=F), bs.bs_embedding_grad(tokens, grad, 300))
    torch.cuda.synchronize()
    errors = []

    def work():
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    y, d = bs.bs_gemv_int4(x, *dev, group=64, out_dtype=F), bs.bs_embedding_grad(tokens, grad, 300)
            stream.synchronize()
            assert same(y, want[0]) and same(d, want[1])
        except Exception as e:  # noqa: BLE001 - reported below
            errors.append(e)

    threads = [threading.Thread(target=work) for _ in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors, errors


def test_captured_graphs_replayed_on_new_inputs():
    """Two graphs of all five operators, captured one after the other and replayed in turn on inputs that change."""
    V, D, T, group = 64, 128, 1200, 32
    w = torch.randn(V, D, generator=_gen(1)).to(DEV)
    tokens = [torch.randint(0, V, (T,), generator=_gen(i)).to(DEV) for i in (2, 3)]

    def step(w, tokens):
        q, s, z = bs.bs_quantize_int4(w, group=group, asymmetric=True)
        rows = bs.bs_embedding(tokens, q, s, z, format="int4", group=group, out_dtype=F)
        y = bs.bs_gemv_int4(rows[:16], q, s, z, group=group, out_dtype=F)
        return rows, y, bs.bs_dequantize_int4(q, s, z, group=group), bs.bs_embedding_grad(tokens, rows, V)

    step(w, tokens[0])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for t in tokens:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(w, t))
        graphs.append(g)
    for round_ in range(3):
        w.copy_(torch.randn(V, D, generator=_gen(10 + round_)))
        tokens[0].copy_(torch.randint(0, V, (T,), generator=_gen(20 + round_)))
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        for t, out in zip(tokens, outs):
            for a, b in zip(out, step(w, t)):
                assert same(a, b)


def test_a_tied_4bit_table_serves_lookup_and_head():
    """Decoding with one 4-bit table: the rows of the last tokens, and the logits of the head that shares it."""
    V, D, group = 1003, 320, 64
    w = _weights(V, D, 31)
    q, s, z = bs.bs_quantize_int4(w.to(DEV), group=group, scale_dtype=BF, asymmetric=True)
    codes, scale, zero = ref.quantize_int4(w, group, True, True)
    tokens = torch.tensor([7, 1002, 0, 7, 500])
    h = bs.bs_embedding(tokens.to(DEV), q, s, z, format="int4", group=group, alpha=D ** 0.5)
    values = ref.values(codes, scale, zero, group)
    assert same(h, torch.from_numpy(ref.lookup(tokens.numpy(), values, D ** 0.5)).to(BF))
    _product_check(h.cpu(), (codes, scale, zero), (q, s, z), group, F)


def test_embedding_into_an_fp8_layer_and_back():
    """A training step's ends: lookup, the FP8 quantisers and GEMM of the next layer, and the table's gradient from the
    layer's input gradient; the gradient of the loss sum(y * r) in the table, against the definition in 64 bits."""
    V, D, N, T = 200, 256, 384, 256
    g = _gen(41)
    table = torch.randn(V, D, generator=g).to(BF).to(DEV)
    w = (torch.randn(N, D, generator=g) * 0.05).to(BF).to(DEV)
    r = torch.randn(T, N, generator=g).to(BF).to(DEV)
    tokens = torch.randint(0, V, (T,), generator=g)
    x = bs.bs_embedding(tokens.to(DEV), table, alpha=2.0)
    qx, sx = bs.bs_quantize_fp8_1x128(x)
    qw, sw = bs.bs_quantize_fp8_128x128(w)
    y = bs.bs_gemm_fp8_blockwise(qx, qw.t(), sx, sw)
    assert y.shape == (T, N) and torch.isfinite(y).all()
    # dx = r W, from the transposed weight codes
    qr, sr = bs.bs_quantize_fp8_1x128(r)
    qwt, swt = bs.bs_quantize_fp8_t(w, "128x128")
    dx = bs.bs_gemm_fp8_blockwise(qr, qwt.t(), sr, swt, out_dtype=F)
    d = _grad_check(tokens, dx.cpu(), V, alpha=2.0, grad_dev=dx)
    # and the whole chain against bf16's own product: e4m3 rounds each factor by at most 2^-4 of it
    exact = r.double().cpu() @ w.double().cpu()
    bound = r.double().abs().cpu() @ w.double().abs().cpu()
    dw, S, _ = ref.lookup_grad(tokens.numpy(), exact.numpy(), V, 2.0)
    _, S, _ = ref.lookup_grad(tokens.numpy(), bound.numpy(), V, 2.0)
    # a factor below the smallest normal code is off by at most half the smallest step of its group, 2^-10 of 448 / amax
    slack = 2 * (2.0**-4) + 2.0**-8
    assert np.all(np.abs(d.cpu().numpy() - dw) <= slack * S + 1e-2 * S.max() * 2.0**-8)
