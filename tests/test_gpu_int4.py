"""GPU parity of the 4-bit weight operators: codes, scales, zero points and values bit for bit
against the oracle, the linear layer against fp64 products."""
import numpy as np
import pytest
import torch

import oracle
from oracle import serving as osv
from w8a8_quantized_gemm_b200 import sq
from w8a8_quantized_gemm_b200 import workloads as wl

from _gpu import dev_bf16, empty, host, host_bits

pytestmark = pytest.mark.gpu

# rows of one tile and of many, a half tile, columns of a short last tile and a short last group
SHAPES = [(8, 16), (16, 32), (24, 80), (40, 272), (256, 256), (328, 1040), (128, 4096)]


def _weight(N, K, seed):
    rng = np.random.default_rng(seed)
    w = rng.normal(0, 0.02, (N, K)).astype(np.float32)
    w[0, :] = 0                       # groups of zeros
    w[1, :] = np.abs(w[1, :])         # one sign only
    w[2, :] = -np.abs(w[2, :])
    w[3, :] = 0.25                    # constant
    w[4, K // 2] = 30.0               # one outlier
    w[5, :] *= 1e-38                  # subnormal scales
    return wl.f32_to_bf16_bits(w)


def _smooth(K, seed):
    return np.random.default_rng(seed).uniform(0.1, 4.0, K).astype(np.float32)


def _packed(N, K, group, asym):
    G = -(-K // group)
    return (torch.full((sq.sq_int4_weight_bytes(N, K),), 0x5A, dtype=torch.uint8, device="cuda"),
            torch.full((G, N), 7.0, dtype=torch.bfloat16, device="cuda"),
            torch.full((G, N), 99, dtype=torch.uint8, device="cuda") if asym else None)


def _up(codes, scale, zero, asym):
    return (torch.from_numpy(osv.int4_pack(codes)).cuda(), dev_bf16(scale),
            torch.from_numpy(zero).cuda() if asym else None)


@pytest.mark.parametrize("asym", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,K", SHAPES)
def test_quant_and_dequant_exact(N, K, group, asym):
    W = _weight(N, K, N + K)
    s = _smooth(K, K)
    for smooth in (None, s):
        Wp, e, z = _packed(N, K, group, asym)
        sq.sq_quant_weight_int4(dev_bf16(W), None if smooth is None else torch.from_numpy(smooth).cuda(), group, Wp, e, z)
        out = empty((N, K), torch.bfloat16)
        sq.sq_dequant_weight_int4(Wp, e, z, group, out)
        sq.sq_sync_status()
        codes, scale, zero = osv.int4_quant(W, smooth, group, asym)
        assert np.array_equal(host(Wp), osv.int4_pack(codes))
        assert np.array_equal(host_bits(e), scale)
        if asym:
            assert np.array_equal(host(z), zero)
        # (code - zero) * scale has at most 13 significant bits: one rounding to bf16
        values = osv.int4_values(codes, scale, zero, group).astype(np.float32)
        assert np.array_equal(host_bits(out), oracle.float_to_bf16(values))


def test_quant_reads_a_column_slice():
    W = _weight(24, 512, 3)
    Wp, e, _ = _packed(24, 272, 64, False)
    sq.sq_quant_weight_int4(dev_bf16(W)[:, 128:400], None, 64, Wp, e)
    codes, scale, _ = osv.int4_quant(W[:, 128:400], None, 64, False)
    assert np.array_equal(host(Wp), osv.int4_pack(codes)) and np.array_equal(host_bits(e), scale)


def _codes(N, K, group, asym, seed):
    rng = np.random.default_rng(seed)
    G = -(-K // group)
    scale = oracle.float_to_bf16(rng.uniform(0.002, 0.02, (G, N)).astype(np.float32))
    zero = rng.integers(0, 16, (G, N), dtype=np.uint8) if asym else np.full((G, N), 8, np.uint8)
    return rng.integers(0, 16, (N, K), dtype=np.uint8), scale, zero


def _check_linear(Y, y, absum, K):
    """|Y - y| <= 2^-8 |y| (half a step of bf16) + the fp32 sums: products are exact, and each of
    the at most K / 16 + K / 32 + 16 additions in a row (16 columns a step, group sums, joined
    parts, bias) rounds or truncates by at most 2^-22 of the largest partial sum. Results below the
    normal range (rows of subnormal scales) are rounded to multiples of bf16's smallest subnormal
    2^-133, off by at most half of it whatever their size, and the fp32 sums by 2^-150 a step:
    2^-133 covers both."""
    err = np.abs(wl.bf16_bits_to_f32(host_bits(Y)).astype(np.float64) - y)
    bound = 2.0 ** -8 * np.abs(y) + (K / 16 + K / 32 + 16) * 2.0 ** -22 * (absum + np.abs(y)) + 2.0 ** -133
    assert np.all(err <= bound), float((err / bound).max())


LINEAR = [(1, 8, 16, 32), (1, 16, 128, 128), (2, 24, 80, 32), (3, 40, 272, 64), (5, 256, 256, 128), (7, 328, 1040, 64),
          (8, 136, 4096, 128), (9, 64, 528, 32), (13, 200, 2064, 128), (16, 512, 1024, 32), (17, 72, 400, 64),
          (31, 128, 3088, 128), (32, 264, 512, 64), (33, 96, 144, 32), (48, 1024, 256, 128), (63, 24, 4112, 64),
          (64, 528, 1296, 128), (1, 8, 65536, 128), (20, 16, 28672, 32)]


@pytest.mark.parametrize("asym", [False, True])
@pytest.mark.parametrize("M,N,K,group", LINEAR)
def test_linear_against_fp64(M, N, K, group, asym):
    codes, scale, zero = _codes(N, K, group, asym, M + N + K)
    rng = np.random.default_rng(K)
    x = rng.normal(0, 1, (M, K)).astype(np.float32)
    x[:, rng.choice(K, 2)] *= 50
    X = wl.f32_to_bf16_bits(x)
    bias = wl.f32_to_bf16_bits(rng.normal(0, 1, N).astype(np.float32)) if (M + N) % 3 else None
    Wp, e, z = _up(codes, scale, zero, asym)
    Y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    sq.sq_int4_linear(dev_bf16(X), Wp, e, z, group, None if bias is None else dev_bf16(bias), Y)
    sq.sq_sync_status()
    y, absum = osv.int4_linear(X, osv.int4_values(codes, scale, zero, group), bias)
    _check_linear(Y, y, absum, K)


@pytest.mark.parametrize("M,N,K", [(4, 5504, 4096), (16, 2048, 8192), (64, 4096, 1024), (1, 11008, 512)])
def test_linear_many_rows(M, N, K):
    """Enough rows for every way the work is split; the same inputs give the same bits."""
    codes, scale, zero = _codes(N, K, 64, True, N)
    X = wl.f32_to_bf16_bits(np.random.default_rng(1).normal(0, 1, (M, K)).astype(np.float32))
    Wp, e, z = _up(codes, scale, zero, True)
    Y, Y2 = empty((M, N), torch.bfloat16), empty((M, N), torch.bfloat16)
    sq.sq_int4_linear(dev_bf16(X), Wp, e, z, 64, None, Y)
    sq.sq_int4_linear(dev_bf16(X), Wp, e, z, 64, None, Y2)
    sq.sq_sync_status()
    y, absum = osv.int4_linear(X, osv.int4_values(codes, scale, zero, 64), None)
    _check_linear(Y, y, absum, K)
    assert torch.equal(Y, Y2)


@pytest.mark.parametrize("M", [3, 4, 9, 16, 17, 40])
def test_linear_nonfinite_tokens_stay_to_themselves(M):
    """A token with a NaN gives NaN, one with an infinity nothing finite that its weight does not
    hide (a code equal to its zero point makes NaN); the other tokens' results are as ever."""
    N, K, group = 48, 400, 64
    codes, scale, zero = _codes(N, K, group, True, M)
    x = np.random.default_rng(M).normal(0, 1, (M, K)).astype(np.float32)
    x[1, 7], x[M - 1, K - 1] = np.nan, -np.inf
    X = wl.f32_to_bf16_bits(x)
    X[1, 7], X[M - 1, K - 1] = 0x7FC0, 0xFF80
    Wp, e, z = _up(codes, scale, zero, True)
    Y = empty((M, N), torch.bfloat16)
    sq.sq_int4_linear(dev_bf16(X), Wp, e, z, group, None, Y)
    sq.sq_sync_status()
    rest = [m for m in range(M) if m not in (1, M - 1)]
    y, absum = osv.int4_linear(X[rest], osv.int4_values(codes, scale, zero, group), None)
    _check_linear(Y[rest], y, absum, K)
    assert bool(torch.isnan(Y[1]).all()) and not bool(torch.isfinite(Y[M - 1]).any())


@pytest.mark.parametrize("M,N,K,group", [(1, 2848, 4128, 128), (2, 2856, 23552, 32), (3, 9480, 1168, 64),
                                         (4, 9480, 13312, 128), (13, 3016, 27872, 64), (16, 4104, 4112, 128),
                                         (38, 4664, 3696, 32), (25, 344, 16704, 64), (64, 1032, 8208, 64),
                                         (18, 4824, 4112, 64), (63, 2040, 12304, 128), (33, 3320, 8192, 32),
                                         (40, 2568, 6160, 128), (64, 29000, 400, 64)])
def test_linear_large(M, N, K, group):
    """Many rows, long rows, both: activations that do not fit shared memory at once, clusters that
    do not all run at once. Every byte is a pair of codes, so the codes are random bytes and their
    integer values come from the (tested) values call with scales of one."""
    G = -(-K // group)
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    Wp = torch.randint(0, 256, (sq.sq_int4_weight_bytes(N, K),), dtype=torch.uint8, device="cuda", generator=gen)
    z = torch.randint(0, 16, (G, N), dtype=torch.uint8, device="cuda", generator=gen)
    e = (torch.rand((G, N), device="cuda", generator=gen) * 0.02 + 0.002).to(torch.bfloat16)
    X = torch.randn((M, K), device="cuda", generator=gen).to(torch.bfloat16)
    codes = empty((N, K), torch.bfloat16)
    sq.sq_dequant_weight_int4(Wp, torch.ones_like(e), z, group, codes)
    values = codes.double() * e.double().t().repeat_interleave(group, 1)[:, :K]
    Y = empty((M, N), torch.bfloat16)
    sq.sq_int4_linear(X, Wp, e, z, group, None, Y)
    sq.sq_sync_status()
    y = (X.double() @ values.t()).cpu().numpy()
    absum = (X.double().abs() @ values.abs().t()).cpu().numpy()
    _check_linear(Y, y, absum, K)


def test_linear_strided_tokens_neighbours_untouched():
    """Tokens read through a wider leading dimension; rows around Y stay as they were."""
    codes, scale, zero = _codes(48, 272, 128, False, 4)
    x = np.random.default_rng(4).normal(0, 1, (5, 400)).astype(np.float32)
    x[:, 272:] = np.nan  # what lies behind a row is never read into a sum
    X = dev_bf16(wl.f32_to_bf16_bits(np.nan_to_num(x)))
    X[:, 272:] = float("nan")
    Wp, e, _ = _up(codes, scale, zero, False)
    buf = torch.full((7, 48), 3.0, dtype=torch.bfloat16, device="cuda")
    sq.sq_int4_linear(X[:, :272], Wp, e, None, 128, None, buf[1:6])
    sq.sq_sync_status()
    y, absum = osv.int4_linear(host_bits(X[:, :272].contiguous()), osv.int4_values(codes, scale, zero, 128), None)
    _check_linear(buf[1:6], y, absum, 272)
    assert bool((buf[0] == 3).all()) and bool((buf[6] == 3).all())


def test_linear_on_a_side_stream_and_in_a_graph():
    codes, scale, zero = _codes(256, 1024, 128, False, 9)
    Wp, e, _ = _up(codes, scale, zero, False)
    rng = np.random.default_rng(0)
    X = dev_bf16(wl.f32_to_bf16_bits(rng.normal(0, 1, (3, 1024)).astype(np.float32)))
    Y, Yg = empty((3, 256), torch.bfloat16), empty((3, 256), torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    sq.sq_int4_linear(X, Wp, e, None, 128, None, Y, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sq.sq_int4_linear(X, Wp, e, None, 128, None, Yg)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(Y, Yg)
    X.copy_(dev_bf16(wl.f32_to_bf16_bits(rng.normal(0, 1, (3, 1024)).astype(np.float32))))
    graph.replay()
    sq.sq_int4_linear(X, Wp, e, None, 128, None, Y)
    sq.sq_sync_status()
    assert torch.equal(Y, Yg)


def test_quantized_weight_through_the_linear():
    """Smoothing, quantization and product together: the smoothed activations times the quantized
    weight differ from the full product by the weight's rounding only."""
    N, K, M, group = 256, 1024, 8, 64
    W, s = _weight(N, K, 8), _smooth(K, 8)
    x = np.random.default_rng(8).normal(0, 1, (M, K)).astype(np.float32)
    X = wl.f32_to_bf16_bits(x / s)
    for asym in (False, True):
        Wp, e, z = _packed(N, K, group, asym)
        sq.sq_quant_weight_int4(dev_bf16(W), torch.from_numpy(s).cuda(), group, Wp, e, z)
        Y = empty((M, N), torch.bfloat16)
        sq.sq_int4_linear(dev_bf16(X), Wp, e, z, group, None, Y)
        sq.sq_sync_status()
        values = osv.int4_values(*osv.int4_quant(W, s, group, asym), group)
        y, absum = osv.int4_linear(X, values, None)
        _check_linear(Y, y, absum, K)


def test_binding_refusals():
    Wp, e, z = _packed(16, 128, 64, True)
    X, Y = empty((2, 128), torch.bfloat16), empty((2, 16), torch.bfloat16)
    for args, err in (((X, Wp[:-1], e, z, 64, None, Y), ValueError), ((X, Wp, e[:1], z, 64, None, Y), ValueError),
                      ((X, Wp, e.float(), z, 64, None, Y), TypeError), ((X.float(), Wp, e, z, 64, None, Y), TypeError),
                      ((X, Wp, e, z, 64, None, Y.t()), (ValueError, sq.SqError)), ((X.t(), Wp, e, z, 64, None, Y), ValueError),
                      ((X, Wp, e, z, 0, None, Y), ValueError), ((X, Wp, e, z, 64, e[0, :8], Y), ValueError)):
        with pytest.raises(err):
            sq.sq_int4_linear(*args)
    big = empty((65, 128), torch.bfloat16)
    with pytest.raises(sq.SqError):
        sq.sq_int4_linear(big, Wp, e, z, 64, None, empty((65, 16), torch.bfloat16))
