"""The 4-bit linear layer of up to 4 tokens on the int8 instructions, which take a token as integers
of 23 bits and a power of two: weights with rows enough that this kernel takes them."""
import numpy as np
import pytest
import torch

import oracle
from oracle import serving as osv
from w8a8_quantized_gemm_b200 import sq
from w8a8_quantized_gemm_b200 import workloads as wl

from _gpu import dev_bf16, empty, host_bits

pytestmark = pytest.mark.gpu


def _rows(M, more=0):
    """Weight rows from which on the int8 instructions are used: 1.2 row tiles of 16 an SM for one and two
    tokens, 4 for three and four."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return 16 * (-(-6 * sms // 5) if M <= 2 else 4 * sms) + more


def _weight(N, K, group, asym, seed, low=0.002, high=0.02):
    rng = np.random.default_rng(seed)
    G = -(-K // group)
    scale = oracle.float_to_bf16(rng.uniform(low, high, (G, N)).astype(np.float32))
    zero = rng.integers(0, 16, (G, N), dtype=np.uint8) if asym else np.full((G, N), 8, np.uint8)
    codes = rng.integers(0, 16, (N, K), dtype=np.uint8)
    up = (torch.from_numpy(osv.int4_pack(codes)).cuda(), dev_bf16(scale), torch.from_numpy(zero).cuda() if asym else None)
    return up, osv.int4_values(codes, scale, zero, group)


def _run(X, weight, group, bias, N, stream=None):
    Y = torch.full((X.shape[0], N), float("nan"), dtype=torch.bfloat16, device="cuda")
    sq.sq_int4_linear(X, *weight, group, bias, Y, stream=stream)
    return Y


def _check(Y, X, values, bias):
    """Half a step of bf16 (2^-8 of the result, 2^-134 where it is subnormal, another 2^-134 for the two
    powers of two), half a unit of each element's integer (2^-22 of its token's largest, for
    elements below 2^-14 of that), and the fp32 sums: exact integers within a group, then at most
    K / 32 + 32 additions in a row (groups, warps, digits, bias) at 2^-23 of the sum of absolute
    products, whose three digits' parts are at most 3 times that."""
    y, absum = osv.int4_linear(X, values, bias)
    x = np.abs(wl.bf16_bits_to_f32(X).astype(np.float64))
    top = x.max(1, keepdims=True)
    unit = np.where(x < 2.0 ** -14 * top, 2.0 ** -22 * top, 0.0) @ np.abs(values).T
    K = X.shape[1]
    err = np.abs(wl.bf16_bits_to_f32(host_bits(Y)).astype(np.float64) - y)
    bound = 2.0 ** -8 * np.abs(y) + 2.0 ** -133 + (unit + 3 * (K / 32 + 32) * 2.0 ** -23 * (absum + np.abs(y))) * (1 + 2.0 ** -8)
    assert np.all(err <= bound), float((err / bound).max())


@pytest.mark.parametrize("M", [1, 2, 4])
def test_tiny_tokens(M):
    """Tokens far below and in the subnormal range are integers of as many bits as any other."""
    N, K, group = _rows(M), 144, 64
    weight, values = _weight(N, K, group, False, M, 0.5, 2.0)
    rng = np.random.default_rng(M)
    for p in (-90, -99, -104, -112, -119, -126, -131):
        X = wl.f32_to_bf16_bits((rng.normal(0, 1, (M, K)) * 2.0 ** p).astype(np.float32))
        Y = _run(dev_bf16(X), weight, group, None, N)
        sq.sq_sync_status()
        _check(Y, X, values, None)


@pytest.mark.parametrize("M", [1, 4])
def test_elements_far_below_the_largest(M):
    """Elements of 2^-10 to 2^-26 of their token's largest, of whose weights one in sixteen is zero: only
    the small ones are seen there."""
    N, K, group = _rows(M), 272, 32
    (Wp, e, z), values = _weight(N, K, group, True, 9)
    rng = np.random.default_rng(M)
    x = rng.normal(0, 1, (M, K)) * 2.0 ** rng.uniform(-26, -10, (M, K))
    x[:, 5] = rng.uniform(1, 2, M) * 2.0 ** rng.integers(-60, 60, M)
    X = wl.f32_to_bf16_bits((x * np.where(np.arange(K) == 5, 1, x[:, 5:6])).astype(np.float32))
    Y = _run(dev_bf16(X), (Wp, e, z), group, None, N)
    sq.sq_sync_status()
    _check(Y, X, values, None)


@pytest.mark.parametrize("M", [1, 2, 4])
@pytest.mark.parametrize("scale,token", [(2.0 ** 99, 2.0 ** -60), (2.0 ** 60, 2.0 ** 40), (2.0 ** -120, 2.0 ** -9), (2.0 ** -132, 2.0 ** 30)])
def test_scales_far_from_one(M, scale, token):
    """Scales up to 2^100 and down to bf16's smallest, tokens that bring the results back into range."""
    N, K, group = _rows(M), 1040, 64
    weight, values = _weight(N, K, group, True, M, scale, 1.9 * scale)
    X = wl.f32_to_bf16_bits((np.random.default_rng(M).normal(0, 1, (M, K)) * token).astype(np.float32))
    Y = _run(dev_bf16(X), weight, group, None, N)
    sq.sq_sync_status()
    _check(Y, X, values, None)


@pytest.mark.parametrize("asym", [False, True])
@pytest.mark.parametrize("M,more,K,group", [(1, 0, 144, 32), (1, 8, 1040, 64), (1, 40, 4096, 128), (2, 8, 272, 64),
                                            (2, 0, 2064, 128), (2, 24, 80, 32), (3, 8, 272, 128), (3, 0, 144, 32),
                                            (4, 0, 528, 64), (4, 24, 400, 128), (4, 8, 16, 32)])
def test_against_fp64(M, more, K, group, asym):
    """Codes with and without zero points, bias, columns of outliers, tokens read through a wider row whose
    rest is NaN; half tiles of rows, short last tiles and groups of columns."""
    N = _rows(M, more)
    weight, values = _weight(N, K, group, asym, M + K)
    rng = np.random.default_rng(K)
    x = rng.normal(0, 1, (M, K)).astype(np.float32)
    x[:, rng.choice(K, 2)] *= 60
    X = wl.f32_to_bf16_bits(x)
    bias = wl.f32_to_bf16_bits(rng.normal(0, 1, N).astype(np.float32)) if (K // 16 + M) % 2 else None
    wide = torch.full((M, K + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :K] = dev_bf16(X)
    Y = _run(wide[:, :K], weight, group, None if bias is None else dev_bf16(bias), N)
    Y2 = _run(dev_bf16(X), weight, group, None if bias is None else dev_bf16(bias), N)
    sq.sq_sync_status()
    _check(Y, X, values, bias)
    assert torch.equal(Y, Y2)


@pytest.mark.parametrize("asym", [False, True])
@pytest.mark.parametrize("M,more,K,group", [(1, 0, 65536, 128), (2, 8, 40016, 64), (3, 8, 28672, 128), (4, 8, 20016, 32),
                                            (1, 11008, 4096, 64), (2, 4096, 8192, 32)])
def test_long_rows_and_many_rows(M, more, K, group, asym):
    """Tokens that shared memory does not hold at once, and several row tiles a team."""
    N, G = _rows(M, more), -(-K // group)
    gen = torch.Generator(device="cuda").manual_seed(M + K)
    Wp = torch.randint(0, 256, (sq.sq_int4_weight_bytes(N, K),), dtype=torch.uint8, device="cuda", generator=gen)
    z = torch.randint(0, 16, (G, N), dtype=torch.uint8, device="cuda", generator=gen) if asym else None
    e = (torch.rand((G, N), device="cuda", generator=gen) * 0.02 + 0.002).to(torch.bfloat16)
    X = torch.randn((M, K), device="cuda", generator=gen)
    X[:, torch.randperm(K, device="cuda", generator=gen)[:6]] *= 40
    X = X.to(torch.bfloat16)
    bias = torch.randn(N, device="cuda", generator=gen).to(torch.bfloat16)
    codes = empty((N, K), torch.bfloat16)
    sq.sq_dequant_weight_int4(Wp, torch.ones_like(e), z, group, codes)
    Y = _run(X, (Wp, e, z), group, bias, N)
    sq.sq_sync_status()
    values = codes.double() * e.double().t().repeat_interleave(group, 1)[:, :K]
    y = (X.double() @ values.t() + bias.double()).cpu().numpy()
    absum = (X.double().abs() @ values.abs().t()).cpu().numpy()
    x = X.double().abs()
    top = x.amax(1, keepdim=True)
    unit = (torch.where(x < 2.0 ** -14 * top, 2.0 ** -22 * top, 0.0) @ values.abs().t()).cpu().numpy()
    err = np.abs(wl.bf16_bits_to_f32(host_bits(Y)).astype(np.float64) - y)
    bound = 2.0 ** -8 * np.abs(y) + (unit + 3 * (K / 32 + 32) * 2.0 ** -23 * (absum + np.abs(y))) * (1 + 2.0 ** -8)
    assert np.all(err <= bound), float((err / bound).max())


@pytest.mark.parametrize("M", [2, 3, 4])
def test_nonfinite_tokens_stay_to_themselves(M):
    """A token with a NaN or an infinity gives NaN, the others are as ever, one of zeros gives the bias."""
    N, K, group = _rows(M), 144, 64
    weight, values = _weight(N, K, group, True, M)
    rng = np.random.default_rng(M)
    X = wl.f32_to_bf16_bits(rng.normal(0, 1, (M, K)).astype(np.float32))
    bias = wl.f32_to_bf16_bits(rng.normal(0, 1, N).astype(np.float32))
    for token, bits in ((0, 0x7FC0), (M - 1, 0xFF80), (1, 0x7F80)):
        bad = X.copy()
        bad[token, 3 + 70 * token % K] = bits
        bad[(token + 1) % M] = 0
        Y = _run(dev_bf16(bad), weight, group, dev_bf16(bias), N)
        sq.sq_sync_status()
        rest = [m for m in range(M) if m != token]
        _check(Y[rest], bad[rest], values, bias)
        assert bool(torch.isnan(Y[token]).all()) and torch.equal(Y[(token + 1) % M], dev_bf16(bias).view(-1))


def test_on_a_side_stream_and_in_a_graph():
    M, K, group = 2, 1040, 128
    N = _rows(M)
    weight, values = _weight(N, K, group, False, 3)
    X = dev_bf16(wl.f32_to_bf16_bits(np.random.default_rng(0).normal(0, 1, (M, K)).astype(np.float32)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        Y = _run(X, weight, group, None, N)
        other = _run(X, weight, group, None, N, stream=side)
    side.synchronize()
    assert torch.equal(Y, other)
    Yg = empty((M, N), torch.bfloat16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sq.sq_int4_linear(X, *weight, group, None, Yg)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(Y, Yg)
    X.mul_(-3)
    graph.replay()
    sq.sq_sync_status()
    _check(Yg, host_bits(X), values, None)


@pytest.mark.parametrize("M", [1, 4])
@pytest.mark.parametrize("place", [0, -1])
def test_nonfinite_scales_stay_in_their_rows(M, place):
    N, K, group = _rows(M, 8), 144, 32
    rng = np.random.default_rng(M)
    scale = oracle.float_to_bf16(rng.uniform(0.002, 0.02, (5, N)).astype(np.float32))
    zero, codes = rng.integers(0, 16, (5, N), dtype=np.uint8), rng.integers(0, 16, (N, K), dtype=np.uint8)
    scale[place, [3, N - 1]], scale[place, 20] = 0x7F80, 0x7FC0  # infinity, NaN
    X = wl.f32_to_bf16_bits(rng.normal(0, 1, (M, K)).astype(np.float32))
    weight = (torch.from_numpy(osv.int4_pack(codes)).cuda(), dev_bf16(scale), torch.from_numpy(zero).cuda())
    Y = _run(dev_bf16(X), weight, group, None, N)
    sq.sq_sync_status()
    assert not bool(torch.isfinite(Y[:, [3, 20, N - 1]]).any())
    rest = np.setdiff1d(np.arange(N), [3, 20, N - 1])
    values = osv.int4_values(codes[rest], scale[:, rest], zero[:, rest], group)
    _check(Y[:, torch.from_numpy(rest).cuda()].contiguous(), X, values, None)
