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
