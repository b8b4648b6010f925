"""Attention over an int8 cache with queries far from one, which it takes as integers of 23 bits and a
power of two for each head."""
import numpy as np
import pytest
import torch

from oracle import serving as osv
from w8a8_quantized_gemm_b200 import sq
from w8a8_quantized_gemm_b200 import workloads as wl

from _gpu import dev_bf16
from test_gpu_kv import _attend, _bits, _check_attention, _filled

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,H,heads,D", [([300, 7], 4, 2, 64), ([1100], 9, 1, 96), ([40, 200], 8, 8, 128), ([90], 16, 1, 256)])
@pytest.mark.parametrize("p", [-132, -126, -115, -104, -99, -90, 40, 100])
def test_queries_of_any_size(lens, H, heads, D, p):
    """Queries of about 2^p and a scale that brings the scores back to one: heads of every size beside
    each other, one of zeros. A head's elements below 2^-14 of its largest are off by at most 2^-22
    of that, less than 2^-22 of the sum of absolute products; the check's bound for the fp32 scores
    allows (D / 8 + 16) times half of that."""
    rng = np.random.default_rng(D + abs(p))
    P, B = 16, len(lens)
    width = -(-max(lens) // P)
    cache, (k, v) = _filled(rng, B * width, heads, P, D, True)
    table = rng.permutation(B * width).reshape(B, width).astype(np.int32)
    q = _bits(rng, B, H, D, scale=2.0 ** p)
    q[:, ::3] = _bits(rng, B, len(range(0, H, 3)), D, scale=2.0 ** min(p + 20, 100))
    q[0, H // 2] = 0
    scale = float(np.float32(2.0 ** min(-p, 126) * D ** -0.5 / 8))
    out, lse = _attend(dev_bf16(q), cache, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), scale)
    sq.sq_sync_status()
    ref = osv.paged_attention(wl.bf16_bits_to_f32(q).astype(np.float64), k, v, table, lens, scale)
    _check_attention(out, lse, ref, D, max(lens))
