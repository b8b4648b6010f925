"""4-bit weights whose scales are not finite, as the quantization of a weight that is not gives them: the
linear layer keeps them to their rows, for every number of tokens alike."""
import numpy as np
import pytest
import torch

from oracle import serving as osv
from w8a8_quantized_gemm_b200 import sq
from w8a8_quantized_gemm_b200 import workloads as wl

from _gpu import dev_bf16, empty, host_bits
from test_gpu_int4 import _check_linear, _codes, _up

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 4, 5, 16, 17, 33, 64])
@pytest.mark.parametrize("K,group", [(144, 32), (208, 64), (256, 128), (400, 64)])
@pytest.mark.parametrize("place", ["first", "last"])
def test_nonfinite_scales_stay_in_their_rows(M, K, group, place):
    """An infinite scale times a group's sum is infinite, its sign the sum's, and nothing of the
    columns behind a short last group is taken into it; a NaN is a NaN."""
    N = 40
    codes, scale, zero = _codes(N, K, group, True, K)
    g = 0 if place == "first" else scale.shape[0] - 1
    zero[g, 3:7] = 4
    codes[3:5, g * group:(g + 1) * group] = 9   # above the zero point, the tokens are positive
    codes[5:7, g * group:(g + 1) * group] = 2
    scale[g, [3, 5]], scale[g, [4, 6]] = 0x7F80, 0x7FC0  # infinity, NaN
    rng = np.random.default_rng(K)
    X = wl.f32_to_bf16_bits(rng.uniform(0.5, 2, (M, K)).astype(np.float32))
    Wp, e, z = _up(codes, scale, zero, True)
    Y = empty((M, N), torch.bfloat16)
    sq.sq_int4_linear(dev_bf16(X), Wp, e, z, group, None, Y)
    sq.sq_sync_status()
    assert bool((Y[:, 3] == float("inf")).all()) and bool((Y[:, 5] == float("-inf")).all())
    assert bool(torch.isnan(Y[:, [4, 6]]).all())
    rest = [n for n in range(N) if not 3 <= n < 7]
    y, absum = osv.int4_linear(X, osv.int4_values(codes[rest], scale[:, rest], zero[:, rest], group), None)
    _check_linear(Y[:, rest].contiguous(), y, absum, K)
