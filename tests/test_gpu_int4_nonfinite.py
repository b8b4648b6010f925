"""4-bit quantization of weights that are not finite: the group shows it, the others are as ever."""
import numpy as np
import pytest
import torch

from w8a8_quantized_gemm_b200 import sq
from w8a8_quantized_gemm_b200 import workloads as wl

from _gpu import dev_bf16, empty
from test_gpu_int4 import _packed, _smooth, _weight

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("asym", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("bad,bits", [("nan", 0x7FC0), ("nan", 0xFFC1), ("inf", 0x7F80), ("inf", 0xFF80)])
@pytest.mark.parametrize("N,K", [(24, 272), (40, 80)])
def test_nonfinite_weights_show_in_their_group(N, K, group, bad, bits, asym):
    W, s = _weight(N, K, 5), _smooth(K, 5)
    where = [(0, 0), (3, K - 1), (9, K // 2), (N - 1, 33)]  # a group of zeros, a short last group, ...

    def run(W, s=s):
        Wp, e, z = _packed(N, K, group, asym)
        sq.sq_quant_weight_int4(dev_bf16(W), torch.from_numpy(s).cuda(), group, Wp, e, z)
        out = empty((N, K), torch.bfloat16)
        sq.sq_dequant_weight_int4(Wp, e, z, group, out)
        sq.sq_sync_status()
        return Wp, e, z, out

    _, e0, z0, clean = run(W)
    W2 = W.copy()
    for n, k in where:
        W2[n, k] = bits
    Wp, e, z, out = run(W2)
    hit = torch.zeros(e.shape, dtype=torch.bool)
    for n, k in where:
        hit[k // group, n] = True
    hit = hit.cuda()
    assert bool((torch.isnan(e) if bad == "nan" else e == float("inf"))[hit].all())
    assert torch.equal(e[~hit], e0[~hit])
    if asym:
        assert torch.equal(z[~hit], z0[~hit]) and int(z.max()) <= 15
    of = hit.t().repeat_interleave(group, 1)[:, :K]
    assert not bool(torch.isfinite(out[of]).any()) and torch.equal(out[~of], clean[~of])
    # and through the linear layer: the rows' results, no others
    X = dev_bf16(wl.f32_to_bf16_bits(np.random.default_rng(1).uniform(0.5, 2, (3, K)).astype(np.float32)))
    Y = empty((3, N), torch.bfloat16)
    sq.sq_int4_linear(X, Wp, e, z, group, None, Y)
    sq.sq_sync_status()
    rows = hit.any(0)
    assert not bool(torch.isfinite(Y[:, rows]).any()) and bool(torch.isfinite(Y[:, ~rows]).all())


@pytest.mark.parametrize("asym", [False, True])
def test_nan_smoothing_factor_shows(asym):
    """A NaN in s is in every row's group."""
    N, K, group = 16, 128, 32
    s = _smooth(K, 1)
    s[70] = np.nan
    Wp, e, z = _packed(N, K, group, asym)
    sq.sq_quant_weight_int4(dev_bf16(_weight(N, K, 2)), torch.from_numpy(s).cuda(), group, Wp, e, z)
    sq.sq_sync_status()
    assert bool(torch.isnan(e[2]).all()) and bool(torch.isfinite(e[[0, 1, 3]]).all())
