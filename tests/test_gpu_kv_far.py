"""The paged cache with pages beyond 2^32 elements and bytes from its start."""
import numpy as np
import pytest
import torch

from oracle import serving as osv
from w8a8_quantized_gemm_b200 import sq
from w8a8_quantized_gemm_b200 import workloads as wl

from _gpu import dev_bf16, host, host_bits
from test_gpu_kv import _attend, _bits, _check_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("P", [8, 32])
def test_far_pages(int8, P):
    """Page 3 starts more than 2^32 elements behind page 0, in int8 the scales' page too: rows one by one
    (pages of 8 tokens) and as a run (pages of 32), attended to and appended."""
    rng = np.random.default_rng(P)
    D, pages = 64, 4
    stride = (1 << 32) // 3 // 16 * 16 + 4096
    assert 3 * stride > 2 ** 32 and stride % 16 == 0
    scale_stride = (1 << 32) // 4 // 3 + 64  # four bytes each
    assert 3 * scale_stride * 4 > 2 ** 32
    row = P * D
    buf = torch.empty(3 * stride + 2 * row, dtype=torch.int8 if int8 else torch.bfloat16, device="cuda")
    views = [torch.as_strided(buf, (pages, 1, P, D), (stride, row, D, 1), off) for off in (0, row)]
    scales = [None, None]
    if int8:
        codes = rng.integers(-127, 128, (2, pages, 1, P, D)).astype(np.int8)
        sc = rng.uniform(0.005, 0.02, (2, pages, 1, P)).astype(np.float32)
        sbuf = torch.empty(3 * scale_stride + 2 * P, device="cuda")
        scales = [torch.as_strided(sbuf, (pages, 1, P), (scale_stride, P, 1), off) for off in (0, P)]
        values = [codes[n].astype(np.float64) * sc[n].astype(np.float64)[..., None] for n in range(2)]
        for n in range(2):
            views[n].copy_(torch.from_numpy(codes[n]).cuda())
            scales[n].copy_(torch.from_numpy(sc[n]).cuda())
    else:
        bits = [_bits(rng, pages, 1, P, D) for _ in range(2)]
        values = [wl.bf16_bits_to_f32(b).astype(np.float64) for b in bits]
        for n in range(2):
            views[n].copy_(dev_bf16(bits[n]).view(pages, 1, P, D))
    cache = sq.KvCache(views[0], views[1], *scales)
    table, lens = np.array([[3, 1, 0, 2]], np.int32), [4 * P - 2]
    q = _bits(rng, 1, 2, D)
    out, lse = _attend(dev_bf16(q), cache, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), 0.125)
    sq.sq_sync_status()
    _check_attention(out, lse, osv.paged_attention(wl.bf16_bits_to_f32(q).astype(np.float64), *values, table, lens, 0.125),
                     D, lens[0])
    x = _bits(rng, 2, 1, D)
    slots = torch.tensor([3 * P + P - 1, 3 * P], dtype=torch.int32, device="cuda")
    dx = dev_bf16(x).view(2, 1, D)
    sq.sq_rope_kv_append(None, dx, dx, None, None, None, slots, cache, None)
    sq.sq_sync_status()
    for n in range(2):
        got = views[n][3, 0, [P - 1, 0]]
        if int8:
            want, s = osv.kv_codes(wl.bf16_bits_to_f32(x).reshape(2, D))
            assert np.array_equal(host(got), want) and np.array_equal(host(scales[n][3, 0, [P - 1, 0]]), s)
        else:
            assert np.array_equal(host_bits(got).reshape(2, D), x.reshape(2, D))
        for page in (0, 1, 2):  # the others are as they were
            t = views[n][page, 0].double()
            t = t * scales[n][page, 0].double()[:, None] if int8 else t
            assert np.array_equal(t.cpu().numpy(), values[n][page, 0])
