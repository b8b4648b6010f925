"""The operators of a decode step one after another, as a layer's attention block uses them: 4-bit
qkv projection, rotation and append, paged attention, then the output projection with 4-bit and
with 8-bit weights; captured as a graph, replayed with new tokens, each step checked against fp64
(or the exact codes) of what the operator before it left."""
import numpy as np
import pytest
import torch

import oracle
from oracle import serving as osv
from w8a8_quantized_gemm_b200 import sq
from w8a8_quantized_gemm_b200 import workloads as wl

from _gpu import dev_bf16, empty, host, host_bits
from test_gpu_int4 import _check_linear
from test_gpu_kv import _check_attention, _new_cache, _tables

pytestmark = pytest.mark.gpu


def _f64(bits):
    return wl.bf16_bits_to_f32(bits).astype(np.float64)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("B", [1, 4, 5, 17, 64])
def test_decode_block(B, int8):
    H, heads, D, P, hidden, group, steps = 4, 2, 64, 16, 272, 64, 19
    rng = np.random.default_rng(B)

    def bits(*shape, scale=1.0):
        return wl.f32_to_bf16_bits((rng.normal(0, 1, shape) * scale).astype(np.float32))

    def up(a):
        return torch.from_numpy(np.ascontiguousarray(a)).cuda()

    # weights, quantized once
    w_qkv, w_out = bits((H + 2 * heads) * D, hidden, scale=0.06), bits(hidden, H * D, scale=0.06)
    bias = bits((H + 2 * heads) * D)
    packed = []
    for w in (w_qkv, w_out):
        N, K = w.shape
        G = -(-K // group)
        p = (empty(sq.sq_int4_weight_bytes(N, K), torch.uint8), empty((G, N), torch.bfloat16),
             empty((G, N), torch.uint8))
        sq.sq_quant_weight_int4(dev_bf16(w), None, group, *p)
        packed.append(p)
    values = [osv.int4_values(osv.int4_unpack(host(p[0]), *w.shape), host_bits(p[1]), host(p[2]), group)
              for p, w in zip(packed, (w_qkv, w_out))]
    w8, e8 = empty((hidden, H * D), torch.int8), empty(hidden, torch.float32)
    ones = torch.ones(H * D, device="cuda")
    sq.sq_smooth_quant_weight(dev_bf16(w_out), ones, sq.SQ_PER_CHANNEL, w8, e8,
                              sq.workspace(sq.SQ_OP_SMOOTH_QUANT_WEIGHT, 0, hidden, H * D))
    # state: the last row of a batch of several is padding
    live = B - 1 if B > 1 else 1
    table = rng.permutation(2 * B).reshape(B, 2).astype(np.int32)
    cache = _new_cache(2 * B, heads, P, D, int8)
    cos, sin = (up(t) for t in _tables(32, D))
    x = torch.zeros((B, hidden), dtype=torch.bfloat16, device="cuda")
    pos, slots, lens = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(3))
    dt, ws = up(table), sq.workspace(sq.SQ_OP_PAGED_ATTENTION, B, H, D)
    gws = sq.workspace(sq.SQ_OP_INT8_GEMM_DEQUANT, B, hidden, H * D)
    qkv, att = empty((B, H + 2 * heads, D), torch.bfloat16), empty((B, H, D), torch.bfloat16)
    q1 = torch.zeros((B, H, D), dtype=torch.bfloat16, device="cuda")
    y4, y8 = empty((B, hidden), torch.bfloat16), empty((B, hidden), torch.bfloat16)
    a8, d8 = empty((B, H * D), torch.int8), empty(B, torch.float32)
    b_dev = dev_bf16(bias)

    def step():
        sq.sq_int4_linear(x, *packed[0], group, b_dev, qkv.view(B, -1))
        sq.sq_rope_kv_append(qkv[:, :H], qkv[:, H:H + heads], qkv[:, H + heads:], cos, sin, pos, slots, cache, q1)
        sq.sq_paged_attention(q1, cache, dt, lens, D ** -0.5, att, ws=ws)
        sq.sq_int4_linear(att.view(B, -1), *packed[1], group, None, y4)
        sq.sq_quant_act_per_token(att.view(B, -1), ones, a8, d8)
        sq.sq_int8_gemm_dequant(a8, w8, d8, e8, sq.SQ_PER_CHANNEL, None, y8, ws=gws)

    def stage(n):
        x.copy_(dev_bf16(bits(B, hidden)))
        pos.fill_(n)
        slots.copy_(up(np.where(np.arange(B) < live, table[:, n // P] * P + n % P, -1).astype(np.int32)))
        lens.copy_(up(np.where(np.arange(B) < live, n + 1, 0).astype(np.int32)))

    stage(0)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(1, steps):
        stage(n)
        graph.replay()
    sq.sq_sync_status()
    # ---- the last step, operator by operator
    y, absum = osv.int4_linear(host_bits(x), values[0], bias)
    _check_linear(qkv.view(B, -1), y, absum, hidden)
    n = steps - 1
    c, s = (t.cpu().numpy()[[n] * live] for t in (cos, sin))
    rot = osv.rotate(wl.bf16_bits_to_f32(host_bits(qkv))[:live, :H + heads], c, s, False)
    assert np.array_equal(host_bits(q1)[:live], oracle.float_to_bf16(rot[:, :H]))
    vals = []
    for i in range(2):
        t = cache.tensors[i].double()
        if int8:
            t = t * torch.nan_to_num(cache.tensors[2 + i]).double()[..., None]
        vals.append(np.nan_to_num(t.cpu().numpy()))
    if int8:
        want, scale = osv.kv_codes(rot[:, H:])
        page, row = table[:live, n // P], n % P
        assert np.array_equal(host(cache.tensors[0])[page, :, row], want)
        assert np.array_equal(host(cache.tensors[2])[page, :, row], scale)
    now = [steps if b < live else 0 for b in range(B)]
    ref = osv.paged_attention(_f64(host_bits(q1)), *vals, table, now, D ** -0.5)
    _check_attention(att, None, ref, D, steps)
    a_bits = host_bits(att).reshape(B, -1)
    y, absum = osv.int4_linear(a_bits, values[1], None)
    _check_linear(y4, y, absum, H * D)
    codes, d = oracle.quant_act_per_token(a_bits, np.ones(H * D, np.float32))
    assert np.array_equal(host(a8), codes) and np.array_equal(host(d8), d)
    y = oracle.int8_gemm(codes, host(w8)) * d.astype(np.float64)[:, None] * host(e8).astype(np.float64)
    # two fp32 products, then half a step of bf16
    assert np.all(np.abs(_f64(host_bits(y8)) - y) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(y) + 2.0 ** -133)
