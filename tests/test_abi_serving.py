"""The 4-bit weight and paged-cache entry points without a GPU: sizes, refusals (before
anything is launched), and the oracle's own pins."""
import ctypes as C

import numpy as np
import pytest
import torch

import oracle
from oracle import serving as osv
from w8a8_quantized_gemm_b200 import sq
from w8a8_quantized_gemm_b200 import workloads as wl

FAKE = 1 << 20  # a 16-byte-aligned non-null address; never dereferenced on these paths
INV, ALIGN, WS = sq.SQ_ERR_INVALID, sq.SQ_ERR_ALIGN, sq.SQ_ERR_WORKSPACE


def test_int4_weight_bytes():
    assert sq.sq_int4_weight_bytes(16, 128) == 1024
    assert sq.sq_int4_weight_bytes(8, 16) == 1024          # padded to a tile
    assert sq.sq_int4_weight_bytes(24, 144) == 4 * 1024
    assert sq.sq_int4_weight_bytes(4096, 4096) == 4096 * 4096 // 2
    assert sq.sq_int4_weight_bytes(0, 128) == 0 and sq.sq_int4_weight_bytes(16, -1) == 0


@pytest.mark.parametrize("bad,code", [
    (dict(W=None), INV), (dict(W=FAKE + 8), ALIGN), (dict(N=12), INV), (dict(N=0), INV), (dict(K=24), INV),
    (dict(K=65552), INV), (dict(ld=32), INV), (dict(ld=68), ALIGN), (dict(s=FAKE + 4), ALIGN), (dict(group=16), INV),
    (dict(group=0), INV), (dict(group=256), INV), (dict(Wp=None), INV), (dict(Wp=FAKE + 8), ALIGN),
    (dict(e=None), INV), (dict(e=FAKE + 2), ALIGN), (dict(z=FAKE + 8), ALIGN)])
def test_quant_weight_int4_refusals(bad, code):
    a = dict(W=FAKE, N=16, K=64, ld=64, s=FAKE, group=64, Wp=FAKE, e=FAKE, z=FAKE)
    a.update(bad)
    assert sq.lib().sq_quant_weight_int4(a["W"], a["N"], a["K"], a["ld"] if "ld" in bad else a["K"], a["s"],
                                         a["group"], a["Wp"], a["e"], a["z"], None) == code
    assert "sq_quant_weight_int4" in sq.sq_last_error()


@pytest.mark.parametrize("bad,code", [(dict(out=None), INV), (dict(out=FAKE + 8), ALIGN), (dict(N=4), INV),
                                      (dict(group=48), INV), (dict(Wp=None), INV), (dict(e=None), INV)])
def test_dequant_weight_int4_refusals(bad, code):
    a = dict(N=16, K=64, group=64, Wp=FAKE, e=FAKE, z=None, out=FAKE)
    a.update(bad)
    assert sq.lib().sq_dequant_weight_int4(a["Wp"], a["e"], a["z"], a["group"], a["N"], a["K"], a["out"], None) == code


@pytest.mark.parametrize("bad,code", [
    (dict(X=None), INV), (dict(X=FAKE + 2), ALIGN), (dict(M=0), INV), (dict(M=65), INV), (dict(K=40), INV),
    (dict(ld=56), INV), (dict(ld=68), ALIGN), (dict(N=20), INV), (dict(N=0), INV), (dict(group=65), INV),
    (dict(Wp=None), INV), (dict(e=None), INV), (dict(bias=FAKE + 2), ALIGN), (dict(Y=None), INV),
    (dict(Y=FAKE + 8), ALIGN)])
def test_int4_linear_refusals(bad, code):
    a = dict(X=FAKE, M=3, K=64, ld=64, N=16, group=64, Wp=FAKE, e=FAKE, z=None, bias=FAKE, Y=FAKE)
    a.update(bad)
    assert sq.lib().sq_int4_linear(a["X"], a["M"], a["K"], a["ld"], a["Wp"], a["e"], a["z"], a["group"], a["bias"],
                                   a["Y"], a["N"], None) == code


def _cache(**kw):
    a = dict(type=sq.SQ_KV_INT8, reserved=0, k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, num_pages=10, heads=2,
             page_size=16, head_dim=64, page_stride=2 * 16 * 64, scale_page_stride=32)
    a.update(kw)
    return sq._KvCacheStruct(*a.values())


BAD_CACHES = [
    (dict(type=2), INV), (dict(reserved=1), INV), (dict(k=None), INV), (dict(v=FAKE + 8), ALIGN),
    (dict(k_scale=None), INV), (dict(v_scale=FAKE + 4), ALIGN), (dict(type=sq.SQ_KV_BF16), INV),
    (dict(head_dim=80), INV), (dict(heads=0), INV), (dict(heads=1025), INV), (dict(page_size=24), INV),
    (dict(page_size=0), INV), (dict(page_size=2048), INV), (dict(num_pages=0), INV), (dict(num_pages=1 << 27), INV),
    (dict(page_stride=2032), INV), (dict(page_stride=2056), ALIGN), (dict(scale_page_stride=31), INV)]


def _append(cache, **kw):
    a = dict(q=FAKE, ldq=256, k=FAKE, ldk=128, v=FAKE, ldv=128, T=3, H=4, cos=FAKE, sin=FAKE, max_pos=8, rot=64,
             pairs=0, positions=FAKE, slots=FAKE)
    out = kw.pop("q_out", 2 * FAKE)
    a.update(kw)
    return sq.lib().sq_rope_kv_append(*a.values(), C.byref(cache) if cache is not None else None, out, None)


def _attend(cache, **kw):
    a = dict(q=FAKE, ldq=256, B=3, H=4)
    b = dict(table=FAKE, ld=5, pages=5, lens=FAKE, window=0, scale=0.125, out=FAKE, lse=FAKE, ws=FAKE, ws_bytes=1 << 40)
    for k, v in kw.items():
        (a if k in a else b)[k] = v
    b["scale"] = C.c_float(b["scale"])
    return sq.lib().sq_paged_attention(*a.values(), C.byref(cache) if cache is not None else None, *b.values(), None)


@pytest.mark.parametrize("bad,code", BAD_CACHES)
def test_cache_refusals(bad, code):
    assert _append(_cache(**bad)) == code
    assert _attend(_cache(**bad)) == code


@pytest.mark.parametrize("bad,code", [
    (dict(q=None), INV), (dict(q_out=None), INV), (dict(H=0), INV), (dict(H=-1, q=None, q_out=None), INV),
    (dict(H=2000), INV), (dict(ldq=248), INV), (dict(ldq=260), ALIGN), (dict(ldk=120), INV), (dict(ldv=132), ALIGN),
    (dict(k=None), INV), (dict(v=FAKE + 2), ALIGN), (dict(T=0), INV), (dict(q_out=FAKE, ldq=512), INV),
    (dict(q_out=FAKE + 8), ALIGN), (dict(rot=8), INV), (dict(rot=80), INV), (dict(rot=-16), INV), (dict(cos=None), INV),
    (dict(sin=FAKE + 4), ALIGN), (dict(positions=None), INV), (dict(positions=FAKE + 2), ALIGN), (dict(max_pos=0), INV),
    (dict(slots=None), INV)])
def test_append_refusals(bad, code):
    assert _append(_cache(), **bad) == code


@pytest.mark.parametrize("bad,code", [
    (dict(q=None), INV), (dict(ldq=128), INV), (dict(ldq=260), ALIGN), (dict(B=0), INV), (dict(B=65536), INV),
    (dict(H=0), INV), (dict(H=3), INV), (dict(H=1026), INV), (dict(table=None), INV), (dict(table=FAKE + 1), ALIGN),
    (dict(ld=4), INV), (dict(pages=0), INV), (dict(pages=1 << 27, ld=1 << 27), INV), (dict(lens=None), INV), (dict(window=-1), INV),
    (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV), (dict(out=None), INV), (dict(out=FAKE + 8), ALIGN),
    (dict(lse=FAKE + 2), ALIGN)])
def test_attention_refusals(bad, code):
    assert _attend(_cache(), **bad) == code


def test_null_cache_refused():
    assert _append(None) == INV and _attend(None) == INV


def test_attention_workspace_refusals():
    need = sq.sq_workspace_size(sq.SQ_OP_PAGED_ATTENTION, 3, 4, 64)
    assert sq.sq_workspace_size(sq.SQ_OP_PAGED_ATTENTION, 0, 4, 64) == 0
    if need:
        assert _attend(_cache(), ws_bytes=need - 1) == WS
        assert _attend(_cache(), ws=None) == WS
        assert _attend(_cache(), ws=FAKE + 8) == ALIGN


def test_binding_refuses_cpu_tensors():
    w = torch.zeros(16, 64, dtype=torch.bfloat16)
    e = torch.zeros(1, 16, dtype=torch.bfloat16)
    p = torch.zeros(1024, dtype=torch.uint8)
    with pytest.raises(TypeError):
        sq.sq_quant_weight_int4(w, None, 64, p, e)
    with pytest.raises(TypeError):
        sq.sq_int4_linear(w, p, e, None, 64, None, torch.zeros(16, 16, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        sq.KvCache(torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        sq.KvCache(torch.zeros(4, 2, 16, 64), torch.zeros(4, 2, 16, 64))


# ---------------------------------------------------------------- the oracle's pins
def test_oracle_int4_by_hand():
    """A group whose scale is exactly 1: absmax 7, ties to even, both ends of the range."""
    w = np.zeros((8, 32), np.float32)
    w[0, :7] = [7.0, -7.0, 2.5, 3.5, -2.5, 0.4, -0.6]
    codes, scale, zero = osv.int4_quant(wl.f32_to_bf16_bits(w), None, 32, False)
    assert list(codes[0, :8]) == [15, 1, 10, 12, 6, 8, 7, 8] and np.all(codes[1:] == 8)
    assert oracle.bf16_to_float(scale)[0, 0] == 1.0 and np.all(scale[0, 1:] == 0) and np.all(zero == 8)
    # with zero points: range -5 .. 10 has scale 1 and zero point 5
    w[0, :4] = [-5.0, 10.0, 0.0, 4.5]
    w[0, 4:7] = 0
    codes, scale, zero = osv.int4_quant(wl.f32_to_bf16_bits(w), None, 32, True)
    assert zero[0, 0] == 5 and list(codes[0, :4]) == [0, 15, 5, 9]
    v = osv.int4_values(codes, scale, zero, 32)
    assert list(v[0, :4]) == [-5.0, 10.0, 0.0, 4.0] and np.all(v[1:] == 0)


@pytest.mark.parametrize("asym", [False, True])
def test_oracle_int4_error_is_half_a_step(asym):
    rng = np.random.default_rng(5)
    W = wl.f32_to_bf16_bits(rng.normal(0, 0.02, (16, 272)).astype(np.float32))
    codes, scale, zero = osv.int4_quant(W, None, 128, asym)
    v = osv.int4_values(codes, scale, zero, 128)
    w = wl.bf16_bits_to_f32(W).astype(np.float64)
    e = np.repeat(oracle.bf16_to_float(scale).T.astype(np.float64), 128, 1)[:, :272]
    # half a step, and at the ends what rounding the scale (2^-8) and the zero point moved: the
    # largest value is at most 15 steps of the unrounded scale
    assert np.all(np.abs(v - w) <= e * (0.5 + (0.5 if asym else 0) + 15 * 2.0 ** -8))


def test_oracle_int4_layout_round_trip():
    rng = np.random.default_rng(1)
    codes = rng.integers(0, 16, (40, 272), dtype=np.uint8)
    packed = osv.int4_pack(codes)
    assert packed.size == sq.sq_int4_weight_bytes(40, 272)
    assert np.array_equal(osv.int4_unpack(packed, 40, 272), codes)
    byte, shift = osv.int4_place(16, 128)
    assert np.unique(byte * 8 + shift).size == 2048  # every nibble of a tile once
    # the header's formula at one place: row 9, column 77
    assert byte[9, 77] == (36 + 38 % 4) * 16 + 2 * 4 + 1 * 2 + 4 % 2 and shift[9, 77] == 4


def test_oracle_rotation_keeps_norms_and_differences():
    """Rotated products depend on the positions' difference only."""
    rng = np.random.default_rng(2)
    x = rng.normal(size=(1, 2, 64)).astype(np.float32)
    ang = np.arange(40)[:, None] * 100.0 ** (-np.arange(16) / 16)
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    for pairs in (False, True):
        def at(p):
            return osv.rotate(x, cos[p:p + 1], sin[p:p + 1], pairs).astype(np.float64)
        assert np.array_equal(at(7)[..., 32:], x[..., 32:])
        assert np.allclose(np.linalg.norm(at(7), axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-6)
        assert np.allclose((at(7)[0, 0] * at(12)[0, 1]).sum(), (at(20)[0, 0] * at(25)[0, 1]).sum(), rtol=1e-5)


def test_oracle_attention_by_hand():
    """Equal scores average the values; a window and a page out of range drop tokens."""
    k = np.zeros((3, 1, 2, 64))
    v = np.arange(6, dtype=np.float64).reshape(3, 1, 2, 1) * np.ones(64)
    q = np.ones((3, 1, 64))
    table = np.array([[2, 0], [1, 7], [0, 0]])
    out, lse, _, _ = osv.paged_attention(q, k, v, table, [3, 4, 0], 1.0)
    assert out[0, 0, 0] == pytest.approx((4 + 5 + 0) / 3) and lse[0, 0] == pytest.approx(np.log(3))
    assert out[1, 0, 0] == pytest.approx(2.5) and np.all(out[2] == 0) and lse[2, 0] == -np.inf
    out, _, _, _ = osv.paged_attention(q, k, v, table, [3, 4, 0], 1.0, window=2)
    assert out[0, 0, 0] == pytest.approx(2.5)
