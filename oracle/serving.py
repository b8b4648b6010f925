"""CPU oracle of the 4-bit weight linear and the paged key-value cache (numpy, from the
formulas of include/sq.h; shares no code with the GPU path).

Codes, scales and rotated values follow the definition's fp32 operations one by one and are
exact; products, softmax and sums are fp64. bf16 arrays are uint16 bit patterns.
"""
from __future__ import annotations

import numpy as np

from . import bf16_to_float, float_to_bf16

F32_MAX = np.finfo(np.float32).max


def _recip(top, bottom):
    """min(top / bottom, FLT_MAX) in fp32, 0 where bottom is 0."""
    with np.errstate(divide="ignore", over="ignore"):
        r = np.minimum(np.float32(top) / bottom, F32_MAX)
    return np.where(bottom > 0, r, np.float32(0)).astype(np.float32)


# ---------------------------------------------------------------- 4-bit weights
def int4_quant(W, s, group, asym):
    """codes uint8 [N, K], scale bf16 bits [G, N], zero uint8 [G, N] (all 8 when symmetric)."""
    w = bf16_to_float(W)
    if s is not None:
        w = (w * np.asarray(s, np.float32)).astype(np.float32)
    N, K = w.shape
    G = -(-K // group)
    codes, scale, zero = np.empty((N, K), np.uint8), np.empty((G, N), np.uint16), np.full((G, N), 8, np.uint8)
    for j in range(G):
        v = w[:, j * group:(j + 1) * group]
        if asym:
            lo, hi = np.minimum(v.min(1), np.float32(0)), np.maximum(v.max(1), np.float32(0))
            e = (hi - lo) / np.float32(15)
        else:
            e = np.abs(v).max(1) / np.float32(7)
        scale[j] = float_to_bf16(e)
        r = _recip(1, bf16_to_float(scale[j]))
        if asym:
            zero[j] = np.clip(np.rint(-lo * r), 0, 15)
        z = zero[j].astype(np.float32)[:, None]
        codes[:, j * group:(j + 1) * group] = np.clip(np.rint(v * r[:, None]) + z, 0, 15)
    return codes, scale, zero


def int4_place(N, K):
    """Byte index and nibble shift in the packed codes of every [n, k]."""
    n, k = np.arange(N)[:, None], np.arange(K)[None, :]
    r, c = n % 16, k % 128
    tile = n // 16 * -(-K // 128) + k // 128
    byte = tile * 1024 + (4 * r + c // 2 % 4) * 16 + c // 32 * 4 + c % 2 * 2 + c // 16 % 2
    return byte, np.broadcast_to(c // 8 % 2 * 4, byte.shape)


def int4_pack(codes):
    N, K = codes.shape
    Np, Kp = -(-N // 16) * 16, -(-K // 128) * 128
    full = np.full((Np, Kp), 8, np.uint8)
    full[:N, :K] = codes
    byte, shift = int4_place(Np, Kp)
    out = np.zeros(Np * Kp // 2, np.uint8)
    np.bitwise_or.at(out, byte.ravel(), (full.astype(np.uint8) << shift.astype(np.uint8)).ravel())
    return out


def int4_unpack(packed, N, K):
    byte, shift = int4_place(N, K)
    return (packed[byte] >> shift.astype(np.uint8)) & 15


def int4_values(codes, scale, zero, group):
    """(code - zero) * scale, exact in fp64."""
    K = codes.shape[1]
    z = np.repeat(zero.T.astype(np.float64), group, 1)[:, :K]
    e = np.repeat(bf16_to_float(scale).T.astype(np.float64), group, 1)[:, :K]
    return (codes.astype(np.float64) - z) * e


def int4_linear(X, values, bias):
    """(Y fp64, sum of absolute products per output)."""
    x = bf16_to_float(X).astype(np.float64)
    y = x @ values.T
    if bias is not None:
        y = y + bf16_to_float(bias).astype(np.float64)
    return y, np.abs(x) @ np.abs(values).T


# ---------------------------------------------------------------- paged key-value cache
def rotate(x, cos, sin, interleaved):
    """fp32 rows x [T, heads, D], cos and sin [T, rot/2] of the tokens: every operation rounded."""
    y = np.array(x, np.float32, copy=True)
    half = cos.shape[1]
    if interleaved:
        ia, ib = np.arange(0, 2 * half, 2), np.arange(1, 2 * half, 2)
    else:
        ia, ib = np.arange(half), np.arange(half, 2 * half)
    c, s = cos[:, None, :].astype(np.float32), sin[:, None, :].astype(np.float32)
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia] = (a * c).astype(np.float32) - (b * s).astype(np.float32)
    y[..., ib] = (b * c).astype(np.float32) + (a * s).astype(np.float32)
    return y


def kv_codes(y):
    """int8 codes and fp32 scales of fp32 rows [..., D]."""
    a = np.abs(y).max(-1)
    r = _recip(127, a)
    codes = np.clip(np.rint(y * r[..., None]), -128, 127).astype(np.int8)
    return codes, (a / np.float32(127)).astype(np.float32)


def paged_attention(q, k, v, table, lens, scale, window=0):
    """q fp64 [B, H, D]; k, v fp64 values of the cache [pages, heads, page_size, D]. Returns out,
    lse, and for error bounds the largest sum of absolute products of a score and
    sum_t p_t |v_t|."""
    B, H, D = q.shape
    heads, P = k.shape[1], k.shape[2]
    out, lse = np.zeros((B, H, D)), np.full((B, H), -np.inf)
    most, absv = np.zeros((B, H)), np.zeros((B, H, D))
    for b in range(B):
        n = int(min(max(lens[b], 0), table.shape[1] * P))
        t = np.arange(max(0, n - window) if window else 0, n)
        page = table[b, t // P]
        ok = (page >= 0) & (page < k.shape[0])
        t, page = t[ok], page[ok]
        if not t.size:
            continue
        for h in range(H):
            kk, vv = k[page, h // (H // heads), t % P], v[page, h // (H // heads), t % P]
            s = scale * (kk @ q[b, h])
            m = s.max()
            p = np.exp(s - m)
            lse[b, h] = m + np.log(p.sum())
            p /= p.sum()
            out[b, h] = p @ vv
            absv[b, h] = p @ np.abs(vv)
            most[b, h] = (np.abs(kk) @ np.abs(q[b, h])).max() * abs(scale)
    return out, lse, most, absv
