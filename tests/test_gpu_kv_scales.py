"""Attention over an int8 cache whose tokens' value scales are far apart, zero or not finite: the
softmax and its log-sum-exp are the keys' alone, whatever the values are."""
import numpy as np
import pytest
import torch

from oracle import serving as osv
from w8a8_quantized_gemm_b200 import sq
from w8a8_quantized_gemm_b200 import workloads as wl

from _gpu import dev_bf16, host, host_bits
from test_gpu_kv import _attend, _bits

pytestmark = pytest.mark.gpu


def _case(seed, lens, H, heads, D, vs):
    """A cache of random keys and of values with the scales vs [tokens], one run of pages after another."""
    rng = np.random.default_rng(seed)
    P = 16
    need = [-(-n // P) for n in lens]
    pages = sum(need)
    codes = rng.integers(64, 128, (2, pages, heads, P, D)).astype(np.int8) * rng.choice([-1, 1], (2, pages, heads, P, D)).astype(np.int8)
    sc = rng.uniform(0.005, 0.02, (2, pages, heads, P)).astype(np.float32)
    sc[1] = vs(rng, (pages, heads, P)).astype(np.float32)
    table = np.zeros((len(lens), max(need)), np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = np.arange(at, at + n)
        at += n
    t = [torch.from_numpy(a).cuda() for a in (codes[0], codes[1], sc[0], sc[1])]
    q = _bits(rng, len(lens), H, D)
    out, lse = _attend(dev_bf16(q), sq.KvCache(*t), torch.from_numpy(table).cuda(),
                       torch.tensor(lens, dtype=torch.int32).cuda(), D ** -0.5)
    sq.sq_sync_status()
    with np.errstate(invalid="ignore"):
        k, v = (codes[n].astype(np.float64) * sc[n].astype(np.float64)[..., None] for n in range(2))
        ref = osv.paged_attention(wl.bf16_bits_to_f32(q).astype(np.float64), k, v, table, lens, D ** -0.5)
    return out, lse, ref, D, max(lens)


def _rel(most, D, longest):
    """As for scales near one (fp32 scores, two 16-bit parts of a probability, sums over the tokens),
    and, since a maximum moved by scales lies up to 2^7 from the scores and 2^8 from another part's,
    differences rounded by 2^-18 and, for the parts' factors, by 2^-17: both times ln 2 in the
    exponential, together below 2^-16."""
    return 2 * (D / 8 + 16) * 2.0 ** -23 * most + 2.0 ** -18 + 2 * (longest / 64 + 128) * 2.0 ** -23 + 2.0 ** -16


SHAPES = [([5], 2, 1, 64), ([700], 4, 2, 128), ([3000, 40, 1], 16, 1, 64), ([64, 333], 3, 3, 96), ([900, 31], 2, 1, 256)]


@pytest.mark.parametrize("lens,H,heads,D", SHAPES)
@pytest.mark.parametrize("low,high", [(0, 40), (-100, 0), (100, 120), (-100, 120)])
def test_scales_far_apart(lens, H, heads, D, low, high):
    """Scales of 2^low to 2^high. No code is zero, so that every element has the largest token's part
    and the bound may count from it."""
    out, lse, (o, l, most, absv), D, longest = _case(
        abs(D + low), lens, H, heads, D, lambda rng, shape: 2.0 ** rng.uniform(low, high, shape))
    rel = _rel(most, D, longest)
    got = wl.bf16_bits_to_f32(host_bits(out)).astype(np.float64)
    err = np.abs(got - o)
    bound = 2.0 ** -8 * np.abs(o) + rel[..., None] * absv * (1 + 2.0 ** -8)
    assert np.all(err <= bound), float((err / bound).max())
    g = host(lse).astype(np.float64)
    # below 2^-19 of the largest, a token may vanish beside scales of 2^121
    allowed = rel + 2.0 ** -22 * (np.abs(l) + most) + (longest * 2.0 ** (high - 140) if high > 100 else 0)
    assert np.all(np.abs(g - l) <= allowed), float((np.abs(g - l) / allowed).max())


@pytest.mark.parametrize("lens,H,heads,D", SHAPES)
@pytest.mark.parametrize("bad", [0.0, np.inf, np.nan])
@pytest.mark.parametrize("where", ["first", "last", "every"])
def test_lse_beside_scales_of_zero_and_not_finite(lens, H, heads, D, bad, where):
    """One token's scale, or all: the log-sum-exp is as ever. Scales that are not finite show in out."""
    def vs(rng, shape):
        s = rng.uniform(0.005, 0.02, shape)
        if where == "every":
            s[:] = bad
        elif where == "first":
            s[0, :, 0] = bad
        else:  # the last token of the first sequence
            s[(lens[0] - 1) // 16, :, (lens[0] - 1) % 16] = bad
        return s

    out, lse, (o, l, most, absv), D, longest = _case(D, lens, H, heads, D, vs)
    rel = _rel(most, D, longest)
    g = host(lse).astype(np.float64)
    assert np.all(np.abs(g - l) <= rel + 2.0 ** -22 * (np.abs(l) + most))
    got = wl.bf16_bits_to_f32(host_bits(out)).astype(np.float64)
    fine = np.isfinite(o)
    assert np.array_equal(np.isfinite(got), fine)
    err = np.abs(got - np.where(fine, o, 0))[fine]
    assert np.all(err <= (2.0 ** -8 * np.abs(o) + rel[..., None] * absv * (1 + 2.0 ** -8))[fine])
