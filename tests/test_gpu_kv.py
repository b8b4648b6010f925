"""GPU parity of the paged key-value cache: the append bit for bit against the oracle, the
attention against fp64, and both together as a decoding loop uses them."""
import numpy as np
import pytest
import torch

import oracle
from oracle import serving as osv
from w8a8_quantized_gemm_b200 import sq
from w8a8_quantized_gemm_b200 import workloads as wl

from _gpu import dev_bf16, empty, host, host_bits

pytestmark = pytest.mark.gpu


def _bits(rng, *shape, scale=1.0):
    return wl.f32_to_bf16_bits((rng.normal(0, 1, shape) * scale).astype(np.float32))


def _new_cache(pages, heads, P, D, int8, fill=None):
    if int8:
        k = torch.full((2, pages, heads, P, D), 77, dtype=torch.int8, device="cuda")
        s = torch.full((2, pages, heads, P), float("nan"), device="cuda")
        return sq.KvCache(k[0], k[1], s[0], s[1])
    k = torch.full((2, pages, heads, P, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    return sq.KvCache(k[0], k[1])


def _tables(max_pos, rot):
    ang = np.arange(max_pos)[:, None] * 10000.0 ** (-np.arange(rot // 2) * 2 / max(rot, 1))
    return np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)


def _attend(q, cache, table, lens, scale, window=0, lse=True, out=None, ws=None):
    B, H, D = q.shape
    out = torch.full((B, H, D), float("nan"), dtype=torch.bfloat16, device="cuda") if out is None else out
    l = torch.full((B, H), float("nan"), device="cuda") if lse else None
    ws = sq.workspace(sq.SQ_OP_PAGED_ATTENTION, B, H, D) if ws is None else ws
    sq.sq_paged_attention(q, cache, table, lens, scale, out, lse=l, window=window, ws=ws)
    return out, l


# ---------------------------------------------------------------- append
APPEND = [  # T, H, heads, D, rot, page_size
    (1, 4, 1, 64, 64, 1), (1, 32, 8, 128, 128, 16), (3, 6, 2, 96, 96, 8), (7, 0, 3, 64, 32, 16), (5, 8, 8, 256, 128, 4),
    (33, 3, 3, 96, 48, 32), (64, 8, 1, 128, 0, 64), (130, 1, 1, 64, 16, 128), (17, 40, 5, 128, 80, 2),
    (257, 2, 2, 256, 256, 64)]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("T,H,heads,D,rot,P", APPEND)
def test_append_exact(T, H, heads, D, rot, P, pairs, int8):
    rng = np.random.default_rng(T + H + D + rot)
    qkv = _bits(rng, T, (H + 2 * heads) * D)
    qkv.reshape(T, H + 2 * heads, D)[T // 2, -1] = 0  # a value row of zeros
    pages = -(-T // P) + 3
    cache = _new_cache(pages, heads, P, D, int8)
    before = [None if t is None else t.clone() for t in cache.tensors]
    slots = rng.permutation(pages * P)[:T].astype(np.int32)
    pos = rng.integers(0, 500, T).astype(np.int32)
    if T > 4:
        slots[2] = -1  # a padding token
        pos[2] = 10 ** 6
    cos, sin = _tables(500, rot)
    dev = dev_bf16(qkv).view(T, H + 2 * heads, D)
    q_out = torch.full((T, H, D), 5.0, dtype=torch.bfloat16, device="cuda") if H else None
    up = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    sq.sq_rope_kv_append(dev[:, :H] if H else None, dev[:, H:H + heads], dev[:, H + heads:], up(cos) if rot else None,
                         up(sin) if rot else None, up(pos) if rot else None, up(slots), cache, q_out, interleaved=pairs)
    sq.sq_sync_status()
    x = wl.bf16_bits_to_f32(qkv).reshape(T, H + 2 * heads, D)
    keep = slots >= 0
    c, s = (cos[np.where(keep, pos, 0)], sin[np.where(keep, pos, 0)]) if rot else (cos[[0] * T], sin[[0] * T])
    turned = osv.rotate(x[:, :H + heads], c, s, pairs)
    if H:
        want = oracle.float_to_bf16(turned[:, :H])
        got = host_bits(q_out)
        assert np.array_equal(got[keep], want[keep])
        assert np.all(got[~keep] == oracle.float_to_bf16(np.float32(5.0)))
    for n, y in ((0, turned[:, H:]), (1, x[:, H + heads:])):
        want, scales = before[n].clone(), None
        page, off = slots[keep] // P, slots[keep] % P
        if int8:
            codes, sc = osv.kv_codes(y[keep])
            scales = before[2 + n].clone()
            want[page, :, off] = torch.from_numpy(codes).cuda()
            scales[page, :, off] = torch.from_numpy(sc).cuda()
            assert torch.equal(cache.tensors[2 + n].view(torch.int32), scales.view(torch.int32))
        else:
            want[page, :, off] = dev_bf16(oracle.float_to_bf16(y[keep]))
        # everything else in the cache is as it was, bit for bit
        assert torch.equal(cache.tensors[n].view(torch.int8), want.view(torch.int8))


def test_append_in_place_and_interleaved_storage():
    """q rotated in place; keys and values in one tensor [pages, 2, heads, page_size, D]."""
    rng = np.random.default_rng(3)
    T, H, heads, D, P = 9, 4, 2, 128, 4
    q, k, v = dev_bf16(_bits(rng, T, H, D)), dev_bf16(_bits(rng, T, heads, D)), dev_bf16(_bits(rng, T, heads, D))
    both = torch.zeros(4, 2, heads, P, D, dtype=torch.bfloat16, device="cuda")
    cos, sin = (torch.from_numpy(t).cuda() for t in _tables(64, D))
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    slots = torch.arange(T, dtype=torch.int32, device="cuda") + 3
    want_q = empty((T, H, D), torch.bfloat16)
    plain = _new_cache(4, heads, P, D, False)
    sq.sq_rope_kv_append(q, k, v, cos, sin, pos, slots, plain, want_q)
    cache = sq.KvCache(both[:, 0], both[:, 1])
    sq.sq_rope_kv_append(q, k, v, cos, sin, pos, slots, cache, q)
    sq.sq_sync_status()
    assert torch.equal(q, want_q)
    for n in range(2):
        a, b = both[:, n].transpose(1, 2).reshape(-1, heads, D), plain.tensors[n].transpose(1, 2).reshape(-1, heads, D)
        assert torch.equal(a[3:3 + T], b[3:3 + T]) and bool((a[:3] == 0).all())


@pytest.mark.parametrize("what", ["slot", "position", "negative position"])
def test_append_out_of_range_is_skipped_and_reported(what):
    rng = np.random.default_rng(1)
    T, D, P = 4, 64, 8
    k = dev_bf16(_bits(rng, T, 1, D))
    cache = _new_cache(2, 1, P, D, True)
    before = [t.clone() for t in cache.tensors]
    cos, sin = (torch.from_numpy(t).cuda() for t in _tables(32, D))
    pos, slots = np.arange(T, dtype=np.int32), np.arange(T, dtype=np.int32)
    if what == "slot":
        slots[2] = 2 * P
    else:
        pos[2] = 32 if what == "position" else -1
    sq.sq_rope_kv_append(None, k, k, cos, sin, torch.from_numpy(pos).cuda(), torch.from_numpy(slots).cuda(), cache, None)
    with pytest.raises(sq.SqError) as ei:
        sq.sq_sync_status()
    assert ei.value.status == sq.SQ_ERR_BOUNDS
    sq.sq_sync_status()  # cleared
    for t, b in zip((host(t) for t in cache.tensors), (host(t) for t in before)):
        assert t[0, :, 2].tobytes() == b[0, :, 2].tobytes()
        assert t[0, :, 3].tobytes() != b[0, :, 3].tobytes()
        assert t[1].tobytes() == b[1].tobytes()


# ---------------------------------------------------------------- attention
def _filled(rng, pages, heads, P, D, int8, scale=1.0):
    """A cache of random contents and its fp64 values."""
    if int8:
        codes = rng.integers(-127, 128, (2, pages, heads, P, D)).astype(np.int8)
        sc = rng.uniform(0.005, 0.02, (2, pages, heads, P)).astype(np.float32)
        t = [torch.from_numpy(codes[n]).cuda() for n in range(2)] + [torch.from_numpy(sc[n]).cuda() for n in range(2)]
        return sq.KvCache(*t), [codes[n].astype(np.float64) * sc[n].astype(np.float64)[..., None] for n in range(2)]
    bits = [_bits(rng, pages, heads, P, D, scale=scale) for _ in range(2)]
    return (sq.KvCache(dev_bf16(bits[0]), dev_bf16(bits[1])),
            [wl.bf16_bits_to_f32(b).astype(np.float64) for b in bits])


def _check_attention(out, lse, ref, D, longest):
    """fp32 scores: D/8 + 16 additions and scalings of at most 2^-23 of the sum of absolute products
    (e); probabilities exp(s - m) inherit twice that, plus 2^-20 of the exponential, of their split
    into two bf16 parts and of the joins' factors; sums over the tokens: at most longest/64 + 128
    additions in a row at 2^-23; out is rounded once, by at most 2^-8 of itself. A probability below
    fp32's normal range, 2^-126, may vanish, whatever is left of the row: with a dominant token of
    value exactly 0 (a zero code) nothing else is left, so `longest` such probabilities times a
    value (below 8 in these caches) are allowed absolutely."""
    o, l, most, absv = ref
    e = (D / 8 + 16) * 2.0 ** -23 * most
    rel = 2 * e + 2.0 ** -18 + 2 * (longest / 64 + 128) * 2.0 ** -23
    got = wl.bf16_bits_to_f32(host_bits(out)).astype(np.float64)
    err = np.abs(got - o)
    bound = 2.0 ** -8 * np.abs(o) + rel[..., None] * absv * (1 + 2.0 ** -8) + longest * 2.0 ** -126 * 8
    assert np.all(err <= bound), float(np.nanmax(err / np.maximum(bound, 1e-300)))
    if lse is not None:
        g = host(lse).astype(np.float64)
        empty_row = np.isneginf(l)
        assert np.array_equal(np.isneginf(g), empty_row)
        ok = ~empty_row
        assert np.all(np.abs(g[ok] - l[ok]) <= rel[ok] + 2.0 ** -22 * (np.abs(l[ok]) + most[ok]))


ATTEND = [  # lens, H, heads, D, page_size, window
    ([1], 1, 1, 64, 1, 0), ([1], 4, 1, 128, 16, 0), ([2, 15, 16, 17], 8, 2, 64, 16, 0), ([33, 0, 1, 64], 6, 3, 96, 8, 0),
    ([100, 31, 250], 16, 2, 128, 32, 0), ([700], 8, 1, 128, 64, 0), ([5, 300], 12, 1, 64, 4, 0),
    ([65, 129, 0, 0, 7], 2, 2, 256, 16, 0), ([511, 512, 513], 16, 1, 256, 128, 0), ([40, 90], 9, 3, 96, 2, 0),
    ([200, 10, 64], 8, 8, 128, 16, 1), ([200, 10, 64], 8, 4, 64, 1, 50), ([513, 1, 100], 32, 2, 128, 16, 129),
    ([1500, 16, 1499], 24, 1, 64, 512, 1000), ([0], 4, 2, 64, 16, 0), ([77], 48, 1, 96, 16, 33)]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("lens,H,heads,D,P,window", ATTEND)
def test_attention_against_fp64(lens, H, heads, D, P, window, int8):
    rng = np.random.default_rng(sum(lens) + H + D + P)
    B, width = len(lens), -(-max(max(lens), 1) // P) + 1
    need = [-(-n // P) for n in lens]
    pages = sum(need) + 2
    cache, (k, v) = _filled(rng, pages, heads, P, D, int8)
    order, table, at = rng.permutation(pages), np.full((B, width), -9, np.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    # what lies behind a sequence's end in its last page is never used: poison it
    for b, n in enumerate(lens):
        if n % P:
            page = int(table[b, n // P])
            for t in cache.tensors:
                if t is not None:
                    t[page, :, n % P:] = 127 if t.dtype == torch.int8 else float("nan")
    q = _bits(rng, B, H, D)
    out, lse = _attend(dev_bf16(q), cache, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                       D ** -0.5, window)
    sq.sq_sync_status()
    ref = osv.paged_attention(wl.bf16_bits_to_f32(q).astype(np.float64), k, v, table, lens, D ** -0.5, window)
    _check_attention(out, lse, ref, D, max(lens))
    assert bool((out[torch.tensor(lens) == 0] == 0).all())


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("lens,H,heads,D,P", [
    ([20000], 8, 2, 128, 16), ([9000, 3, 4000, 1, 0, 700], 16, 4, 64, 32), ([130] * 300, 4, 2, 64, 16),
    ([7] * 40 + [5000], 5, 5, 96, 8), ([3000, 2999], 64, 4, 256, 64)])
def test_attention_long_and_ragged(lens, H, heads, D, P, int8):
    """Lengths that are split over many blocks, many short ones, both; the same inputs give the
    same bits, and the workspace serves one call after another."""
    rng = np.random.default_rng(len(lens) + D)
    B, width = len(lens), -(-max(lens) // P)
    pages = 700
    cache, (k, v) = _filled(rng, pages, heads, P, D, int8)
    table = rng.integers(0, pages, (B, width)).astype(np.int32)  # pages may be shared
    q = _bits(rng, B, H, D)
    dq, dt, dl = dev_bf16(q), torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    ws = sq.workspace(sq.SQ_OP_PAGED_ATTENTION, B, H, D)
    out, lse = _attend(dq, cache, dt, dl, D ** -0.5, ws=ws)
    again, lse2 = _attend(dq, cache, dt, dl, D ** -0.5, ws=ws)
    sq.sq_sync_status()
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    ref = osv.paged_attention(wl.bf16_bits_to_f32(q).astype(np.float64), k, v, table, lens, D ** -0.5)
    _check_attention(out, lse, ref, D, max(lens))


@pytest.mark.parametrize("int8", [False, True])
def test_attention_large_scores(int8):
    """Scores of several hundred: only differences to the maximum are exponentiated; a negative
    scale turns the order round."""
    rng = np.random.default_rng(6)
    cache, (k, v) = _filled(rng, 12, 2, 16, 64, int8)
    q = _bits(rng, 2, 4, 64, scale=30)
    table = rng.integers(0, 12, (2, 12)).astype(np.int32)
    lens = [190, 77]
    for scale in (1.0, -1.0, 0.0):
        out, lse = _attend(dev_bf16(q), cache, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                           scale)
        sq.sq_sync_status()
        ref = osv.paged_attention(wl.bf16_bits_to_f32(q).astype(np.float64), k, v, table, lens, scale)
        _check_attention(out, lse, ref, 64, 190)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("lens,H", [([40], 4), ([700, 33], 4), ([2000], 24)])
def test_attention_nonfinite_query_stays_in_its_head(lens, H, int8):
    rng = np.random.default_rng(H)
    B, D, P = len(lens), 64, 16
    table = np.arange(B * 125, dtype=np.int32).reshape(B, 125)
    cache, (k, v) = _filled(rng, B * 125, 2, P, D, int8)
    q = _bits(rng, B, H, D)
    clean = wl.bf16_bits_to_f32(q).astype(np.float64)
    q[0, 1, 5], q[B - 1, H - 1, 63] = 0x7FC0, 0x7F80  # NaN, infinity
    out, lse = _attend(dev_bf16(q), cache, torch.from_numpy(table).cuda(),
                       torch.tensor(lens, dtype=torch.int32).cuda(), D ** -0.5)
    sq.sq_sync_status()
    for b, h in ((0, 1), (B - 1, H - 1)):
        assert bool(torch.isnan(out[b, h]).all()) and bool(torch.isnan(lse[b, h]))
    keep = np.ones((B, H), bool)
    keep[0, 1] = keep[B - 1, H - 1] = False
    o, l, most, absv = osv.paged_attention(clean, k, v, table, lens, D ** -0.5)
    mask = torch.from_numpy(keep).cuda()
    _check_attention(out[mask], lse[mask], (o[keep], l[keep], most[keep], absv[keep]), D, max(lens))


@pytest.mark.parametrize("int8", [False, True])
def test_attention_bad_pages_and_lengths(int8):
    """A page out of range hides its tokens, lengths are cut to the table; both are reported."""
    rng = np.random.default_rng(2)
    cache, (k, v) = _filled(rng, 6, 1, 16, 64, int8)
    table = np.array([[0, 6, 2], [3, -1, -1], [4, 5, 1], [-2, 9, 0]], np.int32)
    lens = np.array([48, 40, 1000, 32], np.int32)
    q = _bits(rng, 4, 2, 64)
    ws = sq.workspace(sq.SQ_OP_PAGED_ATTENTION, 4, 2, 64)
    out, lse = _attend(dev_bf16(q), cache, torch.from_numpy(table).cuda(), torch.from_numpy(lens).cuda(), 0.125, ws=ws)
    with pytest.raises(sq.SqError) as ei:
        sq.sq_sync_status()
    assert ei.value.status == sq.SQ_ERR_BOUNDS
    ref = osv.paged_attention(wl.bf16_bits_to_f32(q).astype(np.float64), k, v, table, lens, 0.125)
    _check_attention(out, lse, ref, 64, 48)
    assert bool((out[3] == 0).all()) and bool(torch.isneginf(lse[3]).all())
    # the next call with the same workspace is sound
    ok = np.array([[0, 1, 2]] * 4, np.int32)
    out, lse = _attend(dev_bf16(q), cache, torch.from_numpy(ok).cuda(),
                       torch.tensor([48, -5, 1, 20], dtype=torch.int32).cuda(), 0.125, ws=ws)
    with pytest.raises(sq.SqError):
        sq.sq_sync_status()
    ref = osv.paged_attention(wl.bf16_bits_to_f32(q).astype(np.float64), k, v, ok, [48, 0, 1, 20], 0.125)
    _check_attention(out, lse, ref, 64, 48)


def test_attention_far_pages():
    """Pages whose byte offsets pass 32 bits: the strided view of a large allocation."""
    rng = np.random.default_rng(4)
    stride = (1 << 31) // 2 + 4096  # elements; page 3 starts beyond 2^32 bytes of int8
    buf = torch.empty(3 * stride + 16 * 64, dtype=torch.int8, device="cuda")
    views = [torch.as_strided(buf, (4, 1, 8, 64), (stride, 512, 64, 1), off) for off in (0, 512)]
    codes = rng.integers(-127, 128, (2, 4, 1, 8, 64)).astype(np.int8)
    for n in range(2):
        views[n].copy_(torch.from_numpy(codes[n]).cuda())
    sc = rng.uniform(0.005, 0.02, (2, 4, 1, 8)).astype(np.float32)
    cache = sq.KvCache(views[0], views[1], torch.from_numpy(sc[0]).cuda(), torch.from_numpy(sc[1]).cuda())
    k, v = (codes[n].astype(np.float64) * sc[n].astype(np.float64)[..., None] for n in range(2))
    table, lens = np.array([[3, 1, 0, 2]], np.int32), [30]
    q = _bits(rng, 1, 2, 64)
    out, lse = _attend(dev_bf16(q), cache, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), 0.125)
    sq.sq_sync_status()
    _check_attention(out, lse, osv.paged_attention(wl.bf16_bits_to_f32(q).astype(np.float64), k, v, table, lens, 0.125),
                     64, 30)
    # and the append writes there
    x = dev_bf16(_bits(rng, 1, 1, 64))
    sq.sq_rope_kv_append(None, x, x, None, None, None, torch.tensor([3 * 8 + 7], dtype=torch.int32, device="cuda"), cache,
                         None)
    sq.sq_sync_status()
    want, _ = osv.kv_codes(wl.bf16_bits_to_f32(host_bits(x)).reshape(1, 1, 64))
    assert np.array_equal(host(views[1][3, 0, 7]), want[0, 0])


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("int8", [False, True])
def test_decode_loop(int8):
    """A prompt of uneven lengths appended in one call, then steps of one token per sequence with a
    padded batch row, each append followed by the attention, captured once as a graph and replayed;
    checked against fp64 attention over the values the cache stands for."""
    rng = np.random.default_rng(11)
    H, heads, D, P, max_pages = 8, 2, 64, 8, 8
    lens = [19, 1, 40]
    B = len(lens) + 1  # the last row is padding
    cache = _new_cache(B * max_pages, heads, P, D, int8)
    table = rng.permutation(B * max_pages).reshape(B, max_pages).astype(np.int32)
    cos, sin = (torch.from_numpy(t).cuda() for t in _tables(64, D))
    pos = np.concatenate([np.arange(n) for n in lens]).astype(np.int32)
    seq = np.repeat(np.arange(len(lens)), lens)
    slots = (table[seq, pos // P] * P + pos % P).astype(np.int32)
    T = pos.size
    qkv = dev_bf16(_bits(rng, T, H + 2 * heads, D))
    q_out = empty((T, H, D), torch.bfloat16)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    sq.sq_rope_kv_append(qkv[:, :H], qkv[:, H:H + heads], qkv[:, H + heads:], cos, sin, up(pos), up(slots), cache, q_out)

    dt = up(table)
    ws = sq.workspace(sq.SQ_OP_PAGED_ATTENTION, B, H, D)
    step = dev_bf16(_bits(rng, B, H + 2 * heads, D))
    d_pos, d_slots, d_len = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(3))
    q1, out, lse = empty((B, H, D), torch.bfloat16), empty((B, H, D), torch.bfloat16), empty((B, H), torch.float32)
    q1.zero_()

    def one():
        sq.sq_rope_kv_append(step[:, :H], step[:, H:H + heads], step[:, H + heads:], cos, sin, d_pos, d_slots, cache, q1)
        sq.sq_paged_attention(q1, cache, dt, d_len, D ** -0.5, out, lse=lse, ws=ws)

    def stage(n):
        p = np.array([m + n for m in lens] + [0], np.int32)
        s = np.array([table[b, p[b] // P] * P + p[b] % P for b in range(len(lens))] + [-1], np.int32)
        step.copy_(dev_bf16(_bits(rng, B, H + 2 * heads, D)))
        d_pos.copy_(up(p))
        d_slots.copy_(up(s))
        d_len.copy_(up(np.array([m + n + 1 for m in lens] + [0], np.int32)))

    graph = None
    for n in range(5):
        stage(n)
        if n == 2:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                one()
        if graph is not None:
            graph.replay()
        else:
            one()
        sq.sq_sync_status()
        vals = []
        for i in range(2):
            x = cache.tensors[i].double()
            if int8:
                x = x * torch.nan_to_num(cache.tensors[2 + i]).double()[..., None]
            vals.append(np.nan_to_num(x.cpu().numpy()))
        now = [m + n + 1 for m in lens] + [0]
        ref = osv.paged_attention(wl.bf16_bits_to_f32(host_bits(q1)).astype(np.float64), *vals, table, now, D ** -0.5)
        _check_attention(out, lse, ref, D, max(now))


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("B,longest,holes", [(33, 200, False), (1000, 40, True), (2500, 20, True), (5000, 3, False)])
def test_attention_many_sequences(B, longest, holes, int8):
    """More sequences than lanes, and than lanes squared, with empty ones among them, long runs of
    them and at both ends."""
    rng = np.random.default_rng(B)
    H, heads, D, P = 2, 1, 64, 8
    cache, (k, v) = _filled(rng, 100, heads, P, D, int8)
    lens = rng.integers(0 if holes else 1, longest + 1, B)
    if holes:
        lens[:40] = lens[-70:] = lens[B // 2:B // 2 + 100] = 0
    table = rng.integers(0, 100, (B, -(-longest // P))).astype(np.int32)
    q = _bits(rng, B, H, D)
    out, lse = _attend(dev_bf16(q), cache, torch.from_numpy(table).cuda(), torch.from_numpy(lens.astype(np.int32)).cuda(),
                       D ** -0.5)
    sq.sq_sync_status()
    ref = osv.paged_attention(wl.bf16_bits_to_f32(q).astype(np.float64), k, v, table, list(lens), D ** -0.5)
    _check_attention(out, lse, ref, D, longest)


def test_one_workspace_for_calls_of_any_shape():
    """The counters of a large batch lie where an earlier call of another shape, head dimension or
    cache type left none of its partial sums: one workspace, sized for the largest."""
    rng = np.random.default_rng(21)
    ws = sq.workspace(sq.SQ_OP_PAGED_ATTENTION, 300, 64, 64)
    for B, H, heads, D, n, int8 in [(1, 8, 1, 256, 3000, False), (300, 64, 32, 64, 40, True), (2, 32, 8, 128, 2500, True),
                                    (300, 8, 2, 96, 70, False), (1, 64, 4, 256, 4000, True), (260, 64, 64, 64, 17, False)]:
        cache, (k, v) = _filled(rng, 200, heads, 16, D, int8)
        lens = [max(1, n - 7 * (b % 5)) for b in range(B)]
        table = rng.integers(0, 200, (B, -(-n // 16))).astype(np.int32)
        q = _bits(rng, B, H, D)
        out, lse = _attend(dev_bf16(q), cache, torch.from_numpy(table).cuda(),
                           torch.tensor(lens, dtype=torch.int32).cuda(), D ** -0.5, ws=ws)
        sq.sq_sync_status()
        ref = osv.paged_attention(wl.bf16_bits_to_f32(q).astype(np.float64), k, v, table, lens, D ** -0.5)
        _check_attention(out, lse, ref, D, n)


def test_nonfinite_keys_and_values_show_in_an_int8_cache():
    """A NaN or an infinity in an appended row is kept as its scale: attention over that token gives
    NaN for the key head's queries and for no others."""
    x = torch.randn(3, 2, 64, device="cuda").to(torch.bfloat16)
    bad_k, bad_v = x.clone(), x.clone()
    bad_k[1, 0, 5] = float("nan")
    bad_v[2, 1, 63] = float("inf")
    cache = _new_cache(1, 2, 16, 64, True)
    idx = torch.arange(3, dtype=torch.int32, device="cuda")
    sq.sq_rope_kv_append(None, bad_k, bad_v, None, None, None, idx, cache, None)
    ks, vs = cache.tensors[2][0, :, :3], cache.tensors[3][0, :, :3]
    assert bool(torch.isnan(ks[0, 1])) and int(torch.isfinite(ks).sum()) == 5
    assert bool(torch.isinf(vs[1, 2])) and int(torch.isfinite(vs).sum()) == 5
    q = torch.randn(1, 4, 64, device="cuda").to(torch.bfloat16)
    for n, finite in ((1, [True] * 4), (2, [False, False, True, True]), (3, [False] * 4)):
        out, _ = _attend(q, cache, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                         torch.tensor([n], dtype=torch.int32, device="cuda"), 0.125)
        assert [bool(torch.isfinite(out[0, h]).all()) for h in range(4)] == finite
    sq.sq_sync_status()


def test_two_streams_with_their_own_workspaces():
    rng = np.random.default_rng(12)
    cache, (k, v) = _filled(rng, 200, 2, 16, 128, True)
    streams, runs = [torch.cuda.Stream() for _ in range(2)], []
    for n in range(2):
        q = _bits(rng, 3, 8, 128)
        table, lens = rng.integers(0, 200, (3, 100)).astype(np.int32), [1600, 900 + n, 33]
        runs.append((q, table, lens, dev_bf16(q), torch.from_numpy(table).cuda(),
                     torch.tensor(lens, dtype=torch.int32).cuda(), empty((3, 8, 128), torch.bfloat16),
                     sq.workspace(sq.SQ_OP_PAGED_ATTENTION, 3, 8, 128)))
    torch.cuda.synchronize()
    for _ in range(10):
        for st, r in zip(streams, runs):
            sq.sq_paged_attention(r[3], cache, r[4], r[5], 128 ** -0.5, r[6], ws=r[7], stream=st)
    torch.cuda.synchronize()
    sq.sq_sync_status()
    for r in runs:
        ref = osv.paged_attention(wl.bf16_bits_to_f32(r[0]).astype(np.float64), k, v, r[1], r[2], 128 ** -0.5)
        _check_attention(r[6], None, ref, 128, max(r[2]))


def test_binding_refusals():
    cache = _new_cache(4, 2, 8, 64, True)
    q, t, n = empty((3, 4, 64), torch.bfloat16), torch.zeros(3, 4, dtype=torch.int32, device="cuda"), \
        torch.ones(3, dtype=torch.int32, device="cuda")
    out, ws = empty((3, 4, 64), torch.bfloat16), sq.workspace(sq.SQ_OP_PAGED_ATTENTION, 3, 4, 64)
    for args, kw, err in (((q.float(), cache, t, n, 1.0, out), {}, TypeError), ((q, cache, t.long(), n, 1.0, out), {}, TypeError),
                          ((q, cache, t[:2], n, 1.0, out), {}, ValueError), ((q, cache, t, n[:2], 1.0, out), {}, ValueError),
                          ((q, cache, t, n, 1.0, out[:2]), {}, ValueError), ((q[..., :32], cache, t, n, 1.0, out), {}, ValueError),
                          ((q[:, :3], cache, t, n, 1.0, out[:, :3].contiguous()), {}, sq.SqError),
                          ((q, cache, t, n, float("nan"), out), {}, sq.SqError)):
        with pytest.raises(err):
            sq.sq_paged_attention(*args, ws=ws, **kw)
    k = empty((3, 2, 64), torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        sq.sq_rope_kv_append(None, k, k, None, None, None, slots, cache, out)
    with pytest.raises(ValueError):
        sq.sq_rope_kv_append(None, k[:, :1], k[:, :1], None, None, None, slots, cache, None)
    with pytest.raises(ValueError):
        sq.KvCache(cache.tensors[0], cache.tensors[1])
    with pytest.raises(TypeError):
        sq.KvCache(cache.tensors[0], cache.tensors[1], cache.tensors[2].double(), cache.tensors[3].double())
