"""What is measured of the 4-bit weight linear and the paged key-value cache operators.

Each case is one pass of one operator:

* ``int4_weight``: group quantization of a smoothed weight to 4 bits, read back as bf16 values;
* ``int4_linear``: the product of a few tokens with a 4-bit weight;
* ``kv_append``: rotation of queries and keys by position, keys and values into a paged cache;
* ``paged_attention``: attention of one new token per sequence over that cache.

The module's ``own`` says which side ``run`` computes: the operators' plain form in torch
operations of 32 bits, or the framework's kernels.
"""
import math
import random

import torch

own = False

DEV = "cuda"
FLT_MAX = 3.4028234663852886e38


def listed():
    return [
        # quantizing an attention projection's weight at load time, symmetric codes
        dict(name="int4_weight_4096x4096", op="int4_weight", N=4096, K=4096, group=128, asym=False),
        # the largest feed-forward weight, small groups with zero points
        dict(name="int4_weight_28672x8192", op="int4_weight", N=28672, K=8192, group=64, asym=True),
        # decoding for one user: an attention projection (latency)
        dict(name="int4_linear_1x4096x4096", op="int4_linear", M=1, N=4096, K=4096, group=128, asym=False, bias=False),
        # a small batch on a feed-forward up-projection, the finest groups, with bias
        dict(name="int4_linear_5x11008x4096", op="int4_linear", M=5, N=11008, K=4096, group=32, asym=True, bias=True),
        # a serving batch on the largest feed-forward weight (bandwidth)
        dict(name="int4_linear_16x28672x8192", op="int4_linear", M=16, N=28672, K=8192, group=128, asym=True, bias=False),
        # the largest decode batch on a square projection
        dict(name="int4_linear_64x8192x8192", op="int4_linear", M=64, N=8192, K=8192, group=64, asym=False, bias=True),
        # one decode step of a batch of 64 sequences: each appends its token (latency)
        dict(name="kv_append_64_int8", op="kv_append", T=64, H=32, Hkv=8, D=128, R=128, P=16, int8=True, pairs=False),
        # a long prompt, eight queries to a key head, int8 cache
        dict(name="kv_append_8192_int8", op="kv_append", T=8192, H=64, Hkv=8, D=128, R=128, P=64, int8=True,
             pairs=False),
        # an odd prompt, as many key heads as query heads, adjacent pairs, half of the head rotated, bf16 cache
        dict(name="kv_append_2047_bf16", op="kv_append", T=2047, H=32, Hkv=32, D=128, R=64, P=128, int8=False,
             pairs=True),
        # one user with a long context: the split over the length (latency)
        dict(name="attention_1x8192_int8", op="paged_attention", B=1, L=8192, H=32, Hkv=8, D=128, P=16, int8=True,
             window=0),
        # a serving batch of ragged lengths (bandwidth)
        dict(name="attention_64x8192_int8", op="paged_attention", B=64, L=8192, H=64, Hkv=8, D=128, P=64, int8=True,
             window=0),
        # an odd batch of short contexts, one key head to each query head, bf16 cache with a sliding window
        dict(name="attention_13x1500_bf16", op="paged_attention", B=13, L=1500, H=32, Hkv=32, D=64, P=32, int8=False,
             window=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("int4_weight", "int4_linear", "int4_linear", "kv_append", "paged_attention", "paged_attention"))
    if op in ("int4_weight", "int4_linear"):
        K = 16 * _log(rng, 16, 1792)                      # 256 .. 28672
        N = 8 * _log(rng, 32, min(3584, 29360128 // K))   # 256 .. 28672, N * K at most that of 28672 x 8192
        c = dict(op=op, N=N, K=K, group=rng.choice((32, 64, 128)), asym=rng.random() < 0.5)
        if op == "int4_linear":
            c.update(M=_log(rng, 1, 64), bias=rng.random() < 0.5)
        return c
    D = rng.choice((64, 96, 128, 256))
    Hkv = rng.choice((1, 2, 4, 8, 16, 32))
    H = Hkv * rng.choice((1, 2, 3, 4, 6, 7, 8, 12, 16))
    while H > 64:
        H = Hkv * rng.choice((1, 2, 3, 4, 8, 12, 16))
    c = dict(op=op, H=H, Hkv=Hkv, D=D, P=rng.choice((1, 8, 16, 32, 64, 128)), int8=rng.random() < 0.6)
    if op == "kv_append":
        T = _log(rng, 1, min(8192, 8192 * 80 * 128 // ((H + 2 * Hkv) * D)))
        c.update(T=T, R=16 * rng.randint(1, D // 16), pairs=rng.random() < 0.5)
        return c
    L = _log(rng, 1, 32768)
    # cache bytes at most those of 64 sequences of 8192 tokens with 8 heads of 128 bytes
    B = _log(rng, 1, max(1, min(256, (64 * 8192 * 8 * 128) // (L * Hkv * D * (1 if c["int8"] else 2)))))
    c.update(L=L, B=B, window=rng.choice((0, 0, 1 + rng.randrange(4096))))
    return c


def lengths(case):
    """The sequences' lengths, a matter of the case alone: the first is the longest."""
    r = random.Random("%(B)d sequences of up to %(L)d tokens" % case)
    return [case["L"]] + [1 + int((case["L"] - 1) * (0.25 + 0.75 * r.random())) for _ in range(case["B"] - 1)]


def work(case):
    op = case["op"]
    if op in ("int4_weight", "int4_linear"):
        N, K = case["N"], case["K"]
        groups = -(-K // case["group"])
        codes = N * K / 2 + N * groups * (3 if case["asym"] else 2)
        if op == "int4_weight":  # the weight is read, its codes written and read, its values written
            return {"bytes": 2 * N * K + 4 * K + 2 * codes + 2 * N * K, "flops": 4.0 * N * K}
        M = case["M"]
        return {"bytes": codes + 2 * M * K + 2 * M * N + (2 * N if case["bias"] else 0), "flops": 2.0 * M * N * K}
    H, Hkv, D = case["H"], case["Hkv"], case["D"]
    row = D + 4 if case["int8"] else 2 * D  # a token's key (or value) of one head in the cache
    if op == "kv_append":
        T = case["T"]
        return {"bytes": T * (2 * (H + 2 * Hkv) * D + 2 * H * D + 2 * Hkv * row + 4 * case["R"] + 8),
                "flops": 3.0 * T * (H + Hkv) * case["R"]}
    seen = sum(min(n, case["window"] or n) for n in lengths(case))
    return {"bytes": 2 * seen * Hkv * row + 4 * case["B"] * H * D, "flops": 4.0 * seen * H * D}


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return {"case": case, **globals()["_prepare_" + case["op"]](case, g)}


def _normal(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def _prepare_int4_weight(c, g):
    N, K = c["N"], c["K"]
    G = -(-K // c["group"])
    return dict(
        W=_normal(g, N, K, scale=0.02),
        s=torch.exp(torch.randn(K, generator=g, device=DEV) * 0.5),  # smoothing factors
        Wp=torch.empty(packed_bytes(N, K), dtype=torch.uint8, device=DEV),
        w_scale=torch.empty(G, N, dtype=torch.bfloat16, device=DEV),
        w_zero=torch.empty(G, N, dtype=torch.uint8, device=DEV) if c["asym"] else None,
        W_out=torch.empty(N, K, dtype=torch.bfloat16, device=DEV),
    )


def _prepare_int4_linear(c, g):
    M, N, K = c["M"], c["N"], c["K"]
    G = -(-K // c["group"])
    zero = torch.randint(5, 11, (G, N), generator=g, device=DEV, dtype=torch.uint8) if c["asym"] else None
    codes = torch.randn(N, K, generator=g, device=DEV, dtype=torch.float16).mul_(2.6).add_(8).round_().clamp_(0, 15)
    X = torch.randn(M, K, generator=g, device=DEV)
    X[:, torch.randperm(K, generator=g, device=DEV)[:6]] *= 40.0  # outlier channels of the activations
    return dict(
        X=X.to(torch.bfloat16),
        Wp=pack(codes.to(torch.uint8)),
        w_scale=(torch.rand(G, N, generator=g, device=DEV) * 0.01 + 0.005).to(torch.bfloat16),
        w_zero=zero,
        bias=_normal(g, N) if c["bias"] else None,
        Y=torch.empty(M, N, dtype=torch.bfloat16, device=DEV),
    )


def _cache(c, g, pages):
    shape = (pages, c["Hkv"], c["P"], c["D"])
    if not c["int8"]:
        return dict(k_cache=_normal(g, *shape), v_cache=_normal(g, *shape), k_scale=None, v_scale=None)
    codes = [torch.randn(shape, generator=g, device=DEV, dtype=torch.float16).mul_(36).clamp_(-127, 127).to(torch.int8)
             for _ in range(2)]
    scales = [torch.rand(shape[:3], generator=g, device=DEV) * 0.02 + 0.02 for _ in range(2)]
    return dict(k_cache=codes[0], v_cache=codes[1], k_scale=scales[0], v_scale=scales[1])


def _prepare_kv_append(c, g):
    T, H, Hkv, D, R, P = (c[k] for k in ("T", "H", "Hkv", "D", "R", "P"))
    qkv = _normal(g, T, (H + 2 * Hkv) * D)  # the fused projection's output
    heads = qkv.view(T, H + 2 * Hkv, D)
    pages = -(-T // P)
    first = int(torch.randint(0, 100000, (1,), generator=g, device=DEV))
    angle = (torch.arange(first + T, device=DEV, dtype=torch.float64)[:, None]
             * 10000.0 ** (-torch.arange(R // 2, device=DEV, dtype=torch.float64) * 2 / R))
    table = torch.randperm(pages, generator=g, device=DEV)
    t = torch.arange(T, device=DEV)
    state = dict(
        q=heads[:, :H], k=heads[:, H:H + Hkv], v=heads[:, H + Hkv:],
        cos=angle.cos().float(), sin=angle.sin().float(),
        positions=(first + t).to(torch.int32),
        slots=(table[t // P] * P + t % P).to(torch.int32),
        q_out=torch.zeros(T, H, D, dtype=torch.bfloat16, device=DEV),
        **_cache(c, g, pages),
    )
    if c["int8"]:  # where the values that the cache stands for are read back
        state["k_read"], state["v_read"] = (torch.empty(state["k_cache"].shape, dtype=torch.bfloat16, device=DEV)
                                            for _ in range(2))
    return state


def _prepare_paged_attention(c, g):
    B, H, D, P = c["B"], c["H"], c["D"], c["P"]
    n = lengths(c)
    need = [-(-x // P) for x in n]
    pages = sum(need)
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    width = max(need)
    start = torch.tensor([sum(need[:b]) for b in range(B)], device=DEV)
    col = torch.arange(width, device=DEV)
    # rows behind a sequence's last page point at any page
    at = torch.where(col < torch.tensor(need, device=DEV)[:, None], start[:, None] + col, 0)
    return dict(
        q=_normal(g, B, H, D),
        block_table=order[at].contiguous(),
        seq_lens=torch.tensor(n, dtype=torch.int32, device=DEV),
        out=torch.empty(B, H, D, dtype=torch.bfloat16, device=DEV),
        lse=torch.empty(B, H, dtype=torch.float32, device=DEV),
        **_cache(c, g, pages),
    )


# ------------------------------------------------------------------ the packed 4-bit layout

# Tiles of 16 rows by 128 columns, 1024 bytes each, rows and columns padded with code 8. A tile
# holds 16-byte units [row / 8][row % 8][column / 2 % 4]; a unit holds, in this order, the
# columns' bits [column / 32][column % 2][column / 16 % 2] as bytes, whose low nibble has the
# column with column / 8 % 2 == 0 and whose high nibble the one with 1.


def packed_bytes(N, K):
    return (-(-N // 16)) * (-(-K // 128)) * 1024


def pack(codes):
    N, K = codes.shape
    Nt, Kb = -(-N // 16), -(-K // 128)
    full = torch.full((Nt * 16, Kb * 128), 8, dtype=torch.uint8, device=codes.device)
    full[:N, :K] = codes
    #                     0   1  2  3   4  5  6  7  8
    v = full.view(Nt, 2, 8, Kb, 4, 2, 2, 4, 2).permute(0, 3, 1, 2, 7, 4, 8, 5, 6)
    return (v[..., 0] | (v[..., 1] << 4)).reshape(-1)


def unpack(Wp, N, K):
    Nt, Kb = -(-N // 16), -(-K // 128)
    b = Wp.view(Nt, Kb, 2, 8, 4, 4, 2, 2)
    v = torch.stack((b & 15, b >> 4), -1).permute(0, 2, 3, 1, 5, 7, 8, 4, 6)
    return v.reshape(Nt * 16, Kb * 128)[:N, :K]


# ------------------------------------------------------------------ one pass


def run(state):
    return globals()[("_own_" if own else "_plain_") + state["case"]["op"]](state)


def _by_group(t, group, K):
    """[G, N] per-group values as [N, K]."""
    return t.t().repeat_interleave(group, 1)[:, :K]


def _values(codes, scale, zero, group):
    K = codes.shape[1]
    z = 8.0 if zero is None else _by_group(zero.float(), group, K)
    return (codes.float() - z) * _by_group(scale.float(), group, K)


def _plain_int4_weight(st):
    c, group = st["case"], st["case"]["group"]
    N, K = c["N"], c["K"]
    w = st["W"].float() * st["s"]
    v = torch.nn.functional.pad(w, (0, -K % group)).view(N, -1, group)
    if c["asym"]:
        lo, hi = v.amin(2).clamp(max=0), v.amax(2).clamp(min=0)
        span, steps = hi - lo, 15.0
    else:
        span, steps = v.abs().amax(2), 7.0
    scale = (span / torch.full_like(span, steps)).to(torch.bfloat16)
    r = torch.where(scale > 0, (torch.ones_like(span) / scale.float()).clamp(max=FLT_MAX), 0.0)
    zero = None
    if c["asym"]:
        zero = (-lo * r).round().clamp(0, 15)
        q = ((v * r[:, :, None]).round() + zero[:, :, None]).clamp(0, 15) - zero[:, :, None]
        zero = zero.t().to(torch.uint8)
    else:
        q = (v * r[:, :, None]).round().clamp(-8, 7)
    values = (q * scale.float()[:, :, None]).view(N, -1)[:, :K].to(torch.bfloat16)
    return {"values": values, "scale": scale.t(), "zero": zero}


def _plain_int4_linear(st):
    c = st["case"]
    w = _values(unpack(st["Wp"], c["N"], c["K"]), st["w_scale"], st["w_zero"], c["group"])
    y = st["X"].float() @ w.t()
    if st["bias"] is not None:
        y = y + st["bias"].float()
    return y.to(torch.bfloat16)


def _rotate(x, cos, sin, R, pairs):
    """x [T, heads, D] by the angles of its tokens, cos and sin [T, R / 2]."""
    x = x.float()
    c, s = cos[:, None], sin[:, None]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if pairs else (x[..., :R // 2], x[..., R // 2:R])
    a, b = a * c - b * s, b * c + a * s
    turned = torch.stack((a, b), -1).flatten(2) if pairs else torch.cat((a, b), -1)
    return torch.cat((turned, x[..., R:]), -1)


def _plain_kv_append(st):
    c = st["case"]
    cos, sin = st["cos"][st["positions"]], st["sin"][st["positions"]]
    st["q_out"].copy_(_rotate(st["q"], cos, sin, c["R"], c["pairs"]))
    page, off = st["slots"] // c["P"], st["slots"] % c["P"]
    for x, cache, scales in ((_rotate(st["k"], cos, sin, c["R"], c["pairs"]), st["k_cache"], st["k_scale"]),
                             (st["v"].float(), st["v_cache"], st["v_scale"])):
        if c["int8"]:
            a = x.abs().amax(-1)
            steps = torch.full_like(a, 127.0)
            r = torch.where(a > 0, (steps / a).clamp(max=FLT_MAX), 0.0)
            scales[page, :, off] = a / steps
            x = (x * r[..., None]).round().clamp(-128, 127)
        cache[page, :, off] = x.to(cache.dtype)
    return _cache_values(st)


def _cache_values(st):
    k, v = st["k_cache"], st["v_cache"]
    if st["case"]["int8"]:
        k = torch.mul(k, st["k_scale"][..., None], out=st["k_read"])
        v = torch.mul(v, st["v_scale"][..., None], out=st["v_read"])
    return {"q": st["q_out"], "k": k, "v": v}


def _plain_paged_attention(st):
    c = st["case"]
    B, H, Hkv, D = c["B"], c["H"], c["Hkv"], c["D"]

    def rows(cache, scales):
        x = cache[st["block_table"]].float()  # [B, pages, Hkv, P, D]
        if scales is not None:
            x = x * scales[st["block_table"]][..., None]
        return x.transpose(1, 2).reshape(B, Hkv, -1, D)

    k, v = rows(st["k_cache"], st["k_scale"]), rows(st["v_cache"], st["v_scale"])
    s = (st["q"].float().view(B, Hkv, H // Hkv, D) @ k.transpose(2, 3)) * D ** -0.5
    t = torch.arange(s.shape[-1], device=DEV)
    n = st["seq_lens"][:, None]
    seen = (t < n) & (t >= n - (c["window"] or c["L"]))
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / total
    return {"out": out.view(B, H, D).to(torch.bfloat16), "lse": (m + torch.log(total)).view(B, H)}


# ------------------------------------------------------------------ the framework's operators


def _own_int4_weight(st):
    from w8a8_quantized_gemm_b200 import sq
    group = st["case"]["group"]
    sq.sq_quant_weight_int4(st["W"], st["s"], group, st["Wp"], st["w_scale"], st["w_zero"])
    sq.sq_dequant_weight_int4(st["Wp"], st["w_scale"], st["w_zero"], group, st["W_out"])
    return {"values": st["W_out"], "scale": st["w_scale"], "zero": st["w_zero"]}


def _own_int4_linear(st):
    from w8a8_quantized_gemm_b200 import sq
    return sq.sq_int4_linear(st["X"], st["Wp"], st["w_scale"], st["w_zero"], st["case"]["group"], st["bias"], st["Y"])


def _handle(st, sq):
    """The cache's descriptor, which a program makes once for its cache."""
    if "cache" not in st:
        st["cache"] = sq.KvCache(st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"])
    return st["cache"]


def _own_kv_append(st):
    from w8a8_quantized_gemm_b200 import sq
    sq.sq_rope_kv_append(st["q"], st["k"], st["v"], st["cos"], st["sin"], st["positions"], st["slots"],
                         _handle(st, sq), st["q_out"], interleaved=st["case"]["pairs"])
    return _cache_values(st)


def _own_paged_attention(st):
    from w8a8_quantized_gemm_b200 import sq
    c = st["case"]
    if "ws" not in st:  # a program's workspace, made once
        st["ws"] = sq.workspace(sq.SQ_OP_PAGED_ATTENTION, c["B"], c["H"], c["D"], DEV)
    sq.sq_paged_attention(st["q"], _handle(st, sq), st["block_table"], st["seq_lens"], c["D"] ** -0.5, st["out"],
                          lse=st["lse"], window=c["window"], ws=st["ws"])
    return {"out": st["out"], "lse": st["lse"]}


# ------------------------------------------------------------------ the definitions in 64 bits


def exact(case, seed):
    return globals()["_exact_" + case["op"]](prepare(case, seed))


def _exact_int4_weight(st):
    """Group by group; scales and reciprocals are what the definition says, numbers of bf16 and of 32 bits."""
    c, group = st["case"], st["case"]["group"]
    N, K = c["N"], c["K"]
    values, scales, zeros = torch.empty(N, K, dtype=torch.float64, device=DEV), [], []
    for k in range(0, K, group):
        w = st["W"][:, k:k + group].double() * st["s"][k:k + group].double()
        if c["asym"]:
            lo, hi = w.min(1).values.clamp(max=0), w.max(1).values.clamp(min=0)
            e = ((hi - lo) / 15).float().bfloat16().double()
        else:
            e = (w.abs().max(1).values / 7).float().bfloat16().double()
        r = (1 / e).float().double()
        r = torch.where(e > 0, r.clamp(max=FLT_MAX), torch.zeros_like(r))
        if c["asym"]:
            z = torch.round(-lo * r).clamp(0, 15)
            q = (torch.round(w * r[:, None]) + z[:, None]).clamp(0, 15) - z[:, None]
            zeros.append(z.to(torch.uint8))
        else:
            q = torch.round(w * r[:, None]).clamp(-8, 7)
        values[:, k:k + group] = q * e[:, None]
        scales.append(e)
    return {"values": values, "scale": torch.stack(scales), "zero": torch.stack(zeros) if c["asym"] else None}


def _exact_int4_linear(st):
    """Column block by column block of 32, each code read from where the layout puts it."""
    c, group = st["case"], st["case"]["group"]
    M, N, K = c["M"], c["N"], c["K"]
    Kb = -(-K // 128)
    n = torch.arange(N, device=DEV)[:, None]
    y = torch.zeros(M, N, dtype=torch.float64, device=DEV)
    for k0 in range(0, K, 1024):
        k = torch.arange(k0, min(K, k0 + 1024), device=DEV)[None, :]
        unit = ((n // 16 * Kb + k // 128) * 64 + n % 16 * 4 + k // 2 % 4) * 16
        byte = st["Wp"][unit + k % 128 // 32 * 4 + k % 2 * 2 + k // 16 % 2].to(torch.int16)
        q = (byte >> (k // 8 % 2 * 4).to(torch.int16)) & 15
        g = k[0] // group
        z = st["w_zero"][g].t().double() if c["asym"] else 8.0
        y += st["X"][:, k0:k0 + 1024].double() @ ((q.double() - z) * st["w_scale"][g].t().double()).t()
    return y + st["bias"].double() if c["bias"] else y


def _exact_kv_append(st):
    c = st["case"]
    R, D = c["R"], c["D"]
    i = torch.arange(D, device=DEV)
    if c["pairs"]:
        mate, angle, sign = i ^ 1, i // 2, torch.where(i % 2 == 0, -1.0, 1.0)
    else:
        mate, angle, sign = (i + R // 2) % max(R, 1), i % max(R // 2, 1), torch.where(i < R // 2, -1.0, 1.0)
    mate, angle = torch.where(i < R, mate, i), torch.where(i < R, angle, 0)
    at = st["positions"].long()
    cos = torch.where(i < R, st["cos"].double()[at][:, angle], 1.0)[:, None]
    sin = torch.where(i < R, st["sin"].double()[at][:, angle] * sign, 0.0)[:, None]

    def turn(x):
        x = x.double()
        return x * cos + x[..., mate] * sin

    slots = st["slots"].long()
    res = {"q": turn(st["q"])}
    for name, x in (("k", turn(st["k"])), ("v", st["v"].double())):
        full = st[name + "_cache"].double()
        if c["int8"]:
            full = full * st[name + "_scale"].double()[..., None]
            a = x.abs().amax(-1, keepdim=True)
            x = torch.round(x * torch.where(a > 0, 127 / a, 0.0)).clamp(-128, 127) * (a / 127)
        full = full.transpose(1, 2).reshape(-1, c["Hkv"], D)  # by slot
        full[slots] = x
        res[name] = full.view(-1, c["P"], c["Hkv"], D).transpose(1, 2)
    return res


def _exact_paged_attention(st):
    c = st["case"]
    H, Hkv, D = c["H"], c["Hkv"], c["D"]
    outs, lses = [], []
    for b, n in enumerate(lengths(c)):
        first = max(0, n - c["window"]) if c["window"] else 0
        t = torch.arange(first, n, device=DEV)
        page, off = st["block_table"][b].long()[t // c["P"]], t % c["P"]
        k, v = (st[x + "_cache"][page, :, off].double() for x in "kv")  # [n, Hkv, D]
        if c["int8"]:
            k, v = (x * st[y + "_scale"][page, :, off].double()[..., None] for x, y in ((k, "k"), (v, "v")))
        s = torch.einsum("hgd,thd->hgt", st["q"][b].double().view(Hkv, H // Hkv, D), k) / math.sqrt(D)
        lse = torch.logsumexp(s, -1)
        outs.append(torch.einsum("hgt,thd->hgd", torch.exp(s - lse[..., None]), v).reshape(H, D))
        lses.append(lse.reshape(H))
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}
