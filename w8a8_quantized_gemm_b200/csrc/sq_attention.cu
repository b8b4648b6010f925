// Attention of one new token per sequence over a paged key-value cache, bf16 or int8.
//   s_t = scale * (q . k_t),  out = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m)
// "SmoothQuant量化实战" §5.2 (KV-cache INT8 with per-token, per-head scales).
//
// Every key and value is read once for all query heads of its key head: at 4 to 16 flops a
// byte the call is bound by the bytes of the cache. The work is cut into tiles of 16 tokens of
// one key head; all tiles, in the order (sequence, key head, token), form one line that is
// dealt out evenly: each CTA (one per SM) gets a contiguous piece of it and each of its warps a
// contiguous piece of that, whatever the sequences' lengths. A warp works by itself: it brings
// its tiles into its own ring of shared memory with asynchronous copies, several tiles ahead,
// and keeps the running maximum m, the sum l and the unnormalised output of the 8 (or 16) query
// heads in registers. Only where a piece ends inside a key head's tiles is the state joined with
// its neighbours': within the CTA in shared memory, between CTAs through the workspace, where
// the last CTA to arrive adds the parts up in the order of the line. So results do not depend
// on which CTA is last.
//
// Matrix instructions (16x8x16, bf16 in, fp32 sums): scores are K (16 tokens x head_dim) times
// q^T (head_dim x 8 heads), outputs V^T (16 elements x 16 tokens) times p^T (16 tokens x 8
// heads): tokens and elements fill the 16 rows, heads the 8 columns. int8 codes become bf16
// exactly in registers: with s the sign bit of a byte, 128 + (low 7 bits) and 128 + 128 s are
// both bf16 numbers made by one logic operation each, and their difference is the code. The
// fp32 probabilities (times a token's value scale) enter as two bf16 parts, high and low, so
// that the rounding of out to bf16 is the only one that counts.
#include "sq_internal.h"
#include "sq_ptx.cuh"

#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

namespace sq {
namespace {

constexpr int kTile = 16;  // tokens

struct AttnParams {
  const uint16_t* q;
  int64_t ldq;
  int B, H;
  KvView c;
  const int32_t* table;
  int64_t ld_table, max_pages;
  const int32_t* seq_lens;
  int64_t window;
  float scale;  // times log2(e)
  uint16_t* out;
  float* lse;
  float* parts;        // [CTAs][2][heads of a unit * (head_dim + 2)]
  unsigned* counters;  // [B * units of a sequence]
  unsigned* status;
  int group;   // query heads of a key head
  int blocks;  // units of a key head: group / (8 NT), rounded up
};

template <int D_, bool INT8_, int NT_, int WARPS_, int STAGES_>
struct Shape {
  static constexpr int D = D_, NT = NT_, WARPS = WARPS_, STAGES = STAGES_;
  static constexpr bool INT8 = INT8_;
  static constexpr int kRowBytes = D * (INT8 ? 1 : 2);
  static constexpr int kRow = kRowBytes + 16;  // an odd number of 16-byte units: no bank conflicts
  static constexpr int kHalf = kTile * kRow;
  static constexpr int kStage = 2 * kHalf + (INT8 ? 8 * kTile : 0) + 16;  // K, V, scales, the valid tokens' mask
  static constexpr int kRing = STAGES * kStage;
  static constexpr int kHeads = 8 * NT;
  static constexpr int kPart = kHeads * (D + 2);  // floats: output, maximum, sum
  static constexpr size_t kSmem = WARPS * (static_cast<size_t>(kRing) + kPart * 4);
  static_assert(kRing >= kPart * 4, "a warp's last partial state is kept in its ring");
  static_assert(kSmem <= 232448 - 1024, "shared memory of an SM");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(valid ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldmatrix_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}
// The signed bytes 0 and 2 of w as a bf16 pair, exactly.
__device__ __forceinline__ uint32_t bytes_to_bf16(uint32_t w) {
  const uint32_t a = (w & 0x007F007Fu) | 0x43004300u, b = (w & 0x00800080u) | 0x43004300u;
  const __nv_bfloat162 r =
      __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// exp2(a - b) of two running maxima; nothing came before a maximum of -inf.
__device__ __forceinline__ float shrink(float a, float b) { return a == -INFINITY ? 0.0f : exp2_approx(a - b); }

// The tokens lo <= t < len that sequence b attends to, and its tiles first <= i < last.
struct Range {
  int64_t lo, len;
  int first, last;
};
__device__ __forceinline__ Range range_of(const AttnParams& p, int b) {
  Range r;
  r.len = __ldg(p.seq_lens + b);
  r.len = min(max(r.len, int64_t(0)), p.max_pages << p.c.page_shift);
  r.lo = p.window > 0 && r.len > p.window ? r.len - p.window : 0;
  r.first = static_cast<int>(r.lo / kTile);
  r.last = r.len > 0 ? static_cast<int>((r.len + kTile - 1) / kTile) : r.first;
  return r;
}

// A place on the line of tiles.
struct Cursor {
  Range r;
  int b, unit, tile;
  int64_t unit_pos;  // place of the unit's first tile
  __device__ __forceinline__ void next(const AttnParams& p, int units) {
    if (++tile < r.last) return;
    unit_pos += r.last - r.first;
    if (++unit == units) {
      unit = 0;
      do {
        if (++b >= p.B) return;
        r = range_of(p, b);
      } while (r.first == r.last);
    }
    tile = r.first;
  }
};

// Sum over the warp of a 64-bit count.
__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The place `at` (< the number of tiles) as a cursor: prefix sums over 32 sequences at a time.
__device__ __forceinline__ Cursor cursor_at(const AttnParams& p, int units, int64_t at, int lane) {
  Cursor c;
  int64_t base = 0;
  for (int b0 = 0;; b0 += 32) {
    Range r{};
    if (b0 + lane < p.B) r = range_of(p, b0 + lane);
    const int64_t n = static_cast<int64_t>(r.last - r.first) * units;
    int64_t incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const unsigned past = __ballot_sync(0xffffffffu, at < base + incl);
    if (past != 0) {
      const int src = __ffs(past) - 1;
      const int64_t start = base + __shfl_sync(0xffffffffu, incl - n, src);
      c.b = b0 + src;
      c.r = range_of(p, c.b);
      const int per = c.r.last - c.r.first;
      c.unit = static_cast<int>((at - start) / per);
      c.unit_pos = start + static_cast<int64_t>(c.unit) * per;
      c.tile = c.r.first + static_cast<int>(at - c.unit_pos);
      return c;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
}

template <typename S>
__global__ void __launch_bounds__(S::WARPS * 32, 1) paged_attention_kernel(const AttnParams p) {
  constexpr int D = S::D, NT = S::NT, W = S::WARPS, kSteps = D / 16;
  constexpr bool INT8 = S::INT8;
  griddep_wait();
  griddep_launch_dependents();
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int64_t s_unit[2 * W][3];  // of a warp's partial states: unit, its first place, the place after its last
  __shared__ unsigned s_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int units = p.c.heads * p.blocks;
  uint8_t* ring = smem + warp * S::kRing;
  float* own_part = reinterpret_cast<float*>(smem + W * S::kRing) + warp * S::kPart;
  const uint32_t ring32 = smem_u32(ring);

  // this CTA's and this warp's piece of the line
  int64_t total = 0;
  for (int b = lane; b < p.B; b += 32) {
    const Range r = range_of(p, b);
    if (blockIdx.x == 0 && warp == 0 && r.len != __ldg(p.seq_lens + b)) atomicOr(p.status, kErrIndex);
    total += static_cast<int64_t>(r.last - r.first) * units;
  }
  total = warp_sum(total);
  const int64_t ctas = min(static_cast<int64_t>(gridDim.x), (total + W - 1) / W);
  const bool works = blockIdx.x < ctas;
  const int64_t cta0 = works ? total * blockIdx.x / ctas : 0, cta1 = works ? total * (blockIdx.x + 1) / ctas : 0;
  const int64_t p0 = cta0 + (cta1 - cta0) * warp / W, p1 = cta0 + (cta1 - cta0) * (warp + 1) / W;
  if (lane < 2) s_unit[2 * warp + lane][0] = -1;
  __syncwarp();

  if (p0 < p1) {
    Cursor load = cursor_at(p, units, p0, lane), cur = load;
    const int n = static_cast<int>(p1 - p0);
    const int shift = p.c.page_shift;
    // page table entries window .. window + 63 of sequence window_b, one of each half per lane
    int window = 0, window_b = -1, pages0 = 0, pages1 = 0;
    auto entry = [&](int b, int64_t i) {
      return i < p.max_pages ? __ldg(p.table + b * p.ld_table + i) : -1;
    };
    auto issue = [&](int stage) {
      const int64_t tok = static_cast<int64_t>(load.tile) * kTile + (lane & 15);
      const int first_page = static_cast<int>((static_cast<int64_t>(load.tile) * kTile) >> shift);
      const int last_page = static_cast<int>((static_cast<int64_t>(load.tile) * kTile + kTile - 1) >> shift);
      if (load.b != window_b || first_page < window || last_page >= window + 64) {
        window = first_page;
        window_b = load.b;
        pages0 = entry(load.b, static_cast<int64_t>(window) + lane);
        pages1 = entry(load.b, static_cast<int64_t>(window) + 32 + lane);
      } else if (first_page >= window + 32) {
        window += 32;
        pages0 = pages1;
        pages1 = entry(load.b, static_cast<int64_t>(window) + 32 + lane);
      }
      const int at = static_cast<int>(tok >> shift) - window;
      const int e0 = __shfl_sync(0xffffffffu, pages0, at & 31), e1 = __shfl_sync(0xffffffffu, pages1, at & 31);
      const int64_t page = at < 32 ? e0 : e1;
      const bool in = tok >= load.r.lo && tok < load.r.len;
      const bool valid = in && page >= 0 && page < p.c.num_pages;
      if (in && !valid) atomicOr(p.status, kErrIndex);
      const unsigned mask = __ballot_sync(0xffffffffu, valid) & 0xFFFFu;
      const int64_t row = (static_cast<int64_t>(load.unit / p.blocks) << shift) + (tok & ((1 << shift) - 1));
      const int64_t off = valid ? (page * p.c.page_stride + row * D) * (INT8 ? 1 : 2) : 0;
      const uint32_t dst = ring32 + stage * S::kStage;
      constexpr int kChunks = S::kRowBytes / 16;
#pragma unroll
      for (int i = 0; i < kTile * kChunks / 32; ++i) {
        const int r = (i * 32 + lane) / kChunks, ch = (i * 32 + lane) % kChunks;
        const int64_t o = __shfl_sync(0xffffffffu, off, r) + ch * 16;
        const bool ok = (mask >> r) & 1;
        cp_async16(dst + r * S::kRow + ch * 16, static_cast<const uint8_t*>(p.c.k) + o, ok);
        cp_async16(dst + S::kHalf + r * S::kRow + ch * 16, static_cast<const uint8_t*>(p.c.v) + o, ok);
      }
      if (INT8) {
        const float* sc = lane < 16 ? p.c.k_scale : p.c.v_scale;
        cp_async4(dst + 2 * S::kHalf + lane * 4, sc + (valid ? page * p.c.scale_page_stride + row : 0), valid);
      }
      if (lane == 0) *reinterpret_cast<unsigned*>(ring + stage * S::kStage + S::kStage - 16) = mask;
      load.next(p, units);
    };

#pragma unroll
    for (int s = 0; s < S::STAGES - 1; ++s) {
      if (s < n) issue(s);
      cp_async_commit();
    }

    uint32_t qf[NT][kSteps][2];
    float o[NT][kSteps][4], m[NT][2], l[NT][2];
    int stage = 0, free_stage = S::STAGES - 1;
    bool fresh = true, from_start = false;
    for (int i = 0; i < n; ++i) {
      cp_async_wait<S::STAGES - 2>();
      __syncwarp();
      if (i + S::STAGES - 1 < n) issue(free_stage);
      cp_async_commit();
      const int kvh = cur.unit / p.blocks, hb = cur.unit % p.blocks;
      if (fresh) {  // the unit's queries; columns past its heads are zero
        from_start = cur.tile == cur.r.first;
        fresh = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int hl = hb * S::kHeads + nt * 8 + g;
          const uint16_t* qr = p.q + cur.b * p.ldq + (static_cast<int64_t>(kvh) * p.group + hl) * D;
#pragma unroll
          for (int j = 0; j < kSteps; ++j) {
            if (INT8) {  // the order in which a byte row's words give their even and odd codes
              uint2 w = make_uint2(0, 0);
              if (hl < p.group) w = __ldg(reinterpret_cast<const uint2*>(qr + 16 * j + 4 * t));
              qf[nt][j][0] = __byte_perm(w.x, w.y, 0x5410);
              qf[nt][j][1] = __byte_perm(w.x, w.y, 0x7632);
            } else {
              qf[nt][j][0] = hl < p.group ? __ldg(reinterpret_cast<const uint32_t*>(qr + 16 * j + 2 * t)) : 0u;
              qf[nt][j][1] = hl < p.group ? __ldg(reinterpret_cast<const uint32_t*>(qr + 16 * j + 8 + 2 * t)) : 0u;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][j][e] = 0.0f;
          }
          m[nt][0] = m[nt][1] = -INFINITY;
          l[nt][0] = l[nt][1] = 0.0f;
        }
      }
      const uint32_t src = ring32 + stage * S::kStage;
      const uint8_t* src_p = ring + stage * S::kStage;
      const uint32_t frag = src + (lane & 15) * S::kRow + (lane >> 4) * 16;

      // scores of 16 tokens x 8 heads: c0 (token g, head 2t), c1 (g, 2t + 1), c2, c3 (g + 8)
      float s[NT][2][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][0][e] = s[nt][1][e] = 0.0f;
#pragma unroll
      for (int j = 0; j < S::kRowBytes / 32; ++j) {
        uint32_t r[4];
        ldmatrix(r, frag + j * 32);
        if (INT8) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t a0 = bytes_to_bf16(r[2 * h]), a1 = bytes_to_bf16(r[2 * h + 1]);
            const uint32_t a2 = bytes_to_bf16(r[2 * h] >> 8), a3 = bytes_to_bf16(r[2 * h + 1] >> 8);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_bf16(s[nt][h], a0, a1, a2, a3, qf[nt][2 * j + h][0], qf[nt][2 * j + h][1]);
          }
        } else {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_bf16(s[nt][j & 1], r[0], r[1], r[2], r[3], qf[nt][j][0], qf[nt][j][1]);
        }
      }
      float ks0 = p.scale, ks1 = p.scale, vs0 = 1.0f, vs1 = 1.0f;
      if (INT8) {
        const float* sc = reinterpret_cast<const float*>(src_p + 2 * S::kHalf);
        ks0 *= sc[g];
        ks1 *= sc[g + 8];
        vs0 = sc[16 + g];
        vs1 = sc[24 + g];
      }
      const unsigned mask = *reinterpret_cast<const unsigned*>(src_p + S::kStage - 16);
      const bool ok0 = (mask >> g) & 1, ok1 = (mask >> (g + 8)) & 1;
      uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = (s[nt][0][e] + s[nt][1][e]) * (e < 2 ? ks0 : ks1);
        if (!ok0) x[0] = x[1] = -INFINITY;
        if (!ok1) x[2] = x[3] = -INFINITY;
        float mn[2] = {fmaxf(x[0], x[2]), fmaxf(x[1], x[3])};
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) {
          mn[0] = fmaxf(mn[0], __shfl_xor_sync(0xffffffffu, mn[0], w));
          mn[1] = fmaxf(mn[1], __shfl_xor_sync(0xffffffffu, mn[1], w));
        }
        const bool grows = mn[0] > m[nt][0] || mn[1] > m[nt][1];
        if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float top = fmaxf(m[nt][e], mn[e]), f = shrink(m[nt][e], top);
            m[nt][e] = top;
            l[nt][e] *= f;
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
              o[nt][j][e] *= f;
              o[nt][j][e + 2] *= f;
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float top = m[nt][e & 1];
          x[e] = exp2_approx(x[e] - (top == -INFINITY ? 0.0f : top));
          l[nt][e & 1] += x[e];
          x[e] *= e < 2 ? vs0 : vs1;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t hi = pack_bf16(x[2 * h], x[2 * h + 1]);
          const uint32_t lo = pack_bf16(x[2 * h] - __uint_as_float(hi << 16), x[2 * h + 1] - __uint_as_float(hi & 0xFFFF0000u));
          ph[nt][h] = transpose8x8(hi);
          pl[nt][h] = transpose8x8(lo);
        }
      }
#pragma unroll
      for (int j = 0; j < S::kRowBytes / 32; ++j) {
        uint32_t r[4];
        ldmatrix_t(r, frag + S::kHalf + j * 32);
        if (INT8) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t a0 = bytes_to_bf16(r[2 * h]), a1 = bytes_to_bf16(r[2 * h] >> 8);
            const uint32_t a2 = bytes_to_bf16(r[2 * h + 1]), a3 = bytes_to_bf16(r[2 * h + 1] >> 8);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_bf16(o[nt][2 * j + h], a0, a1, a2, a3, ph[nt][0], ph[nt][1]);
              mma_bf16(o[nt][2 * j + h], a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
            }
          }
        } else {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_bf16(o[nt][j], r[0], r[2], r[1], r[3], ph[nt][0], ph[nt][1]);
            mma_bf16(o[nt][j], r[0], r[2], r[1], r[3], pl[nt][0], pl[nt][1]);
          }
        }
      }
      free_stage = stage;
      stage = stage + 1 == S::STAGES ? 0 : stage + 1;

      const bool ends = cur.tile + 1 == cur.r.last;
      if (ends || i + 1 == n) {
        fresh = true;
        const bool whole = from_start && ends;
        // a state that began inside its unit is the warp's first and goes beside the ring, one
        // that breaks off is its last and goes into the ring, where no copy is in flight any more
        float* part = from_start ? reinterpret_cast<float*>(ring) : own_part;
        if (!whole) {
          __syncwarp();
          if (lane == 0) {
            int64_t* u = s_unit[2 * warp + (from_start ? 1 : 0)];
            u[0] = static_cast<int64_t>(cur.b) * units + cur.unit;
            u[1] = cur.unit_pos;
            u[2] = cur.unit_pos + (cur.r.last - cur.r.first);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float sum = l[nt][e];
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
            const int hi = nt * 8 + 2 * t + e, hl = hb * S::kHeads + hi;  // head in the unit, in its group
            const int h = kvh * p.group + hl;
            const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
            uint16_t* out = p.out + (static_cast<int64_t>(cur.b) * p.H + h) * D;
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
              const int d0 = 16 * j + (INT8 ? 2 * g : g), d1 = INT8 ? d0 + 1 : d0 + 8;
              const float v0 = o[nt][j][e], v1 = o[nt][j][e + 2];
              if (!whole) {
                part[hi * D + d0] = v0;
                part[hi * D + d1] = v1;
              } else if (hl < p.group) {
                if (INT8) {
                  *reinterpret_cast<uint32_t*>(out + d0) = pack_bf16(v0 * inv, v1 * inv);
                } else {
                  out[d0] = __bfloat16_as_ushort(__float2bfloat16_rn(v0 * inv));
                  out[d1] = __bfloat16_as_ushort(__float2bfloat16_rn(v1 * inv));
                }
              }
            }
            if (g == 0) {
              if (!whole) {
                part[S::kHeads * D + hi] = m[nt][e];
                part[S::kHeads * (D + 1) + hi] = sum;
              } else if (hl < p.group && p.lse != nullptr) {
                p.lse[static_cast<int64_t>(cur.b) * p.H + h] =
                    sum != 0.0f ? (m[nt][e] + log2f(sum)) * 0.693147180559945309f : -INFINITY;
              }
            }
          }
        }
      }
      cur.next(p, units);
    }
    cp_async_wait<0>();
  }
  __syncthreads();

  // the k-th partial state (warp k / 2) in shared memory
  auto part_of = [&](int k) -> const float* {
    return k & 1 ? reinterpret_cast<const float*>(smem + (k >> 1) * S::kRing)
                 : reinterpret_cast<const float*>(smem + W * S::kRing) + (k >> 1) * S::kPart;
  };
  // one element of a whole unit
  auto write_out = [&](int64_t unit, int hi, int d, float acc, float top, float sum) {
    const int64_t b = unit / units;
    const int u = static_cast<int>(unit % units), hl = u % p.blocks * S::kHeads + hi;
    if (hl >= p.group) return;
    const int64_t h = b * p.H + static_cast<int64_t>(u / p.blocks) * p.group + hl;
    p.out[h * D + d] = __bfloat16_as_ushort(__float2bfloat16_rn(sum != 0.0f ? acc / sum : 0.0f));
    if (d == 0 && p.lse != nullptr) p.lse[h] = sum != 0.0f ? (top + log2f(sum)) * 0.693147180559945309f : -INFINITY;
  };


  // ---- joining within the CTA: parts of one unit follow each other in the order of the line.
  // What is whole then is written out; at most two units reach beyond the CTA's piece (its
  // first and its last), and leave a part in the workspace.
  int64_t open_unit[2] = {-1, -1}, open_first[2], open_end[2];
  for (int k = 0; k < 2 * W;) {
    const int64_t unit = s_unit[k][0];
    int k1 = k + 1;
    if (unit >= 0) {
      while (k1 < 2 * W && (s_unit[k1][0] < 0 || s_unit[k1][0] == unit)) ++k1;
      const int64_t first = s_unit[k][1], end = s_unit[k][2];
      const bool whole = first >= cta0 && end <= cta1;
      const int side = first >= cta0 ? 1 : 0;
      if (!whole) open_unit[side] = unit, open_first[side] = first, open_end[side] = end;
      float* to = p.parts + (static_cast<int64_t>(blockIdx.x) * 2 + side) * S::kPart;
      for (int i = threadIdx.x; i < S::kHeads * D; i += W * 32) {
        const int hi = i / D;
        float top = -INFINITY, sum = 0.0f, acc = 0.0f;
        for (int j = k; j < k1; ++j)
          if (s_unit[j][0] == unit) top = fmaxf(top, part_of(j)[S::kHeads * D + hi]);
        for (int j = k; j < k1; ++j) {
          if (s_unit[j][0] != unit) continue;
          const float* part = part_of(j);
          const float f = shrink(part[S::kHeads * D + hi], top);
          sum = fmaf(f, part[S::kHeads * (D + 1) + hi], sum);
          acc = fmaf(f, part[i], acc);
        }
        if (whole) {
          write_out(unit, hi, i % D, acc, top, sum);
        } else {
          to[i] = acc;
          if (i % D == 0) to[S::kHeads * D + hi] = top, to[S::kHeads * (D + 1) + hi] = sum;
        }
      }
    }
    k = k1;
  }

  // ---- joining across CTAs: the last one to bring its part adds them all up in order.
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    if (open_unit[side] < 0) continue;  // uniform over the CTA
    const int64_t unit = open_unit[side];
    const int64_t c0 = ((open_first[side] + 1) * ctas - 1) / total, c1 = (open_end[side] * ctas - 1) / total;
    const int count = static_cast<int>(c1 - c0 + 1);
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
      const bool last = atomicAdd(p.counters + unit, 1u) == static_cast<unsigned>(count - 1);
      if (last) p.counters[unit] = 0;  // as the next call needs it
      s_last = last;
    }
    __syncthreads();
    if (s_last) {
      __threadfence();
      // part of CTA c0 + k: its last unit (side 1) in the CTA where the unit starts, else its first
      auto part = [&](int k) { return p.parts + ((c0 + k) * 2 + (k == 0 ? 1 : 0)) * S::kPart; };
      float* factor = reinterpret_cast<float*>(smem);  // [heads][count]; the rings are done with
      float* sums = factor + S::kHeads * count;        // [heads]
      for (int hi = warp; hi < S::kHeads; hi += W) {
        float top = -INFINITY, sum = 0.0f;
        for (int k = lane; k < count; k += 32) top = fmaxf(top, __ldcg(part(k) + S::kHeads * D + hi));
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
        for (int k = lane; k < count; k += 32) {
          const float f = shrink(__ldcg(part(k) + S::kHeads * D + hi), top);
          factor[hi * count + k] = f;
          sum = fmaf(f, __ldcg(part(k) + S::kHeads * (D + 1) + hi), sum);
        }
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
        if (lane == 0) sums[hi] = sum, sums[S::kHeads + hi] = top;
      }
      __syncthreads();
      for (int i = threadIdx.x * 4; i < S::kHeads * D; i += W * 32 * 4) {
        const int hi = i / D;
        float4 acc = make_float4(0, 0, 0, 0);
#pragma unroll 8
        for (int k = 0; k < count; ++k) {
          const float4 v = __ldcg(reinterpret_cast<const float4*>(part(k) + i));
          const float f = factor[hi * count + k];
          acc.x = fmaf(f, v.x, acc.x);
          acc.y = fmaf(f, v.y, acc.y);
          acc.z = fmaf(f, v.z, acc.z);
          acc.w = fmaf(f, v.w, acc.w);
        }
        const float top = sums[S::kHeads + hi], sum = sums[hi];
        write_out(unit, hi, i % D, acc.x, top, sum);
        write_out(unit, hi, i % D + 1, acc.y, top, sum);
        write_out(unit, hi, i % D + 2, acc.z, top, sum);
        write_out(unit, hi, i % D + 3, acc.w, top, sum);
      }
    }
  }

  // ---- sequences without tokens
  for (int b0 = (blockIdx.x * W + warp) * 32; b0 < p.B; b0 += gridDim.x * W * 32) {
    bool none = false;
    if (b0 + lane < p.B) {
      const Range r = range_of(p, b0 + lane);
      none = r.first == r.last;
    }
    for (unsigned left = __ballot_sync(0xffffffffu, none); left != 0; left &= left - 1) {
      const int64_t b = b0 + __ffs(left) - 1;
      for (int i = lane; i < p.H * D / 8; i += 32)
        reinterpret_cast<uint4*>(p.out + b * p.H * D)[i] = make_uint4(0, 0, 0, 0);
      if (p.lse != nullptr)
        for (int i = lane; i < p.H; i += 32) p.lse[b * p.H + i] = -INFINITY;
    }
  }
}

// ---------------------------------------------------------------- launch
constexpr int kMaxCtas = 160;  // one per SM

int cta_count() {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return std::min(sms, kMaxCtas);
}

size_t round256(size_t v) { return (v + 255) & ~size_t(255); }

template <typename S>
cudaError_t launch_shape(AttnParams p, const PagedAttentionArgs& a, cudaStream_t stream) {
  p.blocks = (p.group + S::kHeads - 1) / S::kHeads;
  auto kernel = paged_attention_kernel<S>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(S::kSmem));
  if (e != cudaSuccess) return e;
  return launch_kernel(kernel, dim3(static_cast<unsigned>(cta_count())), dim3(S::WARPS * 32), S::kSmem, stream, true, p);
}

}  // namespace

// Arrival counters (at most one per query head), then two parts per CTA of up to 16 heads.
size_t paged_attention_workspace_bytes(int64_t B, int64_t H, int64_t D) {
  return round256(static_cast<size_t>(B) * static_cast<size_t>(H) * 4) +
         static_cast<size_t>(kMaxCtas) * 2 * 16 * (static_cast<size_t>(D) + 2) * 4;
}

cudaError_t launch_paged_attention(const PagedAttentionArgs& a, cudaStream_t stream) {
  AttnParams p{};
  p.q = a.q;
  p.ldq = a.ldq;
  p.B = static_cast<int>(a.B);
  p.H = static_cast<int>(a.H);
  p.c = a.cache;
  p.table = a.table;
  p.ld_table = a.ld_table;
  p.max_pages = a.max_pages;
  p.seq_lens = a.seq_lens;
  p.window = a.window;
  p.scale = a.scale * 1.44269504088896341f;
  p.out = a.out;
  p.lse = a.lse;
  p.counters = static_cast<unsigned*>(a.ws);
  p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + round256(static_cast<size_t>(a.B) * a.H * 4));
  p.status = a.status;
  p.group = static_cast<int>(a.H) / a.cache.heads;
  const bool wide = p.group > 8;  // 16 query heads at a time: keys and values are read half as often
  if (a.cache.int8) {
    switch (a.cache.head_dim) {
      case 64: return wide ? launch_shape<Shape<64, true, 2, 8, 8>>(p, a, stream) : launch_shape<Shape<64, true, 1, 8, 8>>(p, a, stream);
      case 96: return wide ? launch_shape<Shape<96, true, 2, 8, 5>>(p, a, stream) : launch_shape<Shape<96, true, 1, 8, 6>>(p, a, stream);
      case 128: return wide ? launch_shape<Shape<128, true, 2, 8, 4>>(p, a, stream) : launch_shape<Shape<128, true, 1, 8, 5>>(p, a, stream);
      default: return launch_shape<Shape<256, true, 1, 4, 5>>(p, a, stream);
    }
  }
  switch (a.cache.head_dim) {
    case 64: return wide ? launch_shape<Shape<64, false, 2, 8, 5>>(p, a, stream) : launch_shape<Shape<64, false, 1, 8, 5>>(p, a, stream);
    case 96: return wide ? launch_shape<Shape<96, false, 2, 8, 3>>(p, a, stream) : launch_shape<Shape<96, false, 1, 8, 3>>(p, a, stream);
    case 128: return wide ? launch_shape<Shape<128, false, 2, 4, 5>>(p, a, stream) : launch_shape<Shape<128, false, 1, 4, 5>>(p, a, stream);
    default: return launch_shape<Shape<256, false, 1, 3, 4>>(p, a, stream);
  }
}

}  // namespace sq
