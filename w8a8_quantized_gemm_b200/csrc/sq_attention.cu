// Attention of one new token per sequence over a paged key-value cache, bf16 or int8.
//   s_t = scale * (q . k_t),  out = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m)
// "SmoothQuant量化实战" §5.2 (KV-cache INT8 with per-token, per-head scales).
//
// Every key and value is read once for all query heads of its key head: at 4 to 16 flops a
// byte the call is bound by the bytes of the cache, behind the latency of two warps' instructions a
// scheduler, where it is long (64 sequences of up to 8192, 8 key heads of 128, 64 query heads: 126
// us, 5.5 TB/s of int8 cache, for some milliseconds at 1965 MHz; 147 us, 4.7 TB/s, for seconds,
// which the power limit brings to 1700 MHz; inputs that change from call to call take the same, and
// full lengths 5.7 TB/s of 1109 MB at 1965 MHz) and by the chain of
// dependent steps where it is short (one such sequence, 32 query heads: 13.3 us: page table,
// tile and queries 4, scores and values of two tiles 3, the joins 4). The work is cut into
// tiles of 16 or 32 tokens of one key head; all tiles, in the order (sequence, key head, token),
// form one line that is dealt out evenly: each CTA (one per SM) gets a contiguous piece of it and
// each of its warps a contiguous piece of that, whatever the sequences' lengths. A warp works by
// itself: it brings
// its tiles into its own ring of shared memory with asynchronous copies, several tiles ahead,
// and keeps the running maximum m, the sum l and the unnormalised output of the 8 (or 16) query
// heads in registers. Only where a piece ends inside a key head's tiles is the state joined with
// its neighbours': within the CTA in shared memory, between CTAs through the workspace, where
// the last CTA to arrive adds the parts up in the order of the line. So results do not depend
// on which CTA is last.
//
// Matrix instructions: scores are K (16 tokens x head_dim) times q^T (head_dim x 8 heads), outputs
// V^T (16 elements x 16 tokens) times p^T (16 tokens x 8 heads): tokens and elements fill the 16
// rows, heads the 8 columns, all sums fp32 (int8 scores: int32). A bf16 cache takes 16x8x16
// instructions as it is. For an int8 cache, turning codes into 16-bit floats costs more
// instructions than all the rest, so
//   - scores use the 16x8x32 int8 instructions: a query, scaled by a power of two to 23 bits,
//     is split into three signed bytes and the three exact products are put together again
//     (elements down to 2^-14 of the head's largest are exact, smaller ones off by at most 2^-22 of it);
//   - values become fp16 exactly: (byte ^ 0x80) + 1024 has the byte's bits as its mantissa, one
//     logic operation, and 1152 less is the code.
// The probabilities enter as a high and a low 16-bit part (two bf16 numbers carry 16 bits, two fp16
// numbers 22), so that the rounding of out to bf16 is the only one that counts; their sum is of
// the whole ones. For an int8 cache they carry the token's value scale vs: what is
// subtracted is then the running maximum of s + log2(vs), less kShift, which keeps the products
// within [0, 2^kShift], in fp16's range whatever the scales, and the exponentials alone, whose sum
// is the softmax's, in fp32's: from 2^(kShift - 121) (bf16 values are below 2^128, their scales below
// 2^121) to 2^(kShift - kFloor) a token, where kFloor stands for the log2 of smaller scales, of zero
// and of scales that are not finite.
#include "sq_internal.h"
#include "sq_ptx.cuh"
#include "sq_rows.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

namespace sq {
namespace {

struct AttnParams {
  const uint16_t* q;
  int64_t ldq;
  int B, H;
  KvView c;
  const int32_t* table;
  int64_t ld_table;
  int max_pages, max_len;  // max_len: what the table's rows can hold, at most 2^31 - 1
  const int32_t* seq_lens;
  int window;   // 2^31 - 1: the whole sequence
  float scale;  // times log2(e)
  uint16_t* out;
  float* lse;
  float* parts;        // [CTAs][2][heads of a unit * (head_dim + 2)]
  unsigned* counters;  // [B * units of a sequence]
  unsigned* status;
  int group;   // query heads of a key head
  int blocks;  // units of a key head: group / (8 NT), rounded up
};

// D: head dimension; NT: query heads of a unit / 8; MT: tokens of a tile / 16.
template <int D_, bool INT8_, int NT_, int MT_, int WARPS_, int STAGES_>
struct Shape {
  static constexpr int D = D_, NT = NT_, MT = MT_, WARPS = WARPS_, STAGES = STAGES_;
  static constexpr int kTile = 16 * MT;
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
  static_assert(kSmem <= 232448 - 4096, "shared memory of an SM");
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
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_s8(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float log2_approx(float x) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
// The signed bytes 0 and 2 of w as an fp16 pair, exactly: byte + 1152, less 1152.
__device__ __forceinline__ uint32_t bytes_to_f16(uint32_t w) {
  const uint32_t a = (w & 0x00FF00FFu) ^ 0x64806480u, b = 0x64806480u;
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Pairs of values as the sum of a high and a low 16-bit float.
__device__ __forceinline__ void split_f16(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 f = __half22float2(h);
  const __half2 r = __floats2half2_rn(a - f.x, b - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ void split_bf16(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16(a, b);
  lo = pack_bf16(a - bf16_lo(hi), b - bf16_hi(hi));
}
// exp2((a - b) / 2) of two running maxima: its square takes a state to the new one. A sum takes it in
// two steps, since maxima that the scales of values have moved can be further apart than fp32's
// exponents, and the sum's size makes up for it. Nothing came before a maximum of -inf.
__device__ __forceinline__ float shrink_half(float a, float b) {
  return a == -INFINITY ? 0.0f : exp2_approx(0.5f * (a - b));
}
constexpr float kShift = 14.0f, kFloor = -90.0f;  // int8 cache: see above

constexpr int kMaxCtas = 160;  // one per SM

// The tokens lo <= t < len that sequence b attends to, and its tiles first <= i < last.
struct Range {
  int lo, len, first, last;
};
template <typename S>
__device__ __forceinline__ Range range_of(const AttnParams& p, int b) {
  Range r;
  r.len = min(max(__ldg(p.seq_lens + b), 0), p.max_len);
  r.lo = r.len > p.window ? r.len - p.window : 0;
  r.first = static_cast<unsigned>(r.lo) / S::kTile;
  r.last = r.len > 0 ? static_cast<int>((static_cast<unsigned>(r.len) + S::kTile - 1) / S::kTile) : r.first;
  return r;
}

// A place on the line of tiles.
template <typename S>
struct Cursor {
  Range r;
  int b, kvh, hb, tile;  // sequence, key head, block of its query heads
  int64_t unit_pos;      // place of the unit's first tile
  __device__ __forceinline__ void next(const AttnParams& p) {
    if (++tile < r.last) return;
    unit_pos += r.last - r.first;
    if (++hb == p.blocks) {
      hb = 0;
      if (++kvh == p.c.heads) {
        kvh = 0;
        do {
          if (++b >= p.B) return;
          r = range_of<S>(p, b);
        } while (r.first == r.last);
      }
    }
    tile = r.first;
  }
};

// a / b of counts, which nearly always fit 32 bits (a 64-bit division costs ten times as much).
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// The tiles (of all units) of `count` sequences a lane from `first` on, and up to the lane's end;
// the range of the last one.
template <typename S>
struct Scan {
  Range r;
  int64_t n, upto;
  __device__ __forceinline__ Scan(const AttnParams& p, int units, int first, int count, int lane) : r{}, n(0) {
#pragma unroll 4
    for (int b = first; b < min(first + count, p.B); ++b) {
      r = range_of<S>(p, b);
      n += static_cast<int64_t>(r.last - r.first) * units;
    }
    upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
  }
};

// The place `at` (< the number of tiles) as a cursor, from a scan of `each` sequences a lane: the
// lane's, then the sequence among the lane's.
template <typename S>
__device__ __forceinline__ Cursor<S> cursor_at(const AttnParams& p, int units, const Scan<S>& scan, int each,
                                               int64_t at, int lane) {
  Cursor<S> c;
  int src = __ffs(__ballot_sync(0xffffffffu, at < scan.upto)) - 1;
  int64_t start = __shfl_sync(0xffffffffu, scan.upto - scan.n, src);
  Range r = scan.r;
  c.b = src * each;
  while (each > 1) {
    const Scan<S> s(p, units, c.b + lane, 1, lane);
    const unsigned past = __ballot_sync(0xffffffffu, at < start + s.upto);
    if (past != 0) {
      src = __ffs(past) - 1;
      start += __shfl_sync(0xffffffffu, s.upto - s.n, src);
      r = s.r;
      c.b += src;
      break;
    }
    start += __shfl_sync(0xffffffffu, s.upto, 31);
    c.b += 32;
  }
  c.r.lo = __shfl_sync(0xffffffffu, r.lo, src);
  c.r.len = __shfl_sync(0xffffffffu, r.len, src);
  c.r.first = __shfl_sync(0xffffffffu, r.first, src);
  c.r.last = __shfl_sync(0xffffffffu, r.last, src);
  const int per = c.r.last - c.r.first;
  const int unit = static_cast<int>(divide(at - start, per));
  c.kvh = unit / p.blocks;
  c.hb = unit % p.blocks;
  c.unit_pos = start + static_cast<int64_t>(unit) * per;
  c.tile = c.r.first + static_cast<int>(at - c.unit_pos);
  return c;
}

template <typename S>
__global__ void __launch_bounds__(S::WARPS * 32, 1) paged_attention_kernel(const AttnParams p) {
  constexpr int D = S::D, NT = S::NT, MT = S::MT, W = S::WARPS, kSteps = D / 16, kTile = S::kTile;
  constexpr unsigned kAll = kTile == 32 ? 0xFFFFFFFFu : 0xFFFFu;
  constexpr bool INT8 = S::INT8;
  griddep_wait();
  griddep_launch_dependents();
  extern __shared__ __align__(16) uint8_t smem[];
  // a warp's partial states (2 w: the one that began inside its unit, 2 w + 1: the one that breaks
  // off): unit or -1, sequence, key head, block; the unit's first place and the one after its last
  __shared__ int4 s_unit[2 * W];
  __shared__ int64_t s_span[2 * W][2];
  __shared__ float s_factor[2 * W][S::kHeads], s_sum[2 * W][S::kHeads], s_top[2 * W][S::kHeads];
  __shared__ int64_t s_from[2];
  __shared__ int s_count[2];
  __shared__ bool s_last[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int units = p.c.heads * p.blocks;
  uint8_t* ring = smem + warp * S::kRing;
  float* own_part = reinterpret_cast<float*>(smem + W * S::kRing) + warp * S::kPart;
  const uint32_t ring32 = smem_u32(ring);

  // this CTA's and this warp's piece of the line
  const int each = (p.B + 31) / 32;
  const Scan<S> scan(p, units, lane * each, each, lane);
  const int64_t total = __shfl_sync(0xffffffffu, scan.upto, 31);
  const int64_t ctas = min(static_cast<int64_t>(gridDim.x), divide(total + W - 1, W));
  const bool works = blockIdx.x < ctas;
  const int64_t cta0 = works ? divide(total * blockIdx.x, ctas) : 0;
  const int64_t cta1 = works ? divide(total * (blockIdx.x + 1), ctas) : 0;
  const int64_t p0 = cta0 + divide((cta1 - cta0) * warp, W), p1 = cta0 + divide((cta1 - cta0) * (warp + 1), W);
  if (lane < 2) s_unit[2 * warp + lane].x = -1;
  __syncwarp();

  if (p0 < p1) {
    Cursor<S> load = cursor_at<S>(p, units, scan, each, p0, lane), cur = load;
    const int n = static_cast<int>(p1 - p0);
    const int shift = p.c.page_shift;
    // page table entries win .. win + 63 of sequence win_b, one of each half per lane
    int win = 0, win_b = -1, pages0 = 0, pages1 = 0;
    auto entry = [&](int b, int i) {
      return i < p.max_pages && SQ_GUARD(b < p.B && i >= 0) ? __ldg(p.table + b * p.ld_table + i) : -1;
    };
    const bool paged = (1 << shift) >= kTile;  // a tile lies in one page, its rows one after another
    constexpr int kChunks = S::kRowBytes / 16, kCopies = kTile * kChunks / 32;
    // place of copy i of this lane: row (32 i + lane) / kChunks
    auto in_stage = [&](int i) {
      return static_cast<uint32_t>((i * 32 + lane) / kChunks * S::kRow + (i * 32 + lane) % kChunks * 16);
    };
    auto issue = [&](int stage) {
      const int tok0 = load.tile * kTile;
      const int first_page = tok0 >> shift, last_page = (tok0 + (kTile - 1)) >> shift;
      if (load.b != win_b || first_page < win || last_page >= win + 64) {
        win = first_page;
        win_b = load.b;
        pages0 = entry(win_b, win + lane);
        pages1 = entry(win_b, win + 32 + lane);
      } else if (first_page >= win + 32) {
        win += 32;
        pages0 = pages1;
        pages1 = entry(win_b, win + 32 + lane);
      }
      const uint32_t dst = ring32 + stage * S::kStage;
      const uint8_t *k = static_cast<const uint8_t*>(p.c.k), *v = static_cast<const uint8_t*>(p.c.v);
      const int64_t row0 = static_cast<int64_t>(load.kvh) << shift;
      unsigned mask = kAll;
      const int one = __shfl_sync(0xffffffffu, pages0, (first_page - win) & 31);
      if (paged && first_page < win + 32 && tok0 >= load.r.lo && tok0 + kTile <= load.r.len && one >= 0 &&
          one < p.c.num_pages) {
        // whole tile: contiguous
        const int64_t row = row0 + (tok0 & ((1 << shift) - 1));
        const int64_t off = (p.c.page_stride * one + row * D) * (INT8 ? 1 : 2) + lane * 16;
        k += off;
        v += off;
        const int64_t bytes = p.c.elements() * (INT8 ? 1 : 2);
#pragma unroll
        for (int i = 0; i < kCopies; ++i)
          cp_async16(dst + in_stage(i), k + i * 512, SQ_GUARD(within(k + i * 512, 16, p.c.k, bytes)));
#pragma unroll
        for (int i = 0; i < kCopies; ++i)
          cp_async16(dst + S::kHalf + in_stage(i), v + i * 512, SQ_GUARD(within(v + i * 512, 16, p.c.v, bytes)));
        if (INT8) {
          const int64_t at = p.c.scale_page_stride * one + row;
          if (kTile == 32) {
            const bool ok = SQ_GUARD(within(p.c.k_scale + at, 32, p.c.k_scale, p.c.scales()));
            cp_async4(dst + 2 * S::kHalf + lane * 4, p.c.k_scale + at + lane, ok);
            cp_async4(dst + 2 * S::kHalf + 128 + lane * 4, p.c.v_scale + at + lane, ok);
          } else {
            cp_async4(dst + 2 * S::kHalf + lane * 4, (lane < 16 ? p.c.k_scale : p.c.v_scale) + at + (lane & 15),
                      SQ_GUARD(within(p.c.k_scale + at, 16, p.c.k_scale, p.c.scales())));
          }
        }
      } else {
        // row by row: lane r (mod the tile) looks up row r
        const int tok = tok0 + (lane & (kTile - 1)), at = (tok >> shift) - win;
        const int e0 = __shfl_sync(0xffffffffu, pages0, at & 31), e1 = __shfl_sync(0xffffffffu, pages1, at & 31);
        const int64_t page = at < 32 ? e0 : e1;
        const bool in = tok >= load.r.lo && tok < load.r.len;
        const bool valid = in && page >= 0 && page < p.c.num_pages;
        if (in && !valid) atomicOr(p.status, kErrIndex);
        mask = __ballot_sync(0xffffffffu, valid) & kAll;
        const int64_t row = row0 + (tok & ((1 << shift) - 1));
        const int64_t off = valid ? (page * p.c.page_stride + row * D) * (INT8 ? 1 : 2) : 0;
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
          const int r = (i * 32 + lane) / kChunks, ch = (i * 32 + lane) % kChunks;
          const int64_t o = __shfl_sync(0xffffffffu, off, r) + ch * 16;
          const bool ok = ((mask >> r) & 1) && SQ_GUARD(within(k + o, 16, k, p.c.elements() * (INT8 ? 1 : 2)));
          cp_async16(dst + in_stage(i), k + o, ok);
          cp_async16(dst + S::kHalf + in_stage(i), v + o, ok);
        }
        if (INT8) {
          const int64_t sat = valid ? page * p.c.scale_page_stride + row : 0;
          if (kTile == 32 || lane < 16)
            cp_async4(dst + 2 * S::kHalf + (lane & (kTile - 1)) * 4, p.c.k_scale + sat,
                      valid && SQ_GUARD(within(p.c.k_scale + sat, 1, p.c.k_scale, p.c.scales())));
          if (kTile == 32 || lane >= 16)
            cp_async4(dst + 2 * S::kHalf + (kTile + (lane & (kTile - 1))) * 4, p.c.v_scale + sat,
                      valid && SQ_GUARD(within(p.c.k_scale + sat, 1, p.c.k_scale, p.c.scales())));
        }
      }
      if (lane == 0) *reinterpret_cast<unsigned*>(ring + stage * S::kStage + S::kStage - 16) = mask;
      load.next(p);
    };

    // the queries' operand fragments: bf16 pairs, or the three bytes' words; per head the factor
    // that turns an int8 score into an exponent of 2
    constexpr int kParts = INT8 ? 3 : 1, kWords = INT8 ? D / 32 : D / 16;
    uint32_t qf[NT][kParts][kWords][2];
    float o[NT][kSteps][4], m[NT][2], l[NT][2], factor[NT][2];
    int stage = 0, load_stage = 0;
    bool fresh = true, from_start = false;
    for (int i = 1 - S::STAGES; i < n; ++i) {
      const int kvh = cur.kvh, hb = cur.hb;
      if (i >= 0 && fresh) {  // the unit's queries; columns past its heads are zero
        from_start = cur.tile == cur.r.first;
        fresh = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int hl = hb * S::kHeads + nt * 8 + g;
          const uint16_t* qr = p.q + cur.b * p.ldq + (static_cast<int64_t>(kvh) * p.group + hl) * D;
          if (INT8) {
            uint2 w[kWords][2];
            uint32_t top = 0;  // bf16 without their signs are in the order of their bits, infinity and NaN last
#pragma unroll
            for (int j = 0; j < kWords; ++j)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                w[j][h] = make_uint2(0, 0);
                if (hl < p.group) w[j][h] = __ldg(reinterpret_cast<const uint2*>(qr + 32 * j + 16 * h + 4 * t));
              }
#pragma unroll
            for (int j = 0; j < kWords; ++j)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                top = __vmaxu2(__vmaxu2(top, w[j][h].x & 0x7FFF7FFFu), w[j][h].y & 0x7FFF7FFFu);
            top = max(top >> 16, top & 0xFFFFu);
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // 2^up brings the largest, which may be subnormal, between 2^21 and 2^22: two factors, since up
            // is -106 to 155. Integers cannot carry infinity or NaN, so the head's scores become NaN
            const int up = top >= 0x80u ? 22 + 126 - static_cast<int>(top >> 7) : 123 + __clz(static_cast<int>(top));
            const int up0 = min(up, 120), up1 = up - up0;
            const float mul = __uint_as_float(static_cast<uint32_t>(127 + up0) << 23);
            const float mul1 = __uint_as_float(static_cast<uint32_t>(127 + up1) << 23);
#pragma unroll
            for (int j = 0; j < kWords; ++j)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                // round to an integer in the low mantissa bits (1.5 * 2^23 added), then bytes with
                // carries: the three low bytes of v + 0x808080, each less 128, are the signed digits
                constexpr uint32_t kBytes = 0x00808080u - 0x4B400000u;
                const float x[4] = {bf16_lo(w[j][h].x), bf16_hi(w[j][h].x), bf16_lo(w[j][h].y), bf16_hi(w[j][h].y)};
                uint32_t v[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] = __float_as_uint(__fmaf_rn(x[c] * mul1, mul, 12582912.0f)) + kBytes;
#pragma unroll
                for (int d = 0; d < 3; ++d) {
                  const uint32_t pick = d == 0 ? 0x0062u : d == 1 ? 0x0051u : 0x0040u;
                  qf[nt][d == 0 ? 0 : d == 1 ? kParts / 2 : kParts - 1][j][h] =
                      __byte_perm(__byte_perm(v[0], v[1], pick), __byte_perm(v[2], v[3], pick), 0x5410) ^ 0x80808080u;
                }
              }
            const float back =
                top < 0x7F80u ? p.scale * __uint_as_float(static_cast<uint32_t>(127 - up0) << 23) : NAN;
            const float factor_g = back * __uint_as_float(static_cast<uint32_t>(127 - up1) << 23);
            factor[nt][0] = __shfl_sync(0xffffffffu, factor_g, 8 * t);
            factor[nt][1] = __shfl_sync(0xffffffffu, factor_g, 8 * t + 4);
          } else {
#pragma unroll
            for (int j = 0; j < kWords; ++j)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                qf[nt][0][j][h] =
                    hl < p.group ? __ldg(reinterpret_cast<const uint32_t*>(qr + 16 * j + 8 * h + 2 * t)) : 0u;
            factor[nt][0] = factor[nt][1] = p.scale;
          }
#pragma unroll
          for (int j = 0; j < kSteps; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][j][e] = 0.0f;
          m[nt][0] = m[nt][1] = -INFINITY;
          l[nt][0] = l[nt][1] = 0.0f;
        }
      }
      // the next tile's copies go where the previous tile was; the first rounds only start copies
      cp_async_wait<S::STAGES - 2>();
      __syncwarp();
      if (i + S::STAGES - 1 < n) issue(load_stage);
      cp_async_commit();
      load_stage = load_stage + 1 == S::STAGES ? 0 : load_stage + 1;
      if (i < 0) continue;
      const uint32_t src = ring32 + stage * S::kStage;
      const uint8_t* src_p = ring + stage * S::kStage;
      const uint32_t frag = src + (lane & 15) * S::kRow + (lane >> 4) * 16;

      // scores of 16 tokens x 8 heads: c0 (token g, head 2t), c1 (g, 2t + 1), c2, c3 (g + 8)
      float x[MT][NT][4];
      if constexpr (INT8) {
        int c[MT][NT][3][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 12; ++e) c[mt][nt][e / 4][e % 4] = 0;
#pragma unroll
        for (int j = 0; j < kWords; ++j)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            uint32_t r[4];
            ldmatrix(r, frag + mt * 16 * S::kRow + j * 32);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int d = 0; d < 3; ++d) mma_s8(c[mt][nt][d], r, qf[nt][d][j][0], qf[nt][d][j][1]);
          }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[mt][nt][e] = fmaf(static_cast<float>(c[mt][nt][0][e] * 256 + c[mt][nt][1][e]), 256.0f,
                                  static_cast<float>(c[mt][nt][2][e]));
      } else {
        float c[MT][NT][2][4];  // two sums side by side, so that no instruction waits for the one before it
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 8; ++e) c[mt][nt][e / 4][e % 4] = 0.0f;
#pragma unroll
        for (int j = 0; j < kWords; ++j)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            uint32_t r[4];
            ldmatrix(r, frag + mt * 16 * S::kRow + j * 32);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_bf16(c[mt][nt][j & 1], r[0], r[1], r[2], r[3], qf[nt][0][j][0], qf[nt][0][j][1]);
          }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[mt][nt][e] = c[mt][nt][0][e] + c[mt][nt][1][e];
      }
      const unsigned mask = *reinterpret_cast<const unsigned*>(src_p + S::kStage - 16);
      const float* sc = reinterpret_cast<const float*>(src_p + 2 * S::kHalf);
      // per token of this lane (rows g and g + 8 of each 16): the key's scale, the value's and its log2
      float ks[MT][2], vs[MT][2], lv[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = mt * 16 + h * 8 + g;
          ks[mt][h] = INT8 ? sc[row] : 1.0f;
          vs[mt][h] = INT8 ? sc[kTile + row] : 1.0f;
          lv[mt][h] = INT8 ? fmaxf(log2_approx(vs[mt][h]), kFloor) : 0.0f;
          if (INT8 && lv[mt][h] == INFINITY) lv[mt][h] = kFloor;
        }
      uint32_t ph[MT][NT][2], pl[MT][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float mn[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float& v = x[mt][nt][e];
            v *= INT8 ? factor[nt][e & 1] * ks[mt][e / 2] : factor[nt][e & 1];
            if (mask != kAll && !((mask >> (mt * 16 + (e / 2) * 8 + g)) & 1)) v = -INFINITY;
            mn[e & 1] = fmaxf(mn[e & 1], v + lv[mt][e / 2]);
          }
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) {
          mn[0] = fmaxf(mn[0], __shfl_xor_sync(0xffffffffu, mn[0], w));
          mn[1] = fmaxf(mn[1], __shfl_xor_sync(0xffffffffu, mn[1], w));
        }
        if (INT8) mn[0] -= kShift, mn[1] -= kShift;
        const bool grows = mn[0] > m[nt][0] || mn[1] > m[nt][1];
        if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float top = fmaxf(m[nt][e], mn[e]), half = shrink_half(m[nt][e], top), f = half * half;
            m[nt][e] = top;
            l[nt][e] = l[nt][e] * half * half;
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
              o[nt][j][e] *= f;
              o[nt][j][e + 2] *= f;
            }
          }
        }
        const float top[2] = {m[nt][0] == -INFINITY ? 0.0f : m[nt][0], m[nt][1] == -INFINITY ? 0.0f : m[nt][1]};
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float e0 = exp2_approx(x[mt][nt][2 * h] - top[0]), e1 = exp2_approx(x[mt][nt][2 * h + 1] - top[1]);
            l[nt][0] += e0;
            l[nt][1] += e1;
            uint32_t hi, lo;
            if (INT8)
              split_f16(e0 * vs[mt][h], e1 * vs[mt][h], hi, lo);
            else
              split_bf16(e0, e1, hi, lo);
            ph[mt][nt][h] = transpose8x8(hi);
            pl[mt][nt][h] = transpose8x8(lo);
          }
        }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int j = 0; j < S::kRowBytes / 32; ++j) {
          uint32_t r[4];
          ldmatrix_t(r, frag + S::kHalf + mt * 16 * S::kRow + j * 32);
          if constexpr (INT8) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t a0 = bytes_to_f16(r[2 * h]), a1 = bytes_to_f16(r[2 * h] >> 8);
              const uint32_t a2 = bytes_to_f16(r[2 * h + 1]), a3 = bytes_to_f16(r[2 * h + 1] >> 8);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma_f16(o[nt][2 * j + h], a0, a1, a2, a3, ph[mt][nt][0], ph[mt][nt][1]);
                mma_f16(o[nt][2 * j + h], a0, a1, a2, a3, pl[mt][nt][0], pl[mt][nt][1]);
              }
            }
          } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_bf16(o[nt][j], r[0], r[2], r[1], r[3], ph[mt][nt][0], ph[mt][nt][1]);
              mma_bf16(o[nt][j], r[0], r[2], r[1], r[3], pl[mt][nt][0], pl[mt][nt][1]);
            }
          }
        }
      }
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
            const int slot = 2 * warp + (from_start ? 1 : 0);
            s_unit[slot] = make_int4(cur.b * units + kvh * p.blocks + hb, cur.b, kvh, hb);
            s_span[slot][0] = cur.unit_pos;
            s_span[slot][1] = cur.unit_pos + (cur.r.last - cur.r.first);
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
                if (SQ_GUARD(hi < S::kHeads && d1 < D)) part[hi * D + d0] = v0, part[hi * D + d1] = v1;
              } else if (hl < p.group && SQ_GUARD(d1 < D && within(out, D, p.out, static_cast<int64_t>(p.B) * p.H * D))) {
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
              } else if (hl < p.group && p.lse != nullptr && SQ_GUARD(cur.b < p.B && h < p.H)) {
                p.lse[static_cast<int64_t>(cur.b) * p.H + h] =
                    sum != 0.0f ? (m[nt][e] + log2f(sum)) * 0.693147180559945309f : -INFINITY;
              }
            }
          }
        }
      }
      cur.next(p);
    }
    cp_async_wait<0>();
  }
  __syncthreads();

  // the k-th partial state in shared memory
  auto part_of = [&](int k) -> const float* {
    return k & 1 ? reinterpret_cast<const float*>(smem + (k >> 1) * S::kRing)
                 : reinterpret_cast<const float*>(smem + W * S::kRing) + (k >> 1) * S::kPart;
  };
  // elements d .. d + 3 of head hi of a whole unit
  auto write_out = [&](int4 u, int hi, int d, float4 acc, float top, float sum) {
    const int64_t h = static_cast<int64_t>(u.y) * p.H + u.z * p.group + u.w * S::kHeads + hi;
    const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
    if (!SQ_GUARD(h >= 0 && h < static_cast<int64_t>(p.B) * p.H && d + 4 <= D)) return;
    *reinterpret_cast<uint2*>(p.out + h * D + d) =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    if (d == 0 && p.lse != nullptr) p.lse[h] = sum != 0.0f ? (top + log2f(sum)) * 0.693147180559945309f : -INFINITY;
  };
  auto add = [](float4& acc, float f, float4 v) {
    acc.x = fmaf(f, v.x, acc.x);
    acc.y = fmaf(f, v.y, acc.y);
    acc.z = fmaf(f, v.z, acc.z);
    acc.w = fmaf(f, v.w, acc.w);
  };

  // ---- joining within the CTA: parts of one unit follow each other in the order of the line.
  // What is whole then is written out; at most two units reach beyond the CTA's piece (side 0:
  // its first, begun before it, side 1: its last) and leave a part in the workspace.
  static_assert(2 * W <= 32, "one lane per part");
  const int my_unit = lane < 2 * W ? s_unit[lane].x : -1;
  const unsigned parts = __ballot_sync(0xffffffffu, my_unit >= 0), below = parts & ((1u << lane) - 1u);
  const int before = __shfl_sync(0xffffffffu, my_unit, below != 0 ? 31 - __clz(below) : 0);
  const unsigned heads_of_groups = __ballot_sync(0xffffffffu, my_unit >= 0 && (below == 0 || before != my_unit));
  // every part's factor exp2(its maximum - its unit's): a warp per head, a lane per part, and
  // scans that stop at a unit's first part (seg0), whose last one (seg1) then has the whole
  const int seg0 = 31 - __clz(heads_of_groups & (0xffffffffu >> (31 - lane)));
  const unsigned later = heads_of_groups & ~(0xffffffffu >> (31 - lane));
  const int seg1 = later != 0 ? __ffs(later) - 2 : 31;
  for (int hi = warp; hi < S::kHeads; hi += W) {
    const bool mine = my_unit >= 0;
    const float m = mine ? part_of(lane)[S::kHeads * D + hi] : -INFINITY;
    const float l = mine ? part_of(lane)[S::kHeads * (D + 1) + hi] : 0.0f;
    float top = m;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float v = __shfl_up_sync(0xffffffffu, top, o);
      if (lane - o >= seg0) top = fmaxf(top, v);
    }
    top = __shfl_sync(0xffffffffu, top, seg1);
    const float half = shrink_half(m, top), f = half * half;
    float sum = l * half * half;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane - o >= seg0) sum += v;
    }
    sum = __shfl_sync(0xffffffffu, sum, seg1);
    if (mine) s_factor[lane][hi] = f, s_top[lane][hi] = top, s_sum[lane][hi] = sum;
  }
  __syncthreads();
  auto heads_of = [&](int4 u) { return min(S::kHeads, p.group - u.w * S::kHeads); };
  int open[2] = {-1, -1};  // the part that starts the unit left open
  int turn = warp;         // all units' heads go to the warps in turn: this one's next in the unit
  for (unsigned left = heads_of_groups; left != 0; left &= left - 1) {
    const int k0 = __ffs(left) - 1;
    const int k1 = (left & (left - 1)) != 0 ? __ffs(left & (left - 1)) - 1 : 2 * W;
    const bool begun = s_span[k0][0] < cta0, whole = !begun && s_span[k0][1] <= cta1;
    if (!whole) open[0] = begun ? k0 : open[0], open[1] = begun ? open[1] : k0;
    float* to = p.parts + (static_cast<int64_t>(blockIdx.x) * 2 + (begun ? 0 : 1)) * S::kPart;
    const int4 unit = s_unit[k0];
    const int heads = heads_of(unit);
    for (; turn < heads; turn += W) {
      const float top = s_top[k0][turn], sum = s_sum[k0][turn];
      for (int d = lane * 4; d < D; d += 128) {
        float4 acc = make_float4(0, 0, 0, 0);
        for (int j = k0; j < k1; ++j)
          if ((parts >> j) & 1)
            add(acc, s_factor[j][turn], *reinterpret_cast<const float4*>(part_of(j) + turn * D + d));
        if (whole)
          write_out(unit, turn, d, acc, top, sum);
        else if (SQ_GUARD(within(to + turn * D + d, 4, p.parts, static_cast<int64_t>(kMaxCtas) * 2 * S::kPart)))
          *reinterpret_cast<float4*>(to + turn * D + d) = acc;
      }
      if (!whole && lane == 0) to[S::kHeads * D + turn] = top, to[S::kHeads * (D + 1) + turn] = sum;
    }
    turn -= heads;
  }

  // ---- joining across CTAs: the last one to bring its part adds them all up in order.
  if (open[0] >= 0 || open[1] >= 0) {  // uniform over the CTA
    __threadfence();
    __syncthreads();
    if (lane == 0 && warp < 2) {
      const int at = warp == 0 ? open[0] : open[1];
      bool last = false;
      if (at >= 0) {
        const int64_t c0 = divide((s_span[at][0] + 1) * ctas - 1, total);
        const int count = static_cast<int>(divide(s_span[at][1] * ctas - 1, total) - c0) + 1;
        unsigned* counter = p.counters + s_unit[at].x;
        if (SQ_GUARD(c0 >= 0 && c0 + count <= ctas && within(counter, 1, p.counters, static_cast<int64_t>(p.B) * p.H)))
          last = atomicAdd(counter, 1u) == static_cast<unsigned>(count - 1);
        if (last) *counter = 0;  // as the next call needs it
        s_from[warp] = c0;
        s_count[warp] = count;
      }
      s_last[warp] = last;
    }
    __syncthreads();
    __threadfence();
  } else if (threadIdx.x < 2) {
    s_last[threadIdx.x] = false;
  }
  __syncthreads();
  if (s_last[0] || s_last[1]) {  // uniform over the CTA
    // all warps for the one side, or half of them for each
    const bool both = s_last[0] && s_last[1];
    const int side = both ? static_cast<int>(warp >= W / 2) : static_cast<int>(s_last[1]);
    const int warp0 = both && side == 1 ? W / 2 : 0;
    const int warps = !both ? W : side == 0 ? W / 2 : W - W / 2;
    const int first = ((warp - warp0) * 32 + lane) * 4, step = warps * 128;
    const int4 unit = s_unit[side == 0 ? open[0] : open[1]];
    const int count = s_count[side];
    // part of the k-th CTA: side 1 in the one where the unit starts, side 0 in the others
    const float* parts0 = p.parts + s_from[side] * 2 * S::kPart;
    auto part = [&](int k) { return parts0 + (2 * k + (k == 0 ? 1 : 0)) * S::kPart; };
    // the states come a batch of parts at a time, the first while the factors are found
    constexpr int kBatch = 16;
    const int heads = heads_of(unit);
    float4 state[kBatch];
    auto load_batch = [&](int k0, int i) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (k0 + k < count) state[k] = __ldcg(reinterpret_cast<const float4*>(part(k0 + k) + i));
    };
    if (first < heads * D) load_batch(0, first);
    // factors [heads][count], where the rings were
    static_assert(S::kSmem >= 2 * S::kHeads * kMaxCtas * 4, "both sides' factors");
    float* factor = reinterpret_cast<float*>(smem) + side * (S::kHeads * kMaxCtas);
    for (int hi = warp - warp0; hi < heads; hi += warps) {
      auto top_of = [&](int k) { return k < count ? __ldcg(part(k) + S::kHeads * D + hi) : -INFINITY; };
      auto sum_of = [&](int k) { return k < count ? __ldcg(part(k) + S::kHeads * (D + 1) + hi) : 0.0f; };
      const float m = top_of(lane), l = sum_of(lane);
      float top = m;
      for (int k = lane + 32; k < count; k += 32) top = fmaxf(top, top_of(k));
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
      float sum = 0.0f;
      for (int k = lane; k < count; k += 32) {
        const float half = shrink_half(k == lane ? m : top_of(k), top);
        factor[hi * count + k] = half * half;
        sum += (k == lane ? l : sum_of(k)) * half * half;
      }
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      if (lane == 0) s_sum[side][hi] = sum, s_top[side][hi] = top;
    }
    __syncthreads();
    for (int i = first; i < heads * D; i += step) {
      const int hi = i / D;
      float4 acc = make_float4(0, 0, 0, 0);
      for (int k0 = 0; k0 < count; k0 += kBatch) {
        if (k0 > 0 || i > first) load_batch(k0, i);
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (k0 + k < count) add(acc, factor[hi * count + k0 + k], state[k]);
      }
      write_out(unit, hi, i % D, acc, s_top[side][hi], s_sum[side][hi]);
    }
  }

  // ---- sequences without tokens
  for (int b0 = (blockIdx.x * W + warp) * 32; b0 < p.B; b0 += gridDim.x * W * 32) {
    bool none = false;
    if (b0 + lane < p.B) {
      const Range r = range_of<S>(p, b0 + lane);
      none = r.first == r.last;
      if (r.len != __ldg(p.seq_lens + b0 + lane)) atomicOr(p.status, kErrIndex);
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

int cta_count() {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return std::min(sms, kMaxCtas);
}

template <typename S>
cudaError_t launch_shape(AttnParams p, cudaStream_t stream) {
  p.blocks = (p.group + S::kHeads - 1) / S::kHeads;
  auto kernel = paged_attention_kernel<S>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(S::kSmem));
  if (e != cudaSuccess) return e;
  return launch_kernel(kernel, dim3(static_cast<unsigned>(cta_count())), dim3(S::WARPS * 32), S::kSmem, stream, true,
                       p);
}

}  // namespace

// Two parts per CTA of up to 16 heads of up to 256, then the arrival counters (at most one per query
// head): at the same place whatever the shape, so that calls of different shapes, one after another
// on one workspace, find the counters at zero.
constexpr size_t kPartsBytes = static_cast<size_t>(kMaxCtas) * 2 * 16 * (256 + 2) * 4;

size_t paged_attention_workspace_bytes(int64_t B, int64_t H) {
  return kPartsBytes + static_cast<size_t>(B) * static_cast<size_t>(H) * 4;
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
  p.max_pages = static_cast<int>(a.max_pages);
  p.max_len = static_cast<int>(std::min<int64_t>(a.max_pages << a.cache.page_shift, INT32_MAX));
  p.seq_lens = a.seq_lens;
  p.window = a.window == 0 ? INT32_MAX : static_cast<int>(std::min<int64_t>(a.window, INT32_MAX));
  p.scale = a.scale * 1.44269504088896341f;
  p.out = a.out;
  p.lse = a.lse;
  p.parts = static_cast<float*>(a.ws);
  p.counters = reinterpret_cast<unsigned*>(static_cast<uint8_t*>(a.ws) + kPartsBytes);
  p.status = a.status;
  p.group = static_cast<int>(a.H) / a.cache.heads;
  // 16 query heads at a time where a key head has more than 8: keys and values are read half as
  // often (32 sequences of up to 8192, 4 key heads of 128, int8, 16 query heads each: 62 us, by
  // eights 74). Warps rather than stages, since a warp's instructions wait for one another: us at
  // 32 sequences of up to 4096 and 8 key heads, 8 warps of 2 tiles each against 4 of 5: 128 bf16
  // 64 / 77, 256 int8 74 / 98. Tiles of 32 tokens for int8, whose part per tile is the larger: 64
  // sequences of up to 8192, 8 key heads of 128: 128 us, of 16 tokens 163.
  const bool wide = p.group > 8;
  if (a.cache.int8) {
    switch (a.cache.head_dim) {
      case 64: return wide ? launch_shape<Shape<64, true, 2, 2, 8, 4>>(p, stream)
                           : launch_shape<Shape<64, true, 1, 2, 12, 3>>(p, stream);
      case 96: return wide ? launch_shape<Shape<96, true, 2, 2, 8, 2>>(p, stream)
                           : launch_shape<Shape<96, true, 1, 2, 10, 2>>(p, stream);
      case 128: return wide ? launch_shape<Shape<128, true, 2, 2, 8, 2>>(p, stream)
                            : launch_shape<Shape<128, true, 1, 2, 8, 2>>(p, stream);
      default: return launch_shape<Shape<256, true, 1, 1, 8, 2>>(p, stream);
    }
  }
  switch (a.cache.head_dim) {
    case 64: return wide ? launch_shape<Shape<64, false, 2, 2, 8, 2>>(p, stream)
                         : launch_shape<Shape<64, false, 1, 2, 8, 2>>(p, stream);
    case 96: return wide ? launch_shape<Shape<96, false, 2, 1, 10, 2>>(p, stream)
                         : launch_shape<Shape<96, false, 1, 1, 12, 2>>(p, stream);
    case 128: return wide ? launch_shape<Shape<128, false, 2, 1, 8, 2>>(p, stream)
                          : launch_shape<Shape<128, false, 1, 1, 8, 2>>(p, stream);
    default: return launch_shape<Shape<256, false, 1, 1, 4, 2>>(p, stream);
  }
}

}  // namespace sq
