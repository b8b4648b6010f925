// 4-bit weights with group scales: quantization, the values they stand for, and the linear
// layer of a few tokens. "SmoothQuant量化实战" §2.4 and §6.1 (weight-only W4A16 beside W8A8).
//
// A tile is 16 rows x 128 columns in 1024 bytes; lane (g = lane / 4, t = lane % 4) of a warp
// owns its 16-byte units of rows g and g + 8: for the 32-column block a (a = 0..3) the word a,
// whose nibble 4 e + i is the code of column 32 a + 8 i + 2 t + e. Such a word masked with
// 0x000F000F, shifted by 0, 4, 8, 12, gives the lane's column pairs (2t, 2t + 1) of the four
// 8-column chunks: the A fragments of two 16x8x16 matrix instructions.
#include "sq_internal.h"
#include "sq_ptx.cuh"
#include "sq_rows.cuh"

#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>

namespace sq {
namespace {

constexpr int kInt4Threads = 256;
constexpr int kTileBytes = 1024;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Packed bf16 pair arithmetic on 32-bit words.
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r =
      __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r =
      __hmul2_rn(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// The larger and the smaller one, or NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// bf16 pair of 128 + z: 0x4300 is 128, whose mantissa counts in ones.
__device__ __forceinline__ uint32_t zero_pair(uint32_t z) { return 0x43004300u | z | (z << 16); }

__device__ __forceinline__ void ldmatrix(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool valid) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES),
                 "r"(valid ? BYTES : 0)
                 : "memory");
}

// ---------------------------------------------------------------- quantization
// One warp per tile, over the row tiles of one 128-column block. The tile comes as it is into the
// warp's ring of shared memory (asynchronous 16-byte copies, two tiles ahead); loading it as
// 8x8 matrices then gives each lane the column pairs of rows g and g + 8 that its 16-byte units
// hold the codes of, so nothing has to be exchanged: a word of codes is four pairs shifted
// together. A group of 32 columns belongs to the four lanes of a quad, and lane t of it takes
// the two divisions for the block a = t. Bound by instructions as much as by HBM (2.6 bytes an
// element): products are packed pairs, a code's rounding is an addition of 1.5 * 2^23 (the
// product is below 23 in magnitude, even where a subnormal scale is half a step off), and its
// zero point and clamp one packed 16-bit operation per pair. 28672 x 8192 with zero points, groups
// of 64: 123 us, 4.9 TB/s; 4096 x 4096, groups of 128: 11 us.
constexpr int kQuantRing = 3, kQuantRow = 256 + 16, kQuantSlot = 16 * kQuantRow;

template <int G, bool ASYM>
__global__ void __launch_bounds__(kInt4Threads, 2)
int4_quant_kernel(const uint16_t* __restrict__ W, int64_t N, int64_t K, int64_t ldw, const float* __restrict__ s,
                  uint8_t* __restrict__ Wp, uint16_t* __restrict__ scale, uint8_t* __restrict__ zero) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int kSpan = G / 32;  // 32-column blocks of a group
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, quad = lane & ~3;
  const int64_t Nt = (N + 15) / 16, Kb = (K + 127) / 128;
  const int64_t kb = blockIdx.x;
  const int cols = static_cast<int>(K - kb * 128 < 128 ? K - kb * 128 : 128);
  uint64_t sv[16];  // smoothing factors of this lane's column pairs 8 c + 2 t
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    sv[c] = rows::f2_pack(1.0f, 1.0f);
    if (s != nullptr && c * 8 < cols)
      sv[c] = __ldg(reinterpret_cast<const unsigned long long*>(s + kb * 128 + c * 8 + 2 * t));
  }
  const int64_t step = static_cast<int64_t>(gridDim.y) * (kInt4Threads / 32);
  int64_t rt = static_cast<int64_t>(blockIdx.y) * (kInt4Threads / 32) + (threadIdx.x >> 5);
  const uint32_t ring = smem_u32(smem) + (threadIdx.x >> 5) * kQuantRing * kQuantSlot;
  int64_t next = rt;
  auto fetch = [&](int slot) {  // lane: 16 bytes of rows lane / 16 + 2 i
    if (next < Nt) {
      const int64_t n0 = next * 16 + lane / 16;
      const uint16_t* src = W + n0 * ldw + kb * 128 + lane % 16 * 8;
      const uint32_t dst = ring + slot * kQuantSlot + lane / 16 * kQuantRow + lane % 16 * 16;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool in = n0 + 2 * i < N && lane % 16 * 8 < cols;
        cp_async<16>(dst + 2 * i * kQuantRow, in ? src + 2 * i * ldw : W, in);
      }
      next += step;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kQuantRing - 1; ++i) fetch(i);
  int slot = 0, free_slot = kQuantRing - 1;
  for (; rt < Nt; rt += step) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kQuantRing - 2) : "memory");
    __syncwarp();  // every lane's copies are there, and the slot before is read
    fetch(free_slot);
    const uint32_t src = ring + slot * kQuantSlot + (lane & 7) * kQuantRow + (lane >> 3) * 16;
    free_slot = slot;
    slot = slot + 1 == kQuantRing ? 0 : slot + 1;
    const bool inside = rt * 16 + 16 <= N && cols == 128;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t n = rt * 16 + h * 8 + g;
      uint64_t v[16];      // w' of this lane's pairs
      float hi[4], lo[4];  // per 32-column block: max |w'| (symmetric), or max and min with 0
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        uint32_t w[4];
        ldmatrix(w, src + h * 8 * kQuantRow + a * 64);
        hi[a] = lo[a] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[4 * a + i] = rows::f2_mul(rows::f2_pack(bf16_lo(w[i]), bf16_hi(w[i])), sv[4 * a + i]);
          float x, y;
          rows::f2_unpack(v[4 * a + i], x, y);
          hi[a] = ASYM ? max_nan(hi[a], max_nan(x, y)) : max_nan(hi[a], max_nan(fabsf(x), fabsf(y)));
          if (ASYM) lo[a] = min_nan(lo[a], min_nan(x, y));
        }
      }
#pragma unroll
      for (int a = 0; a < 4; a += kSpan) {
#pragma unroll
        for (int i = 1; i < kSpan; ++i) {
          hi[a] = max_nan(hi[a], hi[a + i]);
          lo[a] = min_nan(lo[a], lo[a + i]);
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          hi[a] = max_nan(hi[a], __shfl_xor_sync(0xffffffffu, hi[a], o));
          if (ASYM) lo[a] = min_nan(lo[a], __shfl_xor_sync(0xffffffffu, lo[a], o));
        }
#pragma unroll
        for (int i = 1; i < kSpan; ++i) hi[a + i] = hi[a], lo[a + i] = lo[a];
      }
      // this lane's block: t
      const float top = t & 2 ? (t & 1 ? hi[3] : hi[2]) : (t & 1 ? hi[1] : hi[0]);
      const float low = t & 2 ? (t & 1 ? lo[3] : lo[2]) : (t & 1 ? lo[1] : lo[0]);
      const __nv_bfloat16 e = __float2bfloat16_rn(ASYM ? __fdiv_rn(__fsub_rn(top, low), 15.0f) : __fdiv_rn(top, 7.0f));
      const float ef = __bfloat162float(e);
      const float my_r = ef > 0.0f ? fminf(__fdiv_rn(1.0f, ef), FLT_MAX) : 0.0f;
      int my_z = 8;
      if (ASYM) my_z = static_cast<int>(fminf(fmaxf(rintf(__fmul_rn(-low, my_r)), 0.0f), 15.0f));
      if (t % kSpan == 0 && t * 32 < cols && n < N) {
        const int64_t gr = kb * (128 / G) + t / kSpan;
        if (SQ_GUARD(within(scale + gr * N + n, 1, scale, (K + G - 1) / G * N))) {
          scale[gr * N + n] = __bfloat16_as_ushort(e);
          if (ASYM) zero[gr * N + n] = static_cast<uint8_t>(my_z);
        }
      }
      uint32_t word[4];
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const float r = __shfl_sync(0xffffffffu, my_r, quad | a);
        const uint32_t zz =
            ASYM ? static_cast<uint32_t>(__shfl_sync(0xffffffffu, my_z, quad | a)) * 0x00010001u : 0x00080008u;
        const uint64_t r2 = rows::f2_pack(r, r);
        word[a] = 0;
#pragma unroll
        for (int i = 3; i >= 0; --i) {
          float x, y;
          rows::f2_unpack(rows::f2_mul(v[4 * a + i], r2), x, y);
          const uint32_t q = __byte_perm(__float_as_uint(x + 12582912.0f), __float_as_uint(y + 12582912.0f), 0x5410);
          uint32_t code = __viaddmin_s16x2_relu(q, zz, 0x000F000Fu);  // clamp(q + z, 0, 15)
          if (!inside && (n >= N || a * 32 + i * 8 >= cols)) code = 0x00080008u;
          word[a] = word[a] * 16 + code;
        }
      }
      uint8_t* to = Wp + (rt * Kb + kb) * kTileBytes + (h * 32 + lane) * 16;
      if (SQ_GUARD(within(to, 16, Wp, Nt * Kb * kTileBytes)))
        __stcs(reinterpret_cast<uint4*>(to), make_uint4(word[0], word[1], word[2], word[3]));
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// ---------------------------------------------------------------- values
// The reverse: each lane collects its 8 columns' nibbles from its quad and writes 16 bytes.
// code - zero is exact in bf16 (128 + code minus 128 + zero), so the product with the scale
// is rounded once. Bound by HBM: 28672 x 8192 105 us, 5.7 TB/s; 4096 x 4096 7.8 us.
template <int G, bool ASYM>
__global__ void __launch_bounds__(kInt4Threads, 4)
int4_dequant_kernel(const uint8_t* __restrict__ Wp, const uint16_t* __restrict__ scale,
                    const uint8_t* __restrict__ zero, int64_t N, int64_t K, uint16_t* __restrict__ out) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t Nt = (N + 15) / 16, Kb = (K + 127) / 128;
  const int64_t kb = blockIdx.x, step = static_cast<int64_t>(gridDim.y) * (kInt4Threads / 32);
  for (int64_t rt = static_cast<int64_t>(blockIdx.y) * (kInt4Threads / 32) + (threadIdx.x >> 5); rt < Nt; rt += step) {
    uint4 unit[2];
    uint32_t e[2][128 / G], z[2][128 / G];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t n = rt * 16 + h * 8 + g;
      unit[h] = __ldcs(reinterpret_cast<const uint4*>(Wp + (rt * Kb + kb) * kTileBytes + (h * 32 + lane) * 16));
#pragma unroll
      for (int j = 0; j < 128 / G; ++j) {
        e[h][j] = 0;
        z[h][j] = 8;
        if (n < N && kb * 128 + j * G < K) {
          const int64_t at = (kb * (128 / G) + j) * N + n;
          e[h][j] = __ldg(scale + at);
          if (ASYM) z[h][j] = __ldg(zero + at);
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t n = rt * 16 + h * 8 + g;
      const uint32_t word[4] = {unit[h].x, unit[h].y, unit[h].z, unit[h].w};
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const int64_t k = kb * 128 + a * 32 + t * 8;
        const uint32_t e2 = e[h][a * 32 / G] * 0x00010001u, zp = ASYM ? zero_pair(z[h][a * 32 / G]) : 0x43084308u;
        uint32_t w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          w[u] = __shfl_sync(0xffffffffu, word[a], (lane & ~3) | u) >> (4 * t);
          w[u] = mul_bf16x2(sub_bf16x2((w[u] & 0x000F000Fu) | 0x43004300u, zp), e2);
        }
        if (n < N && k < K && SQ_GUARD(within(out + n * K + k, 8, out, N * K)))
          __stcs(reinterpret_cast<uint4*>(out + n * K + k), make_uint4(w[0], w[1], w[2], w[3]));
      }
    }
  }
}

// ---------------------------------------------------------------- linear layer
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float2 ld_cluster_f32x2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

struct LinearParams {
  const uint16_t* X;
  int64_t ldx, N;
  const uint8_t* Wp;
  const uint16_t* scale;
  const uint8_t* zero;
  const uint16_t* bias;
  uint16_t* Y;
  int M, K, Kb, groups;
};

// ---- up to 4 tokens: int8 matrix instructions.
// Making bf16 of 4-bit codes costs a logic operation, most of a shift and a subtraction per pair;
// for a few tokens that is most of the work, and it bounds the kernel (measured: 230 instructions
// for a 1024-byte block, 41 us at 1 x 28672 x 8192 whatever the copies do). Bytes are cheaper: a
// word of eight codes masked with 0x0F0F0F0F, and shifted once, is two operands of four. So the
// activations become integers instead, once: a token, scaled by a power of two to 23 bits, is
// split into three signed bytes, three columns of the 16x8x32 instructions (elements down to
// 2^-14 of the token's largest are exact, smaller ones off by at most 2^-22 of it). Products and a
// group's sums are exact integers, and so is the zero point's part,
//   sum_k x_k (code - zero) = sum_k x_k code - zero * sum_k x_k,
// with the group's sums of x taken beforehand. A group's result is scaled and added in fp32.
//
// Rows too long for shared memory come in chunks of columns, if every team has one tile only (its
// sums stay in registers meanwhile).
//
// Teams of `kw` warps: each team on a row tile of its own, then on the next that is due (all
// teams of the grid in turn); within a tile the warps take pairs of 128-column blocks in turn.
// Every lane brings its own fragments into its warp's ring with asynchronous copies, across tiles
// and with nothing to wait for but the copies. The team meets once a tile to add its warps' sums
// up in order. One token: 28672 x 8192 27 us (4.5 TB/s), 8192 x 8192 10.4 us, 4096 x 4096 4.9 us (launch,
// first bytes and join).
constexpr int kTeamWarps = 16;  // of a CTA, one CTA per SM
constexpr int kTeamTokens = 4;
constexpr int64_t kSmemMax = 232448;

struct TeamParams {
  LinearParams p;
  int kw;         // warps of a team
  int rounds;     // tiles of a team
  int ring;       // slots of a warp's ring, 2 to 4
  int Kp;         // pairs of column blocks, the second of the last one may lie past K
  int cp;         // pairs whose activations are in shared memory at a time: all, or a multiple of kw
  int col_bytes;  // of a column of them
};

template <int G, bool ASYM>
constexpr int team_slot_bytes() {  // a pair of blocks: codes, 16 scales and 16 zero points per group
  return 2 * (kTileBytes + 128 / G * (ASYM ? 48 : 32));
}

__device__ __forceinline__ void mma_u8s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Where the rings begin: copies to odd multiples of 16 bytes cost more (2 x 8192 x 28672 35 us, 40 from
// there).
template <int G>
__host__ __device__ constexpr int team_ring_at(int tokens, int col_bytes, int cp, int nt) {
  return (3 * tokens * col_bytes + cp * (256 / G) * nt * 8 * 4 + 127) / 128 * 128;
}

// NT: columns / 8; column 3 m + d is byte d (0 the highest) of token m.
template <int NT, int G, bool ASYM>
__global__ void __launch_bounds__(kTeamWarps * 32, 1) int4_team_kernel(const TeamParams q) {
  constexpr int kGroups = 256 / G, kSlot = team_slot_bytes<G, ASYM>(), kCols = NT * 8;
  constexpr int kScales = 2 * kTileBytes, kZeros = kScales + kGroups * 32;
  const LinearParams& p = q.p;
  extern __shared__ __align__(128) uint8_t aligned_smem[];
  uint8_t* smem = aligned_smem;
  __shared__ uint32_t s_top[kTeamWarps];
  __shared__ float s_mul[kTeamTokens][2], s_back[kTeamTokens][2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int teams = kTeamWarps / q.kw, team = warp / q.kw, kw = warp % q.kw;
  const int Nt = static_cast<int>((p.N + 15) / 16), step = gridDim.x * teams;
  // tiles go to the SMs in turn; warps left over from the teams have none
  const int rt0 = team < teams ? static_cast<int>(blockIdx.x + gridDim.x * team) : Nt;
  // the weight does not depend on the kernel before in a decode step: its way into L2 starts
  // before waiting for that kernel (a hint, safe even if that kernel wrote the weight)
  if (kw == 0 && lane == 0 && rt0 < Nt)
    bulk_prefetch_l2(p.Wp + static_cast<int64_t>(rt0) * p.Kb * kTileBytes,
                     static_cast<uint32_t>(min(p.Kb, 2 * q.kw * q.ring)) * kTileBytes);
  griddep_wait();
  griddep_launch_dependents();

  // shared memory: columns of bytes | [groups][kCols] sums of a group's bytes | rings | partial sums
  // (with one tile per team, partial sums where the columns were)
  const int sums_at = 3 * p.M * q.col_bytes, ring_at = team_ring_at<G>(p.M, q.col_bytes, q.cp, NT);
  const uint32_t ring32 = smem_u32(smem) + ring_at + warp * q.ring * kSlot;
  int* sums = reinterpret_cast<int*>(smem + sums_at);
  float* part =  // [2][warps][kCols][16]
      reinterpret_cast<float*>(smem + (q.rounds == 1 ? 0 : ring_at + kTeamWarps * q.ring * kSlot));

  // ---- the next pair to bring
  int load_rt = kw < q.Kp ? rt0 : Nt, load_kp = kw;
  const uint8_t* load_src = p.Wp + (static_cast<int64_t>(rt0) * p.Kb + 2 * kw) * kTileBytes + lane * 16;
  const int64_t tile_jump = static_cast<int64_t>(step) * p.Kb * kTileBytes;
  // this lane's part of a pair's scales: kScaleLanes lanes of kScaleBytes; of its zero points: 4 bytes
  constexpr int kScaleBytes = G == 32 ? 8 : 4, kLanesPerGroup = 32 / kScaleBytes;
  constexpr int kScaleLanes = kGroups * kLanesPerGroup;
  const int e_group = lane / kLanesPerGroup, e_row = lane % kLanesPerGroup * (kScaleBytes / 2);
  const int z_group = lane / 4, z_row = lane % 4 * 4;
  const int64_t e_step = static_cast<int64_t>(q.kw) * kGroups * p.N;
  const uint16_t* e_src;  // this lane's scales of pair load_kp, there in pairs before e_end
  const uint8_t* z_src = nullptr;  // and zero points, before z_end
  int e_end, z_end;
  auto locate = [&]() {  // in the tile load_rt from pair load_kp on
    const int64_t e_n = static_cast<int64_t>(load_rt) * 16 + e_row, z_n = static_cast<int64_t>(load_rt) * 16 + z_row;
    e_src = p.scale + static_cast<int64_t>(load_kp * kGroups + e_group) * p.N + e_n;
    if (ASYM) z_src = p.zero + static_cast<int64_t>(load_kp * kGroups + z_group) * p.N + z_n;
    e_end = e_n < p.N ? (p.groups - e_group + kGroups - 1) / kGroups : 0;
    z_end = z_n < p.N ? (p.groups - z_group + kGroups - 1) / kGroups : 0;
  };
  locate();
  auto fetch = [&](int slot) {
    if (load_rt < Nt) {
      const uint32_t dst = ring32 + slot * kSlot;
      const bool second = 2 * load_kp + 1 < p.Kb;
      const bool codes = SQ_GUARD(
          within(load_src, second ? 1552 : 528, p.Wp, static_cast<int64_t>(Nt) * p.Kb * kTileBytes));
      cp_async<16>(dst + lane * 16, load_src, codes);
      cp_async<16>(dst + 512 + lane * 16, load_src + 512, codes);
      cp_async<16>(dst + 1024 + lane * 16, load_src + (second ? 1024 : 0), second && codes);
      cp_async<16>(dst + 1536 + lane * 16, load_src + (second ? 1536 : 0), second && codes);
      if (lane < kScaleLanes) {
        const bool in = load_kp < e_end && SQ_GUARD(within(e_src, kScaleBytes / 2, p.scale, p.groups * p.N));
        cp_async<kScaleBytes>(dst + kScales + lane * kScaleBytes, in ? e_src : p.scale, in);
      }
      if (ASYM && lane < 4 * kGroups) {
        const bool in = load_kp < z_end && SQ_GUARD(within(z_src, 4, p.zero, p.groups * p.N));
        cp_async<4>(dst + kZeros + lane * 4, in ? z_src : p.zero, in);
      }
      load_kp += q.kw;
      load_src += 2 * q.kw * kTileBytes;
      e_src += e_step;
      if (ASYM) z_src += e_step;
      if (load_kp >= q.Kp) {  // on to the team's next tile
        load_src += tile_jump - static_cast<int64_t>(load_kp - kw) * 2 * kTileBytes;
        load_kp = kw;
        load_rt += step;
        locate();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int i = 0; i < q.ring - 1; ++i) fetch(i);

  // ---- activations to bytes: the tokens' largest values, each by an equal share of the warps
  const int share = kTeamWarps / p.M;  // warps of a token
  if (warp < share * p.M) {
    const uint16_t* x = p.X + warp / share * p.ldx;
    uint32_t top = 0;  // bf16 without their signs are in the order of their bits, infinity and NaN last
#pragma unroll 4
    for (int k = (warp % share * 32 + lane) * 8; k < p.K; k += share * 256) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(x + k));
      top = __vmaxu2(__vmaxu2(top, v.x & 0x7FFF7FFFu), __vmaxu2(v.y & 0x7FFF7FFFu, v.z & 0x7FFF7FFFu));
      top = __vmaxu2(top, v.w & 0x7FFF7FFFu);
    }
    top = max(top >> 16, top & 0xFFFFu);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) s_top[warp] = top;
  }
  __syncthreads();
  if (threadIdx.x < p.M) {
    uint32_t top = 0;
    for (int w = 0; w < share; ++w) top = max(top, s_top[threadIdx.x * share + w]);
    // 2^up brings the largest, which may be subnormal, between 2^21 and 2^22: two factors, since up is
    // -106 to 155. Integers cannot carry infinity or NaN, so the token's results become NaN
    const int up = top >= 0x80u ? 22 + 126 - static_cast<int>(top >> 7) : 123 + __clz(static_cast<int>(top));
    const int up0 = min(up, 120), up1 = up - up0;
    s_mul[threadIdx.x][0] = __uint_as_float(static_cast<uint32_t>(127 + up0) << 23);
    s_mul[threadIdx.x][1] = __uint_as_float(static_cast<uint32_t>(127 + up1) << 23);
    // (of sums in units of the highest digit)
    s_back[threadIdx.x][0] = __uint_as_float(top < 0x7F80u ? static_cast<uint32_t>(143 - up0) << 23 : 0x7FC00000u);
    s_back[threadIdx.x][1] = __uint_as_float(static_cast<uint32_t>(127 - up1) << 23);
  }
  __syncthreads();
  // then 8 elements per thread and step; a warp takes a pair of blocks: 8 words of 32 columns x 4 quad lanes
  auto to_bytes = [&](int first, int pairs) {
    for (int i = warp; i < p.M * pairs; i += kTeamWarps) {
      const int m = i / pairs, kp = i % pairs, word = (first + kp) * 8 + lane / 4;
      const float mul = s_mul[m][0], mul1 = s_mul[m][1];
      const uint16_t* src = p.X + m * p.ldx + word * 32 + t * 2;
      uint32_t v[8];  // columns 2 t, 2 t + 1 of each 8
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t x = word * 32 + c * 8 < p.K ? __ldg(reinterpret_cast<const uint32_t*>(src + c * 8)) : 0u;
        // round to an integer in the low mantissa bits (1.5 * 2^23 added), then bytes with carries:
        // the three low bytes of v + 0x808080, each less 128, are the signed digits
        v[2 * c] = __float_as_uint(__fmaf_rn(bf16_lo(x) * mul1, mul, 12582912.0f)) + (0x00808080u - 0x4B400000u);
        v[2 * c + 1] = __float_as_uint(__fmaf_rn(bf16_hi(x) * mul1, mul, 12582912.0f)) + (0x00808080u - 0x4B400000u);
      }
#pragma unroll
      for (int d = 0; d < 3; ++d) {
        // the order of a word's codes: low nibbles are columns 2t, 16 + 2t, 2t + 1, 17 + 2t, high ones 8 more
        const uint32_t pick = d == 0 ? 0x0062u : d == 1 ? 0x0051u : 0x0040u;
        uint32_t b0 = __byte_perm(__byte_perm(v[0], v[4], pick), __byte_perm(v[1], v[5], pick), 0x5410);
        uint32_t b1 = __byte_perm(__byte_perm(v[2], v[6], pick), __byte_perm(v[3], v[7], pick), 0x5410);
        b0 ^= 0x80808080u;
        b1 ^= 0x80808080u;
        const int col = 3 * m + d, at = col * q.col_bytes + (2 * kp + lane / 16) * 128 + t * 32 + lane / 4 % 4 * 8;
        *reinterpret_cast<uint2*>(smem + at) = make_uint2(b0, b1);
        int sum = __dp4a(static_cast<int>(b0), 0x01010101, __dp4a(static_cast<int>(b1), 0x01010101, 0));
#pragma unroll
        for (int o = 1; o < G / 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane % (G / 8) == 0) sums[(kp * kGroups + lane / (G / 8)) * kCols + col] = sum;
      }
    }
  };

  // B fragments: column 8 nt + g, this lane's 32 bytes of a block; columns past 3 M repeat the last
  // one and nothing reads their results
  const uint8_t* x_col[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) x_col[nt] = smem + min(nt * 8 + g, 3 * p.M - 1) * q.col_bytes + t * 32;
  float acc[NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.0f;
  int side = 0, slot = 0, free_slot = q.ring - 1;
  int rt = rt0;
  for (int round = 0; round < q.rounds; ++round, rt += step) {
    for (int first = 0; first < q.Kp; first += q.cp) {
      const int pairs = min(q.cp, q.Kp - first);
      if (round == 0) {  // (more than one chunk: there is one round)
        if (first > 0) __syncthreads();  // the chunk before is read
        to_bytes(first, pairs);
        __syncthreads();
      }
#pragma unroll 1
      for (int kp = rt < Nt ? kw : pairs; kp < pairs; kp += q.kw) {
        if (q.ring == 4)
          asm volatile("cp.async.wait_group 2;" ::: "memory");
        else if (q.ring == 3)
          asm volatile("cp.async.wait_group 1;" ::: "memory");
        else
          asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncwarp();  // every lane's copies are there, and the slot before is read
        fetch(free_slot);
        const uint8_t* src = smem + ring_at + warp * q.ring * kSlot + slot * kSlot;
        const uint16_t* es = reinterpret_cast<const uint16_t*>(src + kScales) + g;
        const uint8_t* zs = src + kZeros + g;
        const int* sx = sums + kp * kGroups * kCols + 2 * t;
        free_slot = slot;
        slot = slot + 1 == q.ring ? 0 : slot + 1;
        int d[NT][4];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const uint4 u0 = *reinterpret_cast<const uint4*>(src + b * 1024 + lane * 16);
          const uint4 u1 = *reinterpret_cast<const uint4*>(src + b * 1024 + 512 + lane * 16);
          const uint32_t lo[4] = {u0.x, u0.y, u0.z, u0.w}, hi[4] = {u1.x, u1.y, u1.z, u1.w};
          uint32_t x[NT][4];  // of two words
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            const int gr = (b * 128 + a * 32) / G;
            if (a % 2 == 0) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const uint4 v = *reinterpret_cast<const uint4*>(x_col[nt] + (2 * kp + b) * 128 + a * 8);
                x[nt][0] = v.x; x[nt][1] = v.y; x[nt][2] = v.z; x[nt][3] = v.w;
              }
            }
            if (a * 32 % G == 0) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) d[nt][0] = d[nt][1] = d[nt][2] = d[nt][3] = 0;
            }
            const uint32_t a0 = lo[a] & 0x0F0F0F0Fu, a1 = hi[a] & 0x0F0F0F0Fu;
            const uint32_t a2 = (lo[a] >> 4) & 0x0F0F0F0Fu, a3 = (hi[a] >> 4) & 0x0F0F0F0Fu;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_u8s8(d[nt], a0, a1, a2, a3, x[nt][a % 2 * 2], x[nt][a % 2 * 2 + 1]);
            if ((a + 1) * 32 % G == 0) {
              const float e0 = bf16_lo(es[gr * 16]), e1 = bf16_lo(es[gr * 16 + 8]);
              const int z0 = ASYM ? zs[gr * 16] : 8, z1 = ASYM ? zs[gr * 16 + 8] : 8;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const int2 sm = *reinterpret_cast<const int2*>(sx + gr * kCols + nt * 8);
                acc[nt][0] = fmaf(static_cast<float>(d[nt][0] - z0 * sm.x), e0, acc[nt][0]);
                acc[nt][1] = fmaf(static_cast<float>(d[nt][1] - z0 * sm.y), e0, acc[nt][1]);
                acc[nt][2] = fmaf(static_cast<float>(d[nt][2] - z1 * sm.x), e1, acc[nt][2]);
                acc[nt][3] = fmaf(static_cast<float>(d[nt][3] - z1 * sm.y), e1, acc[nt][3]);
              }
            }
          }
        }
      }
    }
    if (q.rounds == 1) __syncthreads();  // the columns are read, the sums may take their place
    if (rt >= Nt) continue;
    // [team][warp][columns][16] sums; the other side is free once the team has met again
    float* mine = part + (side * kTeamWarps + warp) * kCols * 16;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        mine[(nt * 8 + 2 * t + (c & 1)) * 16 + g + (c & 2) * 4] = acc[nt][c];
        acc[nt][c] = 0.0f;
      }
    if (q.kw == 1)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(q.kw * 32) : "memory");
    const float* all = part + (side * kTeamWarps + team * q.kw) * kCols * 16;
    for (int i = kw * 32 + lane; i < p.M * 8; i += q.kw * 32) {
      const int m = i / 8, r = i % 8 * 2;
      const int64_t n = static_cast<int64_t>(rt) * 16 + r;
      if (n >= p.N) continue;
      float y0 = 0.0f, y1 = 0.0f;
      for (int k = 0; k < q.kw; ++k) {
        const float* c = all + (k * kCols + 3 * m) * 16 + r;
        const float2 v0 = *reinterpret_cast<const float2*>(c), v1 = *reinterpret_cast<const float2*>(c + 16);
        const float2 v2 = *reinterpret_cast<const float2*>(c + 32);
        y0 += fmaf(fmaf(v2.x, 0x1p-8f, v1.x), 0x1p-8f, v0.x);
        y1 += fmaf(fmaf(v2.y, 0x1p-8f, v1.y), 0x1p-8f, v0.y);
      }
      y0 = y0 * s_back[m][0] * s_back[m][1];
      y1 = y1 * s_back[m][0] * s_back[m][1];
      if (p.bias != nullptr) {
        const uint32_t b = __ldg(reinterpret_cast<const uint32_t*>(p.bias + n));
        y0 += bf16_lo(b);
        y1 += bf16_hi(b);
      }
      if (SQ_GUARD(within(p.Y + m * p.N + n, 2, p.Y, p.M * p.N)))
        *reinterpret_cast<__nv_bfloat162*>(p.Y + m * p.N + n) = __floats2bfloat162_rn(y0, y1);
    }
    side ^= q.rounds > 1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Shared memory of a team launch; see the kernel's layout.
template <int G, bool ASYM>
int64_t team_smem(const TeamParams& q, int nt) {
  const int64_t cols = nt * 8, sums = kTeamWarps * cols * 64;
  const int64_t rest = team_ring_at<G>(q.p.M, q.col_bytes, q.cp, nt) + kTeamWarps * q.ring * team_slot_bytes<G, ASYM>();
  return q.rounds == 1 ? std::max(rest, sums) : rest + 2 * sums;
}

// Slots and chunks: all columns at once with as many slots as fit, or, with one tile per team, the
// largest chunks beside three slots (at least 8 pairs, else the other kernel is as fast).
template <int G, bool ASYM>
bool team_fits(TeamParams* q, int nt) {
  const int64_t most = kSmemMax - 1024;
  auto fits = [&](int ring, int cp) {
    q->ring = ring;
    q->cp = cp;
    q->col_bytes = cp * 256 + 16;  // an odd number of 16-byte units: no bank conflicts
    return team_smem<G, ASYM>(*q, nt) <= most;
  };
  for (int ring = 4; ring >= 2; --ring)
    if (fits(ring, q->Kp)) return true;
  if (q->rounds > 1) return false;
  for (int cp = q->Kp / q->kw * q->kw; cp >= 8; cp -= q->kw)
    if (fits(3, cp)) return true;
  return false;
}

// Warps of a team. A round of tiles takes an SM the time of its bytes, but a tile never less than
// its team's warps need for it, about a tenth of the SM's bandwidth each; teams with more than
// one tile wait for their slowest warp at each. Among equals the larger team, which is done sooner
// with a small weight. Measured, us, one token, teams of 2 / 4 / 8 / 16 warps: 4096 x 4096
// 5.3 / 4.8 / 4.9 / 5.6 (8 taken), 11008 x 4096 7.1 / 7.5 / 7.8 / 9.6 (3 taken, 6.9),
// 28672 x 8192 27.0 / 26.7 / 26.2 / 31.7 (1 taken, 26.9: 3% off the best).
int team_warps(int64_t Nt, int sms, int Kp) {
  const int64_t tiles = (Nt + sms - 1) / sms;  // of an SM
  int best = 1;
  double least = 1e30;
  for (int kw = 1; kw <= kTeamWarps && kw <= Kp; ++kw) {
    const int64_t teams = kTeamWarps / kw, rounds = (tiles + teams - 1) / teams;
    const double slow = 10.0 / kw;
    double cost = static_cast<double>(rounds - 1) * std::max<double>(teams, slow) +
                  std::max<double>(tiles - (rounds - 1) * teams, slow);
    if (kw > 1 && rounds > 1) cost += 0.3 * rounds;
    if (cost <= least) least = cost, best = kw;
  }
  return best;
}

template <int NT, int G, bool ASYM>
cudaError_t launch_team(const TeamParams& q, int sms, cudaStream_t stream) {
  auto kernel = int4_team_kernel<NT, G, ASYM>;
  const int smem = static_cast<int>(team_smem<G, ASYM>(q, NT));
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t ctas = std::min<int64_t>(sms, (q.p.N + 15) / 16);
  return launch_kernel(kernel, dim3(static_cast<unsigned>(ctas)), dim3(kTeamWarps * 32), smem, stream, true, q);
}

// ---- up to 16 tokens: bf16 matrix instructions.
// The weight rows are the 16 rows of 16x8x16 instructions, 8 NT tokens their columns. Codes become
// bf16 exactly (128 + code, minus 128 + zero); a group's fp32 sum is scaled and added to the
// total. Teams and rings as above; the activations come in chunks of `cp` pairs of column blocks
// for all teams of a CTA, one chunk ahead, and where there are too few row tiles for that the
// CTAs of a cluster share the columns and add their sums up, in order, through distributed
// shared memory. 16 x 28672 x 8192 55 us (2.3 TB/s), 8 x 28672 x 8192 43.5, 5 x 11008 x 4096 12.2:
// no unit is full (integer pipe 51%, 0.55 instructions a cycle); bound by waiting, most of it at the
// block barrier of each chunk, with 12 or 13 of the 16 warps at work where an SM has as many tiles,
// and then for instructions before.
struct WideParams {
  LinearParams p;
  int split;    // CTAs of a cluster
  int kw;       // warps of a team
  int ring;     // slots of a warp's ring, 2 to 4
  int Kp;       // pairs of column blocks
  int cp;       // of a chunk, a multiple of kw
  int rounds;   // tiles of a team
  int buffers;  // of chunks
  unsigned int* status;
};

template <int NT, int G, bool ASYM>
__global__ void __launch_bounds__(kTeamWarps * 32, 1) int4_wide_kernel(const WideParams q) {
  constexpr int W = kTeamWarps, kThreads = W * 32, kGroups = 256 / G, kSlot = team_slot_bytes<G, ASYM>();
  constexpr int kScales = 2 * kTileBytes, kZeros = kScales + kGroups * 32;
  const LinearParams& p = q.p;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(8) uint64_t s_there[2];  // a chunk's copies are there
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int teams = W / q.kw, team = warp / q.kw, kw = warp % q.kw;
  const int rank = blockIdx.x % q.split, cluster = blockIdx.x / q.split, clusters = gridDim.x / q.split;
  const int Nt = static_cast<int>((p.N + 15) / 16), step = clusters * teams;
  const int rt0 = team < teams ? cluster + clusters * team : Nt;
  const int kp0 = static_cast<int>(static_cast<int64_t>(q.Kp) * rank / q.split);
  const int kp1 = static_cast<int>(static_cast<int64_t>(q.Kp) * (rank + 1) / q.split);
  if (kw == 0 && lane == 0 && rt0 < Nt)  // as above
    bulk_prefetch_l2(p.Wp + (static_cast<int64_t>(rt0) * p.Kb + 2 * kp0) * kTileBytes,
                     static_cast<uint32_t>(min(p.Kb - 2 * kp0, 2 * q.kw * q.ring)) * kTileBytes);
  if (threadIdx.x == 0) {
    mbar_init(&s_there[0], kThreads);
    mbar_init(&s_there[1], kThreads);
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();

  // shared memory: chunks of activations | rings | partial sums
  const int x_row = q.cp * 512 + 16, x_bytes = p.M * x_row;  // rows of an odd number of 16-byte units
  const uint32_t smem32 = smem_u32(smem);
  const int ring_at = q.buffers * x_bytes + warp * q.ring * kSlot;
  const uint32_t ring32 = smem32 + ring_at;
  float* part = reinterpret_cast<float*>(smem + q.buffers * x_bytes + W * q.ring * kSlot);  // [warps][M][16]

  int load_rt = kp0 + kw < kp1 ? rt0 : Nt, load_kp = kp0 + kw;
  const uint8_t* load_src = p.Wp + (static_cast<int64_t>(rt0) * p.Kb + 2 * load_kp) * kTileBytes + lane * 16;
  const int64_t tile_jump = static_cast<int64_t>(step) * p.Kb * kTileBytes;
  constexpr int kScaleBytes = G == 32 ? 8 : 4, kLanesPerGroup = 32 / kScaleBytes;
  constexpr int kScaleLanes = kGroups * kLanesPerGroup;
  const int e_group = lane / kLanesPerGroup, e_row = lane % kLanesPerGroup * (kScaleBytes / 2);
  const int z_group = lane / 4, z_row = lane % 4 * 4;
  const int64_t e_step = static_cast<int64_t>(q.kw) * kGroups * p.N;
  const uint16_t* e_src;  // this lane's scales of pair load_kp, there in pairs before e_end
  const uint8_t* z_src = nullptr;  // and zero points, before z_end
  int e_end, z_end;
  auto locate = [&]() {  // in the tile load_rt from pair load_kp on
    const int64_t e_n = static_cast<int64_t>(load_rt) * 16 + e_row, z_n = static_cast<int64_t>(load_rt) * 16 + z_row;
    e_src = p.scale + static_cast<int64_t>(load_kp * kGroups + e_group) * p.N + e_n;
    if (ASYM) z_src = p.zero + static_cast<int64_t>(load_kp * kGroups + z_group) * p.N + z_n;
    e_end = e_n < p.N ? (p.groups - e_group + kGroups - 1) / kGroups : 0;
    z_end = z_n < p.N ? (p.groups - z_group + kGroups - 1) / kGroups : 0;
  };
  locate();
  auto fetch = [&](int slot) {
    if (load_rt < Nt) {
      const uint32_t dst = ring32 + slot * kSlot;
      const bool second = 2 * load_kp + 1 < p.Kb;
      const bool codes = SQ_GUARD(
          within(load_src, second ? 1552 : 528, p.Wp, static_cast<int64_t>(Nt) * p.Kb * kTileBytes));
      cp_async<16>(dst + lane * 16, load_src, codes);
      cp_async<16>(dst + 512 + lane * 16, load_src + 512, codes);
      cp_async<16>(dst + 1024 + lane * 16, load_src + (second ? 1024 : 0), second && codes);
      cp_async<16>(dst + 1536 + lane * 16, load_src + (second ? 1536 : 0), second && codes);
      if (lane < kScaleLanes) {
        const bool in = load_kp < e_end && SQ_GUARD(within(e_src, kScaleBytes / 2, p.scale, p.groups * p.N));
        cp_async<kScaleBytes>(dst + kScales + lane * kScaleBytes, in ? e_src : p.scale, in);
      }
      if (ASYM && lane < 4 * kGroups) {
        const bool in = load_kp < z_end && SQ_GUARD(within(z_src, 4, p.zero, p.groups * p.N));
        cp_async<4>(dst + kZeros + lane * 4, in ? z_src : p.zero, in);
      }
      load_kp += q.kw;
      load_src += 2 * q.kw * kTileBytes;
      e_src += e_step;
      if (ASYM) z_src += e_step;
      if (load_kp >= kp1) {
        load_src += tile_jump - static_cast<int64_t>(load_kp - kp0 - kw) * 2 * kTileBytes;
        load_kp = kp0 + kw;
        load_rt += step;
        locate();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // chunk c of this CTA's columns into a buffer; each thread's copies report to the buffer's barrier
  auto bring = [&](int c, int buffer) {
    const uint32_t dst = smem32 + buffer * x_bytes;
    const int k0 = (kp0 + c * q.cp) * 256, cols = min(q.cp, kp1 - kp0 - c * q.cp) * 32;  // of 8 columns
    for (int m = warp; m < p.M; m += W)
      for (int i = lane; i < cols; i += 32) {
        const bool in = k0 + i * 8 < p.K;
        cp_async<16>(dst + m * x_row + i * 16, p.X + m * p.ldx + (in ? k0 + i * 8 : 0),
                     in && SQ_GUARD(k0 >= 0 && k0 + i * 8 + 8 <= p.K));
      }
    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(&s_there[buffer])) : "memory");
  };

  const int chunks = (kp1 - kp0 + q.cp - 1) / q.cp, steps = q.rounds * chunks;
  const bool resident = chunks <= 2;  // each chunk stays in a buffer of its own
  bring(0, 0);
#pragma unroll 1
  for (int i = 0; i < q.ring - 1; ++i) fetch(i);

  uint32_t x_lane[NT];  // this lane's row for loading fragments; columns past M repeat the last token, unread
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) x_lane[nt] = smem32 + min(nt * 8 + (lane & 7), p.M - 1) * x_row + (lane >> 3) * 16;
  float acc[NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.0f;
  int slot = 0, free_slot = q.ring - 1, chunk = 0, rt = rt0;
  unsigned phase = 0;  // bit b: parity of buffer b's next chunk
  for (int s = 0; s < steps; ++s) {
    __syncthreads();  // the chunk before is read
    if (s + 1 < steps && (!resident || s + 1 < chunks)) bring(chunk + 1 < chunks ? chunk + 1 : 0, (s + 1) & 1);
    const int buffer = resident ? chunk : s & 1;
    if (!resident || s < chunks) {
      if (!mbar_wait_bounded(&s_there[buffer], (phase >> buffer) & 1, kDefaultWaitLimitNs) && lane == 0)
        atomicOr(q.status, kErrProducerWait);
      phase ^= 1u << buffer;
    }
    const int here = min(q.cp, kp1 - kp0 - chunk * q.cp);  // pairs of the chunk
    if (rt < Nt) {
#pragma unroll 1
      for (int j = kw; j < here; j += q.kw) {
        if (q.ring == 4)
          asm volatile("cp.async.wait_group 2;" ::: "memory");
        else if (q.ring == 3)
          asm volatile("cp.async.wait_group 1;" ::: "memory");
        else
          asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncwarp();  // every lane's copies are there, and the slot before is read
        fetch(free_slot);
        const uint8_t* src = smem + ring_at + slot * kSlot;
        const uint16_t* es = reinterpret_cast<const uint16_t*>(src + kScales) + g;
        const uint8_t* zs = src + kZeros + g;
        free_slot = slot;
        slot = slot + 1 == q.ring ? 0 : slot + 1;
        const uint32_t x_at = buffer * x_bytes + j * 512;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const uint4 u0 = *reinterpret_cast<const uint4*>(src + b * 1024 + lane * 16);
          const uint4 u1 = *reinterpret_cast<const uint4*>(src + b * 1024 + 512 + lane * 16);
          const uint32_t lo[4] = {u0.x, u0.y, u0.z, u0.w}, hi[4] = {u1.x, u1.y, u1.z, u1.w};
          float d[NT][4];
          uint32_t z0 = 0x43084308u, z1 = 0x43084308u;
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            const int gr = (b * 128 + a * 32) / G * 16;
            if (a * 32 % G == 0) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) d[nt][0] = d[nt][1] = d[nt][2] = d[nt][3] = 0.0f;
              if (ASYM) {
                z0 = zero_pair(zs[gr]);
                z1 = zero_pair(zs[gr + 8]);
              }
            }
            uint32_t f[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              f[h][0] = sub_bf16x2(((lo[a] >> (8 * h)) & 0x000F000Fu) | 0x43004300u, z0);
              f[h][1] = sub_bf16x2(((hi[a] >> (8 * h)) & 0x000F000Fu) | 0x43004300u, z1);
              f[h][2] = sub_bf16x2(((lo[a] >> (8 * h + 4)) & 0x000F000Fu) | 0x43004300u, z0);
              f[h][3] = sub_bf16x2(((hi[a] >> (8 * h + 4)) & 0x000F000Fu) | 0x43004300u, z1);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              uint32_t x[4];
              ldmatrix(x, x_lane[nt] + x_at + b * 256 + a * 64);
              mma_bf16(d[nt], f[0], x[0], x[1]);
              mma_bf16(d[nt], f[1], x[2], x[3]);
            }
            if ((a + 1) * 32 % G == 0) {
              const float e0 = bf16_lo(es[gr]), e1 = bf16_lo(es[gr + 8]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                acc[nt][0] = fmaf(d[nt][0], e0, acc[nt][0]);
                acc[nt][1] = fmaf(d[nt][1], e0, acc[nt][1]);
                acc[nt][2] = fmaf(d[nt][2], e1, acc[nt][2]);
                acc[nt][3] = fmaf(d[nt][3], e1, acc[nt][3]);
              }
            }
          }
        }
      }
    }
    if (++chunk < chunks) continue;
    chunk = 0;
    // ---- the tiles of this round are done: partial sums of every warp, then each CTA of the
    // cluster finishes its share of the outputs
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int m = nt * 8 + 2 * t + (e & 1);
        if (m < p.M) part[(warp * p.M + m) * 16 + g + (e & 2) * 4] = acc[nt][e];
        acc[nt][e] = 0.0f;
      }
    if (q.split > 1)
      cluster_sync();
    else
      __syncthreads();
    const int64_t tile0 = cluster + static_cast<int64_t>(s / chunks) * step;  // the first team's tile
    for (int i = threadIdx.x * q.split + rank; i < teams * p.M * 8; i += kThreads * q.split) {
      const int r = i % 8 * 2, m = i / 8 % p.M, tm = i / 8 / p.M;
      const int64_t row = (tile0 + clusters * tm) * 16 + r;
      if (row >= p.N) continue;
      float y0 = 0.0f, y1 = 0.0f;
      const float* at = part + (tm * q.kw * p.M + m) * 16 + r;
      if (q.split == 1) {
#pragma unroll 4
        for (int k = 0; k < q.kw; ++k) {
          const float2 v = *reinterpret_cast<const float2*>(at + k * p.M * 16);
          y0 += v.x;
          y1 += v.y;
        }
      } else {
        for (int c = 0; c < q.split; ++c) {
          const uint32_t remote = mapa_shared(at, c);
#pragma unroll 4
          for (int k = 0; k < q.kw; ++k) {
            const float2 v = ld_cluster_f32x2(remote + k * p.M * 64);
            y0 += v.x;
            y1 += v.y;
          }
        }
      }
      if (p.bias != nullptr) {
        const uint32_t b = __ldg(reinterpret_cast<const uint32_t*>(p.bias + row));
        y0 += bf16_lo(b);
        y1 += bf16_hi(b);
      }
      if (SQ_GUARD(within(p.Y + m * p.N + row, 2, p.Y, p.M * p.N)))
        *reinterpret_cast<__nv_bfloat162*>(p.Y + m * p.N + row) = __floats2bfloat162_rn(y0, y1);
    }
    if (q.split > 1) cluster_sync();  // the sums are read: they may be overwritten, or the CTA may end
    rt += step;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int NT, int G, bool ASYM>
cudaError_t launch_wide(const LinearParams& p, int sms, unsigned int* status, cudaStream_t stream) {
  constexpr int W = kTeamWarps, kSlot = team_slot_bytes<G, ASYM>();
  WideParams q{};
  q.p = p;
  q.Kp = (p.Kb + 1) / 2;
  q.status = status;
  const int64_t Nt = (p.N + 15) / 16;
  // The shape of the launch by its estimated time in us, fitted to about 100 measured ones (34 sizes,
  // 1 to 16 tokens; 9% off in the root mean square): a warp alone takes 0.41 for a pair of blocks, all
  // warps of an SM together 0.098 a pair, the larger of the two sums and 0.28 of the smaller count;
  // the activations come at 74 KB a us, a chunk of them costs 0.26 where chunks take turns, a round
  // of tiles 0.74, a cluster of two 1.3 and of four 4 (of eight more than it saves).
  double least = 1e30;
  size_t smem = 0;
  for (int split = 1; split <= 4 && split <= q.Kp; split *= 2) {
    const int64_t clusters = std::min<int64_t>(cluster_slots(sms, split), Nt), tiles = (Nt + clusters - 1) / clusters;
    const int pairs = (q.Kp + split - 1) / split;
    for (int kw = 1; kw <= W && kw <= pairs; ++kw) {
      const int64_t teams = W / kw, rounds = (tiles + teams - 1) / teams;
      const double x_kb = 0.5 * static_cast<double>(rounds) * pairs * p.M;
      const double alone = 0.41 * static_cast<double>(rounds) * ((pairs + kw - 1) / kw);
      const double together = 0.098 * static_cast<double>(tiles) * pairs;
      const double base = std::max(alone, together) + 0.28 * std::min(alone, together) + x_kb / 74 +
                          0.74 * static_cast<double>(rounds) + (split == 4 ? 4.0 : split == 2 ? 1.3 : 0.0);
      if (base >= least) continue;
      // the largest chunks, up to all columns, that leave three slots for every ring
      const int64_t room = kSmemMax - 1024 - static_cast<int64_t>(W) * p.M * 64;
      for (int ring = 4; ring >= 2; --ring) {
        const int64_t left = room - W * ring * kSlot, row = 512;
        int64_t all = (pairs + kw - 1) / kw * kw;
        int buffers = 1;
        if (p.M * (all * row + 16) > left) {
          buffers = 2;
          all = (left / 2 / p.M - 16) / row / kw * kw;
        }
        if (all < kw || (ring > 2 && buffers == 2 && all * p.M < 64)) continue;
        const double turns = buffers == 2 ? 0.26 * static_cast<double>(rounds) * ((pairs + all - 1) / all) : 0.0;
        if (base + turns >= least) break;
        least = base + turns;
        q.split = split;
        q.kw = kw;
        q.ring = ring;
        q.cp = static_cast<int>(all);
        q.rounds = static_cast<int>(rounds);
        q.buffers = buffers;
        smem = static_cast<size_t>(buffers * p.M * (all * row + 16) + W * ring * kSlot + W * p.M * 64);
        break;
      }
    }
  }
  const int64_t clusters = std::min<int64_t>(cluster_slots(sms, q.split), Nt);
  auto kernel = int4_wide_kernel<NT, G, ASYM>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_kernel_clustered(kernel, dim3(static_cast<unsigned>(clusters * q.split)), dim3(W * 32), smem, stream,
                                 true, static_cast<unsigned>(q.split), q);
}

template <int G, bool ASYM>
cudaError_t launch_linear(const LinearParams& p, unsigned int* status, cudaStream_t stream) {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  // Every CTA of the int8 kernel makes bytes of all activations, which takes enough row tiles to pay.
  // Measured (us, int8 / bf16 kernel) at 0.2, 1, 1.4, 3.5, 4.6 and 12 tiles an SM (448 x 13376, 2472 x
  // 22560, 3232 x 12112, 8192 x 8192, 11008 x 4096, 28672 x 8192): 1 token 7.9 / 7.1, 16 / 15,
  // 9.3 / 10.4, 10.4 / 14.6, 7.6 / 10.0, 26 / 41; 4 tokens 16 / 7.6, 32 / 16, 17 / 12, 18 / 16, 10.7 / 11.5,
  // 35 / 43.
  const int64_t Nt = (p.N + 15) / 16;
  if (p.M <= kTeamTokens && 5 * Nt >= (p.M <= 2 ? 6 : 20) * static_cast<int64_t>(sms)) {
    TeamParams q;
    q.p = p;
    q.Kp = (p.Kb + 1) / 2;
    const int64_t ctas = std::min<int64_t>(sms, Nt);
    q.kw = team_warps(Nt, sms, q.Kp);
    const int64_t teams = ctas * (kTeamWarps / q.kw);
    q.rounds = static_cast<int>((Nt + teams - 1) / teams);
    const int nt = (3 * p.M + 7) / 8;
    if (team_fits<G, ASYM>(&q, nt)) {
      return nt == 1 ? launch_team<1, G, ASYM>(q, sms, stream) : launch_team<2, G, ASYM>(q, sms, stream);
    }
  }
  if (p.M <= 8) return launch_wide<1, G, ASYM>(p, sms, status, stream);
  return launch_wide<2, G, ASYM>(p, sms, status, stream);
}

// Grid of the two tile kernels: one column block per x, row tiles over y so that about `per_sm`
// CTAs per SM exist and each column block's factors are read by few of them.
dim3 tile_grid(int64_t N, int64_t K, int per_sm) {
  const int64_t Kb = (K + 127) / 128, rows = ((N + 15) / 16 + kInt4Threads / 32 - 1) / (kInt4Threads / 32);
  const int64_t y = std::max<int64_t>(1, std::min<int64_t>(rows, (148 * per_sm + Kb - 1) / Kb));
  return dim3(static_cast<unsigned>(Kb), static_cast<unsigned>(y));
}

template <int G>
cudaError_t launch_quant_g(const uint16_t* W, int64_t N, int64_t K, int64_t ldw, const float* s, uint8_t* Wp,
                           uint16_t* scale, uint8_t* zero, cudaStream_t stream) {
  auto kernel = zero != nullptr ? int4_quant_kernel<G, true> : int4_quant_kernel<G, false>;
  constexpr int smem = kInt4Threads / 32 * kQuantRing * kQuantSlot;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kernel, tile_grid(N, K, 4), dim3(kInt4Threads), smem, stream, true, W, N, K, ldw, s, Wp, scale,
                       zero);
}

template <int G>
cudaError_t launch_dequant_g(const uint8_t* Wp, const uint16_t* scale, const uint8_t* zero, int64_t N, int64_t K,
                             uint16_t* out, cudaStream_t stream) {
  auto kernel = zero != nullptr ? int4_dequant_kernel<G, true> : int4_dequant_kernel<G, false>;
  return launch_kernel(kernel, tile_grid(N, K, 8), dim3(kInt4Threads), 0, stream, true, Wp, scale, zero, N, K, out);
}

}  // namespace

size_t int4_weight_bytes(int64_t N, int64_t K) {
  return static_cast<size_t>((N + 15) / 16) * static_cast<size_t>((K + 127) / 128) * kTileBytes;
}

cudaError_t launch_int4_quant(const uint16_t* W, int64_t N, int64_t K, int64_t ldw, const float* s, int group,
                              uint8_t* Wp, uint16_t* scale, uint8_t* zero, cudaStream_t stream) {
  if (group == 32) return launch_quant_g<32>(W, N, K, ldw, s, Wp, scale, zero, stream);
  return group == 64 ? launch_quant_g<64>(W, N, K, ldw, s, Wp, scale, zero, stream)
                     : launch_quant_g<128>(W, N, K, ldw, s, Wp, scale, zero, stream);
}

cudaError_t launch_int4_dequant(const uint8_t* Wp, const uint16_t* scale, const uint8_t* zero, int group, int64_t N,
                                int64_t K, uint16_t* out, cudaStream_t stream) {
  if (group == 32) return launch_dequant_g<32>(Wp, scale, zero, N, K, out, stream);
  return group == 64 ? launch_dequant_g<64>(Wp, scale, zero, N, K, out, stream)
                     : launch_dequant_g<128>(Wp, scale, zero, N, K, out, stream);
}

cudaError_t launch_int4_linear(const Int4LinearArgs& a, cudaStream_t stream) {
  // Measured (us; these kernels / tcgen05): 8 x 28672 x 8192 43 / 58, 16 x 28672 x 8192 55 / 58,
  // 16 x 11008 x 4096 15 / 17, 32 x 28672 x 8192 79 / 63, 64 x 4096 x 4096 45 / 12
  if (a.M > 16) return launch_int4_linear_tc(a, stream);
  LinearParams p{};
  p.X = a.X;
  p.ldx = a.ldx;
  p.N = a.N;
  p.Wp = a.Wp;
  p.scale = a.scale;
  p.zero = a.zero;
  p.bias = a.bias;
  p.Y = a.Y;
  p.M = static_cast<int>(a.M);
  p.K = static_cast<int>(a.K);
  p.Kb = (p.K + 127) / 128;
  p.groups = (p.K + a.group - 1) / a.group;
  if (a.zero != nullptr) {
    if (a.group == 32) return launch_linear<32, true>(p, a.status, stream);
    return a.group == 64 ? launch_linear<64, true>(p, a.status, stream) : launch_linear<128, true>(p, a.status, stream);
  }
  if (a.group == 32) return launch_linear<32, false>(p, a.status, stream);
  return a.group == 64 ? launch_linear<64, false>(p, a.status, stream) : launch_linear<128, false>(p, a.status, stream);
}

}  // namespace sq
