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
// bf16 pair of 128 + z: 0x4300 is 128, whose mantissa counts in ones.
__device__ __forceinline__ uint32_t zero_pair(uint32_t z) { return 0x43004300u | z | (z << 16); }

// ---------------------------------------------------------------- quantization
// One warp per tile, over the row tiles of one 128-column block. Lane (g, t) reads the
// columns 32 a + 8 t .. + 7 of rows g and g + 8 (16-byte loads, 64 contiguous bytes per row),
// so a group of 32 columns belongs to the four lanes of a quad, and two exchanges between
// them put the codes where the layout wants them.
template <bool ASYM>
__global__ void __launch_bounds__(kInt4Threads)
int4_quant_kernel(const uint16_t* __restrict__ W, int64_t N, int64_t K, int64_t ldw, const float* __restrict__ s,
                  int group, uint8_t* __restrict__ Wp, uint16_t* __restrict__ scale, uint8_t* __restrict__ zero) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t Nt = (N + 15) / 16, Kb = (K + 127) / 128;
  const int64_t kb = blockIdx.x;
  const int span = group / 32;  // 32-column blocks of a group
  float sv[4][8];
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int64_t k = kb * 128 + a * 32 + t * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) sv[a][i] = 1.0f;
    if (s != nullptr && k < K) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(s + k)), y = __ldg(reinterpret_cast<const float4*>(s + k + 4));
      sv[a][0] = x.x; sv[a][1] = x.y; sv[a][2] = x.z; sv[a][3] = x.w;
      sv[a][4] = y.x; sv[a][5] = y.y; sv[a][6] = y.z; sv[a][7] = y.w;
    }
  }
  const int64_t rt0 = static_cast<int64_t>(blockIdx.y) * (kInt4Threads / 32) + (threadIdx.x >> 5);
  for (int64_t rt = rt0; rt < Nt; rt += static_cast<int64_t>(gridDim.y) * (kInt4Threads / 32)) {
    uint4 raw[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const int64_t n = rt * 16 + h * 8 + g, k = kb * 128 + a * 32 + t * 8;
        raw[h][a] = (n < N && k < K) ? __ldcs(reinterpret_cast<const uint4*>(W + n * ldw + k)) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t n = rt * 16 + h * 8 + g;
      float hi[4], lo[4];  // per 32-column block: max |w'| (symmetric), or max and min with 0
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const uint32_t w[4] = {raw[h][a].x, raw[h][a].y, raw[h][a].z, raw[h][a].w};
        hi[a] = lo[a] = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float v = __fmul_rn(i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]), sv[a][i]);
          hi[a] = fmaxf(hi[a], ASYM ? v : fabsf(v));
          if (ASYM) lo[a] = fminf(lo[a], v);
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          hi[a] = fmaxf(hi[a], __shfl_xor_sync(0xffffffffu, hi[a], o));
          if (ASYM) lo[a] = fminf(lo[a], __shfl_xor_sync(0xffffffffu, lo[a], o));
        }
      }
      if (span >= 2) {
        hi[0] = hi[1] = fmaxf(hi[0], hi[1]);
        hi[2] = hi[3] = fmaxf(hi[2], hi[3]);
        lo[0] = lo[1] = fminf(lo[0], lo[1]);
        lo[2] = lo[3] = fminf(lo[2], lo[3]);
      }
      if (span == 4) {
        hi[0] = hi[1] = hi[2] = hi[3] = fmaxf(hi[0], hi[2]);
        lo[0] = lo[1] = lo[2] = lo[3] = fminf(lo[0], lo[2]);
      }
      uint32_t word[4];
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const __nv_bfloat16 e = __float2bfloat16_rn(ASYM ? __fdiv_rn(__fsub_rn(hi[a], lo[a]), 15.0f)
                                                         : __fdiv_rn(hi[a], 7.0f));
        const float ef = __bfloat162float(e);
        const float r = ef > 0.0f ? fminf(__fdiv_rn(1.0f, ef), FLT_MAX) : 0.0f;
        int z = 8;
        if (ASYM) z = static_cast<int>(fminf(fmaxf(rintf(__fmul_rn(-lo[a], r)), 0.0f), 15.0f));
        const int64_t k0 = kb * 128 + a * 32;
        if (t == 0 && (a & (span - 1)) == 0 && k0 < K && n < N && SQ_GUARD(k0 / group < (K + group - 1) / group)) {
          scale[k0 / group * N + n] = __bfloat16_as_ushort(e);
          if (ASYM) zero[k0 / group * N + n] = static_cast<uint8_t>(z);
        }
        // codes of this lane's 8 columns: clamping w' r to [-z, 15 - z] before the rounding is
        // the same as clamping the code after it
        const float down = static_cast<float>(-z), up = static_cast<float>(15 - z);
        const uint32_t w[4] = {raw[h][a].x, raw[h][a].y, raw[h][a].z, raw[h][a].w};
        const bool in = n < N && k0 + t * 8 < K;
        uint32_t pair[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float v0 = __fmul_rn(__fmul_rn(bf16_lo(w[u]), sv[a][2 * u]), r);
          const float v1 = __fmul_rn(__fmul_rn(bf16_hi(w[u]), sv[a][2 * u + 1]), r);
          const int q0 = __float2int_rn(fminf(fmaxf(v0, down), up)) + z;
          const int q1 = __float2int_rn(fminf(fmaxf(v1, down), up)) + z;
          pair[u] = in ? static_cast<uint32_t>(q0 | (q1 << 16)) << (4 * t) : 0x00080008u << (4 * t);
        }
        // lane t keeps pair t of all four lanes
        const bool b1 = t & 2, b0 = t & 1;
        uint32_t p0 = b1 ? pair[2] : pair[0], p1 = b1 ? pair[3] : pair[1];
        p0 |= __shfl_xor_sync(0xffffffffu, b1 ? pair[0] : pair[2], 2);
        p1 |= __shfl_xor_sync(0xffffffffu, b1 ? pair[1] : pair[3], 2);
        word[a] = (b0 ? p1 : p0) | __shfl_xor_sync(0xffffffffu, b0 ? p0 : p1, 1);
      }
      *reinterpret_cast<uint4*>(Wp + (rt * Kb + kb) * kTileBytes + (h * 32 + lane) * 16) =
          make_uint4(word[0], word[1], word[2], word[3]);
    }
  }
}

// ---------------------------------------------------------------- values
// The reverse: each lane collects its 8 columns' nibbles from its quad and writes 16 bytes.
// code - zero is exact in bf16 (128 + code minus 128 + zero), so the product with the scale
// is rounded once.
__global__ void __launch_bounds__(kInt4Threads)
int4_dequant_kernel(const uint8_t* __restrict__ Wp, const uint16_t* __restrict__ scale,
                    const uint8_t* __restrict__ zero, int group, int64_t N, int64_t K, uint16_t* __restrict__ out) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t Nt = (N + 15) / 16, Kb = (K + 127) / 128;
  const int64_t kb = blockIdx.x;
  const int64_t rt0 = static_cast<int64_t>(blockIdx.y) * (kInt4Threads / 32) + (threadIdx.x >> 5);
  for (int64_t rt = rt0; rt < Nt; rt += static_cast<int64_t>(gridDim.y) * (kInt4Threads / 32)) {
    uint4 unit[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      unit[h] = __ldcs(reinterpret_cast<const uint4*>(Wp + (rt * Kb + kb) * kTileBytes + (h * 32 + lane) * 16));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t n = rt * 16 + h * 8 + g;
      const uint32_t word[4] = {unit[h].x, unit[h].y, unit[h].z, unit[h].w};
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const int64_t k0 = kb * 128 + a * 32, k = k0 + t * 8;
        uint32_t w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) w[u] = __shfl_sync(0xffffffffu, word[a], (lane & ~3) | u) >> (4 * t);
        if (n < N && k < K) {
          const int64_t at = k0 / group * N + n;
          const uint32_t e = __ldg(scale + at), zp = zero_pair(zero != nullptr ? __ldg(zero + at) : 8u);
#pragma unroll
          for (int u = 0; u < 4; ++u)
            w[u] = mul_bf16x2(sub_bf16x2((w[u] & 0x000F000Fu) | 0x43004300u, zp), e | (e << 16));
          *reinterpret_cast<uint4*>(out + n * K + k) = make_uint4(w[0], w[1], w[2], w[3]);
        }
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
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(valid ? BYTES : 0)
                 : "memory");
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
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
  int split;   // CTAs of a cluster, which share a row block's columns
  int stages;  // 1 when a CTA's columns are one chunk
};

// The tokens' product with the weight streams the codes once: 16x8x16 matrix instructions with
// the weight rows as the 16 rows and up to 8 NT tokens as columns. A CTA takes RW row tiles, its
// 8 / RW warps of a tile take the 128-column blocks in turn; each lane's fragments of a block
// are two 16-byte loads, PF blocks ahead in registers. Activations, scales and zero points of a
// chunk of columns are staged in shared memory by asynchronous copies, one chunk ahead. Codes
// become bf16 exactly (128 + code, minus 128 + zero); a group's fp32 sum is scaled and added to
// the total. Warps of a tile, and the CTAs of a cluster along K, are joined in a fixed order
// through (distributed) shared memory.
template <int NT, int G, bool ASYM, int RW, int PF>
__global__ void __launch_bounds__(kInt4Threads) int4_linear_kernel(const LinearParams p) {
  constexpr int W = kInt4Threads / 32, KW = W / RW, kBlocks = KW * PF, kCols = kBlocks * 128, kRows = RW * 16;
  constexpr int kStride = (kCols + 8) * 2, kGroups = kCols / G;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rw = warp % RW, kw = warp / RW;
  const int rank = blockIdx.x % p.split;
  const int64_t row_block = blockIdx.x / p.split, rt = row_block * RW + rw, n0 = row_block * kRows;
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.Kb) * rank / p.split);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.Kb) * (rank + 1) / p.split);
  const bool rows_in = rt * 16 < p.N;
  const uint8_t* tiles = p.Wp + rt * p.Kb * kTileBytes;
  // the weight does not depend on the kernel before in a decode step: its way into L2 starts
  // before waiting for that kernel (a hint, safe even if that kernel wrote the weight)
  if (rows_in && kw == 0 && lane == 0)
    bulk_prefetch_l2(tiles + static_cast<int64_t>(kb0) * kTileBytes,
                     static_cast<uint32_t>(min(kb1 - kb0, kBlocks)) * kTileBytes);
  griddep_wait();
  griddep_launch_dependents();

  const int x_bytes = (p.M + 1) * kStride, stage_bytes = x_bytes + kGroups * kRows * (ASYM ? 3 : 2);
  const uint32_t smem32 = smem_u32(smem);
  auto stage_in = [&](int kb, int stage) {  // the chunk of columns from block kb on
    const uint32_t dst = smem32 + stage * stage_bytes;
    const int k0 = kb * 128, k1 = min(p.K, kb1 * 128);
    for (int i = threadIdx.x; i < p.M * (kCols / 8); i += kInt4Threads) {
      const int m = i / (kCols / 8), k = i % (kCols / 8) * 8;
      const bool in = k0 + k < k1;
      cp_async<16>(dst + m * kStride + k * 2, p.X + (in ? m * p.ldx + k0 + k : 0), in);
    }
    for (int i = threadIdx.x; i < kGroups * (kRows / 8); i += kInt4Threads) {
      const int gr = k0 / G + i / (kRows / 8), r = i % (kRows / 8) * 8;
      const bool in = gr < p.groups && n0 + r < p.N;
      const int64_t at = in ? gr * p.N + n0 + r : 0;
      cp_async<16>(dst + x_bytes + i * 16, p.scale + at, in);
      if (ASYM) cp_async<8>(dst + x_bytes + kGroups * kRows * 2 + i * 8, p.zero + at, in);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  uint4 w[PF][2];
  auto fetch = [&](int i, int kb) {
    if (rows_in && kb < kb1) {
      const uint4* src = reinterpret_cast<const uint4*>(tiles + static_cast<int64_t>(kb) * kTileBytes) + lane;
      w[i][0] = __ldcs(src);
      w[i][1] = __ldcs(src + 32);
    }
  };
#pragma unroll
  for (int i = 0; i < PF; ++i) {
    w[i][0] = w[i][1] = make_uint4(0, 0, 0, 0);
    fetch(i, kb0 + i * KW + kw);
  }
  stage_in(kb0, 0);
  // row M of each stage: zeros, for the tokens that fill up the last 8
  for (int i = threadIdx.x; i < kStride / 16 * p.stages; i += kInt4Threads)
    *reinterpret_cast<uint4*>(smem + (i / (kStride / 16)) * stage_bytes + p.M * kStride + i % (kStride / 16) * 16) =
        make_uint4(0, 0, 0, 0);

  float acc[NT][4];
  uint32_t x_row[NT];  // this lane's row address for loading the activations' fragments
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[nt][e] = 0.0f;
    x_row[nt] = smem32 + min(nt * 8 + (lane & 7), p.M) * kStride + (lane >> 3) * 16;
  }
  int stage = 0;
  for (int kb = kb0; kb < kb1; kb += kBlocks) {
    if (kb + kBlocks < kb1) {
      stage_in(kb + kBlocks, stage ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncthreads();
    const uint32_t base = stage * stage_bytes;
    const uint16_t* es = reinterpret_cast<const uint16_t*>(smem + base + x_bytes) + rw * 16 + g;
    const uint8_t* zs = smem + base + x_bytes + kGroups * kRows * 2 + rw * 16 + g;
#pragma unroll
    for (int i = 0; i < PF; ++i) {
      const int block = i * KW + kw;  // of the chunk
      if (kb + block < kb1) {
        const uint32_t lo[4] = {w[i][0].x, w[i][0].y, w[i][0].z, w[i][0].w};
        const uint32_t hi[4] = {w[i][1].x, w[i][1].y, w[i][1].z, w[i][1].w};
        float d[NT][4];
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const int gr = (block * 128 + a * 32) / G * kRows;
          const uint32_t z0 = ASYM ? zero_pair(zs[gr]) : 0x43084308u, z1 = ASYM ? zero_pair(zs[gr + 8]) : 0x43084308u;
          if (a * 32 % G == 0) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) d[nt][e] = 0.0f;
          }
          uint32_t f[2][4];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            f[j][0] = sub_bf16x2(((lo[a] >> (8 * j)) & 0x000F000Fu) | 0x43004300u, z0);
            f[j][1] = sub_bf16x2(((hi[a] >> (8 * j)) & 0x000F000Fu) | 0x43004300u, z1);
            f[j][2] = sub_bf16x2(((lo[a] >> (8 * j + 4)) & 0x000F000Fu) | 0x43004300u, z0);
            f[j][3] = sub_bf16x2(((hi[a] >> (8 * j + 4)) & 0x000F000Fu) | 0x43004300u, z1);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            uint32_t x[4];
            ldmatrix(x, x_row[nt] + base + block * 256 + a * 64);
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
      fetch(i, kb + kBlocks + block);
    }
    __syncthreads();
    stage ^= 1;
  }

  // [KW][M][kRows] partial sums in the staging area
  float* part = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int m = nt * 8 + 2 * t + (e & 1);
      if (m < p.M) part[(kw * p.M + m) * kRows + rw * 16 + g + (e & 2) * 4] = acc[nt][e];
    }
  if (p.split > 1)
    cluster_sync();
  else
    __syncthreads();
  const int share = kRows / 2 / p.split;  // row pairs that this CTA of the cluster finishes
  for (int i = threadIdx.x; i < p.M * share; i += kInt4Threads) {
    const int m = i / share, r = (rank * share + i % share) * 2;
    const int64_t n = n0 + r;
    if (n >= p.N) continue;
    float y0 = 0.0f, y1 = 0.0f;
    for (int c = 0; c < p.split; ++c) {
#pragma unroll
      for (int k = 0; k < KW; ++k) {
        const float* at = part + (k * p.M + m) * kRows + r;
        if (p.split > 1) {
          const uint32_t a = mapa_shared(at, c);
          y0 += ld_cluster_f32(a);
          y1 += ld_cluster_f32(a + 4);
        } else {
          y0 += at[0];
          y1 += at[1];
        }
      }
    }
    if (p.bias != nullptr) {
      const uint32_t b = __ldg(reinterpret_cast<const uint32_t*>(p.bias + n));
      y0 += bf16_lo(b);
      y1 += bf16_hi(b);
    }
    const __nv_bfloat162 y = __floats2bfloat162_rn(y0, y1);
    *reinterpret_cast<__nv_bfloat162*>(p.Y + m * p.N + n) = y;
  }
  if (p.split > 1) cluster_sync();  // no CTA leaves while its sums are being read
}

template <int NT, int G, bool ASYM, int RW, int PF>
cudaError_t launch_linear(LinearParams p, cudaStream_t stream) {
  constexpr int kBlocks = kInt4Threads / 32 / RW * PF, kCols = kBlocks * 128, kRows = RW * 16;
  const int64_t blocks = (p.N + kRows - 1) / kRows;
  // split along K until two CTAs per SM exist, as long as every CTA keeps a chunk of columns
  p.split = 1;
  while (p.split < 8 && blocks * p.split < 2 * 148 && p.Kb >= 2 * p.split * kBlocks) p.split *= 2;
  const int most = (p.Kb + p.split - 1) / p.split;
  p.stages = most > kBlocks ? 2 : 1;
  const size_t stage = (p.M + 1) * (kCols + 8) * 2 + kCols / G * kRows * (ASYM ? 3 : 2);
  const size_t smem = std::max(stage * p.stages, static_cast<size_t>(p.M) * kRows * (kInt4Threads / 32 / RW) * 4);
  auto kernel = int4_linear_kernel<NT, G, ASYM, RW, PF>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_kernel_clustered(kernel, dim3(static_cast<unsigned>(blocks * p.split)), dim3(kInt4Threads), smem, stream,
                                 true, static_cast<unsigned>(p.split), p);
}

template <int G, bool ASYM>
cudaError_t launch_linear_g(const LinearParams& p, cudaStream_t stream) {
  if (p.M <= 8) return launch_linear<1, G, ASYM, 1, 4>(p, stream);
  if (p.M <= 16) return launch_linear<2, G, ASYM, 8, 4>(p, stream);
  if (p.M <= 32) return launch_linear<4, G, ASYM, 8, 4>(p, stream);
  return launch_linear<8, G, ASYM, 8, 2>(p, stream);
}

// Grid of the two tile kernels: one column block per x, row tiles over y so that about eight
// CTAs per SM exist and each column block's factors are read by few of them.
dim3 tile_grid(int64_t N, int64_t K) {
  const int64_t Kb = (K + 127) / 128, rows = ((N + 15) / 16 + kInt4Threads / 32 - 1) / (kInt4Threads / 32);
  const int64_t y = std::max<int64_t>(1, std::min<int64_t>(rows, (148 * 8 + Kb - 1) / Kb));
  return dim3(static_cast<unsigned>(Kb), static_cast<unsigned>(y));
}

}  // namespace

size_t int4_weight_bytes(int64_t N, int64_t K) {
  return static_cast<size_t>((N + 15) / 16) * static_cast<size_t>((K + 127) / 128) * kTileBytes;
}

cudaError_t launch_int4_quant(const uint16_t* W, int64_t N, int64_t K, int64_t ldw, const float* s, int group,
                              uint8_t* Wp, uint16_t* scale, uint8_t* zero, cudaStream_t stream) {
  auto kernel = zero != nullptr ? int4_quant_kernel<true> : int4_quant_kernel<false>;
  return launch_kernel(kernel, tile_grid(N, K), dim3(kInt4Threads), 0, stream, false, W, N, K, ldw, s, group, Wp, scale,
                       zero);
}

cudaError_t launch_int4_dequant(const uint8_t* Wp, const uint16_t* scale, const uint8_t* zero, int group, int64_t N,
                                int64_t K, uint16_t* out, cudaStream_t stream) {
  return launch_kernel(int4_dequant_kernel, tile_grid(N, K), dim3(kInt4Threads), 0, stream, false, Wp, scale, zero,
                       group, N, K, out);
}

cudaError_t launch_int4_linear(const Int4LinearArgs& a, cudaStream_t stream) {
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
    if (a.group == 32) return launch_linear_g<32, true>(p, stream);
    return a.group == 64 ? launch_linear_g<64, true>(p, stream) : launch_linear_g<128, true>(p, stream);
  }
  if (a.group == 32) return launch_linear_g<32, false>(p, stream);
  return a.group == 64 ? launch_linear_g<64, false>(p, stream) : launch_linear_g<128, false>(p, stream);
}

}  // namespace sq
