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

// One CTA per row tile and 8 tokens, its warps over the column blocks in turn.
__global__ void __launch_bounds__(kInt4Threads)
int4_linear_kernel(const uint16_t* __restrict__ X, int M, int64_t K, int64_t ldx, const uint8_t* __restrict__ Wp,
                   const uint16_t* __restrict__ scale, const uint8_t* __restrict__ zero, int group,
                   const uint16_t* __restrict__ bias, uint16_t* __restrict__ Y, int64_t N) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float part[kInt4Threads / 32][8][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t Kb = (K + 127) / 128, rt = blockIdx.x;
  const int m = blockIdx.y * 8 + g;
  float acc[4] = {0, 0, 0, 0};
  for (int64_t kb = warp; kb < Kb; kb += kInt4Threads / 32) {
    const uint8_t* tile = Wp + (rt * Kb + kb) * kTileBytes;
    const uint4 u0 = __ldg(reinterpret_cast<const uint4*>(tile) + lane);
    const uint4 u1 = __ldg(reinterpret_cast<const uint4*>(tile) + 32 + lane);
    const uint32_t lo[4] = {u0.x, u0.y, u0.z, u0.w}, hi[4] = {u1.x, u1.y, u1.z, u1.w};
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int64_t k0 = kb * 128 + a * 32;
      if (k0 >= K) break;
      const int64_t n0 = rt * 16 + g, n1 = n0 + 8, row = k0 / group * N;
      const float e0 = n0 < N ? bf16_lo(__ldg(scale + row + n0)) : 0.0f, e1 = n1 < N ? bf16_lo(__ldg(scale + row + n1)) : 0.0f;
      const uint32_t z0 = zero_pair(zero != nullptr && n0 < N ? __ldg(zero + row + n0) : 8u);
      const uint32_t z1 = zero_pair(zero != nullptr && n1 < N ? __ldg(zero + row + n1) : 8u);
      float d[4] = {0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int64_t k = k0 + j * 16 + 2 * t;
        uint32_t af[4];
        af[0] = sub_bf16x2(((lo[a] >> (8 * j)) & 0x000F000Fu) | 0x43004300u, z0);
        af[1] = sub_bf16x2(((hi[a] >> (8 * j)) & 0x000F000Fu) | 0x43004300u, z1);
        af[2] = sub_bf16x2(((lo[a] >> (8 * j + 4)) & 0x000F000Fu) | 0x43004300u, z0);
        af[3] = sub_bf16x2(((hi[a] >> (8 * j + 4)) & 0x000F000Fu) | 0x43004300u, z1);
        const uint16_t* x = X + m * ldx + k;
        const uint32_t b0 = m < M && k < K ? __ldg(reinterpret_cast<const uint32_t*>(x)) : 0u;
        const uint32_t b1 = m < M && k + 8 < K ? __ldg(reinterpret_cast<const uint32_t*>(x + 8)) : 0u;
        mma_bf16(d, af, b0, b1);
      }
      acc[0] = fmaf(d[0], e0, acc[0]);
      acc[1] = fmaf(d[1], e0, acc[1]);
      acc[2] = fmaf(d[2], e1, acc[2]);
      acc[3] = fmaf(d[3], e1, acc[3]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) part[warp][2 * t + (i & 1)][g + (i & 2) * 4] = acc[i];
  __syncthreads();
  if (threadIdx.x < 128) {
    const int r = threadIdx.x & 15, tok = blockIdx.y * 8 + (threadIdx.x >> 4);
    const int64_t n = rt * 16 + r;
    float y = 0.0f;
#pragma unroll
    for (int w = 0; w < kInt4Threads / 32; ++w) y += part[w][threadIdx.x >> 4][r];
    if (tok < M && n < N) {
      if (bias != nullptr) y += bf16_lo(__ldg(bias + n));
      Y[tok * N + n] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
    }
  }
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
  const dim3 grid(static_cast<unsigned>((a.N + 15) / 16), static_cast<unsigned>((a.M + 7) / 8));
  return launch_kernel(int4_linear_kernel, grid, dim3(kInt4Threads), 0, stream, true, a.X, static_cast<int>(a.M), a.K,
                       a.ldx, a.Wp, a.scale, a.zero, a.group, a.bias, a.Y, a.N);
}

}  // namespace sq
