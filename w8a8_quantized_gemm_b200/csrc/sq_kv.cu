// Paged key-value cache: the append of new tokens, with the position rotation on the way.
// "SmoothQuant量化实战" §5.2 (KV-cache INT8 with per-token, per-head scales).
#include "sq_internal.h"
#include "sq_ptx.cuh"
#include "sq_rows.cuh"

#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>

namespace sq {
namespace {

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// The larger one, or NaN: a row with a NaN gets a scale that says so.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// ---------------------------------------------------------------- append
// 128 threads and at most 72 registers: seven CTAs an SM. Measured (us; 8192 tokens of 64 + 16 heads of
// 128, int8; 2047 tokens of 32 + 64 heads, bf16): 256 threads 88 / 25, 128 threads 69 / 21, held to 72
// registers 64 / 20.5 (5.1 and 4.9 TB/s), to 64 registers 62 / 21.5.
constexpr int kAppendThreads = 128;

// head_dim / 16 lanes own a head row (the group of `lanes`, a power of two, has idle ones for
// head_dim 96): each holds 16 elements, which are 8 pairs when its part of the row is rotated,
// whichever way pairs are formed, so the lane's 8 angles stay in registers while its group
// walks over the token's heads. A CTA takes one token, or several when a token has fewer rows
// than the CTA has groups.
template <bool INT8, bool PAIRS>
__global__ void __launch_bounds__(kAppendThreads, 7)
rope_kv_append_kernel(const uint16_t* q, int64_t ldq, const uint16_t* __restrict__ k, int64_t ldk,
                      const uint16_t* __restrict__ v, int64_t ldv, int64_t T, int H, const float* __restrict__ cos_t,
                      const float* __restrict__ sin_t, int64_t max_pos, int rot,
                      const int32_t* __restrict__ positions, const int32_t* __restrict__ slots, KvView c,
                      uint16_t* q_out, int lanes, int groups_per_token, unsigned int* status) {
  griddep_wait();
  griddep_launch_dependents();
  const int D = c.head_dim, groups = kAppendThreads / lanes;
  const int group = threadIdx.x / lanes, i = threadIdx.x % lanes;
  const int64_t tok = static_cast<int64_t>(blockIdx.x) * (groups / groups_per_token) + group / groups_per_token;
  if (tok >= T) return;
  const unsigned quad = lanes == 32 ? 0xffffffffu : ((1u << lanes) - 1u) << (threadIdx.x & 31 & ~(lanes - 1));
  const bool on = 16 * i < D, turn = 16 * i < rot;
  // places of the lane's two runs of 8 elements
  const int p0 = turn && !PAIRS ? 8 * i : 16 * i, p1 = turn && !PAIRS ? rot / 2 + 8 * i : 16 * i + 8;
  const int rows = H + 2 * c.heads;
  // a row's elements, loaded one row ahead; the first do not wait for the slot and the angles
  auto load = [&](int row, uint4 (&r)[2]) {
    r[0] = r[1] = make_uint4(0, 0, 0, 0);
    if (on && row < rows) {
      const uint16_t* src = row < H ? q + tok * ldq + static_cast<int64_t>(row) * D
                            : row < H + c.heads ? k + tok * ldk + static_cast<int64_t>(row - H) * D
                                                : v + tok * ldv + static_cast<int64_t>(row - H - c.heads) * D;
      r[0] = *reinterpret_cast<const uint4*>(src + p0);
      r[1] = *reinterpret_cast<const uint4*>(src + p1);
    }
  };
  int row = group % groups_per_token;
  uint4 ahead[2];
  load(row, ahead);
  const int slot = __ldg(slots + tok);
  if (slot < 0) return;
  const int64_t pos = rot > 0 ? __ldg(positions + tok) : 0;
  const int page = slot >> c.page_shift, off = slot & ((1 << c.page_shift) - 1);
  if (page >= c.num_pages || pos < 0 || (rot > 0 && pos >= max_pos)) {
    if (i == 0 && group % groups_per_token == 0) atomicOr(status, kErrIndex);
    return;
  }
  float cs[8], sn[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) cs[j] = 1.0f, sn[j] = 0.0f;
  if (turn && SQ_GUARD(within(cos_t + pos * (rot / 2) + 8 * i, 8, cos_t, max_pos * (rot / 2)))) {
    const float4* cp = reinterpret_cast<const float4*>(cos_t + pos * (rot / 2) + 8 * i);
    const float4* sp = reinterpret_cast<const float4*>(sin_t + pos * (rot / 2) + 8 * i);
    const float4 c0 = __ldg(cp), c1 = __ldg(cp + 1), s0 = __ldg(sp), s1 = __ldg(sp + 1);
    cs[0] = c0.x; cs[1] = c0.y; cs[2] = c0.z; cs[3] = c0.w; cs[4] = c1.x; cs[5] = c1.y; cs[6] = c1.z; cs[7] = c1.w;
    sn[0] = s0.x; sn[1] = s0.y; sn[2] = s0.z; sn[3] = s0.w; sn[4] = s1.x; sn[5] = s1.y; sn[6] = s1.z; sn[7] = s1.w;
  }
  for (; row < rows; row += groups_per_token) {
    const bool is_q = row < H, is_v = row >= H + c.heads;
    const int head = is_q ? row : is_v ? row - H - c.heads : row - H;
    float x[16];
    sq::rows::widen16(ahead, x);
    load(row + groups_per_token, ahead);
    if (turn && !is_v) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float& a = PAIRS ? x[2 * j] : x[j];
        float& b = PAIRS ? x[2 * j + 1] : x[8 + j];
        const float ya = __fsub_rn(__fmul_rn(a, cs[j]), __fmul_rn(b, sn[j]));
        const float yb = __fadd_rn(__fmul_rn(b, cs[j]), __fmul_rn(a, sn[j]));
        a = ya;
        b = yb;
      }
    }
    if (is_q || !INT8) {
      uint16_t* dst = is_q ? q_out + (tok * H + head) * D
                           : static_cast<uint16_t*>(is_v ? c.v : c.k) + page * c.page_stride +
                                 (static_cast<int64_t>(head) << c.page_shift) * D + static_cast<int64_t>(off) * D;
      if (on && SQ_GUARD(p1 + 8 <= D && within(dst, D, is_q ? q_out : is_v ? c.v : c.k, is_q ? T * H * D : c.elements()))) {
        *reinterpret_cast<uint4*>(dst + p0) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                                         pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
        *reinterpret_cast<uint4*>(dst + p1) = make_uint4(pack_bf16(x[8], x[9]), pack_bf16(x[10], x[11]),
                                                         pack_bf16(x[12], x[13]), pack_bf16(x[14], x[15]));
      }
    } else {
      float a = 0.0f;
#pragma unroll
      for (int j = 0; j < 16; ++j) a = max_nan(a, fabsf(x[j]));
      for (int o = lanes / 2; o > 0; o >>= 1) a = max_nan(a, __shfl_xor_sync(quad, a, o));
      const float r = a > 0.0f ? fminf(__fdiv_rn(127.0f, a), FLT_MAX) : 0.0f;
      const int64_t at = (static_cast<int64_t>(head) << c.page_shift) + off;
      int8_t* dst = static_cast<int8_t*>(is_v ? c.v : c.k) + page * c.page_stride + at * D;
      if (on && SQ_GUARD(p1 + 8 <= D && within(dst, D, is_v ? c.v : c.k, c.elements()))) {
        int e[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) e[j] = __float2int_rn(fminf(fmaxf(__fmul_rn(x[j], r), -128.0f), 127.0f));
        *reinterpret_cast<uint2*>(dst + p0) =
            make_uint2(sq::rows::pack4(e[0], e[1], e[2], e[3]), sq::rows::pack4(e[4], e[5], e[6], e[7]));
        *reinterpret_cast<uint2*>(dst + p1) =
            make_uint2(sq::rows::pack4(e[8], e[9], e[10], e[11]), sq::rows::pack4(e[12], e[13], e[14], e[15]));
      }
      float* to = (is_v ? c.v_scale : c.k_scale) + page * c.scale_page_stride + at;
      if (i == 0 && SQ_GUARD(within(to, 1, is_v ? c.v_scale : c.k_scale, c.scales()))) *to = __fdiv_rn(a, 127.0f);
    }
  }
}

}  // namespace

cudaError_t launch_rope_kv_append(const RopeAppendArgs& a, cudaStream_t stream) {
  int lanes = 4;
  while (lanes * 16 < a.cache.head_dim) lanes *= 2;
  const int groups = kAppendThreads / lanes, rows = a.H + 2 * a.cache.heads;
  int per = 1;
  while (per < rows && per < groups) per *= 2;
  const int64_t tokens = groups / per;
  auto kernel = rope_kv_append_kernel<false, false>;
  if (a.cache.int8)
    kernel = a.interleaved ? rope_kv_append_kernel<true, true> : rope_kv_append_kernel<true, false>;
  else if (a.interleaved)
    kernel = rope_kv_append_kernel<false, true>;
  const dim3 grid(static_cast<unsigned>((a.T + tokens - 1) / tokens));
  return launch_kernel(kernel, grid, dim3(kAppendThreads), 0, stream, true, a.q, a.ldq, a.k, a.ldk, a.v, a.ldv, a.T,
                       a.H, a.cos_t, a.sin_t, a.max_pos, a.rot, a.positions, a.slots, a.cache, a.q_out, lanes, per,
                       a.status);
}

}  // namespace sq
