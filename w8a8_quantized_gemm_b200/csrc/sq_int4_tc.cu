// The 4-bit linear layer for 17 to 64 tokens, on the tensor cores (tcgen05).
//   Y[m,n] = sum_k X[m,k] * (code[n,k] - zero[g,n]) * scale[g,n] + bias[n]
//
// The weight rows are the 128 rows of the instructions, the tokens (up to 64) their columns, so
// that every code is made a bf16 number once for all tokens. 64 x 28672 x 8192 69 us, 64 x 8192 x
// 8192 22.6, of which 4 are the row block's end (the bytes alone would take 20 and 6, the products
// 19 and 5): no unit is full (integer pipe 46%, tensor pipe 24%, half of the issue slots). Bound by
// latency: two warps a scheduler each convert, store, wait for the products, read back and add in
// turn, half of a block's time in the conversion. Warpgroups take the
// 128-column blocks of a row block in turn. A thread
// owns a weight row: its 64 bytes of codes (contiguous in the tiled layout) come by asynchronous
// copies several blocks ahead, become code - zero exactly (128 + code, minus 128 + zero) in the
// order of the columns, and go into tensor memory as operand A; the tokens are operand B, streamed
// by TMA. Products and a group's sums are fp32 in tensor memory, one accumulator per group; the
// warpgroup reads it back, scales it and adds it to its fp32 totals in registers while the
// others' blocks are converted and multiplied. At a row block's end they add up, in order, and so
// do, through distributed shared memory, the CTAs of a cluster that share the columns where there
// are too few row blocks to go round.
#include "sq_internal.h"
#include "sq_ptx.cuh"

#include <cuda_bf16.h>

#include <algorithm>

namespace sq {
namespace {

constexpr int kTileBytes = 1024;
constexpr int kCodeRow = 80;                  // 64 bytes of codes: an odd number of 16-byte units
constexpr int kCodeBytes = 32 * kCodeRow;     // of a warp's rows in a block
constexpr int64_t kSmemMax = 232448;
constexpr uint64_t kAbortWaitNs = 10000000;  // 10 ms: far more than a copy takes

struct TcParams {
  int64_t N;
  const uint8_t* Wp;
  const uint16_t* scale;
  const uint8_t* zero;
  const uint16_t* bias;
  uint16_t* Y;
  int M, K, Kb, groups;
  int split;  // CTAs of a cluster
  int row_blocks;
  unsigned int* status;
};

template <int TOKENS_, int G_>
struct Cfg {
  static constexpr int kTokens = TOKENS_, G = G_;
  // Two warpgroups, a warp for TMA and one per warpgroup for the matrix instructions. (Three of them,
  // with registers handed over by the other warps, were measured no faster: 55 against 58 us at
  // 16 x 28672 x 8192, 28 against 25 us at 64 x 8192 x 8192.)
  static constexpr int kWg = 2, kWorkers = kWg * 128, kThreads = kWorkers + 32 + 32 * kWg;
  // columns of a unit of work: a block, or half of one where its groups' accumulators need the room
  static constexpr int kUnit = 128 + (128 / G) * kTokens <= 256 ? 128 : 64;
  static constexpr int kHalves = 128 / kUnit, kGroups = kUnit / G;
  static constexpr int kAtom = kTokens * 128;  // 64 columns of the tokens, 128-byte swizzle
  static constexpr int kXSlot = kAtom * (kUnit / 64), kXStages = kTokens == 64 ? 4 : 8;
  // a warp's slot: codes, then the rows' scales and zero points per group
  static constexpr int kPer = 128 / G, kScales = kCodeBytes, kZeros = kScales + kPer * 64;
  static constexpr int kCodeSlot = kZeros + kPer * 32, kCodeStages = 5;
  static_assert((kXStages & (kXStages - 1)) == 0, "stages are counted with shifts");
  static constexpr int kPart = kTokens * 128 * 4;
  static constexpr int kX = 0, kCodes = kXStages * kXSlot, kSums = kCodes + 4 * kWg * kCodeStages * kCodeSlot;
  static constexpr int kSmem = kSums + kPart + 1024;  // and the alignment
  static_assert(kSmem <= kSmemMax - 1024, "shared memory of an SM");
  // tensor memory of a warpgroup: accumulators, then two operands
  static constexpr int kA = kGroups * kTokens, kStride = 256;
  static_assert(kA + kUnit <= kStride && kWg * kStride <= 512, "tensor memory");
};

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool valid = true) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES),
                 "r"(valid ? BYTES : 0)
                 : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r =
      __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
template <int THREADS>
__device__ __forceinline__ void workers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

// Cluster-scope arrival on, and wait for, an mbarrier that orders reads of distributed shared memory.
__device__ __forceinline__ void arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ bool wait_cluster_bounded(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  const uint64_t t0 = global_timer_ns();
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred P;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 P, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, P;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if (global_timer_ns() - t0 > limit_ns) return false;
  }
}
__device__ __forceinline__ float2 ld_cluster_f32x2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

struct Shared {
  uint64_t x_full[8], x_empty[8], a_full[2][2], d_full[2], d_free[2], done[2], part_ready, part_free;
  uint32_t tmem;
  volatile uint32_t abort;
};

template <int TOKENS, int G, bool ASYM>
__global__ void __launch_bounds__(Cfg<TOKENS, G>::kThreads, 1)
int4_tc_kernel(const __grid_constant__ CUtensorMap x_map, const TcParams p) {
  using C = Cfg<TOKENS, G>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int kTmaWarp = 4 * C::kWg;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % p.split, cluster = blockIdx.x / p.split, clusters = gridDim.x / p.split;
  const int b0 = static_cast<int>(static_cast<int64_t>(p.Kb) * rank / p.split);
  const int nb = static_cast<int>(static_cast<int64_t>(p.Kb) * (rank + 1) / p.split) - b0;  // blocks of this CTA
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kXStages; ++i) {
      mbar_init(&sh.x_full[i], 1);
      mbar_init(&sh.x_empty[i], 1);
    }
    for (int i = 0; i < C::kWg; ++i) {
      mbar_init(&sh.a_full[i][0], 128);
      mbar_init(&sh.a_full[i][1], 128);
      mbar_init(&sh.d_full[i], 1);
      mbar_init(&sh.d_free[i], 128);
      mbar_init(&sh.done[i], 1);
    }
    mbar_init(&sh.part_ready, p.split);
    mbar_init(&sh.part_free, p.split);
    sh.abort = 0;
    fence_mbar_init();
  }
  if (warp == kTmaWarp) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  if (p.split > 1)
    cluster_sync();  // the peers' barriers are ready
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  griddep_wait();
  griddep_launch_dependents();

  // A wait that gives up is recorded and makes every later one return at once, so that each role
  // runs through its loops without waiting.
  auto wait = [&](uint64_t* bar, uint32_t parity, unsigned code) -> bool {
    if (mbar_try_wait(bar, parity)) return true;
    if (sh.abort) return false;
    if (mbar_wait_bounded(bar, parity, kDefaultWaitLimitNs)) return true;
    sh.abort = 1;
    atomicOr(p.status, code);
    return false;
  };
  // Units of a row block in order: kWg blocks at a time, one per warpgroup; their halves; the warpgroups.
  if (warp >= kTmaWarp) {
    // A whole warp runs each of these loops, so that addresses and descriptors live in uniform
    // registers as the instructions want them (one lane alone took 90 cycles an instruction), and one
    // lane issues.
    const bool one = elect_one();
    if (warp == kTmaWarp) {
      if (one) tma_prefetch_desc(&x_map);
      unsigned n = 0;
      for (int rb = cluster; rb < p.row_blocks; rb += clusters)
        for (int base = 0; base < nb; base += C::kWg)
          for (int h = 0; h < C::kHalves; ++h)
            for (int wg = 0; wg < C::kWg && base + wg < nb; ++wg, ++n) {
              const unsigned s = n % C::kXStages;
              // slot s has been read; where that gives up, nothing more is brought
              if (n >= C::kXStages && !wait(&sh.x_empty[s], (n / C::kXStages - 1) & 1, kErrProducerWait)) continue;
              if (one) {
                const int k0 = (b0 + base + wg) * 128 + h * C::kUnit;
                mbar_arrive_expect_tx(&sh.x_full[s], C::kXSlot);
#pragma unroll
                for (int a = 0; a < C::kUnit / 64; ++a)
                  tma_load_2d(smem + C::kX + s * C::kXSlot + a * C::kAtom, &x_map, &sh.x_full[s], k0 + a * 64, 0,
                              kEvictLast);
              }
              __syncwarp();
            }
      // copies still in flight after a wait gave up end before the CTA does
      if (sh.abort)
        for (int i = 0; i < C::kXStages; ++i) {
          mbar_wait_bounded(&sh.x_full[i], 0, kAbortWaitNs);
          mbar_wait_bounded(&sh.x_full[i], 1, kAbortWaitNs);
        }
    } else {
      // One issuing warp per warpgroup: a unit costs some hundred cycles here, which one warp for all
      // could not keep up with.
      const int wg = warp - kTmaWarp - 1;
      constexpr uint32_t kIdesc = idesc_bf16_f32(128, C::kTokens);
      const uint64_t x_desc = smem_desc_k128(smem_u32(smem + C::kX));
      const uint32_t d0 = tmem + wg * C::kStride;
      unsigned n = 0, u = 0;
      for (int rb = cluster; rb < p.row_blocks; rb += clusters)
        for (int base = 0; base < nb; base += C::kWg) {
          const int all = min(C::kWg, nb - base);
          for (int h = 0; h < C::kHalves; ++h, n += all) {
            if (wg >= all) continue;
            const unsigned s = (n + wg) % C::kXStages;
            wait(&sh.x_full[s], ((n + wg) / C::kXStages) & 1, kErrMmaWait);
            wait(&sh.a_full[wg][u & 1], (u >> 1) & 1, kErrMmaWait);
            if (u > 0) wait(&sh.d_free[wg], (u - 1) & 1, kErrMmaWait);
            tc_fence_after();
            const uint32_t a0 = d0 + C::kA + (u & 1) * (C::kUnit / 2);
            const uint64_t b0 = x_desc + ((s * C::kXSlot) >> 4);  // addresses count in 16 bytes
            if (one && !sh.abort) {
#pragma unroll
              for (int j = 0; j < C::kUnit / 16; ++j)
                mma_ts(d0 + j / (G / 16) * C::kTokens, a0 + j * 8, b0 + (((j / 4) * C::kAtom + (j % 4) * 32) >> 4),
                       kIdesc, j % (G / 16) != 0);
              mma_commit(&sh.d_full[wg]);
              mma_commit(&sh.x_empty[s]);
            }
            __syncwarp();
            ++u;
          }
        }
      if (one) {
        mma_commit(&sh.done[wg]);
        if (!mbar_wait_bounded(&sh.done[wg], 0, kDefaultWaitLimitNs)) atomicOr(p.status, kErrTeardownWait);
      }
    }
  } else {
    const int wg = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t tmem_lane = tmem + wg * C::kStride + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t ring = smem_u32(smem + C::kCodes) + warp * C::kCodeStages * C::kCodeSlot;
    const uint8_t* ring_p = smem + C::kCodes + warp * C::kCodeStages * C::kCodeSlot;
    const int64_t Nt = (p.N + 15) / 16;
    constexpr int kPer = C::kPer;  // groups of a block
    // ---- this warp's blocks: wg, wg + kWg, ... of each row block, codes and factors several ahead.
    // Rows past N take a valid row's bytes and groups past K the last group's zero points: neither is
    // ever used (the tokens are zero there). Scales past K are zero, whatever the last group's is.
    int load_rb = wg < nb ? cluster : p.row_blocks, load_b = wg;
    const int64_t tile_bytes = static_cast<int64_t>(p.Kb) * kTileBytes;
    const uint8_t *src = nullptr, *z_src = nullptr;  // 16 bytes `lane` of this warp's first tile in the next block
    const uint16_t* e_src = nullptr;
    int64_t second = 0;  // from the first tile to the second
    // lane's part of a block's scales: 32 rows per group, kE bytes a lane; and of its zero points, 4 bytes
    constexpr int kE = G == 32 ? 8 : 4, kELanes = 64 / kE;
    const int e_group = lane / kELanes % kPer, z_group = lane / 8 % kPer;
    auto locate = [&]() {  // the next row block
      const int64_t rt = static_cast<int64_t>(load_rb) * 8 + quarter * 2, last = Nt - 1;
      src = p.Wp + (rt < last ? rt : last) * tile_bytes + static_cast<int64_t>(b0 + wg) * kTileBytes + lane * 16;
      second = rt + 1 < Nt ? tile_bytes : 0;
      const int64_t n = static_cast<int64_t>(load_rb) * 128 + quarter * 32, e_row = n + lane % kELanes * (kE / 2),
                    z_row = n + lane % 8 * 4;
      e_src = p.scale + (e_row < p.N ? e_row : 0);
      if (ASYM) z_src = p.zero + (z_row < p.N ? z_row : 0);
    };
    if (load_rb < p.row_blocks) locate();
    auto fetch = [&](int slot) {
      if (load_rb < p.row_blocks) {
        const uint32_t at = ring + slot * C::kCodeSlot;
        const uint32_t dst = at + lane / 4 * kCodeRow + lane % 4 * 16;  // row lane / 4, then 8 on
        if (SQ_GUARD(within(src, second + 528, p.Wp, Nt * tile_bytes))) {
          cp_async<16>(dst, src);
          cp_async<16>(dst + 8 * kCodeRow, src + 512);
          cp_async<16>(dst + 16 * kCodeRow, src + second);
          cp_async<16>(dst + 24 * kCodeRow, src + second + 512);
        }
        const int gr = (b0 + load_b) * kPer;
        if (lane < kPer * kELanes &&
            SQ_GUARD(within(e_src + min(gr + e_group, p.groups - 1) * p.N, kE / 2, p.scale, p.groups * p.N)))
          cp_async<kE>(at + C::kScales + lane * kE, e_src + min(gr + e_group, p.groups - 1) * p.N,
                       gr + e_group < p.groups);
        if (ASYM && lane < kPer * 8 &&
            SQ_GUARD(within(z_src + min(gr + z_group, p.groups - 1) * p.N, 4, p.zero, p.groups * p.N)))
          cp_async<4>(at + C::kZeros + lane * 4, z_src + min(gr + z_group, p.groups - 1) * p.N);
        src += C::kWg * kTileBytes;
        load_b += C::kWg;
        if (load_b >= nb) {
          load_b = wg;
          load_rb += clusters;
          if (load_rb < p.row_blocks) locate();
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int i = 0; i < C::kCodeStages - 1; ++i) fetch(i);

    int slot = 0, free_slot = C::kCodeStages - 1, u = 0;
    uint4 code[4];
    float e[kPer];
    uint32_t z[kPer];
    // the next block's codes and this row's factors into registers
    auto take = [&]() {
      asm volatile("cp.async.wait_group %0;" ::"n"(C::kCodeStages - 2) : "memory");
      __syncwarp();
      fetch(free_slot);
      const uint8_t* at = ring_p + slot * C::kCodeSlot;
#pragma unroll
      for (int c = 0; c < 4; ++c) code[c] = *reinterpret_cast<const uint4*>(at + lane * kCodeRow + c * 16);
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        e[j] = bf16_lo(*reinterpret_cast<const uint16_t*>(at + C::kScales + j * 64 + lane * 2));
        const uint32_t zero = ASYM ? at[C::kZeros + j * 32 + lane] : 8u;
        z[j] = 0x43004300u | zero | (zero << 16);
      }
      free_slot = slot;
      slot = slot + 1 == C::kCodeStages ? 0 : slot + 1;
    };
    // half h of the block as operand A of unit `at`
    auto convert = [&](int h, int at) {
      const uint32_t dst = tmem_lane + C::kA + (at & 1) * (C::kUnit / 2);
#pragma unroll
      for (int q = 0; q < C::kUnit / 64; ++q) {
        uint32_t r[32];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const int a = 2 * q + w;  // of the unit: the block's word a + 2 h
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t lo = a == 0 ? code[c].x : a == 1 ? code[c].y : a == 2 ? code[c].z : code[c].w;
            const uint32_t hi = a == 0 ? code[c].z : code[c].w;
            const uint32_t v = C::kHalves == 2 && h == 1 ? hi : lo;
            const uint32_t zz = C::kHalves == 2 && h == 1 ? z[(a + 2) * 32 / G % kPer] : z[a * 32 / G];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              r[16 * w + 4 * i + c] = sub_bf16x2(((v >> (4 * i)) & 0x000F000Fu) | 0x43004300u, zz);
          }
        }
        tmem_st_32x32b_x32(dst + q * 32, r);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&sh.a_full[wg][at & 1]);  // (one barrier per operand: a thread may be a unit ahead of another)
    };

    float acc[C::kTokens];
#pragma unroll
    for (int m = 0; m < C::kTokens; ++m) acc[m] = 0.0f;
    float* part = reinterpret_cast<float*>(smem + C::kSums);  // [tokens][128 rows]
    int item = 0;
    // The conversion runs one unit ahead of the accumulation: unit u is multiplied meanwhile.
    int left = 0;  // units not converted yet
    for (int rb = cluster; rb < p.row_blocks; rb += clusters) left += (nb - wg + C::kWg - 1) / C::kWg * C::kHalves;
    int next_h = 0, ahead = 0;
    float f[kPer];  // the factors of the block being accumulated
    auto step_ahead = [&]() {
      if (ahead == left) return;
      if (next_h == 0) take();
      if (C::kHalves == 1 || next_h == 0)
        convert(0, ahead);
      else
        convert(1, ahead);
      ++ahead;
      next_h = next_h + 1 == C::kHalves ? 0 : next_h + 1;
    };
    step_ahead();
    for (int rb = cluster; rb < p.row_blocks; rb += clusters, ++item) {
      for (int b = wg; b < nb; b += C::kWg)
#pragma unroll
        for (int h = 0; h < C::kHalves; ++h, ++u) {
          if (h == 0) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) f[j] = e[j];
          }
          step_ahead();
          const bool ok = wait(&sh.d_full[wg], u & 1, kErrEpilogueWait);
          if (!__all_sync(0xffffffffu, ok)) continue;
          tc_fence_after();
#pragma unroll
          for (int j = 0; j < C::kGroups; ++j) {
#pragma unroll
            for (int m = 0; m < C::kTokens; m += 16) {
              uint32_t d[16];
              tmem_ld_32x32b_x16(tmem_lane + j * C::kTokens + m, d);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) acc[m + i] = fmaf(__uint_as_float(d[i]), f[h * C::kGroups + j], acc[m + i]);
            }
          }
          tc_fence_before();
          mbar_arrive(&sh.d_free[wg]);
        }
      // ---- the row block's sums: the warpgroups' in order, then the other CTAs'
      if (p.split > 1 && item > 0 && !sh.abort &&
          !wait_cluster_bounded(&sh.part_free, (item - 1) & 1, kDefaultWaitLimitNs)) {
        sh.abort = 1;
        atomicOr(p.status, kErrEpilogueWait);
      }
      workers_sync<C::kWorkers>();
      // each warpgroup leaves half of its tokens' sums to the other and takes the other's half of its own
      constexpr int kHalf = C::kTokens / 2;
      const bool second = wg == 1;
#pragma unroll
      for (int m = 0; m < kHalf; ++m) part[((second ? 0 : kHalf) + m) * 128 + row] = second ? acc[m] : acc[kHalf + m];
      workers_sync<C::kWorkers>();
#pragma unroll
      for (int m = 0; m < kHalf; ++m) part[((second ? kHalf : 0) + m) * 128 + row] += second ? acc[kHalf + m] : acc[m];
      workers_sync<C::kWorkers>();
#pragma unroll
      for (int m = 0; m < C::kTokens; ++m) acc[m] = 0.0f;
      if (p.split > 1) {
        if (threadIdx.x < p.split) arrive_cluster(mapa_shared(&sh.part_ready, threadIdx.x));
        if (!sh.abort && !wait_cluster_bounded(&sh.part_ready, item & 1, kDefaultWaitLimitNs)) {
          sh.abort = 1;
          atomicOr(p.status, kErrEpilogueWait);
        }
      }
      // this CTA's share of the 64 row pairs, a pair per lane and the tokens over the warps; the loads
      // of a warp's tokens from the other CTAs are under way together
      constexpr int kWarps = C::kWorkers / 32, kPerWarp = C::kTokens / kWarps;
      for (int r = 64 * rank / p.split + lane; r < 64 * (rank + 1) / p.split; r += 32) {
        float2 y[kPerWarp];
#pragma unroll
        for (int j = 0; j < kPerWarp; ++j) y[j] = make_float2(0.0f, 0.0f);
        for (int c = 0; c < p.split; ++c) {
          const uint32_t from = mapa_shared(part + warp * 128 + r * 2, c);
#pragma unroll
          for (int j = 0; j < kPerWarp; ++j) {
            const float2 v = ld_cluster_f32x2(from + j * kWarps * 512);
            y[j].x += v.x;
            y[j].y += v.y;
          }
        }
        const int64_t n = static_cast<int64_t>(rb) * 128 + r * 2;
        if (n >= p.N) continue;
        float2 bias = make_float2(0.0f, 0.0f);
        if (p.bias != nullptr) {
          const uint32_t b = __ldg(reinterpret_cast<const uint32_t*>(p.bias + n));
          bias = make_float2(bf16_lo(b), bf16_hi(b));
        }
#pragma unroll
        for (int j = 0; j < kPerWarp; ++j) {
          const int m = warp + j * kWarps;
          if (m < p.M && SQ_GUARD(within(p.Y + m * p.N + n, 2, p.Y, p.M * p.N)))
            *reinterpret_cast<__nv_bfloat162*>(p.Y + m * p.N + n) =
                __floats2bfloat162_rn(y[j].x + bias.x, y[j].y + bias.y);
        }
      }
      if (p.split > 1) {
        workers_sync<C::kWorkers>();
        if (threadIdx.x < p.split) arrive_cluster(mapa_shared(&sh.part_free, threadIdx.x));
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
  __syncwarp();
  tc_fence_before();
  if (p.split > 1)
    cluster_sync();  // no CTA leaves while its sums are being read
  else
    __syncthreads();
  tc_fence_after();
  if (warp == kTmaWarp) tmem_dealloc(tmem, 512);
}

template <int TOKENS, int G, bool ASYM>
cudaError_t launch_tc(const Int4LinearArgs& a, cudaStream_t stream) {
  using C = Cfg<TOKENS, G>;
  TcParams p{};
  p.N = a.N;
  p.Wp = a.Wp;
  p.scale = a.scale;
  p.zero = a.zero;
  p.bias = a.bias;
  p.Y = a.Y;
  p.M = static_cast<int>(a.M);
  p.K = static_cast<int>(a.K);
  p.Kb = (p.K + 127) / 128;
  p.groups = (p.K + G - 1) / G;
  p.status = a.status;
  p.row_blocks = static_cast<int>((a.N + 127) / 128);
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  // Rounds of row blocks over the clusters, in blocks of columns per CTA, and what a round costs
  // besides: its end, and the exchange of a cluster. Measured, us, clusters of 1 / 2 / 4 / 8:
  // 64 x 8192 x 8192 37 / 22 / 27 / 52, 24 x 2048 x 14336 52 / 29 / 18 / 22 (of 6 14.5), 25 x 344 x
  // 16704 65 / 36 / 23 / 15, 64 x 1024 x 1024 9.4 / 7.6 / 7.1 / 9.2; of 2 / 3: 64 x 5120 x 13824
  // 32 / 24; of 1 / 3: 64 x 28672 x 8192 70 / 74.
  double least = 1e30;
  p.split = 1;
  for (int split = 1; split <= 8 && split <= p.Kb; ++split) {
    const int clusters = cluster_slots(sms, split), rounds = (p.row_blocks + clusters - 1) / clusters;
    const double cost = rounds * ((p.Kb + split - 1) / split + (split > 1 ? 5.0 + 0.7 * split : 3.0));
    if (cost < least) least = cost, p.split = split;
  }
  CUtensorMap map{};
  if (!make_bf16_operand_map(&map, a.X, static_cast<uint64_t>(a.K), static_cast<uint64_t>(a.M),
                     static_cast<uint64_t>(a.ldx) * 2, TOKENS))
    return cudaErrorInvalidValue;
  auto kernel = int4_tc_kernel<TOKENS, G, ASYM>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  const int clusters = std::min(cluster_slots(sms, p.split), p.row_blocks);
  return launch_kernel_clustered(kernel, dim3(static_cast<unsigned>(clusters * p.split)), dim3(C::kThreads), C::kSmem,
                                 stream, true, static_cast<unsigned>(p.split), map, p);
}

template <int TOKENS>
cudaError_t launch_tokens(const Int4LinearArgs& a, cudaStream_t stream) {
  if (a.zero != nullptr) {
    if (a.group == 32) return launch_tc<TOKENS, 32, true>(a, stream);
    return a.group == 64 ? launch_tc<TOKENS, 64, true>(a, stream) : launch_tc<TOKENS, 128, true>(a, stream);
  }
  if (a.group == 32) return launch_tc<TOKENS, 32, false>(a, stream);
  return a.group == 64 ? launch_tc<TOKENS, 64, false>(a, stream) : launch_tc<TOKENS, 128, false>(a, stream);
}

}  // namespace

cudaError_t launch_int4_linear_tc(const Int4LinearArgs& a, cudaStream_t stream) {
  return a.M <= 32 ? launch_tokens<32>(a, stream) : launch_tokens<64>(a, stream);
}

}  // namespace sq
