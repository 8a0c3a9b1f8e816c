// fm_gemm_e4m3_b128: E4M3 x E4M3 with fp32 scales per 128 inputs of a row (a)
// and per 128 x 128 block (w).
//
//   out[i][j] = sum_g sa[i][g] sw[j/128][g] sum_{c in g} a[i][c] w[j][c]
//
// The scales are arbitrary fp32 numbers, so the tensor cores can only sum
// inside a group (K = 128: four kind::f8f6f4 MMAs into a fresh TMEM
// accumulator); the groups are scaled and summed in the registers of the
// epilogue warps.  TMEM holds several accumulators, so the MMAs of a group run
// while the ones before are read.
//
// Operands come by tiled TMA (128-byte rows, SW128), zero-filled outside the
// matrices: ragged m, n and the last group of k need no code of their own.
#include <cuda.h>
#include <cuda_bf16.h>

#include <atomic>
#include <cstdint>

#include "../../include/fm_ops.h"
#include "fm_ops_check.h"
#include "fm_ops_math.cuh"
#include "fm_ptx.cuh"

namespace fm {
namespace {

// Waits that gave up on this device since the library was loaded: their number
// (low half; never cleared, so that no reader takes another's report) and which.
__device__ unsigned long long g_ops_err;
__device__ __forceinline__ void gave_up(unsigned int which) {
  atomicOr(&g_ops_err, (unsigned long long)which << 32);
  atomicAdd(&g_ops_err, 1ull);
}

// The bound of a wait, in SM cycles (about 2 s).  The pipelines' waits take it
// from GemmParams::spin (fm_ops_test_stall); the waits at a kernel's end, for
// what is still on its way to a block's shared memory, always have this one.
constexpr unsigned kSpin = 4000000000u;

struct GemmParams {
  const float *sa, *sw;
  const uint16_t* bias;
  void* out;
  int64_t ldsa, ldsw, ldo;
  int m, n, groups;
  uint8_t f32;
  uint8_t vec;             // rows of `out` start on 16-byte boundaries
  uint8_t stall;           // 0, or the role (FM_STALL_*) that gives up
  unsigned stall_at;       //   at this group of its own count
  unsigned spin;           // bound of the pipeline's waits, cycles
};
// 16 bytes more, beside the two tensor maps, cost 0.4 us of a 5.5 us call.
static_assert(sizeof(GemmParams) <= 80, "kernel parameters");
// How many of its next `count` groups `role` does when it has done `done`: all but
// where it is to give up.  (Outside the loops over groups: a comparison in them
// cost 50 cycles a group.)
__device__ __forceinline__ int groups_of(const GemmParams& p, int role, int count, uint32_t done) {
  if (p.stall != role) return count;
  const uint32_t left = p.stall_at > done ? p.stall_at - done : 0;
  return left < (uint32_t)count ? (int)left : count;
}

// 2-D tiled load of a box of 128-byte rows at (column c0, row c1).
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* tmap, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(tmap), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
      "%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// Whether the phase has completed, without waiting for it (try_wait may sleep
// for microseconds where it never completes: after the last accumulator).
__device__ __forceinline__ bool mbar_peek(uint32_t bar, uint32_t parity) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(bar), "r"(parity)
      : "memory");
  return r != 0;
}
// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// One MMA of a group (kind::f8f6f4, K = 32), ACC 0: a fresh accumulator.
template <int ACC>
__device__ __forceinline__ void mma_e4m3_one(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "n"(ACC)
      : "memory");
}
// Completes `bytes` of the barrier's expected transactions: those of a copy that
// was announced and will not be made.
__device__ __forceinline__ void mbar_complete_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// Waits for the last phase below `end` on each of the `depth` (<= 32) barriers
// from bar0 on that phases 0, 1, ... go round on (a whole warp; a barrier per lane).
__device__ __forceinline__ void await_last(uint32_t bar0, uint32_t depth, uint32_t end, int lane) {
  const uint32_t l = (uint32_t)lane;
  if (l < depth && l < end) {
    const uint32_t last = end - 1 - (end - 1 - l) % depth;
    mbar_wait(bar0 + 8 * l, (last / depth) & 1, kSpin);
  }
  __syncwarp();
}
__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}
__device__ __forceinline__ float bias_at(const GemmParams& p, int j) {
  return p.bias != nullptr && j < p.n ? __uint_as_float((uint32_t)p.bias[j] << 16) : 0.f;
}
__device__ __forceinline__ void store_out1(const GemmParams& p, int i, int j, float v) {
  if (j >= p.n) return;
  if (p.f32)
    static_cast<float*>(p.out)[(int64_t)i * p.ldo + j] = v;
  else
    static_cast<__nv_bfloat16*>(p.out)[(int64_t)i * p.ldo + j] = __float2bfloat16_rn(v);
}
// Channels j .. j + 7 (j a multiple of 8) of row i where p.vec holds, plus the
// bias, rounded once to the output type.
__device__ __forceinline__ void store_out8(const GemmParams& p, int i, int j, const float* v) {
  if (j + 8 > p.n) {
#pragma unroll
    for (int e = 0; e < 8; ++e) store_out1(p, i, j + e, v[e] + bias_at(p, j + e));
    return;
  }
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = v[e] + bias_at(p, j + e);
  const int64_t at = (int64_t)i * p.ldo + j;
  if (p.f32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at);
    o[0] = make_float4(x[0], x[1], x[2], x[3]);
    o[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at) =
        make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  }
}

// As store_out8, of 4 channels (j a multiple of 4).
__device__ __forceinline__ void store_out4(const GemmParams& p, int i, int j, float4 v) {
  v.x += bias_at(p, j);
  v.y += bias_at(p, j + 1);
  v.z += bias_at(p, j + 2);
  v.w += bias_at(p, j + 3);
  const int64_t at = (int64_t)i * p.ldo + j;
  if (j + 4 > p.n) {
    store_out1(p, i, j, v.x);
    store_out1(p, i, j + 1, v.y);
    store_out1(p, i, j + 2, v.z);
  } else if (p.f32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = v;
  } else {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
  }
}

// 4 consecutive scales from group g on (0 past the last); `v4`: 16-byte loads allowed.
__device__ __forceinline__ float4 scales4(const float* s, int g, int groups, bool v4) {
  if (v4 && g + 4 <= groups) return *reinterpret_cast<const float4*>(s + g);
  float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
  if (g < groups) r.x = s[g];
  if (g + 1 < groups) r.y = s[g + 1];
  if (g + 2 < groups) r.z = s[g + 2];
  if (g + 3 < groups) r.w = s[g + 3];
  return r;
}

// ----------------------------------------------------------------- few rows
// A block owns up to 128 rows of `a` (BT of them brought: 16, 32, 64 or 128)
// x 128 output channels, and the blocks of a cluster split the groups of k:
// there are too few tiles to fill the GPU, and the time is that of streaming
// the weights.  The rows are the 128-row operand even when there is one of them:
// the rows behind BT are whatever shared memory holds and give accumulator rows
// nobody reads, and a thread is a row, so a group's factor is one register.
// (With the channels as the 128-row operand the factors differ by column and
// come from shared memory, whose bandwidth M = 128, N <= 128 products use up:
// 830 cycles a group against 380 at 50 rows.)  Each block of the cluster leaves
// its sums in shared memory and adds its share of the tile over all of them in
// rank order.
template <int BT>
struct Few {
  static constexpr int kW = 128 * 128, kStage = kW + BT * 128;
  static constexpr int kStages = BT == 128 ? 6 : 8;
  static constexpr int kTail = (128 - BT) * 128;       // the last stage's rows behind BT
  static constexpr int kBufs = 4;                      // accumulators of 128 columns
  static constexpr int kThreads = 320;                 // TMA, MMA, 8 epilogue warps
  static constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + kTail + 256;
  static_assert(kSmem <= 232448, "227 KB");
  static_assert((size_t)kStages * kStage >= (size_t)BT * 512, "the sums reuse the ring");
};

template <int BT>
__global__ void __launch_bounds__(320, 1)
few_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mw,
           const __grid_constant__ GemmParams p, int split) {
  using C = Few<BT>;
  extern __shared__ uint8_t raw[];
  uint8_t* ring = align1024(raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + (size_t)C::kStages * C::kStage + C::kTail);
  uint64_t* empty = full + C::kStages;
  uint64_t* tfull = empty + C::kStages;  // [kBufs]
  uint64_t* tempty = tfull + C::kBufs;   // [kBufs]
  uint32_t* slot = reinterpret_cast<uint32_t*>(tempty + C::kBufs);
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const unsigned rank = split > 1 ? cluster_rank() : 0, tile = blockIdx.x / (unsigned)split;
  const unsigned rt = (unsigned)((p.m + BT - 1) / BT);
  const int i0 = (int)(tile % rt) * BT, nb = (int)(tile / rt), n0 = nb * 128;
  const int rows = p.m - i0 < BT ? p.m - i0 : BT;
  const int quarters = (rows + 31) / 32;               // TMEM lane quarters with rows of `a`
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < C::kBufs; ++b) {
      mbar_init(smem_u32(&tfull[b]), 1);
      mbar_init(smem_u32(&tempty[b]), 2 * quarters);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *slot, 0);   // known uniform: TMEM addresses need no moves
  grid_dep_launch();
  grid_dep_wait();                           // everything above touches this block's memory only
  const int g0 = (int)((int64_t)p.groups * rank / split), g1 = (int)((int64_t)p.groups * (rank + 1) / split);
  const int count = g1 - g0;

  // In the TMA and MMA warps all lanes run the loop and one elected lane issues,
  // so that addresses and descriptors live in uniform registers.
  if (warp == 0) {
    const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty), ring0 = smem_u32(ring);
    const int end = groups_of(p, rank == 0 ? FM_STALL_TMA0 : rank == 1 ? FM_STALL_TMA1 : -1, count, 0);
    uint32_t s = 0, ph = 1;                  // a fresh barrier's previous phase counts as done
    int it = 0;
    for (; it < end; ++it) {
      if (!__all_sync(0xffffffffu, mbar_wait(empty0 + 8 * s, ph, p.spin))) {
        break;
      }
      if (elect_one()) {
        mbar_arrive_expect_tx(full0 + 8 * s, C::kStage);
        tma_load_2d(ring0 + s * C::kStage, &mw, (g0 + it) * 128, n0, full0 + 8 * s);
        tma_load_2d(ring0 + s * C::kStage + C::kW, &ma, (g0 + it) * 128, i0, full0 + 8 * s);
      }
      __syncwarp();
      if (++s == C::kStages) s = 0, ph ^= 1;
    }
    if (it < count && lane == 0) gave_up(1);
    await_last(full0, C::kStages, (uint32_t)it, lane);   // every issued copy has landed
  } else if (warp == 1) {
    constexpr uint32_t idesc = idesc_e4m3(128, 128);
    const uint64_t d0 = desc_sw128(smem_u32(ring));
    const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty), tfull0 = smem_u32(tfull), tempty0 = smem_u32(tempty);
    const int end = groups_of(p, rank == 0 ? FM_STALL_MMA0 : rank == 1 ? FM_STALL_MMA1 : -1, count, 0);
    uint32_t s = 0, ph = 0, b = 0, bph = 1;
    int it = 0;
    for (; it < end; ++it) {
      if (!__all_sync(0xffffffffu, mbar_wait(tempty0 + 8 * b, bph, p.spin) && mbar_wait(full0 + 8 * s, ph, p.spin))) {
        break;
      }
      tc_fence_after();
      if (elect_one()) {
        const uint64_t wd = d0 + s * (C::kStage >> 4), ad = wd + (C::kW >> 4);
        mma_e4m3_one<0>(tmem + b * 128, ad, wd, idesc);
        mma_e4m3_one<1>(tmem + b * 128, ad + 2, wd + 2, idesc);
        mma_e4m3_one<1>(tmem + b * 128, ad + 4, wd + 4, idesc);
        mma_e4m3_one<1>(tmem + b * 128, ad + 6, wd + 6, idesc);
        mma_commit(tfull0 + 8 * b);
        mma_commit(empty0 + 8 * s);
      }
      __syncwarp();
      if (++s == C::kStages) s = 0, ph ^= 1;
      if (++b == C::kBufs) b = 0, bph ^= 1;
    }
    if (it < count && lane == 0) gave_up(2);
    // every MMA is done and every commit has arrived before TMEM and the ring are given up
    await_last(tfull0, C::kBufs, (uint32_t)it, lane);
    await_last(empty0, C::kStages, (uint32_t)it, lane);
  } else if ((warp & 3) < quarters) {
    const int q4 = warp & 3, h = (warp - 2) >> 2;
    const int row = 32 * q4 + lane;            // TMEM lane: row i0 + row
    const bool live = row < rows;
    const uint32_t ta = tmem + ((uint32_t)(32 * q4) << 16) + h * 64;
    const float* sa = p.sa + (int64_t)(i0 + (live ? row : 0)) * p.ldsa + g0;
    const float* sw = p.sw + (int64_t)nb * p.ldsw + g0;
    const bool v4 = (reinterpret_cast<uintptr_t>(sa) & 15) == 0;
    float acc[64];
#pragma unroll
    for (int c = 0; c < 64; ++c) acc[c] = 0.f;
    const bool w4 = (reinterpret_cast<uintptr_t>(sw) & 15) == 0;
    const uint32_t tfull0 = smem_u32(tfull), tempty0 = smem_u32(tempty);
    bool ok = true, ready = false;             // ready: the next accumulator was seen
    // four groups' scales of this row and of its channels, fetched four groups ahead
    float4 fa = scales4(sa, 0, count, v4), fw = scales4(sw, 0, count, w4);
    uint32_t unit = 0;                         // accumulators used so far: buffer and phase
    static_assert((C::kBufs & (C::kBufs - 1)) == 0, "a power of two");
    for (int it0 = 0; ok && it0 < count; it0 += 4) {
      const float s4[4] = {fa.x * fw.x, fa.y * fw.y, fa.z * fw.z, fa.w * fw.w};
      fa = scales4(sa, it0 + 4, count, v4);
      fw = scales4(sw, it0 + 4, count, w4);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (it0 + u >= count) break;
        const uint32_t b = unit % C::kBufs;
        if (!ready) ok = __all_sync(0xffffffffu, mbar_wait(tfull0 + 8 * b, (unit / C::kBufs) & 1, p.spin));
        if (!ok) {
          if (lane == 0) gave_up(4);
          break;
        }
        tc_fence_after();
        ++unit;
        const float s = s4[u];
        float v[2][32];
        tmem_ld32(ta + b * 128, v[0]);
        tmem_ld32(ta + b * 128 + 32, v[1]);
        tmem_ld_wait();
        // all read: the accumulator goes back, and the sums cover the look at the next
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty0 + 8 * b);
        const bool next = mbar_peek(tfull0 + 8 * (unit % C::kBufs), (unit / C::kBufs) & 1);
#pragma unroll
        for (int e = 0; e < 64; e += 2)
          fma2(acc[e], acc[e + 1], v[e >> 5][e & 31], v[e >> 5][(e & 31) + 1], s, s);
        ready = __all_sync(0xffffffffu, next);
      }
    }
    if (split == 1 && p.vec) {
      if (ok && live) {
#pragma unroll
        for (int c = 0; c < 64; c += 8) store_out8(p, i0 + row, n0 + h * 64 + c, acc + c);
      }
    } else {
      // the ring is free: every MMA that reads it has completed (the last tfull).
      // [row][128], 16-byte pieces swizzled by the row
      float* part = reinterpret_cast<float*>(ring) + row * 128;
      if (live) {
#pragma unroll
        for (int c = 0; c < 16; ++c)
          *reinterpret_cast<float4*>(part + (((h * 16 + c) ^ (row & 31)) << 2)) =
              make_float4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]);
      }
    }
  }
  __syncwarp();
  if (split > 1 || !p.vec) {
    cluster_sync_all();
    if (warp >= 2) {
      const float* part = reinterpret_cast<const float*>(ring);
      if (p.vec) {
        // this rank's share of the tile's rows x 32 pieces of 4 channels, four
        // of them per thread at a time
        constexpr int kThr = C::kThreads - 64;
        const int all = rows * 32, c0 = all * (int)rank / split, c1 = all * ((int)rank + 1) / split;
        const int piece = (int)threadIdx.x & 31, j = n0 + 4 * piece;     // the same for all of a thread's items
        for (int c = c0 - (c0 & 31) + (int)threadIdx.x - 64; c < c1; c += 4 * kThr) {
          float4 sum[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) sum[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int k = 0; k < split; ++k) {
            const uint32_t base = map_shared_rank(smem_u32(part), k);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int i = c + u * kThr, r = i >> 5;
              if (i >= c0 && i < c1) {
                const float4 x = ld_dsmem_f4(base + r * 512 + ((piece ^ (r & 31)) << 4));
                sum[u].x += x.x;
                sum[u].y += x.y;
                sum[u].z += x.z;
                sum[u].w += x.w;
              }
            }
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int i = c + u * kThr;
            if (i >= c0 && i < c1) store_out4(p, i0 + (i >> 5), j, sum[u]);
          }
        }
      } else {
        // rows at any element: a warp takes four rows of this rank's share at a
        // time and stores 32 neighbours of one with each instruction
        const int c0 = rows * (int)rank / split, c1 = rows * ((int)rank + 1) / split;
        float bias[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) bias[q] = bias_at(p, n0 + 32 * q + lane);
        for (int r = c0 + 4 * (warp - 2); r < c1; r += 32) {
          float sum[4][4];
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int q = 0; q < 4; ++q) sum[u][q] = 0.f;
          for (int k = 0; k < split; ++k) {
            const uint32_t base = map_shared_rank(smem_u32(part), k);
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
              for (int q = 0; q < 4; ++q)
                if (r + u < c1)
                  sum[u][q] += ld_dsmem_f1(base + (r + u) * 512 + (((8 * q + (lane >> 2)) ^ ((r + u) & 31)) << 4) +
                                           ((lane & 3) << 2));
          }
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (r + u < c1) store_out1(p, i0 + r + u, n0 + 32 * q + lane, sum[u][q] + bias[q]);
        }
      }
    }
    cluster_sync_all();                        // no block leaves while another reads its sums
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int BT>
cudaError_t launch_few(const CUtensorMap& ma, const CUtensorMap& mw, const GemmParams& p, int split, cudaStream_t st) {
  using C = Few<BT>;
  cudaError_t e = cudaFuncSetAttribute(few_kernel<BT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (((int64_t)p.m + BT - 1) / BT) * (((int64_t)p.n + 127) / 128);
  return launch_op(few_kernel<BT>, (unsigned)(tiles * split), C::kThreads, C::kSmem, split, st, ma, mw, p, split);
}

// ----------------------------------------------------------------- many rows
// A pair of blocks (cluster of 2, cta_group::2) owns a tile of 256 rows of `a`
// x 256 output channels: each block brings its own 128 rows and half of the
// weights (32 KB a group for 128 x 256 x 128 products), which halves the
// operand traffic a 128 x 256 tile of one block would need.  The leader's two
// MMA warps issue M = 256, N = 128 products, one half of the channels each, into
// two TMEM accumulators per half; four epilogue warps per half and block
// scale and sum them, thread = row, so a group's factor is one register.
// Outputs leave through shared memory, by TMA where `out` allows it (other
// rows cost ~4000 cycles a tile more: 34.5 -> 60.1 us at m 12000, k 512, n 4096
// -> 4097).
//
// What bounds it: a group is 512 cycles of products and takes 635 (8192^3 in
// short runs, 2660 TFLOP/s; 500 us sustained, where the power cap sets the
// clock and the library's product without group scales takes 420).  The
// epilogue warps set the pace: two share a scheduler, each reads 128 columns
// and makes 64 packed FMAs a group, and what they do beside that shows: TMEM
// addresses that the compiler does not know to be uniform cost 80 cycles, a
// wait for a barrier that is ready 130, scales fetched group by group 130.
// Without the sums the loop takes 557.  Measured and left: one MMA warp for
// both halves (695 without the sums), N = 256 units, 16 epilogue warps (870),
// 16 columns a load.
struct Wide {
  static constexpr int kA = 128 * 128, kB = 64 * 128, kStage = kA + 2 * kB;
  static constexpr int kStages = 5;
  static constexpr int kSlot = 4096;               // 32 rows x 128 bytes of output
  static constexpr int kThreads = 384;             // 8 epilogue warps, TMA, 2 x MMA, one idle
  static constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + 16 * kSlot + 2 * 256 * 2 + 256;
  static_assert(kSmem <= 232448, "227 KB");
};

__device__ __forceinline__ uint32_t leader_addr(uint32_t a) { return map_shared_rank(a, 0); }
// As tma_load_2d, completing on a barrier of the pair (shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const void* tmap, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(tmap), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_store_2d(const void* tmap, int c0, int c1, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(tmap), "r"(c0),
               "r"(c1), "r"(src)
               : "memory");
}
__device__ __forceinline__ void bulk_commit_group() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
template <int ACC>
__device__ __forceinline__ void mma_e4m3_pair(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "n"(ACC)
      : "memory");
}
// Arrives on `bar` of both blocks of the pair when this thread's MMAs are done.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .b16 m;\n\tmov.b16 m, 3;\n\t"
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(bar)
      : "memory");
}
// Relaxed: what it hands over is a TMEM accumulator whose loads have returned
// (tcgen05.wait::ld), no memory; a release of cluster scope waits for all the
// thread's memory operations and cost ~1000 cycles a group (956 -> 490 us at
// 8192^3).
__device__ __forceinline__ void arrive_at(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// Leaves `value` at `slot` of both blocks and arrives on `ended` of both (a whole warp).
__device__ __forceinline__ void leave_count(uint32_t* slot, uint32_t value, uint64_t* ended, int lane) {
  if (lane < 2) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_shared_rank(smem_u32(slot), (uint32_t)lane)), "r"(value)
                 : "memory");
    mbar_arrive_cluster(smem_u32(ended), (uint32_t)lane);
  }
  __syncwarp();
}
// The end of the pair's pipeline, by the TMA warp of each block: returns when no
// copy and no commit is on its way to this block's shared memory (the leader's:
// to either ring), so that the blocks may leave after one more cluster barrier.
// Where waits gave up the roles have stopped at different groups.  Each leaves
// its count and does nothing more, and what a phase lacks is then made up: the
// other block's copies on the leader's `full`, the other MMA warp's commits on
// `empty`.  A stage is used again only after both have gone by, so at most one
// phase of each barrier is open.
template <int S, int BYTES>
__device__ __forceinline__ void pair_end(uint32_t full0, uint32_t empty0, uint32_t tfull0, uint32_t ended,
                                         const uint32_t* counts, uint32_t rank, int lane) {
  // (a role may still be waiting out its own bound, and one behind it the next)
  if (!__all_sync(0xffffffffu, mbar_wait_cluster(ended, 0, 8ll * kSpin))) return;
  const volatile uint32_t* c = counts;
  const uint32_t i0 = c[0], i1 = c[1], m0 = c[2], m1 = c[3];
  const uint32_t is = i0 < i1 ? i0 : i1, ib = i0 < i1 ? i1 : i0, ms = m0 < m1 ? m0 : m1, mb = m0 < m1 ? m1 : m0;
  if (lane == 0) {
    if (rank == 0)
      for (uint32_t j = is; j < ib; ++j) {
        if (i0 > i1)
          mbar_complete_tx(full0 + 8 * (j % S), BYTES);
        else
          mbar_arrive_expect_tx(full0 + 8 * (j % S), BYTES);
      }
    for (uint32_t j = ms; j < mb; ++j) mbar_arrive(empty0 + 8 * (j % S));
  }
  __syncwarp();
  if (rank == 0) await_last(full0, S, ib, lane);
  await_last(empty0, S, mb, lane);
  await_last(tfull0, 2, m0, lane);
  await_last(tfull0 + 16, 2, m1, lane);
}

// Tiles in bands of 8 row tiles, so that the tiles in flight share operands in L2.
struct TileAt {
  int mt, nt;
};
__device__ __forceinline__ TileAt tile_at(unsigned t, unsigned mts, unsigned nts) {
  const unsigned band = t / (8 * nts), r = t - band * 8 * nts;
  const unsigned h = mts - band * 8 < 8 ? mts - band * 8 : 8;
  return TileAt{(int)(band * 8 + r % h), (int)(r / h)};
}

__global__ void __launch_bounds__(384, 1)
wide_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mw,
            const __grid_constant__ CUtensorMap mo, const __grid_constant__ GemmParams p, int tma_out) {
  using C = Wide;
  extern __shared__ uint8_t raw[];
  uint8_t* ring = align1024(raw);
  uint8_t* slots = ring + (size_t)C::kStages * C::kStage;
  uint16_t* bias_s = reinterpret_cast<uint16_t*>(slots + 16 * C::kSlot);   // [2][256]
  uint64_t* full = reinterpret_cast<uint64_t*>(bias_s + 512);          // the leader's
  uint64_t* empty = full + C::kStages;
  uint64_t* tfull = empty + C::kStages;      // [half][buffer]
  uint64_t* tempty = tfull + 4;              // [half][buffer], the leader's
  uint64_t* ended = tempty + 4;              // four roles of the pair have left their counts:
  uint32_t* counts = reinterpret_cast<uint32_t*>(ended + 1);   // groups brought by each block, multiplied by each MMA warp
  uint32_t* slot = counts + 4;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 2);
    }
    for (int b = 0; b < 4; ++b) {
      mbar_init(smem_u32(&tfull[b]), 1);
      mbar_init(smem_u32(&tempty[b]), 8);
    }
    mbar_init(smem_u32(ended), 4);
    fence_mbar_init();
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();                        // both blocks' barriers exist before any remote arrival
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *slot, 0);   // known uniform: TMEM addresses need no moves
  grid_dep_launch();
  grid_dep_wait();                           // everything above touches this pair's memory only
  const unsigned mts = (unsigned)((p.m + 255) / 256), nts = (unsigned)((p.n + 255) / 256);
  const unsigned tiles = mts * nts, pairs = gridDim.x >> 1, first = blockIdx.x >> 1;

  // 384 threads start with 168 registers: 4 warps keep 40, 8 get 232 (64512 in all)
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 8) {
      const uint32_t empty0 = smem_u32(empty), full0 = smem_u32(full), ring0 = smem_u32(ring), lead0 = leader_addr(full0);
      uint32_t it = 0, s = 0, ph = 1;        // a fresh barrier's previous phase counts as done
      bool ok = true;
      for (unsigned t = first; ok && t < tiles; t += pairs) {
        const TileAt at = tile_at(t, mts, nts);
        const int m0 = at.mt * 256 + (int)rank * 128, n0 = at.nt * 256 + (int)rank * 64;
        const int end = groups_of(p, rank == 0 ? FM_STALL_TMA0 : FM_STALL_TMA1, p.groups, it);
        int g = 0;
        for (; g < end; ++g) {
          if (!__all_sync(0xffffffffu, mbar_wait(empty0 + 8 * s, ph, p.spin))) break;
          if (elect_one()) {
            const uint32_t dst = ring0 + s * C::kStage, bar = lead0 + 8 * s;
            if (rank == 0) mbar_arrive_expect_tx(full0 + 8 * s, 2 * C::kStage);
            tma_load_2d_pair(dst, &ma, g * 128, m0, bar);
            tma_load_2d_pair(dst + C::kA, &mw, g * 128, n0, bar);
            tma_load_2d_pair(dst + C::kA + C::kB, &mw, g * 128, n0 + 128, bar);
          }
          __syncwarp();
          if (++s == C::kStages) s = 0, ph ^= 1;
        }
        it += g;
        ok = g == p.groups;
      }
      if (!ok && lane == 0) gave_up(8);
      leave_count(counts + rank, it, ended, lane);
      pair_end<C::kStages, C::kStage>(full0, empty0, smem_u32(tfull), smem_u32(ended), counts, rank, lane);
    } else if (warp < 11 && rank == 0) {
      // The whole warp runs the loop and one elected lane issues, so that the
      // descriptors live in uniform registers: a lone thread spent ~1000 cycles
      // a group on building and moving them, twice the products' time.
      constexpr uint32_t idesc = idesc_e4m3(256, 128);
      const uint32_t h = warp - 9;
      const uint64_t d0 = desc_sw128(smem_u32(ring)), w0 = desc_sw128(smem_u32(ring) + C::kA + h * C::kB);
      const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty), tfull0 = smem_u32(tfull + 2 * h),
                     tempty0 = smem_u32(tempty + 2 * h), dst0 = tmem + h * 256;
      uint32_t s = 0, ph = 0, b = 0, bph = 1, it = 0;
      bool ok = true;
      for (unsigned t = first; ok && t < tiles; t += pairs) {
        const int end = groups_of(p, h == 0 ? FM_STALL_MMA0 : FM_STALL_MMA1, p.groups, it);
        int g = 0;
        for (; g < end; ++g) {
          if (!__all_sync(0xffffffffu, mbar_wait(full0 + 8 * s, ph, p.spin) && mbar_wait(tempty0 + 8 * b, bph, p.spin)))
            break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t d = dst0 + b * 128;
            const uint64_t ad = d0 + s * (C::kStage >> 4), bd = w0 + s * (C::kStage >> 4);
            mma_e4m3_pair<0>(d, ad, bd, idesc);
            mma_e4m3_pair<1>(d, ad + 2, bd + 2, idesc);
            mma_e4m3_pair<1>(d, ad + 4, bd + 4, idesc);
            mma_e4m3_pair<1>(d, ad + 6, bd + 6, idesc);
            mma_commit_pair(tfull0 + 8 * b);
            mma_commit_pair(empty0 + 8 * s);
          }
          __syncwarp();
          if (++s == C::kStages) s = 0, ph ^= 1;
          if ((b ^= 1) == 0) bph ^= 1;
        }
        it += g;
        ok = g == p.groups;
      }
      if (!ok && lane == 0) gave_up(16);
      leave_count(counts + 2 + h, it, ended, lane);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    const int q4 = warp & 3, h = warp >> 2;
    const uint32_t ta = tmem + ((uint32_t)(32 * q4) << 16) + h * 256;
    const uint32_t tfull0 = smem_u32(&tfull[2 * h]), te0 = leader_addr(smem_u32(&tempty[2 * h]));
    const bool v4 = (reinterpret_cast<uintptr_t>(p.sa) & 15) == 0 && p.ldsa % 4 == 0;
    uint32_t unit = 0;                         // accumulators used so far: buffer and phase
    int par = 0;
    bool ok = true, ready = false;             // ready: the next accumulator was seen
    const bool w4 = (reinterpret_cast<uintptr_t>(p.sw) & 15) == 0 && p.ldsw % 4 == 0;
    // Four groups' scales of this row and of its channels, fetched four groups
    // ahead (a tile's first ones before the tile ahead of it is written out).
    float4 fa, fw;
    const float *sa, *sw;
    auto enter = [&](unsigned t) {
      const TileAt at = tile_at(t, mts, nts);
      const int row = at.mt * 256 + (int)rank * 128 + 32 * q4 + lane, col = at.nt * 256 + h * 128;
      const bool live = row < p.m && col < p.n;
      sa = p.sa + (int64_t)(live ? row : 0) * p.ldsa;
      sw = p.sw + (int64_t)(live ? col >> 7 : 0) * p.ldsw;
      fa = scales4(sa, 0, p.groups, v4);
      fw = scales4(sw, 0, p.groups, w4);
    };
    if (first < tiles) enter(first);
    for (unsigned t = first; t < tiles; t += pairs, par ^= 1) {
      float acc[128];
#pragma unroll
      for (int c = 0; c < 128; ++c) acc[c] = 0.f;
      for (int g0 = 0; g0 < p.groups; g0 += 4) {
        const float s4[4] = {fa.x * fw.x, fa.y * fw.y, fa.z * fw.z, fa.w * fw.w};
        fa = scales4(sa, g0 + 4, p.groups, v4);
        fw = scales4(sw, g0 + 4, p.groups, w4);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (g0 + u >= p.groups) break;
          if (ok && !ready) ok = __all_sync(0xffffffffu, mbar_wait(tfull0 + 8 * (unit & 1), (unit >> 1) & 1, p.spin));
          if (!ok) {
            if (lane == 0) gave_up(32);
            continue;
          }
          tc_fence_after();
          const uint32_t b = unit & 1;
          ++unit;
          const float s = s4[u];
          float v[2][32];
          tmem_ld32(ta + b * 128, v[0]);
          bool next = false;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            tmem_ld_wait();
            if (q < 3) {
              tmem_ld32(ta + b * 128 + (q + 1) * 32, v[(q + 1) & 1]);
            } else {
              // all read: the accumulator goes back before the last sums, and they
              // cover the look at the next one
              tc_fence_before();
              __syncwarp();
              if (lane == 0) arrive_at(te0 + 8 * b);
              next = mbar_peek(tfull0 + 8 * (unit & 1), (unit >> 1) & 1);
            }
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              fma2(acc[q * 32 + e], acc[q * 32 + e + 1], v[q & 1][e], v[q & 1][e + 1], s, s);
          }
          ready = __all_sync(0xffffffffu, next);
        }
      }
      const TileAt here = tile_at(t, mts, nts);
      const int row0 = here.mt * 256 + (int)rank * 128 + 32 * q4, col0 = here.nt * 256 + h * 128;
      uint8_t* stage = slots + warp * 2 * C::kSlot;
      if (t + pairs < tiles) enter(t + pairs);
      if (p.bias != nullptr) {
        const int j = col0 + 32 * q4 + lane;
        uint16_t* bs = bias_s + par * 256 + h * 128;
        bs[32 * q4 + lane] = j < p.n ? p.bias[j] : 0;
        named_bar_sync(1 + h, 128);
#pragma unroll
        for (int c = 0; c < 128; c += 2) {
          const uint32_t f = *reinterpret_cast<const uint32_t*>(bs + c);
          acc[c] += __uint_as_float(f << 16);
          acc[c + 1] += __uint_as_float(f & 0xFFFF0000u);
        }
      }
      // the warp's rows, 128 bytes of them at a time (64 bf16 or 32 fp32
      // columns), as 16-byte pieces swizzled by (row & 7)
      const int sw7 = lane & 7;
      auto flush = [&](int c0, int width) {                // the slots hold columns c0 .. c0 + 2 width - 1
        if (tma_out) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (ok && row0 < p.m && c0 < p.n) tma_store_2d(&mo, c0, row0, smem_u32(stage));
            if (ok && row0 < p.m && c0 + width < p.n) tma_store_2d(&mo, c0 + width, row0, smem_u32(stage + C::kSlot));
            bulk_commit_group();
          }
        } else {
          __syncwarp();
          const int per = width / 32;                      // 2 bf16 or 1 fp32 per lane and row
          for (int r = 0; r < 32 && row0 + r < p.m && ok; ++r) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint32_t word = *reinterpret_cast<const uint32_t*>(stage + half * C::kSlot + r * 128 +
                                                                       (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
              const int j = c0 + half * width + lane * per;
              if (per == 1) {
                if (j < p.n) static_cast<float*>(p.out)[(int64_t)(row0 + r) * p.ldo + j] = __uint_as_float(word);
              } else {
                uint16_t* o = static_cast<uint16_t*>(p.out) + (int64_t)(row0 + r) * p.ldo + j;
                if (j < p.n) o[0] = (uint16_t)word;
                if (j + 1 < p.n) o[1] = (uint16_t)(word >> 16);
              }
            }
          }
          __syncwarp();
        }
      };
      if (tma_out && lane == 0) bulk_wait_read();          // the previous tile's slots have been read
      __syncwarp();
      uint8_t* o = stage + lane * 128;
      if (p.f32) {
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          if (part == 1) {
            if (tma_out && lane == 0) bulk_wait_read();
            __syncwarp();
          }
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float* a = acc + part * 64 + k * 4;
            *reinterpret_cast<float4*>(o + (k >> 3) * C::kSlot + (((k & 7) ^ sw7) << 4)) = make_float4(a[0], a[1], a[2], a[3]);
          }
          flush(col0 + part * 64, 32);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float* a = acc + k * 8;
          *reinterpret_cast<uint4*>(o + (k >> 3) * C::kSlot + (((k & 7) ^ sw7) << 4)) =
              make_uint4(pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]), pack_bf16(a[4], a[5]), pack_bf16(a[6], a[7]));
        }
        flush(col0, 64);
      }
    }
    if (tma_out && lane == 0) bulk_wait_all();
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();
  if (warp == 9) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// Pairs of blocks of wide_kernel that can run at once on the current device; 0
// where it cannot run.
int wide_pairs(int device) {
  static std::atomic<int> known[64];
  if (device >= 0 && device < 64) {
    const int k = known[device].load(std::memory_order_relaxed);
    if (k > 0) return k;
  }
  // the register split of wide_kernel needs the registers the launch brings
  cudaFuncAttributes fa;
  if (cudaFuncGetAttributes(&fa, wide_kernel) != cudaSuccess || fa.numRegs * Wide::kThreads < 40 * 128 + 232 * 256) {
    cudaGetLastError();
    return 0;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(148);
  cfg.blockDim = dim3(Wide::kThreads);
  cfg.dynamicSmemBytes = Wide::kSmem;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, wide_kernel, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    n = sm_count(device) / 2;
  }
  if (device >= 0 && device < 64) known[device].store(n, std::memory_order_relaxed);
  return n;
}

cudaError_t launch_wide(const CUtensorMap& ma, const CUtensorMap& mw, const CUtensorMap& mo, const GemmParams& p,
                        bool tma_out, int device, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(wide_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Wide::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (((int64_t)p.m + 255) / 256) * (((int64_t)p.n + 255) / 256);
  const int pairs = wide_pairs(device);
  if (pairs < 1) return cudaErrorInvalidConfiguration;
  const unsigned grid = 2u * (unsigned)(tiles < pairs ? tiles : pairs);
  return launch_op(wide_kernel, grid, Wide::kThreads, Wide::kSmem, 2, st, ma, mw, mo, p, tma_out ? 1 : 0);
}

// Which kernel, how many rows a block brings and how often k is split: the
// smallest estimated time.  The figures (microseconds) were fitted to sweeps of
// both kernels over 1 .. 16384 rows, 16 .. 8192 channels and 1 .. 128 groups: a
// block of few_kernel
// takes 0.20 a group whatever it holds (one MMA warp's four products, waits and
// commits), a pair of wide_kernel 0.39 for four times as much; adding the sums
// of a split costs by rows and blocks, rows of `out` that do not start on 16
// bytes (`vec` false) cost stores by element, and rows of codes that do not
// start on 128 (`lines` false) two lines of L2 for each 128 codes.  Over another 80
// random sizes the choice is 1.2 % from the best of all on average; at worst 38 %
// (m 3093 n 1390 k 2656, fp32 rows of `out` that do not start on 16 bytes: 31.9
// us, few_kernel 23.1), next 10 % (m 11 n 2713 k 176: 4.3, 3.9 us).
struct Choice {
  bool wide;
  int bt, split;
};
Choice choose(int64_t m, int64_t n, int64_t groups, bool vec, bool lines, int sms) {
  Choice best{false, m <= 16 ? 16 : m <= 32 ? 32 : m <= 64 ? 64 : 128, 1};
  const int64_t tiles = (m + best.bt - 1) / best.bt * ((n + 127) / 128);
  const double rows = m < best.bt ? (double)m : best.bt;
  double least = 1e30;
  for (int s = 1; s <= 8 && s <= groups; s *= 2) {
    // clusters need their blocks on neighbouring SMs: 120 of 148 SMs take clusters of 8, 132 of 4
    const int64_t room = s <= 2 ? sms : s == 4 ? sms * 132 / 148 : sms * 120 / 148;
    const int64_t waves = (tiles * s + room - 1) / room, g = (groups + s - 1) / s;
    const double t = (waves > 1 ? 1.5 + waves * (2.8 + (lines ? 0.24 : 0.42) * g) : 3.3 + (lines ? 0.20 : 0.38) * g) +
                     (s > 1 ? 0.1 * s + rows * (0.016 + 0.001 * s) : 0.0) + (vec ? 0.0 : waves * rows * 0.012 / s);
    if (t < least) least = t, best.split = s;
  }
  const int64_t pairs = sms / 2, waves = (((m + 255) / 256) * ((n + 255) / 256) + pairs - 1) / pairs;
  if (4.6 + waves * (1.1 + 0.39 * groups + (vec ? 0.0 : 2.1)) < least) best.wide = true;
  return best;
}

// fm_ops_test_stall of the calling thread.
struct Stall {
  uint8_t role = FM_STALL_NONE;
  unsigned group = 0, spin = kSpin;
};
thread_local Stall t_stall;

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}

// Codes [rows, k] as boxes of 128 bytes x box_rows, SW128, zeros outside.
bool codes_map(CUtensorMap* map, const uint8_t* p, int64_t ld, int rows, int k, int box_rows) {
  const EncodeFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(rows > 1 ? ld : k)};
  const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
  const cuuint32_t one[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// `out` as boxes of 32 rows x 128 bytes, SW128; false where TMA cannot address it.
bool out_map(CUtensorMap* map, void* p, int64_t ldo, int m, int n, bool f32) {
  const EncodeFn fn = encode_fn();
  const size_t es = f32 ? 4 : 2;
  if (fn == nullptr || ((uintptr_t)p & 15) != 0 || (m > 1 && ((uint64_t)ldo * es) % 16 != 0)) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)n, (cuuint64_t)m};
  const cuuint64_t strides[1] = {m > 1 ? (cuuint64_t)ldo * es : (((cuuint64_t)n * es + 15) & ~(cuuint64_t)15)};
  const cuuint32_t box[2] = {f32 ? 32u : 64u, 32};
  const cuuint32_t one[2] = {1, 1};
  return fn(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p, dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace fm

using fm::OpCheck;

extern "C" {
#pragma GCC visibility push(default)

fm_status fm_gemm_e4m3_b128(const uint8_t* a, int64_t lda, const float* sa, int64_t ldsa, const uint8_t* w, int64_t ldw,
                            const float* sw, int64_t ldsw, const uint16_t* bias, int m, int n, int k, void* out,
                            fm_dtype out_type, int64_t ldo, void* stream) {
  OpCheck c{"fm_gemm_e4m3_b128"};
  fm::set_thread_error("");
  if (out_type != FM_BF16 && out_type != FM_F32)
    return c.fail(FM_ERR_UNSUPPORTED, "out_type %d: FM_BF16 or FM_F32", (int)out_type);
  if (m < 0 || n < 0 || k < 16 || k % 16 != 0)
    return c.fail(FM_ERR_INVALID_ARG, "m %d / n %d / k %d out of range (k a positive multiple of 16)", m, n, k);
  if (m == 0 || n == 0) return FM_OK;
  const int64_t groups = ((int64_t)k + 127) / 128, tiles = (((int64_t)m + 127) / 128) * (((int64_t)n + 127) / 128);
  if (tiles > 0x0FFFFFFF || n > 0x7FFFFF00 || m > 0x7FFFFF00 || k > 0x7FFFFF00)
    return c.fail(FM_ERR_INVALID_ARG, "m %d x n %d x k %d is more than one launch takes", m, n, k);
  FM_TRY(c.rows(a, "a", lda, k, m, 1, 16));
  FM_TRY(c.rows(sa, "sa", ldsa, groups, m, 4, 4));
  FM_TRY(c.rows(w, "w", ldw, k, n, 1, 16));
  FM_TRY(c.rows(sw, "sw", ldsw, groups, (n + 127) / 128, 4, 4));
  if (bias != nullptr) FM_TRY(c.rows(bias, "bias", n, n, 1, 2, 2));
  FM_TRY(c.rows(out, "out", ldo, n, m, out_type == FM_F32 ? 4 : 2, out_type == FM_F32 ? 4 : 2));
  FM_TRY(c.memory());
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const size_t es = out_type == FM_F32 ? 4 : 2;
  const bool vec = ((uintptr_t)out & 15) == 0 && (m <= 1 || ((uint64_t)ldo * es) % 16 == 0);
  const fm::GemmParams p{sa, sw, bias, out, ldsa, ldsw, ldo, m, n, (int)groups, out_type == FM_F32, vec,
                         fm::t_stall.role, fm::t_stall.group, fm::t_stall.spin};
  const bool lines = (((uintptr_t)a | (uintptr_t)w) & 127) == 0 && (m <= 1 || lda % 128 == 0) && (n <= 1 || ldw % 128 == 0);
  const fm::Choice pick = fm::choose(m, n, groups, vec, lines, fm::sm_count(c.device));
  const bool wide = pick.wide;
  const int bt = pick.bt, split = pick.split;
  CUtensorMap ma, mw, mo;
  if (!fm::codes_map(&ma, a, lda, m, k, wide ? 128 : bt) || !fm::codes_map(&mw, w, ldw, n, k, wide ? 64 : 128))
    return c.fail(FM_ERR_CUDA, "the tensor maps of a and w were refused (m %d, n %d, k %d, strides %lld, %lld)", m, n, k,
                  (long long)lda, (long long)ldw);
  if (wide) {
    const bool tma_out = fm::out_map(&mo, out, ldo, m, n, out_type == FM_F32);
    if (!tma_out) mo = ma;
    return c.launched(fm::launch_wide(ma, mw, mo, p, tma_out, c.device, st));
  }
  return c.launched(bt == 16   ? fm::launch_few<16>(ma, mw, p, split, st)
                    : bt == 32 ? fm::launch_few<32>(ma, mw, p, split, st)
                    : bt == 64 ? fm::launch_few<64>(ma, mw, p, split, st)
                               : fm::launch_few<128>(ma, mw, p, split, st));
}

fm_status fm_ops_test_stall(fm_stall role, int group, long long spin_cycles) {
  OpCheck c{"fm_ops_test_stall"};
  fm::set_thread_error("");
  if (role < FM_STALL_NONE || role > FM_STALL_MMA1)
    return c.fail(FM_ERR_INVALID_ARG, "role %d out of range", (int)role);
  if (group < 0 || spin_cycles < 0)
    return c.fail(FM_ERR_INVALID_ARG, "group %d / spin_cycles %lld is negative", group, spin_cycles);
  fm::t_stall.role = (uint8_t)role;
  fm::t_stall.group = (unsigned)group;
  fm::t_stall.spin = spin_cycles == 0 || spin_cycles > fm::kSpin ? fm::kSpin : (unsigned)spin_cycles;
  return FM_OK;
}

fm_status fm_ops_sync(void* stream) {
  OpCheck c{"fm_ops_sync"};
  fm::set_thread_error("");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  FM_TRY(c.launched(cudaStreamIsCapturing(st, &capture)));
  if (capture != cudaStreamCaptureStatusNone)
    return c.fail(FM_ERR_INVALID_ARG, "the stream is being captured: there is nothing to wait for");
  int device = 0;
  FM_TRY(c.launched(cudaGetDevice(&device)));
  // the copy goes by `stream`, behind its products; a capture of another thread
  // is not this call's business
  unsigned long long word = 0;
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  FM_TRY(c.launched(cudaThreadExchangeStreamCaptureMode(&mode)));
  cudaError_t e = cudaMemcpyFromSymbolAsync(&word, fm::g_ops_err, sizeof(word), 0, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  cudaThreadExchangeStreamCaptureMode(&mode);
  FM_TRY(c.launched(e));
  static thread_local unsigned int seen[64];
  unsigned int& last = seen[device & 63];
  const unsigned int count = (unsigned int)word;
  if (count == last) return FM_OK;
  const unsigned int fresh = count - last;
  last = count;
  return c.fail(FM_ERR_TIMEOUT, "%u device-side waits of fm_gemm_e4m3_b128 gave up (kinds so far 0x%x)", fresh,
                (unsigned int)(word >> 32));
}

#pragma GCC visibility pop
}  // extern "C"
