// The E4M3 block-scaled operators of include/fm_ops.h that are bound by memory:
// residual + RMS norm, the gated activation (both quantise their result),
// the weight quantiser and the multi-axis RoPE.  The matrix product is in
// fm_ops_gemm.cu.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "../../include/fm_ops.h"
#include "fm_ops_check.h"
#include "fm_ops_math.cuh"
#include "fm_ptx.cuh"

namespace fm {
namespace {

// ----------------------------------------------------------------- 8 elements at a time
template <typename T>
struct Pack8;
template <>
struct Pack8<uint16_t> {   // bf16 bits
  uint4 r;
  __device__ __forceinline__ void load(const uint16_t* p) { r = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Pack8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ float to_f(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ float to_f(float f) { return f; }
__device__ __forceinline__ void from_f(uint16_t* p, float v) {
  const __nv_bfloat16 b = __float2bfloat16_rn(v);
  *p = *reinterpret_cast<const uint16_t*>(&b);
}
__device__ __forceinline__ void from_f(float* p, float v) { *p = v; }

// ----------------------------------------------------------------- groups of 128 -> codes + scales
// Half a warp holds one group of 128 values, 8 per lane (a piece), and N such
// groups at once.  a' = max(a, 2^-100) keeps 448 / a' finite, so tiny groups
// give codes and not 0 x inf.  The maxima of the N groups are exchanged
// together (the lane bits 8 and 4 tell whose a lane ends up with), so the two
// divisions are made once for all N and not once for each: they and the
// shuffles were a quarter of the instructions of kernels that are bound by them.
constexpr float kTiny = 7.8886090522101181e-31f;   // 2^-100
template <int N>
struct Groups {
  static_assert(N == 1 || N == 2 || N == 4, "");
  float r, s;              // 448 / a' and a' / 448 of group `mine`
  int mine;

  __device__ __forceinline__ Groups(const float (&y)[N][8], int lane) {
    float a[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      a[i] = fabsf(y[i][0]);
#pragma unroll
      for (int e = 1; e < 7; e += 2) a[i] = max_abs3(a[i], y[i][e], y[i][e + 1]);
      a[i] = fmaxf(a[i], fabsf(y[i][7]));
    }
    float m;
    int o = 8;
    mine = 0;
    if constexpr (N == 4) {
      const bool hi = lane & 8;
      const float s0 = hi ? a[0] : a[2], s1 = hi ? a[1] : a[3];
      a[0] = fmaxf(hi ? a[2] : a[0], __shfl_xor_sync(0xffffffffu, s0, 8));
      a[1] = fmaxf(hi ? a[3] : a[1], __shfl_xor_sync(0xffffffffu, s1, 8));
      mine = hi ? 2 : 0;
      o = 4;
    }
    if constexpr (N >= 2) {
      const bool hi = lane & o;
      const float send = hi ? a[0] : a[1];
      m = fmaxf(hi ? a[1] : a[0], __shfl_xor_sync(0xffffffffu, send, o));
      mine += hi ? 1 : 0;
      o >>= 1;
    } else {
      m = a[0];
    }
    for (; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float t = fmaxf(m, kTiny);
    r = m > 0.f ? __fdiv_rn(448.0f, t) : 3e38f;              // (a zero group: any number)
    s = m > 0.f ? __fdiv_rn(t, 448.0f) : 1.0f;
  }
  // Whether this lane is the one that stores the scale of group `mine`.
  static __device__ __forceinline__ bool writer(int lane) { return (lane & (N == 4 ? 3 : N == 2 ? 7 : 15)) == 0; }
  // 448 / a' of group i, for every lane (all lanes call it).
  __device__ __forceinline__ float factor(int i, int lane) const {
    if constexpr (N == 1) return r;
    const int src = (lane & 16) | (N == 4 ? ((i >> 1) << 3) | ((i & 1) << 2) : i << 3);
    return __shfl_sync(0xffffffffu, r, src);
  }
  // The codes of a piece of group i.
  static __device__ __forceinline__ uint2 codes(float (&y)[8], float f) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) mul2(y[e], y[e + 1], f, f);
    return make_uint2(f32x2_to_e4m3x2(y[0], y[1]) | (f32x2_to_e4m3x2(y[2], y[3]) << 16),
                      f32x2_to_e4m3x2(y[4], y[5]) | (f32x2_to_e4m3x2(y[6], y[7]) << 16));
  }
};

// ----------------------------------------------------------------- residual + RMS norm
// A row stays in the registers of its `wpr` warps between the sum of squares
// and the codes: one pass over memory, 8 elements per lane and piece.  Memory
// bounds it: 38.5 us at 16384 x 2048 bf16 with a residual (6.1 TB/s, 95 % of the
// measured copy rate), 43.2 before the groups were divided together.
struct NormParams {
  const void* x;
  const void* res;
  const uint16_t* gain;
  void* h;
  uint8_t* codes;
  float* scales;
  int64_t ldx, ldr, ldh, ldc, lds;
  float offset, eps;
  int rows, d, wpr;
};

template <typename TX, typename TH, int NP>
__global__ void norm_kernel(const NormParams p) {
  __shared__ float part[32];
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int slot = warp / p.wpr;                              // row of this block
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / (32 * p.wpr)) + slot;
  const bool have = row < p.rows;
  const int t = (warp - slot * p.wpr) * 32 + lane;            // thread of the row
  const int pieces = p.d >> 3, step = p.wpr * 32;
  const TX* x = static_cast<const TX*>(p.x) + row * p.ldx;
  const TH* res = static_cast<const TH*>(p.res) + row * p.ldr;

  float v[NP][8];
  float sq = 0.f, sq1 = 0.f;
  {
    Pack8<TX> px[NP];
    Pack8<TH> pr[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int c = t + i * step;
      if (have && c < pieces) {
        px[i].load(x + c * 8);
        if (p.res != nullptr) pr[i].load(res + c * 8);
      }
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int c = t + i * step;
      if (have && c < pieces) {
        px[i].get(v[i]);
        if (p.res != nullptr) {
          float r[8];
          pr[i].get(r);
#pragma unroll
          for (int e = 0; e < 8; e += 2) add2(v[i][e], v[i][e + 1], r[e], r[e + 1]);
        }
        if (p.h != nullptr) store8(static_cast<TH*>(p.h) + row * p.ldh + c * 8, v[i]);
#pragma unroll
        for (int e = 0; e < 8; e += 2) fma2(sq, sq1, v[i][e], v[i][e + 1], v[i][e], v[i][e + 1]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
      }
    }
  }
  sq += sq1;
#pragma unroll
  for (int o = 16; o; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
  if (p.wpr > 1) {
    if (lane == 0) part[warp] = sq;
    __syncthreads();
    sq = 0.f;
    for (int w = 0; w < p.wpr; ++w) sq += part[slot * p.wpr + w];
  }
  const float rstd = rsqrtf(sq / (float)p.d + p.eps);
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int c = t + i * step;
#pragma unroll
    for (int e = 0; e < 8; e += 2) mul2(v[i][e], v[i][e + 1], rstd, rstd);
    if (p.gain != nullptr) {
      Pack8<uint16_t> pg;
      float g[8];
      pg.r = make_uint4(0, 0, 0, 0);
      if (c < pieces) pg.load(p.gain + c * 8);
      pg.get(g);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        add2(g[e], g[e + 1], p.offset, p.offset);
        mul2(v[i][e], v[i][e + 1], g[e], g[e + 1]);
      }
    } else {
      const float g = 1.f + p.offset;
#pragma unroll
      for (int e = 0; e < 8; e += 2) mul2(v[i][e], v[i][e + 1], g, g);
    }
  }
  const Groups<NP> groups(v, lane);
  if (have) {
    const int first = (t & ~15) + groups.mine * step;          // the group's first piece
    if (Groups<NP>::writer(lane) && first < pieces) p.scales[row * p.lds + (first >> 4)] = groups.s;
  }
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int c = t + i * step;
    const uint2 code = Groups<NP>::codes(v[i], groups.factor(i, lane));
    if (have && c < pieces) *reinterpret_cast<uint2*>(p.codes + row * p.ldc + c * 8) = code;
  }
}

template <typename TX, typename TH>
cudaError_t launch_norm(NormParams p, cudaStream_t st) {
  // One piece of 8 per lane and row needs wpr = d / 256 warps; four pieces per
  // lane quarter that.  Few rows are spread over warps (64 x 1024: one piece 2.1,
  // four 2.8 us; 64 x 4096 2.6, 3.1), many keep four pieces, whose groups share
  // their divisions (16384 x 1024: 24.7, 21.0 us; 16384 x 2048 47.3, 38.2; 4096 x
  // 8192 with two 42.8, 38.4).  Around 512 rows the two differ by 10 % either
  // way.  Rows of less than 1024, whose four pieces are partly empty, lose by it
  // (16384 x 128: 6.6, 10.8 us; 16384 x 512 with two 12.0, 14.1).
  const int pieces = p.d >> 3;
  int np = pieces > 32 * 16 * 2 ? 4 : pieces > 32 * 16 ? 2 : 1;
  if (p.rows > 512) np = 4;
  p.wpr = (pieces + 32 * np - 1) / (32 * np);
  const int rpb = p.wpr >= 8 ? 1 : 8 / p.wpr;
  const unsigned grid = (unsigned)(((int64_t)p.rows + rpb - 1) / rpb);
  const int threads = rpb * p.wpr * 32;
  return np == 1   ? launch_op(norm_kernel<TX, TH, 1>, grid, threads, 0, 1, st, p)
         : np == 2 ? launch_op(norm_kernel<TX, TH, 2>, grid, threads, 0, 1, st, p)
                   : launch_op(norm_kernel<TX, TH, 4>, grid, threads, 0, 1, st, p);
}

// ----------------------------------------------------------------- gated activation
struct GatedParams {
  const void* x;
  uint8_t* codes;
  float* scales;
  int64_t ldx, ldc, lds;
  int rows, f;
  int row_pieces;          // pieces of 8 per row, rounded up to whole groups
  int tiles;               // column tiles of blockDim.x pieces per row, or 0:
  int rpb;                 //   so many whole rows per block
};

// act(g) u with both activations as g / (1 + exp(-t)): SiLU has t = g, and
// (1 + tanh(z)) / 2 = 1 / (1 + exp(-2 z)) makes the tanh form of GELU one with
// t = 2 z, without its cancellation for negative z.  2^x and 1/x are the
// approximate instructions (about 2^-22 each; their forms that keep subnormals
// take three more instructions each).  SiLU's exponent is made to 48 bits: what
// t loses to rounding, up to |t| 2^-24, is l, and 2^l = 1 + l ln 2.  GELU's comes
// from three fp32 operations (8 roundings with its constants).  At 16384 x 4096
// bf16 GELU takes 55.2 us (95 % of the measured copy rate; inputs and outputs that
// are not in L2), SiLU 57.5; with expf and a true division, with one row per
// thread and with subnormals it was 96, 77 and 65.
//
// Far negative gates, whose 1 / (1 + 2^t) is no normal fp32 number (t > 125: SiLU
// below -86.6, GELU below -10), come out as 0 or nearly: they are gated_tail's.
// Their values are below 2^-117 |up|, so that they count only in groups whose
// largest value is as far below an |up| of theirs: gated_kernel compares the two
// for each thread and group, and a warp that has such a group makes its rows again
// (1.3 us of GELU's 55.2, 0.4 of SiLU's; a branch per pair of elements cost 6).
constexpr float kLog2e = 1.4426950408889634f;
template <int ACT>
__device__ __forceinline__ void gated_exponent(float g0, float g1, float& t0, float& t1) {   // -t log2(e)
  t0 = g0, t1 = g1;
  if (ACT == FM_ACT_SILU) {
    mul2(t0, t1, -kLog2e, -kLog2e);
  } else {
    constexpr float c = -2.0f * 0.7978845608028654f * kLog2e;
    float w0 = c, w1 = c;
    mul2(t0, t1, g0, g1);
    fma2(w0, w1, t0, t1, c * 0.044715f, c * 0.044715f);
    t0 = g0, t1 = g1;
    mul2(t0, t1, w0, w1);
  }
}
// l ln 2 for SiLU's exponents t of gates g.
__device__ __forceinline__ void silu_rest(float g0, float g1, float t0, float t1, float& l0, float& l1) {
  constexpr float kLo = (float)(1.4426950408889634074 - (double)1.4426950408889634f);
  l0 = -t0, l1 = -t1;
  fma2(l0, l1, g0, g1, -kLog2e, -kLog2e);
  fma2(l0, l1, g0, g1, -kLo, -kLo);
  mul2(l0, l1, 0.6931471805599453f, 0.6931471805599453f);
}
// g u 2^-t (t > 125, where 1 + 2^t is 2^t), 2^-t as two halves so that it may lie
// below fp32's range where the product does not.
template <int ACT>
__device__ __forceinline__ float gated_tail(float g, float u, float t) {
  float h = -0.5f * t;
  asm("ex2.approx.f32 %0, %0;" : "+f"(h));
  float l0 = 0.f, l1 = 0.f;
  if (ACT == FM_ACT_SILU && h > 0.f) silu_rest(g, g, t, t, l0, l1);
  const float y = (g * h) * (u * h);
  return fmaf(-l0, y, y);
}
// (g0, g1) = act(g) u, far gates included where TAIL.
template <int ACT, bool TAIL>
__device__ __forceinline__ void gated2(float& g0, float& g1, float u0, float u1) {
  float t0, t1;
  gated_exponent<ACT>(g0, g1, t0, t1);
  float e0 = t0, e1 = t1;
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e0));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e1));
  if (ACT == FM_ACT_SILU) {
    float l0, l1;
    silu_rest(g0, g1, t0, t1, l0, l1);
    // beyond 2^126 there is nothing to mend, and l may be anything: the limits are 0 and g
    e0 = fabsf(t0) < 126.f ? fmaf(e0, l0, e0) : e0;
    e1 = fabsf(t1) < 126.f ? fmaf(e1, l1, e1) : e1;
  }
  add2(e0, e1, 1.0f, 1.0f);
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e0));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e1));
  const float far0 = g0, far1 = g1;
  mul2(g0, g1, e0, e1);
  mul2(g0, g1, u0, u1);
  if (TAIL && t0 > 125.f) g0 = gated_tail<ACT>(far0, u0, t0);
  if (TAIL && t1 > 125.f) g1 = gated_tail<ACT>(far1, u1, t1);
}

// A far gate's value is below 2^-117 |up|: its code is 0, and its group's scale is
// another's, where |up| 448 / a' is below this (2^-10 is half the smallest code).
constexpr float kTail = 8.1129638414606682e31f;   // 2^106

// U rows per thread, their loads in flight together.
template <typename T, int ACT, int U>
__global__ void __launch_bounds__(256) gated_kernel(const GatedParams p) {
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 31;
  int64_t row;
  int c, stride = 1;
  bool live = true;
  if (p.tiles) {
    row = (int64_t)(blockIdx.x / (unsigned)p.tiles) * U;
    c = (blockIdx.x % (unsigned)p.tiles) * blockDim.x + threadIdx.x;
  } else {
    const int slot = threadIdx.x / p.row_pieces;     // the block's threads are rounded up to whole warps
    live = slot < p.rpb;
    row = (int64_t)blockIdx.x * p.rpb * U + slot;
    c = threadIdx.x - slot * p.row_pieces;
    stride = p.rpb;
  }
  const bool group = live && (c & ~15) * 8 < p.f;      // this half warp's group has elements; this lane's piece may not
  live = live && c * 8 < p.f;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx + (int64_t)c * 8;
  Pack8<T> a[U], b[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (live && row + u * stride < p.rows) {
      a[u].load(x + (int64_t)u * stride * p.ldx);
      if (ACT != FM_ACT_NONE) b[u].load(x + (int64_t)u * stride * p.ldx + p.f);
    }
  }
  float y[U][8], um[U];                               // um: the largest |up| of a piece
#pragma unroll
  for (int u = 0; u < U; ++u) {
    um[u] = 0.f;
    if (live && row + u * stride < p.rows) {
      a[u].get(y[u]);
      if (ACT != FM_ACT_NONE) {
        float v[8];
        b[u].get(v);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          um[u] = max_abs3(um[u], v[e], v[e + 1]);
          gated2<ACT, false>(y[u][e], y[u][e + 1], v[e], v[e + 1]);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[u][e] = 0.f;
    }
  }
  const Groups<U> groups(y, lane);
  if (group) {
    const int64_t r = row + groups.mine * stride;
    if (Groups<U>::writer(lane) && r < p.rows) p.scales[r * p.lds + (c >> 4)] = groups.s;
  }
  bool tail = false;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t r = row + u * stride;
    const float factor = groups.factor(u, lane);
    const uint2 code = Groups<U>::codes(y[u], factor);
    if (live && r < p.rows) *reinterpret_cast<uint2*>(p.codes + r * p.ldc + (int64_t)c * 8) = code;
    tail |= um[u] * factor > kTail;
  }
  if (ACT != FM_ACT_NONE && __any_sync(0xffffffffu, tail)) {        // rare: x is read again
#pragma unroll 1
    for (int u = 0; u < U; ++u) {
      const int64_t r = row + u * stride;
      float z[1][8];
#pragma unroll
      for (int e = 0; e < 8; ++e) z[0][e] = 0.f;
      if (live && r < p.rows) {
        Pack8<T> px;
        float v[8];
        px.load(x + (int64_t)u * stride * p.ldx);
        px.get(z[0]);
        px.load(x + (int64_t)u * stride * p.ldx + p.f);
        px.get(v);
#pragma unroll
        for (int e = 0; e < 8; e += 2) gated2<ACT, true>(z[0][e], z[0][e + 1], v[e], v[e + 1]);
      }
      const Groups<1> one(z, lane);
      if (group && Groups<1>::writer(lane) && r < p.rows) p.scales[r * p.lds + (c >> 4)] = one.s;
      const uint2 code = Groups<1>::codes(z[0], one.r);
      if (live && r < p.rows) *reinterpret_cast<uint2*>(p.codes + r * p.ldc + (int64_t)c * 8) = code;
    }
  }
}

template <typename T, int U>
cudaError_t launch_gated_u(GatedParams p, fm_act act, cudaStream_t st) {
  int threads = 256;
  int64_t grid;
  if (p.row_pieces >= 256) {
    p.tiles = (p.row_pieces + 255) / 256;
    p.rpb = 0;
    grid = ((int64_t)p.rows + U - 1) / U * p.tiles;
  } else {
    p.tiles = 0;
    p.rpb = 256 / p.row_pieces;
    threads = (p.rpb * p.row_pieces + 31) & ~31;
    grid = ((int64_t)p.rows + p.rpb * U - 1) / (p.rpb * U);
  }
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  return act == FM_ACT_SILU        ? launch_op(gated_kernel<T, FM_ACT_SILU, U>, (unsigned)grid, threads, 0, 1, st, p)
         : act == FM_ACT_GELU_TANH ? launch_op(gated_kernel<T, FM_ACT_GELU_TANH, U>, (unsigned)grid, threads, 0, 1, st, p)
                                   : launch_op(gated_kernel<T, FM_ACT_NONE, U>, (unsigned)grid, threads, 0, 1, st, p);
}

template <typename T>
cudaError_t launch_gated(GatedParams p, fm_act act, int sms, cudaStream_t st) {
  p.row_pieces = ((p.f + 127) / 128) * 16;
  // Where there are pieces for several waves of threads, each takes UU of them
  // (SiLU, bf16, f 4096: 592 rows, a quarter of the bound, 4.6 us with one and with
  // four; at the bound 13.2, 11.1; at four times it 45.4, 34.0).
  constexpr int UU = sizeof(T) == 2 ? 4 : 2;
  return (int64_t)p.rows * p.row_pieces >= (int64_t)sms * 2048 * UU ? launch_gated_u<T, UU>(p, act, st)
                                                                    : launch_gated_u<T, 1>(p, act, st);
}

// ----------------------------------------------------------------- weight quantiser
// One block of threads per 128 x 128 block of the weight (a set-up call: two
// reads of the block, the second from L1).
__global__ void __launch_bounds__(256) quantize_weight_kernel(const uint16_t* __restrict__ w, int64_t ldw, int n, int k,
                                                              uint8_t* __restrict__ codes, int64_t ldc,
                                                              float* __restrict__ scales, int64_t lds) {
  __shared__ float part[8];
  grid_dep_launch();
  grid_dep_wait();
  const unsigned gk = (unsigned)((k + 127) / 128);
  const int64_t n0 = (int64_t)(blockIdx.x / gk) * 128;
  const int k0 = (int)(blockIdx.x % gk) * 128;
  const int col = k0 + (threadIdx.x & 127);
  const int r0 = threadIdx.x >> 7;
  float a = 0.f;
  if (col < k)
    for (int r = r0; r < 128 && n0 + r < n; r += 2) a = fmaxf(a, fabsf(to_f(w[(n0 + r) * ldw + col])));
  for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = a;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, part[i]);
  const float s = a > 0.f ? __fdiv_rn(fmaxf(a, kTiny), 448.0f) : 1.0f;
  if (threadIdx.x == 0) scales[(n0 / 128) * lds + blockIdx.x % gk] = s;
  if (col < k)
    for (int r = r0; r < 128 && n0 + r < n; r += 2)
      codes[(n0 + r) * ldc + col] =
          (uint8_t)__nv_cvt_float_to_fp8(__fdiv_rn(to_f(w[(n0 + r) * ldw + col]), s), __NV_SATFINITE, __NV_E4M3);
}

// ----------------------------------------------------------------- multi-axis RoPE
// A block takes whole rows, so that what is in flight is contiguous, and makes
// their cosines and sines once, in shared memory, while its loads are on the
// way: a thread owns V consecutive pairs of kHeads heads of one row.  The angle
// is reduced to a fraction of a turn in 64 bits (positions x frequency pass 2^20
// turns, where fp32 has no digits left).  16384 rows of 16 + 2 + 2 heads of 128
// bf16 take 32 us (81 % of the measured copy rate; registers leave 27 % of the
// warps), 306 rows 2.5.
constexpr int kMaxPairs = 128;
struct RopeParams {
  const void* x;
  const int32_t* pos;
  void *q, *k, *v;
  int64_t ldx, ldp, ldq, ldk, ldv;
  int rows, nq, nkv, hd, n;
  int parts, tb;                      // shares of the heads; rows per block
  double turn[kMaxPairs];             // frequency in turns per position
  uint8_t axis[kMaxPairs];
};

// V consecutive elements, 16 or 2 V / 4 V bytes at a time.
template <int BYTES>
struct Word;
template <>
struct Word<16> { using type = uint4; };
template <>
struct Word<8> { using type = uint2; };
template <>
struct Word<4> { using type = uint32_t; };
template <>
struct Word<2> { using type = uint16_t; };
template <typename T, int V>
struct Run {
  static constexpr int kBytes = V * (int)sizeof(T), kWord = kBytes < 16 ? kBytes : 16;
  using W = typename Word<kWord>::type;
  union {
    W w[kBytes / kWord];
    T e[V];
  };
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kBytes / kWord; ++i) w[i] = reinterpret_cast<const W*>(p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < kBytes / kWord; ++i) reinterpret_cast<W*>(p)[i] = w[i];
  }
};
template <typename T, int V>
__device__ __forceinline__ void copy_v(const T* src, T* dst) {
  Run<T, V> r;
  r.load(src);
  r.store(dst);
}

constexpr int kHeads = 3;
template <typename T, int V>
__global__ void __launch_bounds__(512) rope_kernel(const __grid_constant__ RopeParams p) {
  extern __shared__ float4 table[];
  __shared__ double turn[kMaxPairs];
  __shared__ uint8_t axis[kMaxPairs];
  grid_dep_launch();
  for (int j = threadIdx.x; j < p.n; j += blockDim.x) {
    turn[j] = p.turn[j];
    axis[j] = p.axis[j];
  }
  __syncthreads();
  grid_dep_wait();
  const int n = p.n, hd = p.hd, heads = p.nq + p.nkv;
  const int per = n / V;                                      // threads per row and share of the heads
  const int slot = (int)threadIdx.x / per, j = ((int)threadIdx.x - slot * per) * V;
  const int r = slot / p.parts, part = slot - r * p.parts;
  const int vals = p.v != nullptr ? p.nkv * hd : 0, ve = part * n + j;    // this thread's first value element
  const int size = (p.tb * n + 3) & ~3;
  int buf = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * p.tb; row0 < p.rows; row0 += (int64_t)gridDim.x * p.tb, buf ^= 1) {
    const int here = (int)(p.rows - row0 < p.tb ? p.rows - row0 : p.tb);
    const bool mine = r < here;
    const int64_t row = row0 + (mine ? r : 0);
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    T* q = static_cast<T*>(p.q);
    T* k = static_cast<T*>(p.k);
    if (q != nullptr) q += row * p.ldq;
    if (k != nullptr) k += row * p.ldk - (int64_t)p.nq * hd;
    Run<T, V> a[kHeads], b[kHeads], v;
    auto bring = [&](int h0) {
#pragma unroll
      for (int u = 0; u < kHeads; ++u) {
        const int h = h0 + u * p.parts;
        if (h < heads && (h < p.nq ? q : k) != nullptr) {
          a[u].load(x + h * hd + j);
          b[u].load(x + h * hd + j + n);
        }
      }
    };
    if (mine) bring(part);
    if (mine && ve < vals) v.load(x + heads * hd + ve);
    float* cs = reinterpret_cast<float*>(table) + buf * 2 * size;          // [tb][n] cosines, then the sines
    for (int i = threadIdx.x; i < here * n; i += blockDim.x) {
      const int w = i / n, e = i - w * n;
      const double z = (double)p.pos[(int64_t)axis[e] * p.ldp + row0 + w] * turn[e];
      sincospif(2.0f * (float)(z - rint(z)), &cs[size + i], &cs[i]);
    }
    __syncthreads();                                          // (the other buffer's readers are one barrier behind)
    if (!mine) continue;
    float c[V], s[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      c[e] = cs[r * n + j + e];
      s[e] = cs[size + r * n + j + e];
    }
    auto turn_head = [&](int h, Run<T, V>& lo_, Run<T, V>& hi_) {
      T* out = (h < p.nq ? q : k) + h * hd;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        // spelled out, so that every width rounds alike
        const float lo = to_f(lo_.e[e]), hi = to_f(hi_.e[e]);
        from_f(&lo_.e[e], __fmaf_rn(lo, c[e], -__fmul_rn(hi, s[e])));
        from_f(&hi_.e[e], __fmaf_rn(hi, c[e], __fmul_rn(lo, s[e])));
      }
      lo_.store(out + j);
      hi_.store(out + j + n);
      for (int e = 2 * n + j; e < hd; e += n) copy_v<T, V>(x + h * hd + e, out + e);
    };
    for (int h0 = part; h0 < heads; h0 += kHeads * p.parts) {
      if (h0 != part) bring(h0);
#pragma unroll
      for (int u = 0; u < kHeads; ++u) {
        const int h = h0 + u * p.parts;
        if (h < heads && (h < p.nq ? q : k) != nullptr) turn_head(h, a[u], b[u]);
      }
    }
    T* vo = static_cast<T*>(p.v) + row * p.ldv;
    if (ve < vals) v.store(vo + ve);
    for (int e = ve + p.parts * n; e < vals; e += p.parts * n) copy_v<T, V>(x + heads * hd + e, vo + e);
  }
}

template <typename T>
cudaError_t launch_rope(RopeParams& p, int v, int sms, cudaStream_t st) {
  const int per = p.n / v, heads = p.nq + p.nkv;
  // One head per thread where rows are few, kHeads or a few times that where
  // they fill the GPU: as many shares of the heads as bring 1536 threads to an SM
  // (16 + 2 heads of 128: 306 rows in 18 shares 2.5, in 6 2.7 us; 2048 rows in 6
  // 7.6, in 2 9.5, in 18 10.6; 16384 rows in 2 31.9, in 1 38.4, in 9 45.0).  The
  // choice is off by up to 30 % around 1024 rows (18 shares 5.8, 6 4.5).  Whole
  // rows up to about 128 threads per block (16384 rows: 64 threads 32.1, 128 31.9,
  // 256 38.3).
  int64_t parts = ((int64_t)sms * 1536 + (int64_t)p.rows * per - 1) / ((int64_t)p.rows * per);
  const int64_t most_parts = (int64_t)p.rows * per * heads < (int64_t)sms * 1024 ? heads : (heads + kHeads - 1) / kHeads;
  if (parts > most_parts) parts = most_parts;
  if (parts * per > 512) parts = 512 / per;
  p.parts = parts < 1 ? 1 : (int)parts;
  p.tb = 128 / (p.parts * per);
  if (p.tb < 1) p.tb = 1;
  if ((int64_t)p.rows < (int64_t)p.tb * sms) p.tb = 1;
  const int threads = (p.tb * p.parts * per + 31) & ~31;
  const int64_t tiles = ((int64_t)p.rows + p.tb - 1) / p.tb, most = (int64_t)sms * (2048 / threads);
  const int64_t grid = tiles < most ? tiles : most;
  const size_t smem = 4 * (size_t)((p.tb * p.n + 3) & ~3) * sizeof(float);   // at most 1024 pairs, 16 KB
  return v == 8   ? launch_op(rope_kernel<T, 8>, (unsigned)grid, threads, smem, 1, st, p)
         : v == 4 ? launch_op(rope_kernel<T, 4>, (unsigned)grid, threads, smem, 1, st, p)
         : v == 2 ? launch_op(rope_kernel<T, 2>, (unsigned)grid, threads, smem, 1, st, p)
                  : launch_op(rope_kernel<T, 1>, (unsigned)grid, threads, smem, 1, st, p);
}

// Whether `n` rows at `p` start on `bytes`-byte boundaries (NULL: nothing to ask).
bool rows_on(size_t bytes, const void* p, int64_t ld, size_t elem, int n) {
  return p == nullptr || ((uintptr_t)p % bytes == 0 && (n <= 1 || ((uint64_t)ld * elem) % bytes == 0));
}

}  // namespace

// ----------------------------------------------------------------- argument checks
fm_status OpCheck::fail(fm_status st, const char* fmt, ...) {
  char msg[320];
  const int at = snprintf(msg, sizeof(msg), "%s: ", call);
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg + at, sizeof(msg) - at, fmt, ap);
  va_end(ap);
  set_thread_error(msg);
  return st;
}

fm_status OpCheck::rows(const void* p, const char* name, int64_t ld, int64_t width, int n, size_t elem, size_t align) {
  if (p == nullptr) return fail(FM_ERR_INVALID_ARG, "%s is NULL", name);
  if (n > 1 && ld < width)
    return fail(FM_ERR_INVALID_ARG, "%s: row stride %lld is below the row's %lld elements", name, (long long)ld,
                (long long)width);
  if (((uintptr_t)p % align) != 0 || (n > 1 && ((uint64_t)ld * elem) % align != 0))
    return fail(FM_ERR_INVALID_ARG, "%s: rows must start on %d-byte boundaries", name, (int)align);
  ptr[count] = p;
  ptr_name[count++] = name;
  return FM_OK;
}

fm_status OpCheck::memory() {
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(FM_ERR_CUDA, "no usable current CUDA device (%s)", cudaGetErrorString(e));
  }
  for (int i = 0; i < count; ++i) {
    cudaPointerAttributes at;
    e = cudaPointerGetAttributes(&at, ptr[i]);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return fail(FM_ERR_CUDA, "%s: cudaPointerGetAttributes: %s", ptr_name[i], cudaGetErrorString(e));
    }
    if (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged)
      return fail(FM_ERR_INVALID_ARG, "%s is not device memory", ptr_name[i]);
    if (at.type == cudaMemoryTypeDevice && at.device != device)
      return fail(FM_ERR_INVALID_ARG, "%s is on device %d, the current device is %d", ptr_name[i], at.device, device);
  }
  return FM_OK;
}

fm_status OpCheck::launched(cudaError_t e) {
  if (e == cudaSuccess) return FM_OK;
  cudaGetLastError();
  return fail(FM_ERR_CUDA, "%s", cudaGetErrorString(e));
}

int sm_count(int device) {
  static std::atomic<int> known[64];
  if (device >= 0 && device < 64) {
    const int k = known[device].load(std::memory_order_relaxed);
    if (k > 0) return k;
  }
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || n < 1) {
    cudaGetLastError();
    n = 148;
  }
  if (device >= 0 && device < 64) known[device].store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace fm

using fm::OpCheck;

extern "C" {
#pragma GCC visibility push(default)

fm_status fm_add_rmsnorm_e4m3(const void* x, fm_dtype x_type, int64_t ldx, const void* residual, fm_dtype h_type,
                              int64_t ldr, const uint16_t* gain, float gain_offset, float eps, int rows, int d,
                              void* h_out, int64_t ldh, uint8_t* codes, int64_t ldc, float* scales, int64_t lds,
                              void* stream) {
  OpCheck c{"fm_add_rmsnorm_e4m3"};
  fm::set_thread_error("");
  if ((x_type != FM_BF16 && x_type != FM_F32) || (h_type != FM_BF16 && h_type != FM_F32))
    return c.fail(FM_ERR_UNSUPPORTED, "x_type %d / h_type %d: FM_BF16 or FM_F32", (int)x_type, (int)h_type);
  if (rows < 0 || d < 16 || d > 16384 || d % 16 != 0)
    return c.fail(FM_ERR_INVALID_ARG, "rows %d / d %d out of range (d a multiple of 16, 16 .. 16384)", rows, d);
  if (!(eps >= 0.f)) return c.fail(FM_ERR_INVALID_ARG, "eps must not be negative");
  if (rows == 0) return FM_OK;
  const size_t xs = x_type == FM_F32 ? 4 : 2, hs = h_type == FM_F32 ? 4 : 2;
  FM_TRY(c.rows(x, "x", ldx, d, rows, xs, 16));
  if (residual != nullptr) FM_TRY(c.rows(residual, "residual", ldr, d, rows, hs, 16));
  if (gain != nullptr) FM_TRY(c.rows(gain, "gain", d, d, 1, 2, 16));
  if (h_out != nullptr) FM_TRY(c.rows(h_out, "h_out", ldh, d, rows, hs, 16));
  FM_TRY(c.rows(codes, "codes", ldc, d, rows, 1, 16));
  FM_TRY(c.rows(scales, "scales", lds, (d + 127) / 128, rows, 4, 4));
  FM_TRY(c.memory());
  fm::NormParams p{x, residual, gain, h_out, codes, scales, ldx, ldr, ldh, ldc, lds, gain_offset, eps, rows, d, 0};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (x_type == FM_BF16)
    return c.launched(h_type == FM_BF16 ? fm::launch_norm<uint16_t, uint16_t>(p, st)
                                        : fm::launch_norm<uint16_t, float>(p, st));
  return c.launched(h_type == FM_BF16 ? fm::launch_norm<float, uint16_t>(p, st) : fm::launch_norm<float, float>(p, st));
}

fm_status fm_gated_e4m3(const void* x, fm_dtype x_type, int64_t ldx, fm_act act, int rows, int f, uint8_t* codes,
                        int64_t ldc, float* scales, int64_t lds, void* stream) {
  OpCheck c{"fm_gated_e4m3"};
  fm::set_thread_error("");
  if (x_type != FM_BF16 && x_type != FM_F32)
    return c.fail(FM_ERR_UNSUPPORTED, "x_type %d: FM_BF16 or FM_F32", (int)x_type);
  if (act != FM_ACT_NONE && act != FM_ACT_SILU && act != FM_ACT_GELU_TANH)
    return c.fail(FM_ERR_UNSUPPORTED, "act %d: FM_ACT_NONE, FM_ACT_SILU or FM_ACT_GELU_TANH", (int)act);
  if (rows < 0 || f < 16 || f > (1 << 20) || f % 16 != 0)
    return c.fail(FM_ERR_INVALID_ARG, "rows %d / f %d out of range (f a multiple of 16, 16 .. 2^20)", rows, f);
  if ((int64_t)rows * ((f + 2047) / 2048) > 0x7FFFFFFF)
    return c.fail(FM_ERR_INVALID_ARG, "rows %d x f %d is more than one launch takes", rows, f);
  if (rows == 0) return FM_OK;
  FM_TRY(c.rows(x, "x", ldx, act == FM_ACT_NONE ? f : 2 * (int64_t)f, rows, x_type == FM_F32 ? 4 : 2, 16));
  FM_TRY(c.rows(codes, "codes", ldc, f, rows, 1, 16));
  FM_TRY(c.rows(scales, "scales", lds, (f + 127) / 128, rows, 4, 4));
  FM_TRY(c.memory());
  fm::GatedParams p{x, codes, scales, ldx, ldc, lds, rows, f, 0, 0, 0};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int sms = fm::sm_count(c.device);
  return c.launched(x_type == FM_BF16 ? fm::launch_gated<uint16_t>(p, act, sms, st)
                                      : fm::launch_gated<float>(p, act, sms, st));
}

fm_status fm_quantize_weight_e4m3_b128(const uint16_t* w, int64_t ldw, int n, int k, uint8_t* codes, int64_t ldc,
                                       float* scales, int64_t lds, void* stream) {
  OpCheck c{"fm_quantize_weight_e4m3_b128"};
  fm::set_thread_error("");
  if (n < 0 || k < 0) return c.fail(FM_ERR_INVALID_ARG, "n %d / k %d negative", n, k);
  if (n == 0 || k == 0) return FM_OK;
  const int64_t gn = ((int64_t)n + 127) / 128, gk = ((int64_t)k + 127) / 128;
  if (gn * gk > 0x7FFFFFFF) return c.fail(FM_ERR_INVALID_ARG, "n %d x k %d is more than one launch takes", n, k);
  FM_TRY(c.rows(w, "w", ldw, k, n, 2, 2));
  FM_TRY(c.rows(codes, "codes", ldc, k, n, 1, 1));
  FM_TRY(c.rows(scales, "scales", lds, gk, (int)gn, 4, 4));
  FM_TRY(c.memory());
  return c.launched(fm::launch_op(fm::quantize_weight_kernel, (unsigned)(gn * gk), 256, 0, 1,
                                  static_cast<cudaStream_t>(stream), w, ldw, n, k, codes, ldc, scales, lds));
}

fm_status fm_rope_axes(const void* x, fm_dtype type, int64_t ldx, int rows, int n_q, int n_kv, int head_dim,
                       const int32_t* positions, int64_t ldp, int n_axes, const uint8_t* pair_axis,
                       const double* pair_freq, int n_pairs, void* q_out, int64_t ldq, void* k_out, int64_t ldk,
                       void* v_out, int64_t ldv, void* stream) {
  OpCheck c{"fm_rope_axes"};
  fm::set_thread_error("");
  if (type != FM_BF16 && type != FM_F32) return c.fail(FM_ERR_UNSUPPORTED, "type %d: FM_BF16 or FM_F32", (int)type);
  if (rows < 0 || n_q < 0 || n_kv < 0 || n_q > 1024 || n_kv > 1024)
    return c.fail(FM_ERR_INVALID_ARG, "rows %d / n_q %d / n_kv %d out of range (0 .. 1024 heads)", rows, n_q, n_kv);
  if (head_dim < 2 || head_dim > 256 || head_dim % 2 != 0 || n_pairs < 1 || n_pairs > head_dim / 2)
    return c.fail(FM_ERR_INVALID_ARG, "head_dim %d / n_pairs %d out of range (head_dim even, 2 .. 256; 1 .. head_dim/2 pairs)",
                  head_dim, n_pairs);
  if (n_axes < 1 || n_axes > 8) return c.fail(FM_ERR_INVALID_ARG, "n_axes %d out of range (1 .. 8)", n_axes);
  if (pair_axis == nullptr || pair_freq == nullptr)
    return c.fail(FM_ERR_INVALID_ARG, "pair_axis and pair_freq must be host arrays, not NULL");
  fm::RopeParams p;
  for (int j = 0; j < n_pairs; ++j) {
    if (pair_axis[j] >= n_axes)
      return c.fail(FM_ERR_INVALID_ARG, "pair %d: axis %d of %d", j, (int)pair_axis[j], n_axes);
    if (!std::isfinite(pair_freq[j])) return c.fail(FM_ERR_INVALID_ARG, "pair %d: frequency is not finite", j);
    p.axis[j] = pair_axis[j];
    p.turn[j] = pair_freq[j] * 0.15915494309189535;   // 1 / (2 pi)
  }
  for (int j = n_pairs; j < fm::kMaxPairs; ++j) {
    p.axis[j] = 0;
    p.turn[j] = 0.0;
  }
  if (n_q == 0) q_out = nullptr;
  if (n_kv == 0) k_out = v_out = nullptr;
  if (rows == 0 || (q_out == nullptr && k_out == nullptr && v_out == nullptr)) return FM_OK;
  const size_t es = type == FM_F32 ? 4 : 2;
  const int64_t wq = (int64_t)n_q * head_dim, wk = (int64_t)n_kv * head_dim;
  FM_TRY(c.rows(x, "x", ldx, wq + (v_out != nullptr ? 2 : 1) * wk, rows, es, es));
  FM_TRY(c.rows(positions, "positions", ldp, rows, n_axes, 4, 4));
  if (q_out != nullptr) FM_TRY(c.rows(q_out, "q_out", ldq, wq, rows, es, es));
  if (k_out != nullptr) FM_TRY(c.rows(k_out, "k_out", ldk, wk, rows, es, es));
  if (v_out != nullptr) FM_TRY(c.rows(v_out, "v_out", ldv, wk, rows, es, es));
  FM_TRY(c.memory());
  p.x = x; p.pos = positions; p.q = q_out; p.k = k_out; p.v = v_out;
  p.ldx = ldx; p.ldp = ldp; p.ldq = ldq; p.ldk = ldk; p.ldv = ldv;
  p.rows = rows; p.nq = n_q; p.nkv = n_kv; p.hd = head_dim; p.n = n_pairs; p.parts = p.tb = 1;
  // the widest run that divides the pairs and the head and that every row allows
  int v = 8;
  for (; v > 1; v /= 2) {
    const size_t on = v * es < 16 ? v * es : 16;
    if (head_dim % v == 0 && n_pairs % v == 0 && fm::rows_on(on, x, ldx, es, rows) &&
        fm::rows_on(on, q_out, ldq, es, rows) && fm::rows_on(on, k_out, ldk, es, rows) &&
        fm::rows_on(on, v_out, ldv, es, rows))
      break;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int sms = fm::sm_count(c.device);
  return c.launched(type == FM_BF16 ? fm::launch_rope<uint16_t>(p, v, sms, st) : fm::launch_rope<float>(p, v, sms, st));
}

#pragma GCC visibility pop
}  // extern "C"
