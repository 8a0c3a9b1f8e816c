// fm_gemm_e4m3_b128: E4M3 x E4M3 with fp32 scales per 128 inputs of a row (a)
// and per 128 x 128 block (w).
//
//   out[i][j] = sum_g sa[i][g] sw[j/128][g] sum_{c in g} a[i][c] w[j][c]
//
// The scales are arbitrary fp32 numbers, so the tensor cores can only sum
// inside a group (K = 128: four kind::f8f6f4 MMAs into a fresh TMEM
// accumulator); the groups are scaled and summed in the registers of the
// epilogue warps.  TMEM holds two accumulators, so the MMAs of a group run
// while the one before is read.
//
// Operands come by tiled TMA (128-byte rows, SW128), zero-filled outside the
// matrices: ragged m, n and the last group of k need no code of their own.
#include <cuda.h>
#include <cuda_bf16.h>

#include <cstdint>

#include "../../include/fm_ops.h"
#include "fm_ops_check.h"
#include "fm_ptx.cuh"

namespace fm {
namespace {

// Device-side timeouts since the last fm_ops_sync on this device.
__device__ unsigned int g_ops_err;

constexpr long long kSpin = 4000000000ll;       // ~2 s of SM cycles
constexpr int kStages = 5;
constexpr int kTileA = 128 * 128, kTileW = 128 * 128, kStage = kTileA + kTileW;
constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + 256;
constexpr int kThreads = 192;

struct GemmParams {
  const float *sa, *sw;
  const uint16_t* bias;
  void* out;
  int64_t ldsa, ldsw, ldo;
  int m, n, groups, f32;
};

// 2-D tiled load of a [128 rows][128 bytes] box at (column c0, row c1).
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* tmap, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(tmap), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}

__global__ void __launch_bounds__(kThreads, 1)
gemm_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mw,
            const __grid_constant__ GemmParams p) {
  extern __shared__ uint8_t raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + (size_t)kStages * kStage);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;     // [2]
  uint64_t* tempty = tfull + 2;          // [2]
  uint64_t* drain = tempty + 2;
  uint32_t* slot = reinterpret_cast<uint32_t*>(drain + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&tfull[b]), 1);
      mbar_init(smem_u32(&tempty[b]), 4);
    }
    mbar_init(smem_u32(drain), 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(slot), 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  const unsigned mt = (unsigned)((p.m + 127) / 128);
  const int m0 = (int)(blockIdx.x % mt) * 128, n0 = (int)(blockIdx.x / mt) * 128;

  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      for (; it < p.groups; ++it) {
        const int s = it % kStages;
        if (it >= kStages && !mbar_wait(smem_u32(&empty[s]), ((it / kStages) & 1) ^ 1, kSpin)) {
          atomicOr(&g_ops_err, 1u);
          break;
        }
        const uint32_t dst = smem_u32(ring + (size_t)s * kStage), bar = smem_u32(&full[s]);
        mbar_arrive_expect_tx(bar, kStage);
        tma_load_2d(dst, &ma, it * 128, m0, bar);
        tma_load_2d(dst + kTileA, &mw, it * 128, n0, bar);
      }
      // every issued copy lands before the block may exit
      for (int j = it > kStages ? it - kStages : 0; j < it; ++j)
        mbar_wait(smem_u32(&full[j % kStages]), (j / kStages) & 1, kSpin);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3(128, 128);
      for (int it = 0; it < p.groups; ++it) {
        const int s = it % kStages, b = it & 1;
        if ((it >= 2 && !mbar_wait(smem_u32(&tempty[b]), ((it >> 1) - 1) & 1, kSpin)) ||
            !mbar_wait(smem_u32(&full[s]), (it / kStages) & 1, kSpin)) {
          atomicOr(&g_ops_err, 2u);
          break;
        }
        tc_fence_after();
        const uint32_t a = smem_u32(ring + (size_t)s * kStage);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mma_e4m3(tmem + b * 128, desc_sw128(a + j * 32), desc_sw128(a + kTileA + j * 32), idesc, j != 0);
        mma_commit(smem_u32(&empty[s]));
        mma_commit(smem_u32(&tfull[b]));
      }
      mma_commit(smem_u32(drain));             // every MMA is done before TMEM is released
      mbar_wait(smem_u32(drain), 0, kSpin);
    }
  } else {
    const int row = 32 * (warp & 3) + lane;    // TMEM lane
    const int i = m0 + row;
    const bool valid = i < p.m;
    const uint32_t ta = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const float* sa = p.sa + (int64_t)i * p.ldsa;
    const float* sw = p.sw + (int64_t)(n0 >> 7) * p.ldsw;
    float acc[128];
#pragma unroll
    for (int c = 0; c < 128; ++c) acc[c] = 0.f;
    bool ok = true;
    for (int it = 0; it < p.groups; ++it) {
      const int b = it & 1;
      const float s = valid ? sa[it] * sw[it] : 0.f;
      // every lane of the warp gets the same answer: the barrier is shared
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&tfull[b]), (it >> 1) & 1, kSpin));
      if (!ok) {
        if (lane == 0) atomicOr(&g_ops_err, 4u);
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        float v[16];
        tmem_ld16(ta + b * 128 + q * 16, v);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[q * 16 + e] = fmaf(v[e], s, acc[q * 16 + e]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&tempty[b]));
    }
    if (ok && valid) {
#pragma unroll
      for (int c = 0; c < 128; ++c) {
        const int j = n0 + c;
        if (j < p.n) {
          float v = acc[c];
          if (p.bias != nullptr) v += __uint_as_float((uint32_t)p.bias[j] << 16);
          if (p.f32)
            static_cast<float*>(p.out)[(int64_t)i * p.ldo + j] = v;
          else
            static_cast<__nv_bfloat16*>(p.out)[(int64_t)i * p.ldo + j] = __float2bfloat16_rn(v);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

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

}  // namespace
}  // namespace fm

using fm::OpCheck;

#define FM_TRY(expr)              \
  do {                            \
    const fm_status st_ = (expr); \
    if (st_ != FM_OK) return st_; \
  } while (0)

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
  if (tiles > 0x7FFFFFFF || n > 0x7FFFFF00 || m > 0x7FFFFF00 || k > 0x7FFFFF00)
    return c.fail(FM_ERR_INVALID_ARG, "m %d x n %d x k %d is more than one launch takes", m, n, k);
  FM_TRY(c.rows(a, "a", lda, k, m, 1, 16));
  FM_TRY(c.rows(sa, "sa", ldsa, groups, m, 4, 4));
  FM_TRY(c.rows(w, "w", ldw, k, n, 1, 16));
  FM_TRY(c.rows(sw, "sw", ldsw, groups, (n + 127) / 128, 4, 4));
  if (bias != nullptr) FM_TRY(c.rows(bias, "bias", n, n, 1, 2, 2));
  FM_TRY(c.rows(out, "out", ldo, n, m, out_type == FM_F32 ? 4 : 2, out_type == FM_F32 ? 4 : 2));
  FM_TRY(c.memory());
  CUtensorMap ma, mw;
  if (!fm::codes_map(&ma, a, lda, m, k, 128) || !fm::codes_map(&mw, w, ldw, n, k, 128))
    return c.fail(FM_ERR_CUDA, "the tensor maps of a and w were refused (m %d, n %d, k %d, strides %lld, %lld)", m, n, k,
                  (long long)lda, (long long)ldw);
  FM_TRY(c.launched(cudaFuncSetAttribute(fm::gemm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)fm::kSmem)));
  fm::GemmParams p{sa, sw, bias, out, ldsa, ldsw, ldo, m, n, (int)groups, out_type == FM_F32};
  fm::gemm_kernel<<<(unsigned)tiles, fm::kThreads, fm::kSmem, static_cast<cudaStream_t>(stream)>>>(ma, mw, p);
  return c.launched(cudaGetLastError());
}

fm_status fm_ops_sync(void* stream) {
  OpCheck c{"fm_ops_sync"};
  fm::set_thread_error("");
  FM_TRY(c.launched(cudaStreamSynchronize(static_cast<cudaStream_t>(stream))));
  unsigned int err = 0;
  FM_TRY(c.launched(cudaMemcpyFromSymbol(&err, fm::g_ops_err, sizeof(err))));
  if (err == 0) return FM_OK;
  const unsigned int zero = 0;
  FM_TRY(c.launched(cudaMemcpyToSymbol(fm::g_ops_err, &zero, sizeof(zero))));
  return c.fail(FM_ERR_TIMEOUT, "a device-side wait of fm_gemm_e4m3_b128 gave up (code 0x%x)", err);
}

#pragma GCC visibility pop
}  // extern "C"
