// Argument checks shared by the entry points of include/fm_ops.h.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <utility>

#include "../../include/fm_ops.h"
#include "fm_launch.h"

namespace fm {

struct OpCheck {
  const char* call;
  int device = -1;               // set by memory()
  int count = 0;
  const void* ptr[8] = {};
  const char* ptr_name[8] = {};

  // Sets the thread's error text ("<call>: ...") and returns `st`.
  fm_status fail(fm_status st, const char* fmt, ...);
  // `n` rows of `width` elements of `elem` bytes, `ld` elements apart, start on
  // `align`-byte boundaries (one row: any ld); host arithmetic only.
  fm_status rows(const void* p, const char* name, int64_t ld, int64_t width, int n, size_t elem, size_t align);
  // Every pointer given to rows() is device memory on the current device.
  fm_status memory();
  // FM_OK, or FM_ERR_CUDA with the error's text (and the error cleared).
  fm_status launched(cudaError_t e);
};

// Launches with programmatic dependent launch (every kernel of these operators
// lets its successor start at once and touches memory only after
// griddepcontrol.wait, so set-up overlaps the predecessor's end), in clusters of
// `cluster` blocks.
template <typename... Params, typename... Args>
cudaError_t launch_op(void (*kernel)(Params...), unsigned grid, int block, size_t smem, int cluster, cudaStream_t st,
                      Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3((unsigned)block, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Multiprocessors of `device`.
int sm_count(int device);

}  // namespace fm

// Leaves a call with the first status that is not FM_OK.
#define FM_TRY(expr)              \
  do {                            \
    const fm_status st_ = (expr); \
    if (st_ != FM_OK) return st_; \
  } while (0)
