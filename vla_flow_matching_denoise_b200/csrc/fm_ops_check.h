// Argument checks shared by the entry points of include/fm_ops.h.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

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

// Multiprocessors of `device`.
int sm_count(int device);

}  // namespace fm
