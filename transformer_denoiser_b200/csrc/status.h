// Status codes, the calling thread's error message and the device error word of the
// kernel-level entry points, shared by the files that implement the C ABI.
#pragma once

#include <cuda_runtime.h>

#include "../../include/kimodo.h"
#include "common.cuh"

namespace kd {

// Records the message of a failure on the calling thread and returns `code`.
int set_error(int code, const char* fmt, ...);
void clear_error();
const char* last_error();

bool is_device_memory(const void* p);

// Name of a kernel stage recorded in DevError::where.
const char* where_name(int where);

// Error word of the kernel-level entry points on the current device (no allocation).
DevError* kernel_error_word();

}  // namespace kd

#define KD_CUDA(call)                                                                              \
  do {                                                                                             \
    cudaError_t e_ = (call);                                                                       \
    if (e_ != cudaSuccess)                                                                         \
      return kd::set_error(e_ == cudaErrorMemoryAllocation ? KIMODO_ENOMEM : KIMODO_ECUDA, "%s: %s (%s:%d)", \
                           #call, cudaGetErrorString(e_), __FILE__, __LINE__);                     \
  } while (0)

#define KD_TRY(call)        \
  do {                      \
    int s_ = (call);        \
    if (s_ != KIMODO_OK) return s_; \
  } while (0)
