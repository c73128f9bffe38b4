// Status plumbing of the C ABI (see status.h).
#include "status.h"

#include <stdarg.h>
#include <stdio.h>

#include <mutex>

namespace kd {
namespace {

thread_local char g_message[512] = "";
__device__ DevError g_kernel_error;

}  // namespace

int set_error(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_message, sizeof(g_message), fmt, ap);
  va_end(ap);
  return code;
}

void clear_error() { g_message[0] = 0; }
const char* last_error() { return g_message; }

bool is_device_memory(const void* p) {
  cudaPointerAttributes a;
  if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return a.type == cudaMemoryTypeDevice || a.type == cudaMemoryTypeManaged;
}

const char* where_name(int where) {
  switch (where) {
    case WHERE_GEMM_PRODUCER: return "GEMM TMA producer";
    case WHERE_GEMM_MMA: return "GEMM MMA issuer";
    case WHERE_GEMM_EPILOGUE: return "GEMM epilogue";
    case WHERE_GEMM_DRAIN: return "GEMM MMA drain";
    case WHERE_ATTENTION: return "attention";
    case WHERE_WAIT_SELFTEST: return "wait self-test";
    case WHERE_SCORED_ATTENTION: return "attention with scored masks";
    default: return "unknown stage";
  }
}

// The address of the static word is looked up once per device, with that device current;
// the lookup is serialised for threads that make their first call at the same time.
DevError* kernel_error_word() {
  static std::mutex mu;
  static DevError* p[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (!p[dev]) {
    void* a = nullptr;
    if (cudaGetSymbolAddress(&a, g_kernel_error) != cudaSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    p[dev] = static_cast<DevError*>(a);
  }
  return p[dev];
}

}  // namespace kd
