// The library's own device error word, one per device, for callers that bring none
// (kq_default_info).
#include "kq_internal.cuh"

namespace {
__device__ int32_t default_info;   // 0 until a kernel records an error in it
}

extern "C" int32_t* kq_default_info(void) {
  void* p = nullptr;
  if (kq::cuda_check(cudaGetSymbolAddress(&p, default_info), "kq_default_info") != KQ_OK) {
    (void)cudaGetLastError();
    return nullptr;
  }
  kq::clear_error();
  return static_cast<int32_t*>(p);
}
