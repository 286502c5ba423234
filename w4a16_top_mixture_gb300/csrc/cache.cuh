// The paged key-value cache: the handle, and what its three operators (cache_plan.cu, cache_write.cu,
// cache_attend.cu) get from the C ABI (cache.cu). Layouts and formulas are in include/moe_block.h.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/moe_block.h"

namespace moe {

// records a CUDA runtime error for moe_last_cuda_error and returns MOE_ERR_CUDA (api.cu)
int report_cuda(cudaError_t e, const char* what);

constexpr int CACHE_MAX_REQUESTS = 4096;
constexpr int CACHE_MAX_GROUP = 64;      // query heads to a key-value head

enum : uint32_t {                        // bits of the handle's status word
  CACHE_BAD_WAIT = 1, CACHE_BAD_LENGTH = 2, CACHE_BAD_PAGE = 4, CACHE_BAD_STATE = 8,
};

// the shape as the kernels use it
struct CacheShape {
  int Hq, Hkv, D, page_log2, n_pages, max_pages;
  int rope;                              // rotated elements of a head
  bool bf16, e4m3;                       // activations; cache elements
  float gamma_offset, eps;
};

cudaError_t cache_plan_init();           // once per device: the kernel's shared-memory limit
cudaError_t cache_plan_launch(const CacheShape& S, const moe_cache_plan_t& p, uint32_t* arrivals, uint32_t* status,
                              int num_sms, cudaStream_t st);
cudaError_t cache_write_launch(const CacheShape& S, const moe_cache_write_t& w, const uint64_t* turns,
                               uint32_t* status, int num_sms, cudaStream_t st);

struct CacheAttendState {
  void* workspace;                       // cache_attend_workspace bytes, 16-byte aligned, zeroed once
  uint32_t* status;
  int num_sms;
  uint64_t timeout_ns;                   // of the device's waits
  int skip_copy;
};
size_t cache_attend_workspace(int num_sms);
cudaError_t cache_attend_launch(const CacheShape& S, const moe_cache_attend_t& a, const CacheAttendState& w,
                                cudaStream_t st);

// ---- launches ----
// The three kernels are launched so that they may start while the kernel before them in the stream still ends
// (programmatic dependent launch): each lets its successor start at once, and waits for its predecessor's end before it
// reads or writes device memory. What a predecessor wrote is read past L1 (__ldcg, bulk copies): a line that another
// kernel left in an SM's L1 could be older.
__device__ __forceinline__ void follow_predecessor() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
template <class... P, class... A>
cudaError_t launch_following(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t st,
                             const A&... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(grid);
  c.blockDim = dim3(block);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = a;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

// ---- 16-bit pairs ----
template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if (BF16) return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {   // a in the low half
  uint32_t r;
  if (BF16) *reinterpret_cast<__nv_bfloat162*>(&r) = __floats2bfloat162_rn(a, b);
  else *reinterpret_cast<__half2*>(&r) = __floats2half2_rn(a, b);
  return r;
}
// four e4m3 codes as two pairs of fp16, the lower ones first: exact, NaN kept
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t v, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(v));
}

}  // namespace moe
