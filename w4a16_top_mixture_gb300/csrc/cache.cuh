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
  CACHE_BAD_WAIT = 1, CACHE_BAD_LENGTH = 2, CACHE_BAD_PAGE = 4, CACHE_BAD_STATE = 8, CACHE_BAD_ROWS = 16,
};
constexpr int CACHE_MAX_NEW = 256;       // new tokens of a request in one step

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

// ---- several new tokens of a request ----
cudaError_t cache_tree_launch(const CacheShape& S, const moe_cache_tree_t& t, int max_new, uint32_t* status,
                              cudaStream_t st);

constexpr int CACHE_TREE_COUNTS = 12288;  // bytes of counts at the workspace's start, zeroed once and after a lost wait
struct CacheTreeState {
  void* workspace;                       // cache_attend_tree_workspace bytes
  uint32_t* status;
  int num_sms, max_new;
  uint64_t timeout_ns;                   // of the device's waits
  int skip_copy;
};
size_t cache_attend_tree_workspace(int num_sms, int head_dim);
cudaError_t cache_attend_tree_launch(const CacheShape& S, const moe_cache_attend_tree_t& a, const CacheTreeState& w,
                                     cudaStream_t st);

// Rows of tokens that move from one slot to another, of one request: `rows` positions from `first` on. Position p comes
// from p below `older`, else from older + path[p - older]; its page is `from` before the move and `to` after it, counted
// from the page of `first` on.
constexpr int CACHE_MOVE_SPAN = 20;      // pages that 256 new tokens can lie in, and some
struct alignas(16) CacheMoves {
  int first, rows, older, pad;
  int from[CACHE_MOVE_SPAN], to[CACHE_MOVE_SPAN];
};
cudaError_t cache_pages_init();          // once per device: the kernels' shared-memory limits
cudaError_t cache_keep_launch(const CacheShape& S, const moe_cache_keep_t& k, int max_new, CacheMoves* moves,
                              uint32_t* status, int num_sms, cudaStream_t st);
cudaError_t cache_fork_launch(const CacheShape& S, const moe_cache_fork_t& f, CacheMoves* moves, uint32_t* status,
                              int num_sms, cudaStream_t st);

#ifdef __CUDACC__
// What a step brings of request b: rows lo .. lo + n - 1, its last n tokens of len. left_out: what starts or the length
// say cannot be (reported). A refused request has no new tokens in the cache; lo and n_rows are its rows all the same.
struct NewTokens {
  int lo, rows, n, len;
  bool left_out;
};
__device__ __forceinline__ NewTokens new_tokens_of(const int32_t* starts, const int32_t* slots, const int32_t* lengths,
                                                   int b, int n_rows, long long max_len, int most, uint32_t* bad) {
  NewTokens t;
  t.len = __ldcg(lengths + b);
  t.lo = __ldcg(starts + b);
  const int hi = __ldcg(starts + b + 1);
  t.left_out = false;
  t.rows = 0;
  if (t.lo < 0 || hi < t.lo || hi > n_rows) {
    *bad |= CACHE_BAD_ROWS;
    t.left_out = true;
    t.lo = 0;
  } else {
    t.rows = hi - t.lo;
  }
  t.n = t.rows;
  if (t.rows > 0 && slots && __ldcg(slots + t.lo) < 0) t.n = 0;
  if (t.len < 0 || t.len > max_len || t.len < t.n) {
    *bad |= CACHE_BAD_LENGTH;
    t.left_out = true;
  }
  if (t.n > most) {
    *bad |= CACHE_BAD_ROWS;
    t.left_out = true;
  }
  return t;
}
#endif

// ---- launches ----
// The kernels are launched so that they may start while the kernel before them in the stream still ends
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
