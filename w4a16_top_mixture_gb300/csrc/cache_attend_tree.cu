// Attention of several new tokens of each request over the paged cache (moe_cache_attend_tree).
//
// The simple form: a CTA to a row and query head, four warps that take the tokens in turn, each lane D / 32 elements of
// the head; running maxima and sums, joined in shared memory.
#include "cache.cuh"

namespace moe {
namespace {

constexpr float LOG2E = 1.4426950408889634f;

struct TreeAttendArgs {
  moe_cache_attend_tree_t a;
  int B, rows, Hq, Hkv, group, page_log2, n_pages, most;
  long long max_len;
  float scale;
  uint32_t* status;
};

template <int D, bool BF16, bool E4M3>
__device__ __forceinline__ void load_row(const void* pool, int64_t at, int lane, float (&x)[D / 32]) {
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    const int64_t e = at + i * 64 + lane * 2;
    if (E4M3) {
      const uint16_t c = __ldcg((const unsigned short*)((const uint8_t*)pool + e));
      uint32_t lo, hi;
      e4m3x4_to_f16x4(c, lo, hi);
      const float2 f = unpack2<false>(lo);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    } else {
      const float2 f = unpack2<BF16>(__ldcg((const uint32_t*)((const uint16_t*)pool + e)));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

template <int D, bool BF16, bool E4M3>
__global__ void __launch_bounds__(128) k_tree_simple(const __grid_constant__ TreeAttendArgs A) {
  __shared__ float s_o[4][D], s_m[4], s_l[4];
  const moe_cache_attend_tree_t& a = A.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = blockIdx.x, h = blockIdx.y;
  follow_predecessor();
  int lo = 0, hi = A.B;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldcg(a.starts + mid + 1) > r) hi = mid; else lo = mid + 1;
  }
  if (lo >= A.B) return;
  uint32_t bad = 0;
  const NewTokens t = new_tokens_of(a.starts, a.slots, a.lengths, lo, A.rows, A.max_len, A.most, &bad);
  if (bad && threadIdx.x == 0) atomicOr(A.status, bad);
  const int i = r - t.lo, older = t.len - t.n, g = h / A.group;
  const int len = t.left_out || t.n == 0 ? 0 : t.len;
  float q[D / 32], o[D / 32] = {}, m = -INFINITY, l = 0.f;
  load_row<D, BF16, false>(a.q.p, r * a.q.row_stride + h * a.q.head_stride, lane, q);
  const float scale = A.scale * (E4M3 ? __ldcg(a.k_scale + g) : 1.f);
  for (int p = warp; p < len; p += 4) {
    if (p >= older) {
      const int j = p - older;
      if (!(a.masks ? __ldcg(a.masks + (size_t)r * a.mask_words + (j >> 6)) >> (j & 63) & 1 : j <= i)) continue;
    }
    const int page = __ldcg(a.tables + (size_t)lo * a.table_stride + (p >> A.page_log2));
    const bool in = page >= 0 && page < A.n_pages;
    if (!in && lane == 0) atomicOr(A.status, CACHE_BAD_PAGE);
    const int64_t off = ((int64_t)g << A.page_log2) * D + (int64_t)(p & ((1 << A.page_log2) - 1)) * D;
    float k[D / 32] = {}, v[D / 32] = {}, s = 0.f;
    if (in) {
      load_row<D, BF16, E4M3>(a.k_cache, page * a.k_page_stride + off, lane, k);
      load_row<D, BF16, E4M3>(a.v_cache, page * a.v_page_stride + off, lane, v);
    }
#pragma unroll
    for (int d = 0; d < D / 32; ++d) s += q[d] * k[d];
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, x);
    s *= scale;
    const float top = fmaxf(m, s), w = exp2f(s - top), keep = m == -INFINITY ? 0.f : exp2f(m - top);
    l = l * keep + w;
#pragma unroll
    for (int d = 0; d < D / 32; ++d) o[d] = o[d] * keep + w * v[d];
    m = top;
  }
#pragma unroll
  for (int d = 0; d < D / 32; ++d) s_o[warp][d / 2 * 64 + lane * 2 + d % 2] = o[d];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  __syncthreads();
  const float top = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  float total = 0.f, w[4];
  for (int k = 0; k < 4; ++k) {
    w[k] = s_m[k] == -INFINITY && s_l[k] == 0.f ? 0.f : exp2f(s_m[k] - top);
    total += w[k] * s_l[k];
  }
  for (int d = threadIdx.x; d < D; d += 128) {
    float y = 0.f;
    for (int k = 0; k < 4; ++k) y += w[k] == 0.f ? 0.f : w[k] * s_o[k][d];
    y = total == 0.f ? 0.f : y / total * (E4M3 ? __ldcg(a.v_scale + g) : 1.f);
    if (a.gate.p) {
      const uint16_t c = __ldcg((const unsigned short*)a.gate.p + r * a.gate.row_stride + h * a.gate.head_stride + d);
      y /= 1.f + __expf(-unpack2<BF16>(c).x);
    }
    ((uint16_t*)a.out.p)[r * a.out.row_stride + h * a.out.head_stride + d] = (uint16_t)pack2<BF16>(y, 0.f);
  }
}

template <int D>
cudaError_t run(const CacheShape& S, const TreeAttendArgs& A, cudaStream_t st) {
  auto* k = S.bf16 ? (S.e4m3 ? k_tree_simple<D, true, true> : k_tree_simple<D, true, false>)
                   : (S.e4m3 ? k_tree_simple<D, false, true> : k_tree_simple<D, false, false>);
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(A.rows, A.Hq);
  c.blockDim = dim3(128);
  c.stream = st;
  return cudaLaunchKernelEx(&c, k, A);
}

}  // namespace

size_t cache_attend_tree_workspace(int num_sms, int head_dim) { return 256; }

cudaError_t cache_attend_tree_launch(const CacheShape& S, const moe_cache_attend_tree_t& a, const CacheTreeState& w,
                                     cudaStream_t st) {
  TreeAttendArgs A;
  A.a = a;
  A.B = (int)a.n_requests;
  A.rows = (int)a.n_rows;
  A.Hq = S.Hq;
  A.Hkv = S.Hkv;
  A.group = S.Hq / S.Hkv;
  A.page_log2 = S.page_log2;
  A.n_pages = S.n_pages;
  A.most = a.masks && 64 * (int)a.mask_words < w.max_new ? 64 * (int)a.mask_words : w.max_new;
  A.max_len = (long long)S.max_pages << S.page_log2;
  A.scale = (float)a.scale * LOG2E;
  A.status = w.status;
  return S.D == 64 ? run<64>(S, A, st) : S.D == 128 ? run<128>(S, A, st) : run<256>(S, A, st);
}

}  // namespace moe
