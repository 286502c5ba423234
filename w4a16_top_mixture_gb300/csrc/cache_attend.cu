// Attention of one new token of each request over the paged cache (moe_cache_attend).
#include "cache.cuh"

namespace moe {
namespace {

struct AttendArgs {
  moe_cache_attend_t a;
  int Hq, Hkv, page_log2, n_pages, max_pages;
  float scale;
  uint32_t* status;
};

// One CTA per request and query head, one warp per token in turn: a lane holds D / 32 elements of q and of the
// output, and every warp keeps its own running maximum and sum, joined at the end.
template <int D, bool BF16, bool E4M3>
__global__ void __launch_bounds__(256) k_cache_attend(const __grid_constant__ AttendArgs A) {
  constexpr int E = D / 32;
  __shared__ float s_m[8], s_l[8], s_o[8][D];
  const moe_cache_attend_t& a = A.a;
  const int h = blockIdx.x, b = blockIdx.y, g = h / (A.Hq / A.Hkv);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long max_len = (long long)A.max_pages << A.page_log2;
  int len = a.lengths[b];
  if (len < 0 || len > max_len) {
    if (threadIdx.x == 0) atomicOr(A.status, CACHE_BAD_LENGTH);
    len = len < 0 ? 0 : (int)max_len;
  }
  auto load = [&](const void* pool, long long at, float* x) {
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      float2 f;
      if (E4M3) {
        const uint32_t r = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>((const uint8_t*)pool + at + i));
        f = unpack2<false>(r);
      } else {
        f = unpack2<BF16>(*reinterpret_cast<const uint32_t*>((const uint16_t*)pool + at + i));
      }
      x[i] = f.x;
      x[i + 1] = f.y;
    }
  };
  float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < E; i += 2) {
    const float2 f = unpack2<BF16>(*reinterpret_cast<const uint32_t*>((const uint16_t*)a.q.p + b * a.q.row_stride +
                                                                      h * a.q.head_stride + lane * E + i));
    const float s = A.scale * (E4M3 ? a.k_scale[g] : 1.f);
    q[i] = f.x * s;
    q[i + 1] = f.y * s;
  }
  for (int j = warp; j < len; j += 8) {
    const int page = a.tables[b * a.table_stride + (j >> A.page_log2)];
    const bool bad = page < 0 || page >= A.n_pages;
    if (bad && lane == 0) atomicOr(A.status, CACHE_BAD_PAGE);
    const long long in = ((long long)g << A.page_log2) * D + (long long)(j & ((1 << A.page_log2) - 1)) * D + lane * E;
    float k[E] = {}, v[E] = {};
    if (!bad) {
      load(a.k_cache, page * a.k_page_stride + in, k);
      load(a.v_cache, page * a.v_page_stride + in, v);
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) s = fmaf(q[i], k[i], s);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, x);
    // a maximum of -inf (only scores of -inf so far) counts as 0: the weights are exp(-inf) = 0, not NaN
    const float top = fmaxf(m, s), base = top == -INFINITY ? 0.f : top;
    const float c = __expf(m - base), p = __expf(s - base);
    m = top;
    l = l * c + p;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = o[i] * c + p * v[i];
  }
#pragma unroll
  for (int i = 0; i < E; ++i) s_o[warp][lane * E + i] = o[i];
  if (lane == 0) { s_m[warp] = m; s_l[warp] = l; }
  __syncthreads();
  const int e = threadIdx.x;
  if (e >= D) return;
  float top = -INFINITY, sum = 0.f, y = 0.f;
  for (int w = 0; w < 8; ++w) top = fmaxf(top, s_m[w]);
  for (int w = 0; w < 8 && w < len; ++w) {
    const float c = __expf(s_m[w] - top);
    sum += s_l[w] * c;
    y += s_o[w][e] * c;
  }
  y = len ? y / sum * (E4M3 ? a.v_scale[g] : 1.f) : 0.f;
  auto at = [&](const moe_rows_t& r) { return (uint16_t*)r.p + b * r.row_stride + h * r.head_stride + e; };
  if (a.gate.p) {
    const float x = unpack2<BF16>(*at(a.gate)).x;
    y = y / (1.f + __expf(-x));
  }
  *at(a.out) = (uint16_t)pack2<BF16>(y, 0.f);
}

template <int D>
void launch(const AttendArgs& a, bool bf16, bool e4m3, cudaStream_t st) {
  const dim3 grid(a.Hq, (unsigned)a.a.n_requests);
  if (bf16 && e4m3) k_cache_attend<D, true, true><<<grid, 256, 0, st>>>(a);
  else if (bf16) k_cache_attend<D, true, false><<<grid, 256, 0, st>>>(a);
  else if (e4m3) k_cache_attend<D, false, true><<<grid, 256, 0, st>>>(a);
  else k_cache_attend<D, false, false><<<grid, 256, 0, st>>>(a);
}

}  // namespace

cudaError_t cache_attend_launch(const CacheShape& S, const moe_cache_attend_t& a, uint32_t* status, cudaStream_t st) {
  AttendArgs A;
  A.a = a;
  A.Hq = S.Hq;
  A.Hkv = S.Hkv;
  A.page_log2 = S.page_log2;
  A.n_pages = S.n_pages;
  A.max_pages = S.max_pages;
  A.scale = (float)a.scale;
  A.status = status;
  if (S.D == 64) launch<64>(A, S.bf16, S.e4m3, st);
  else if (S.D == 128) launch<128>(A, S.bf16, S.e4m3, st);
  else launch<256>(A, S.bf16, S.e4m3, st);
  return cudaGetLastError();
}

}  // namespace moe
