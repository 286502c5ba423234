// Block tables and slot maps of a step from the requests' lengths (moe_cache_plan).
//
// Two exclusive scans over the requests decide everything: of the new tokens (where a request's rows start, and so
// whether they fit), then of the pages needed and the pages given back (which entries of the ring of free pages they
// are). What follows is independent for each page and each row. The scans are a few thousand integers, so every CTA
// repeats them and no CTA waits for another: the last one to have read the inputs writes the outputs that may lie in
// place of them.
#include "cache.cuh"

namespace moe {
namespace {

struct PlanArgs {
  moe_cache_plan_t p;
  int B, rows, page_log2, n_pages, max_pages;
  bool in_place;
  uint32_t *arrivals, *status;
};

// exclusive scan of one value per thread over the block; *total: the sum. ws: 33 words
__device__ __forceinline__ unsigned long long block_scan(unsigned long long v, unsigned long long* ws,
                                                         unsigned long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  unsigned long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) ws[warp] = x;
  __syncthreads();
  if (warp == 0) {
    unsigned long long s = lane < nw ? ws[lane] : 0;
    const unsigned long long mine = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xFFFFFFFFu, s, o);
      if (lane >= o) s += y;
    }
    if (lane < nw) ws[lane] = s - mine;
    if (lane == 31) ws[32] = s;
  }
  __syncthreads();
  *total = ws[32];
  return ws[warp] + x - v;
}

// EACH: requests of a thread, side by side, so that all its loads are on their way at once and two scans do
template <int EACH>
__global__ void k_cache_plan(const __grid_constant__ PlanArgs a) {
  extern __shared__ int sm[];
  // per request: the row after its last, its cached tokens, its first page's place among the pages taken (-1: not
  // admitted; -2 - place: its first page's place among the pages given back)
  int *s_end = sm, *s_len = sm + a.B, *s_at = sm + 2 * a.B;
  __shared__ unsigned long long ws[2][33];
  __shared__ int s_refused, s_taken;
  __shared__ bool s_last;
  const moe_cache_plan_t& p = a.p;
  const int ps = 1 << a.page_log2;
  const long long max_len = (long long)a.max_pages << a.page_log2;
  const int tid = threadIdx.x, nth = blockDim.x;
  if (tid == 0) s_refused = s_taken = 0;
  follow_predecessor();
  int head = __ldcg(p.free_state), count = __ldcg(p.free_state + 1);
  int len[EACH], nw[EACH];
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int b = tid * EACH + i;
    len[i] = b < a.B ? __ldcg(p.lengths + b) : 0;
    nw[i] = b < a.B ? (p.new_tokens ? __ldcg(p.new_tokens + b) : 1) : 0;
  }
  if (head < 0 || head >= a.n_pages || count < 0 || count > a.n_pages) {
    head = count = 0;
    if (tid == 0) atomicOr(a.status, CACHE_BAD_STATE);
  }
  // what the ring can take back: all that the requests hold, if no page is in two places
  const int room = a.n_pages - count;
  // where each request's rows end
  unsigned long long sum = 0, total;
#pragma unroll
  for (int i = 0; i < EACH; ++i) sum += nw[i] > 0 ? nw[i] : 0;
  unsigned long long end = block_scan(sum, ws[0], &total);
  // the pages it needs (low half: those that fit take at most n_rows / 16 + B) and gives back (high half: below 2^32
  // but where 2^12 requests hold 2^20 pages each, of a pool's 2^27; then none of them count)
  int held[EACH], need[EACH];
  bool fits[EACH];
  sum = 0;
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int b = tid * EACH + i;
    const long long n = nw[i] > 0 ? nw[i] : 0;
    end += n;
    const bool in = b < a.B, good = len[i] >= 0 && len[i] <= max_len;
    held[i] = good ? (int)(((long long)len[i] + ps - 1) >> a.page_log2) : 0;
    fits[i] = in && good && nw[i] >= 0 && len[i] + n <= max_len && end <= (unsigned long long)a.rows;
    need[i] = fits[i] ? (int)((len[i] + n + ps - 1) >> a.page_log2) - held[i] : 0;
    sum += (unsigned long long)need[i] | (unsigned long long)(uint32_t)(in && nw[i] < 0 ? held[i] : 0) << 32;
    if (in) {
      s_end[b] = (int)(end < 0x7FFFFFFF ? end : 0x7FFFFFFF);
      s_len[b] = len[i];
      if (!good) atomicOr(a.status, CACHE_BAD_LENGTH);
    }
  }
  unsigned long long at = block_scan(sum, ws[1], &total);
  const uint32_t back_total = (uint32_t)(total >> 32);
  int refused = 0, taken = 0;
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int b = tid * EACH + i;
    if (b < a.B) {
      const uint32_t need_at = (uint32_t)at, back_at = (uint32_t)(at >> 32);
      const bool done = nw[i] < 0, ok = fits[i] && (need[i] == 0 || need_at + (uint32_t)need[i] <= (uint32_t)count);
      const int back_to = (int)(back_at < 0x3FFFFFFFu ? back_at : 0x3FFFFFFFu);
      s_at[b] = ok ? (need[i] ? (int)need_at : 0) : done ? -2 - back_to : -1;
      if (ok) taken += need[i];
      else if (!done) ++refused;
      at += (unsigned long long)need[i] | (unsigned long long)(uint32_t)(done ? held[i] : 0) << 32;
    }
  }
  refused = __reduce_add_sync(0xFFFFFFFFu, refused);
  taken = __reduce_add_sync(0xFFFFFFFFu, taken);
  if ((tid & 31) == 0) {
    if (refused) atomicAdd(&s_refused, refused);
    if (taken) atomicAdd(&s_taken, taken);
  }
  __syncthreads();

  // the pages: a warp to a request
  {
    const int lane = tid & 31;
    const int gw = (blockIdx.x * nth + tid) >> 5, n_w = (gridDim.x * nth) >> 5;
    for (int b = gw; b < a.B; b += n_w) {
      const int at = s_at[b], len = s_len[b];
      int32_t* row = p.tables + (size_t)b * p.table_stride;
      if (at >= 0) {
        const int n = s_end[b] - (b ? s_end[b - 1] : 0);
        const int held = (int)(((long long)len + ps - 1) >> a.page_log2);
        const int want = (int)(((long long)len + n + ps - 1) >> a.page_log2);
        for (int j = held + lane; j < want; j += 32)
          row[j] = __ldcg(p.free_pages + ((uint32_t)head + (uint32_t)at + (uint32_t)(j - held)) % (uint32_t)a.n_pages);
      } else if (at <= -2 && len > 0 && len <= max_len) {
        const int back = -2 - at, held = (int)(((long long)len + ps - 1) >> a.page_log2);
        // no further than the ring has room: beyond lie entries that this call's requests take
        const int fit = held < room - back ? held : room - back;
        const uint32_t to = (uint32_t)head + (uint32_t)count + (uint32_t)back;
        for (int j = lane; j < fit; j += 32) p.free_pages[(to + (uint32_t)j) % (uint32_t)a.n_pages] = __ldcg(row + j);
      }
    }
  }
  // the rows
  for (long long r = (long long)blockIdx.x * nth + tid; r < a.rows; r += (long long)gridDim.x * nth) {
    int lo = 0, hi = a.B;              // the first request that ends past row r
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (s_end[mid] > r) hi = mid; else lo = mid + 1;
    }
    int slot = -1, pos = 0;
    if (lo < a.B && s_at[lo] >= 0) {
      const int len = s_len[lo];
      pos = len + (int)(r - (lo ? s_end[lo - 1] : 0));
      const int held = (int)(((long long)len + ps - 1) >> a.page_log2), j = pos >> a.page_log2;
      // a page taken in this call is read where it comes from
      const int page = __ldcg(j < held ? p.tables + (size_t)lo * p.table_stride + j
                                       : p.free_pages + ((uint32_t)head + (uint32_t)s_at[lo] + (uint32_t)(j - held)) %
                                                            (uint32_t)a.n_pages);
      if (page >= 0 && page < a.n_pages) slot = (page << a.page_log2) + (pos & (ps - 1));
      else atomicOr(a.status, CACHE_BAD_PAGE);
    }
    p.slots[r] = slot;
    p.positions[r] = pos;
  }
  // the first CTA writes the rest; what lies in place of inputs, the last to have read them
  if (!a.in_place) {
    if (blockIdx.x) return;
  } else if (gridDim.x > 1) {
    __syncthreads();
    if (tid == 0) {
      __threadfence();
      s_last = atomicAdd(a.arrivals, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
  }
  for (int b = tid; b < a.B; b += nth) {
    const int at = s_at[b], n = s_end[b] - (b ? s_end[b - 1] : 0);
    p.lengths_out[b] = at >= 0 ? s_len[b] + n : at <= -2 ? 0 : s_len[b];
    p.starts[b + 1] = s_end[b];
  }
  if (tid == 0) {
    p.starts[0] = 0;
    p.free_state_out[0] = (int)((uint32_t)(head + s_taken) % (uint32_t)a.n_pages);
    p.free_state_out[1] = count - s_taken + (back_total < (uint32_t)room ? (int)back_total : room);
    p.free_state_out[2] = s_refused;
    if (back_total > (uint32_t)room) atomicOr(a.status, CACHE_BAD_STATE);
    if (a.in_place && gridDim.x > 1) *a.arrivals = 0;
  }
}

}  // namespace

cudaError_t cache_plan_init() {
  cudaError_t e = cudaSuccess;
  for (auto* k : {k_cache_plan<1>, k_cache_plan<2>, k_cache_plan<4>})
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, CACHE_MAX_REQUESTS * 12);
  return e;
}

cudaError_t cache_plan_launch(const CacheShape& S, const moe_cache_plan_t& p, uint32_t* arrivals, uint32_t* status,
                              int num_sms, cudaStream_t st) {
  PlanArgs a;
  a.p = p;
  a.B = (int)p.n_requests;
  a.rows = (int)p.n_rows;
  a.page_log2 = S.page_log2;
  a.n_pages = S.n_pages;
  a.max_pages = S.max_pages;
  a.in_place = p.lengths == p.lengths_out || p.free_state == p.free_state_out;
  a.arrivals = arrivals;
  a.status = status;
  const int each = a.B <= 1024 ? 1 : a.B <= 2048 ? 2 : 4;
  int threads = ((a.B + each - 1) / each + 31) & ~31;
  threads = threads < 128 ? 128 : threads;
  // a CTA for every row of each thread: rows are independent, and the scans cost every CTA alike
  const long long want = ((long long)a.rows + threads - 1) / threads;
  const int grid = (int)(want < 1 ? 1 : want > num_sms ? num_sms : want);
  return launch_following(each == 1 ? k_cache_plan<1> : each == 2 ? k_cache_plan<2> : k_cache_plan<4>, grid, threads,
                          (size_t)a.B * 12, st, a);
}

}  // namespace moe
