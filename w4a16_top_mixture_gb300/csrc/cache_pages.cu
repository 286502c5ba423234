// What stays of a step's new tokens, and requests that share pages (moe_cache_keep, moe_cache_fork).
//
// Both calls decide first, on the requests' few integers, and then move rows of keys and values in every layer's pools.
//   Deciding is one cluster of up to 8 CTAs, a warp to a request in turn. What depends on the order of the requests (who
// gets the pages of the ring's head, where the pages given back go at its tail) are two scans over one integer a request,
// which every CTA of the cluster holds and repeats. A page that several requests give back in one call goes to the ring
// once and at the place of the first of them, whatever the order of the atomics: all take their reference off first; where
// that leaves less than none, all of them put their number's code there as a minimum; the one whose code stayed owns it.
//   Moving is a warp to each request, key-value head and two pools. New tokens only move down, to places before their own, so
// a warp that reads rows in ascending order before it writes them reads each before it is overwritten.
#include <cooperative_groups.h>

#include "cache.cuh"

namespace moe {
namespace {

namespace cg = cooperative_groups;

constexpr int WARPS = 16, THREADS = 32 * WARPS, MAX_CLUSTER = 8;
constexpr int EACH = CACHE_MAX_REQUESTS / THREADS;   // requests of a thread in a scan
constexpr int LOWEST = -0x7FFFFFFF - 1;

// exclusive scan of one value per thread over the block; *total: the sum. ws: 33 words
__device__ __forceinline__ unsigned long long block_scan(unsigned long long v, unsigned long long* ws,
                                                         unsigned long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) ws[warp] = x;
  __syncthreads();
  if (warp == 0) {
    unsigned long long s = lane < WARPS ? ws[lane] : 0;
    const unsigned long long mine = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xFFFFFFFFu, s, o);
      if (lane >= o) s += y;
    }
    if (lane < WARPS) ws[lane] = s - mine;
    if (lane == 31) ws[32] = s;
  }
  __syncthreads();
  *total = ws[32];
  return ws[warp] + x - v;
}

// the ring of free pages, empty where its state cannot be
struct Ring {
  int head, count, n;
  __device__ __forceinline__ Ring(const int32_t* state, int n_pages, uint32_t* bad) : n(n_pages) {
    head = __ldcg(state);
    count = __ldcg(state + 1);
    if (head < 0 || head >= n || count < 0 || count > n) {
      head = count = 0;
      *bad |= CACHE_BAD_STATE;
    }
  }
  __device__ __forceinline__ int at(uint32_t i) const {    // entry i from the head on
    return (int)(((unsigned long long)(uint32_t)head + i) % (uint32_t)n);
  }
};

// In place of the needs: where each request's (or entry's) pages begin among those taken, -1 where it gets none for want
// of them; -2: left out before. A need of 0 is always met. Returns the pages taken; *refused: how many went without.
__device__ __forceinline__ int admit(int* need, int n, int count, unsigned long long* ws, int* sums, int* refused) {
  unsigned long long sum = 0, total;
  int own[EACH];
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int b = threadIdx.x * EACH + i;
    own[i] = b < n ? need[b] : 0;
    sum += own[i] > 0 ? own[i] : 0;
  }
  if (threadIdx.x == 0) sums[0] = sums[1] = 0;
  unsigned long long at = block_scan(sum, ws, &total);
  int taken = 0, out = 0;
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int b = threadIdx.x * EACH + i;
    if (b >= n) break;
    if (own[i] > 0) {
      const bool ok = at + own[i] <= (unsigned long long)count;
      need[b] = ok ? (int)at : -1;
      if (ok) taken += own[i];
      else ++out;
      at += own[i];
    }
  }
  if (taken) atomicAdd(&sums[0], taken);
  if (out) atomicAdd(&sums[1], out);
  __syncthreads();
  *refused = sums[1];
  return sums[0];
}

struct KeepArgs {
  moe_cache_keep_t k;
  int B, rows, page_log2, n_pages, most, local;   // local: requests of a CTA
  bool move;                                      // rows may move: records are written
  long long max_len;
  CacheMoves* moves;
  uint32_t* status;
};

// a request between the phases, in its warp's CTA
struct Kept {
  int len, now;              // tokens before and after
  int page0, rows0;          // first page and row that change, of those that stay
  int older, moved;          // its older tokens; whether new ones move
  uint32_t exchange;         // bit i: page0 + i is exchanged
};

__global__ void __launch_bounds__(THREADS) k_cache_keep(const __grid_constant__ KeepArgs a) {
  extern __shared__ int4 sm4[];
  Kept* s_kept = reinterpret_cast<Kept*>(sm4);
  int* s_need = reinterpret_cast<int*>(s_kept + a.local);
  int* s_give = s_need + a.B;
  __shared__ unsigned long long ws[33];
  __shared__ int sums[2];
  cg::cluster_group cluster = cg::this_cluster();
  const moe_cache_keep_t& k = a.k;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
  const int ps = 1 << a.page_log2;
  const unsigned ALL = 0xFFFFFFFFu;
  uint32_t bad = 0;
  follow_predecessor();
  const Ring ring(k.free_state, a.n_pages, &bad);
  // every CTA has to run before another writes into its shared memory
  cluster.sync();

  // what each request keeps, which of its pages it gives back, and how many fresh ones it needs
  for (int l = warp, b; (b = l * ctas + rank) < a.B; l += WARPS) {
    Kept q;
    q.page0 = q.rows0 = q.older = q.moved = 0;
    q.exchange = 0;
    int n, count = __ldcg(k.counts + b);
    bool out;
    if (k.starts) {
      const NewTokens t = new_tokens_of(k.starts, k.slots, k.lengths, b, a.rows, a.max_len, 0x7FFFFFFF, &bad);
      q.len = t.len;
      n = t.n;
      out = t.left_out;
    } else {
      n = q.len = __ldcg(k.lengths + b);
      out = n < 0 || n > a.max_len;
      if (out) bad |= CACHE_BAD_LENGTH;
    }
    int first_moved = 0x7FFFFFFF;
    if (!out && count >= 0) {
      bool good = count <= n;
      if (good && k.path) {
        good = n <= a.most && count <= k.path_stride;
        const int32_t* path = k.path + (size_t)b * k.path_stride;
        int before = -1;
        for (int i0 = 0; good && i0 < count; i0 += 32) {
          const int i = i0 + lane, v = i < count ? __ldcg(path + i) : n;
          int prev = __shfl_up_sync(ALL, v, 1);
          prev = lane ? prev : before;
          before = __shfl_sync(ALL, v, 31);
          good = __all_sync(ALL, i >= count || (v > prev && v < n));
          const unsigned m = __ballot_sync(ALL, i < count && v != i);
          if (m && first_moved == 0x7FFFFFFF) first_moved = i0 + __ffs(m) - 1;
        }
      }
      if (!good) {
        out = true;
        bad |= CACHE_BAD_ROWS;
      }
    }
    q.now = out ? q.len : count < 0 ? 0 : q.len - n + count;
    q.older = q.len - n;
    if (!out && q.now > 0) {
      q.moved = first_moved < count;
      const int stay = (int)(((long long)q.now + ps - 1) >> a.page_log2);
      q.rows0 = q.moved ? q.older + first_moved : q.now;
      q.page0 = q.moved ? q.rows0 >> a.page_log2 : (q.now & (ps - 1)) ? stay - 1 : stay;
      if (k.refs) {
        const int i = q.page0 + lane;
        const int page = i < stay ? __ldcg(k.tables + (size_t)b * k.table_stride + i) : -1;
        if (i < stay && (page < 0 || page >= a.n_pages)) bad |= CACHE_BAD_PAGE;
        q.exchange = __ballot_sync(ALL, page >= 0 && page < a.n_pages && __ldcg(k.refs + page) > 0);
      }
    }
    if (lane < ctas) cluster.map_shared_rank(s_need, lane)[b] = out ? -2 : __popc(q.exchange);
    if (lane == 0) s_kept[l] = q;
  }
  cluster.sync();
  int refused = 0, taken = 0;
  if (k.refs) taken = admit(s_need, a.B, ring.count, ws, sums, &refused);

  // the table entries that a request gives back, in ascending order, 32 at a time: f(page, whether the lane has one)
  auto leaving = [&](const Kept& q, int b, auto f) {
    const int32_t* row = k.tables + (size_t)b * k.table_stride;
    if (q.exchange) {
      const bool is = q.exchange >> lane & 1;
      f(is ? __ldcg(row + q.page0 + lane) : -1, is);
    }
    const int stay = (int)(((long long)q.now + ps - 1) >> a.page_log2);
    const int held = (int)(((long long)q.len + ps - 1) >> a.page_log2);
    for (int i = stay; i < held; i += 32) f(i + lane < held ? __ldcg(row + i + lane) : -1, i + lane < held);
  };
  auto in_pool = [&](int page) { return page >= 0 && page < a.n_pages; };
  // the pages' references, then whom each page without one is left to
  if (k.refs) {
    for (int l = warp, b; (b = l * ctas + rank) < a.B; l += WARPS)
      if (s_need[b] >= 0) leaving(s_kept[l], b, [&](int page, bool) { if (in_pool(page)) atomicSub(k.refs + page, 1); });
    cluster.sync();
    for (int l = warp, b; (b = l * ctas + rank) < a.B; l += WARPS)
      if (s_need[b] >= 0)
        leaving(s_kept[l], b, [&](int page, bool) {
          if (in_pool(page) && __ldcg(k.refs + page) < 0) atomicMin(k.refs + page, LOWEST + b);
        });
    cluster.sync();
  }
  for (int l = warp, b; (b = l * ctas + rank) < a.B; l += WARPS) {
    int pages = 0;
    if (s_need[b] >= 0)
      leaving(s_kept[l], b, [&](int page, bool is) {
        if (is && !in_pool(page)) bad |= CACHE_BAD_PAGE;
        pages += __popc(__ballot_sync(ALL, in_pool(page) && (!k.refs || __ldcg(k.refs + page) == LOWEST + b)));
      });
    if (lane < ctas) cluster.map_shared_rank(s_give, lane)[b] = pages;
  }
  cluster.sync();
  // where each request's pages go, from the ring's tail on
  unsigned long long given;
  {
    unsigned long long sum = 0;
    int own[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const int b = threadIdx.x * EACH + i;
      own[i] = b < a.B ? s_give[b] : 0;
      sum += own[i];
    }
    unsigned long long at = block_scan(sum, ws, &given);
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const int b = threadIdx.x * EACH + i;
      if (b < a.B) s_give[b] = (int)(at < 0x3FFFFFFF ? at : 0x3FFFFFFF);
      at += own[i];
    }
    __syncthreads();
  }
  const int room = ring.n - ring.count;
  for (int l = warp, b; (b = l * ctas + rank) < a.B; l += WARPS) {
    const Kept q = s_kept[l];
    const int at = s_need[b];
    int32_t* row = k.tables + (size_t)b * k.table_stride;
    if (at >= 0) {
      int to = s_give[b];
      leaving(q, b, [&](int page, bool) {
        const bool mine = in_pool(page) && (!k.refs || __ldcg(k.refs + page) == LOWEST + b);
        const unsigned m = __ballot_sync(ALL, mine);
        if (mine) {
          const int i = to + __popc(m & ((1u << lane) - 1));
          if (i < room) k.free_pages[ring.at((uint32_t)ring.count + (uint32_t)i)] = page;
          if (k.refs) k.refs[page] = 0;
        }
        to += __popc(m);
      });
    }
    if (a.move) {
      CacheMoves* m = a.moves + b;
      const bool some = at >= 0 && (q.moved || q.exchange);
      if (some) {
        // from the start of a page that is exchanged, else from the first row that moves
        const int first = q.exchange & 1 || !q.moved ? q.page0 << a.page_log2 : q.rows0;
        const int stay = (int)(((long long)q.now + ps - 1) >> a.page_log2);
        const int held = (int)(((long long)q.len + ps - 1) >> a.page_log2);
        const int span = q.moved ? held - q.page0 : stay - q.page0;
        const int was = lane < span ? __ldcg(row + q.page0 + lane) : -1;
        const int now = q.exchange >> lane & 1
            ? __ldcg(k.free_pages + ring.at((uint32_t)at + (uint32_t)__popc(q.exchange & ((1u << lane) - 1)))) : was;
        if (lane < CACHE_MOVE_SPAN) {
          m->from[lane] = was;
          m->to[lane] = now;
        }
        if (q.exchange >> lane & 1) row[q.page0 + lane] = now;
        if (lane == 0) *reinterpret_cast<int4*>(m) = make_int4(first, q.now - first, q.older, 0);
      } else if (lane == 0) {
        *reinterpret_cast<int4*>(m) = make_int4(0, 0, 0, 0);
      }
    }
    if (lane == 0) k.lengths_out[b] = at >= 0 ? q.now : q.len;
  }
  bad = __reduce_or_sync(ALL, bad);
  if (bad && lane == 0) atomicOr(a.status, bad);
  if (rank == 0 && threadIdx.x == 0) {
    k.free_state_out[0] = ring.at(taken);
    k.free_state_out[1] = ring.count - taken + (int)(given < (unsigned)room ? given : room);
    k.free_state_out[2] = refused;
    if (given > (unsigned)room) atomicOr(a.status, CACHE_BAD_STATE);
  }
}

struct ForkArgs {
  moe_cache_fork_t f;
  int B, n, page_log2, n_pages;
  long long max_len;
  CacheMoves* moves;
  uint32_t* status;
};

__global__ void __launch_bounds__(THREADS) k_cache_fork(const __grid_constant__ ForkArgs a) {
  extern __shared__ int4 sm4[];
  int* s_first = reinterpret_cast<int*>(sm4);      // [B]: the first entry that names a request
  int* s_len = s_first + a.B;                      // [n]: tokens of the entry's source
  int* s_at = s_len + a.n;                         // [n]: needs, then places among the pages taken, as in admit
  __shared__ unsigned long long ws[33];
  __shared__ int sums[2];
  cg::cluster_group cluster = cg::this_cluster();
  const moe_cache_fork_t& f = a.f;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
  const int ps = 1 << a.page_log2;
  uint32_t bad = 0;
  for (int b = threadIdx.x; b < a.B; b += THREADS) s_first[b] = a.n;
  follow_predecessor();
  const Ring ring(f.free_state, a.n_pages, &bad);
  __syncthreads();
  for (int i = threadIdx.x; i < a.n; i += THREADS) {
    const int src = __ldcg(f.src + i), dst = __ldcg(f.dst + i);
    int len = 0, need = -2;
    if (src >= 0) {
      if (src >= a.B || dst < 0 || dst >= a.B) {
        bad |= CACHE_BAD_ROWS;
      } else {
        len = __ldcg(f.lengths + src);
        atomicMin(s_first + dst, i);
        if (len < 0 || len > a.max_len) bad |= CACHE_BAD_LENGTH;
        else need = (len & (ps - 1)) ? 1 : 0;
        if (__ldcg(f.lengths + dst) != 0) {
          need = -2;
          bad |= CACHE_BAD_ROWS;
        }
      }
    }
    s_len[i] = len;
    s_at[i] = need;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.n; i += THREADS)
    if (s_at[i] >= 0 && s_first[__ldcg(f.dst + i)] != i) {
      s_at[i] = -2;
      bad |= CACHE_BAD_ROWS;
    }
  __syncthreads();
  int refused = 0;
  const int taken = admit(s_at, a.n, ring.count, ws, sums, &refused);
  cluster.sync();                                  // all have read the lengths and the ring's state

  for (int i = rank + ctas * warp; i < a.n; i += ctas * WARPS) {
    const int at = s_at[i], len = s_len[i];
    CacheMoves* m = a.moves + i;
    int part = 0;
    if (at >= 0) {
      const int full = len >> a.page_log2;
      const int32_t* from = f.tables + (size_t)__ldcg(f.src + i) * f.table_stride;
      int32_t* to = f.tables + (size_t)__ldcg(f.dst + i) * f.table_stride;
      for (int j = lane; j < full; j += 32) {
        const int page = __ldcg(from + j);
        to[j] = page;
        if (page >= 0 && page < a.n_pages) atomicAdd(f.refs + page, 1);
        else bad |= CACHE_BAD_PAGE;
      }
      part = len & (ps - 1);
      if (part && lane == 0) {
        const int fresh = __ldcg(f.free_pages + ring.at((uint32_t)at));
        m->from[0] = __ldcg(from + full);
        m->to[0] = to[full] = fresh;
      }
    }
    if (lane == 0) *reinterpret_cast<int4*>(m) = make_int4(part ? len - part : 0, part, 0x7FFFFFFF, 0);
  }
  if (rank == 0)
    for (int b = threadIdx.x; b < a.B; b += THREADS) {
      const int i = s_first[b];
      f.lengths_out[b] = i < a.n && s_at[i] >= 0 ? s_len[i] : __ldcg(f.lengths + b);
    }
  if (bad) atomicOr(a.status, bad);
  if (rank == 0 && threadIdx.x == 0) {
    f.free_state_out[0] = ring.at(taken);
    f.free_state_out[1] = ring.count - taken;
    f.free_state_out[2] = refused;
  }
}

constexpr int POOLS = 64, MOVE_THREADS = 256;

struct MoveArgs {
  const CacheMoves* moves;
  const int32_t* path;               // NULL: positions stay what they are
  int64_t path_stride;
  int n, heads, page_log2, n_pages, vecs_log2, n_pools;   // 2^vecs_log2: 16-byte vectors of a row
  int pairs, chunks;                 // of pools; of a request's rows
  uint32_t* status;
  uint4* pools[POOLS];
  int64_t strides[POOLS];            // of pages, in vectors
};

// A warp moves a request's rows of one head in two pools: what it looks up (the record, the path, the pages, one after
// another) is looked up once for both, and 8 KB of its rows are on their way at once, 256 bytes a lane. Without a path no
// row is both read and written, and a request's rows are cut into chunks of a warp each; with one they are read and written in
// order. 256 requests, 6 rows of 512 bytes in 20 pools each: 28.8 us with the deciding, where a warp to each pool took 42.4.
__global__ void __launch_bounds__(MOVE_THREADS) k_cache_move(const __grid_constant__ MoveArgs a) {
  constexpr int U = 8;
  const int lane = threadIdx.x & 31, ps = 1 << a.page_log2;
  const int col = lane & ((1 << a.vecs_log2) - 1), sub = lane >> a.vecs_log2, side = 32 >> a.vecs_log2;
  const unsigned per = (unsigned)a.heads * a.pairs * a.chunks, items = per * (unsigned)a.n;
  follow_predecessor();
  for (unsigned it = (blockIdx.x * MOVE_THREADS + threadIdx.x) >> 5; it < items; it += gridDim.x * (MOVE_THREADS / 32)) {
    const unsigned b = it / per, rest = it % per, chunk = rest % a.chunks, head = rest / a.chunks % a.heads;
    const unsigned pool = rest / a.chunks / a.heads * 2, second = pool + 1 < (unsigned)a.n_pools ? pool + 1 : pool;
    const CacheMoves* m = a.moves + b;
    const int4 h = __ldcg(reinterpret_cast<const int4*>(m));   // first, rows, older
    if (h.y == 0) continue;
    const int page0 = h.x >> a.page_log2;
    const size_t in_page = (((size_t)head << a.page_log2) << a.vecs_log2) + col;
    uint4 *one = a.pools[pool] + in_page, *two = a.pools[second] + in_page;
    const int64_t stride1 = a.strides[pool], stride2 = a.strides[second];
    for (int r0 = chunk * U * side; r0 < h.y; r0 += a.chunks * U * side) {
      uint4 v[U], w[U];
      int from[U], to[U], sat[U], dat[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + u * side + sub, p = h.x + r;
        to[u] = -1;
        if (r < h.y) {
          const int s = p >= h.z && a.path ? h.z + __ldcg(a.path + (size_t)b * a.path_stride + (p - h.z)) : p;
          from[u] = __ldcg(m->from + (s >> a.page_log2) - page0);
          to[u] = __ldcg(m->to + (p >> a.page_log2) - page0);
          sat[u] = (s & (ps - 1)) << a.vecs_log2;
          dat[u] = (p & (ps - 1)) << a.vecs_log2;
          if (from[u] < 0 || from[u] >= a.n_pages || to[u] < 0 || to[u] >= a.n_pages) {
            atomicOr(a.status, CACHE_BAD_PAGE);
            to[u] = -1;
          } else if (from[u] == to[u] && s == p) {
            to[u] = -1;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (to[u] >= 0) {
          v[u] = __ldcg(one + from[u] * stride1 + sat[u]);
          w[u] = __ldcg(two + from[u] * stride2 + sat[u]);
        }
      __syncwarp();                  // a row may be another lane's to read before it is this one's to write
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (to[u] >= 0) {
          __stcg(one + to[u] * stride1 + dat[u], v[u]);
          if (second != pool) __stcg(two + to[u] * stride2 + dat[u], w[u]);
        }
      __syncwarp();
    }
  }
}

cudaError_t move(const CacheShape& S, const CacheMoves* moves, const int32_t* path, int64_t path_stride, int n,
                 void* const* pools, const int64_t* strides, int n_pools, uint32_t* status, int num_sms, cudaStream_t st) {
  MoveArgs a;
  a.moves = moves;
  a.path = path;
  a.path_stride = path_stride;
  a.n = n;
  a.heads = S.Hkv;
  a.page_log2 = S.page_log2;
  a.n_pages = S.n_pages;
  const int per = S.e4m3 ? 16 : 8;                 // elements of a vector
  a.vecs_log2 = 0;
  while ((per << a.vecs_log2) < S.D) ++a.vecs_log2;
  a.status = status;
  for (int i = 0; i < n_pools; i += POOLS) {
    a.n_pools = n_pools - i < POOLS ? n_pools - i : POOLS;
    for (int j = 0; j < a.n_pools; ++j) {
      a.pools[j] = (uint4*)pools[i + j];
      a.strides[j] = strides[i + j] / per;
    }
    a.pairs = (a.n_pools + 1) / 2;
    // the record's rows: up to a page without a path
    a.chunks = path ? 1 : ((1 << S.page_log2) + 8 * (32 >> a.vecs_log2) - 1) / (8 * (32 >> a.vecs_log2));
    const unsigned long long want = ((unsigned long long)n * a.heads * a.pairs * a.chunks * 32 + MOVE_THREADS - 1) / MOVE_THREADS;
    const unsigned most = num_sms * (2048 / MOVE_THREADS);
    const cudaError_t e = launch_following(k_cache_move, want < most ? (unsigned)want : most, MOVE_THREADS, 0, st, a);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// one cluster: a CTA for every 16 requests, so that a warp has one, up to the portable 8
int cluster_size(int n) {
  int c = 1;
  while (c < MAX_CLUSTER && c * WARPS < n) c *= 2;
  return c;
}
template <class A>
cudaError_t launch_cluster(void (*kernel)(const A), int ctas, size_t smem, cudaStream_t st, const A& args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(ctas);
  c.blockDim = dim3(THREADS);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  cudaLaunchAttribute a[2];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  a[1].id = cudaLaunchAttributeClusterDimension;
  a[1].val.clusterDim.x = ctas;
  a[1].val.clusterDim.y = a[1].val.clusterDim.z = 1;
  c.attrs = a;
  c.numAttrs = 2;
  return cudaLaunchKernelEx(&c, kernel, args);
}
constexpr size_t KEEP_SMEM = (CACHE_MAX_REQUESTS / MAX_CLUSTER + WARPS) * sizeof(Kept) + CACHE_MAX_REQUESTS * 8;
constexpr size_t FORK_SMEM = CACHE_MAX_REQUESTS * 12;

}  // namespace

cudaError_t cache_pages_init() {
  cudaError_t e = cudaFuncSetAttribute(k_cache_keep, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)KEEP_SMEM);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k_cache_fork, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)FORK_SMEM);
  return e;
}

cudaError_t cache_keep_launch(const CacheShape& S, const moe_cache_keep_t& k, int max_new, CacheMoves* moves,
                              uint32_t* status, int num_sms, cudaStream_t st) {
  KeepArgs a;
  a.k = k;
  a.B = (int)k.n_requests;
  a.rows = (int)k.n_rows;
  a.page_log2 = S.page_log2;
  a.n_pages = S.n_pages;
  a.most = max_new;
  a.move = k.path || k.refs;
  a.max_len = (long long)S.max_pages << S.page_log2;
  a.moves = moves;
  a.status = status;
  const int ctas = cluster_size(a.B);
  a.local = (a.B + ctas - 1) / ctas;
  const cudaError_t e = launch_cluster(k_cache_keep, ctas, a.local * sizeof(Kept) + (size_t)a.B * 8, st, a);
  // without a path no row moves but of pages that are exchanged, without refs none is
  if (e != cudaSuccess || !a.move || k.n_pools == 0 || a.B == 0) return e;
  return move(S, moves, k.path, k.path_stride, a.B, k.pools, k.page_strides, (int)k.n_pools, status, num_sms, st);
}

cudaError_t cache_fork_launch(const CacheShape& S, const moe_cache_fork_t& f, CacheMoves* moves, uint32_t* status,
                              int num_sms, cudaStream_t st) {
  ForkArgs a;
  a.f = f;
  a.B = (int)f.n_requests;
  a.n = (int)f.n_entries;
  a.page_log2 = S.page_log2;
  a.n_pages = S.n_pages;
  a.max_len = (long long)S.max_pages << S.page_log2;
  a.moves = moves;
  a.status = status;
  const int ctas = cluster_size(a.n);
  const cudaError_t e = launch_cluster(k_cache_fork, ctas, ((size_t)a.B + 2 * (size_t)a.n) * 4, st, a);
  if (e != cudaSuccess || f.n_pools == 0 || a.n == 0) return e;
  return move(S, moves, nullptr, 0, a.n, f.pools, f.page_strides, (int)f.n_pools, status, num_sms, st);
}

}  // namespace moe
