// Ancestor masks and positions of drafted trees from the tokens' parents (moe_cache_tree).
//
// A row's ancestors are its parent's and the parent itself. Every row holds the ancestors found so far as a mask and the
// next one up; a step ORs the mask of the next one up into its own and takes over that one's next, which doubles how far a
// row has looked: 8 steps do for 256 tokens, and fewer once no row has anyone left to ask. A request is a CTA's, its
// masks in shared memory; the call is bound by its launch and the dependent loads starts - slots - parents.
#include "cache.cuh"

namespace moe {
namespace {

struct TreeArgs {
  moe_cache_tree_t t;
  int B, rows, most;
  long long max_len;
  uint32_t* status;
};

// W: mask words; a thread to a token
template <int W>
__global__ void __launch_bounds__(64 * W) k_cache_tree(const __grid_constant__ TreeArgs a) {
  __shared__ uint64_t s_mask[2][64 * W][W];
  __shared__ int s_up[2][64 * W];
  const moe_cache_tree_t& t = a.t;
  const int i = threadIdx.x;
  follow_predecessor();
  if ((int)blockIdx.x == a.B) {           // rows past the last token
    int from = a.B ? __ldcg(t.starts + a.B) : 0;
    from = from < 0 ? 0 : from;
    for (int r = from + i; r < a.rows; r += 64 * W) {
      t.positions[r] = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) t.masks[(size_t)r * W + w] = 0;
    }
    return;
  }
  uint32_t bad = 0;
  const NewTokens k = new_tokens_of(t.starts, t.slots, t.lengths, blockIdx.x, a.rows, a.max_len, a.most, &bad);
  if (k.left_out || k.n == 0) {
    for (int r = i; r < k.rows; r += 64 * W) {
      t.positions[k.lo + r] = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) t.masks[(size_t)(k.lo + r) * W + w] = 0;
    }
    if (bad && i == 0) atomicOr(a.status, bad);
    return;
  }
  uint64_t mask[W];
  int up = -1;
#pragma unroll
  for (int w = 0; w < W; ++w) mask[w] = 0;
  if (i < k.n) {
    up = __ldcg(t.parents + k.lo + i);
    if (up < -1 || up >= i) {
      up = -1;
      atomicOr(a.status, CACHE_BAD_ROWS);
    }
#pragma unroll
    for (int w = 0; w < W; ++w)
      if (w == i >> 6) mask[w] = 1ull << (i & 63);
  }
  for (int s = 0;; s ^= 1) {
#pragma unroll
    for (int w = 0; w < W; ++w) s_mask[s][i][w] = mask[w];
    s_up[s][i] = up;
    if (!__syncthreads_or(up >= 0)) break;
    if (up >= 0) {
#pragma unroll
      for (int w = 0; w < W; ++w) mask[w] |= s_mask[s][up][w];
      up = s_up[s][up];
    }
  }
  if (i < k.n) {
    int depth = -1;                        // its ancestors and itself, less one
#pragma unroll
    for (int w = 0; w < W; ++w) {
      depth += __popcll(mask[w]);
      t.masks[(size_t)(k.lo + i) * W + w] = mask[w];
    }
    t.positions[k.lo + i] = k.len - k.n + depth;
  }
}

}  // namespace

cudaError_t cache_tree_launch(const CacheShape& S, const moe_cache_tree_t& t, int max_new, uint32_t* status,
                              cudaStream_t st) {
  TreeArgs a;
  a.t = t;
  a.B = (int)t.n_requests;
  a.rows = (int)t.n_rows;
  a.most = max_new < 64 * (int)t.mask_words ? max_new : 64 * (int)t.mask_words;
  a.max_len = (long long)S.max_pages << S.page_log2;
  a.status = status;
  auto* k = t.mask_words == 1 ? k_cache_tree<1> : t.mask_words == 2 ? k_cache_tree<2>
          : t.mask_words == 3 ? k_cache_tree<3> : k_cache_tree<4>;
  return launch_following(k, a.B + 1, 64 * (int)t.mask_words, 0, st, a);
}

}  // namespace moe
