// C ABI of the paged key-value cache (declared in include/moe_block.h): argument checks, the handle's device memory
// and dispatch. No call throws or aborts; every failure is a negative status.
#include <cuda_runtime.h>
#include <math.h>
#include <new>
#include <stdio.h>
#include <stdlib.h>

#include "cache.cuh"

using namespace moe;

struct moe_cache {
  moe_cache_config_t cfg;
  CacheShape S;
  int dev = 0, num_sms = 0;
  uint8_t* mem = nullptr;                // one allocation: control words, the frequencies (1 KB), the workspace
  uint32_t *status = nullptr, *arrivals = nullptr;
  uint64_t* turns = nullptr;
  uint8_t* workspace = nullptr;          // of the attention: counts, partial results
  size_t workspace_bytes = 0;
  uint64_t timeout_ns = 500ull * 1000 * 1000;
  int skip_copy = 0;
  // of moe_cache_reserve: the rows that calls move, the tree attention's workspace
  int max_new = 0;
  uint8_t* reserved = nullptr;
};

namespace {

constexpr int CTL_WORDS = 64;
constexpr double MAX_SCALE = 2.35e38;    // of the attention, which multiplies it by log2(e) in fp32

int check_config(const moe_cache_config_t& c, CacheShape* S) {
  if (c.n_kv_heads < 1 || c.n_kv_heads > 256 || c.n_heads < 1 || c.n_heads % c.n_kv_heads ||
      c.n_heads / c.n_kv_heads > CACHE_MAX_GROUP)
    return MOE_ERR_UNSUPPORTED;
  if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) return MOE_ERR_UNSUPPORTED;
  int lg = 4;
  while (lg < 8 && (1 << lg) != c.page_size) ++lg;
  if ((1 << lg) != c.page_size) return MOE_ERR_UNSUPPORTED;
  if (c.n_pages < 1 || c.max_pages < 1 || ((int64_t)c.n_pages << lg) > INT32_MAX ||
      ((int64_t)c.max_pages << lg) > INT32_MAX)
    return MOE_ERR_UNSUPPORTED;
  if (c.max_requests < 1 || c.max_requests > CACHE_MAX_REQUESTS) return MOE_ERR_UNSUPPORTED;
  // the attention numbers its tiles, of 64 tokens or more for each head, in 31 bits
  if (((int64_t)c.max_pages << lg) * c.max_requests > ((int64_t)1 << 36) / c.n_heads) return MOE_ERR_UNSUPPORTED;
  if (c.act_dtype != MOE_DTYPE_F16 && c.act_dtype != MOE_DTYPE_BF16) return MOE_ERR_UNSUPPORTED;
  if (c.cache_dtype != c.act_dtype && c.cache_dtype != MOE_DTYPE_E4M3) return MOE_ERR_UNSUPPORTED;
  if (c.rope_dim < 0 || c.rope_dim > c.head_dim || c.rope_dim % 16) return MOE_ERR_UNSUPPORTED;
  if (c.rope_dim && !(c.rope_theta > 1.0 && isfinite(c.rope_theta))) return MOE_ERR_UNSUPPORTED;
  if (!isfinite(c.gamma_offset) || !(c.norm_eps >= 0.f) || !isfinite(c.norm_eps)) return MOE_ERR_UNSUPPORTED;
  S->Hq = c.n_heads;
  S->Hkv = c.n_kv_heads;
  S->D = c.head_dim;
  S->page_log2 = lg;
  S->n_pages = c.n_pages;
  S->max_pages = c.max_pages;
  S->rope = c.rope_dim;
  S->bf16 = c.act_dtype == MOE_DTYPE_BF16;
  S->e4m3 = c.cache_dtype == MOE_DTYPE_E4M3;
  S->gamma_offset = c.gamma_offset;
  S->eps = c.norm_eps;
  return MOE_OK;
}

bool aligned(const void* p, int n) { return p && ((uintptr_t)p & (n - 1)) == 0; }
// strides and their products with the rows and pages are bounded, so that every offset in bytes fits 62 bits
bool within(int64_t v, int bits) { return v > -((int64_t)1 << bits) && v < (int64_t)1 << bits; }
constexpr int64_t FARTHEST = (int64_t)1 << 60;
bool rows_ok(const moe_rows_t& r, int64_t n) {
  return aligned(r.p, 16) && r.row_stride % 8 == 0 && r.head_stride % 8 == 0 && within(r.row_stride, 40) &&
         within(r.head_stride, 30) && llabs(r.row_stride) <= FARTHEST / n;
}
// a pool: 16-byte aligned, pages that do not overlap, whole rows of D and whole lines of 128 bytes apart
bool pool_ok(const CacheShape& S, const void* p, int64_t page_stride) {
  return aligned(p, 16) && page_stride >= ((int64_t)S.Hkv << S.page_log2) * S.D && page_stride < (int64_t)1 << 38 &&
         page_stride <= FARTHEST / S.n_pages && page_stride % S.D == 0 &&
         (S.e4m3 ? page_stride : 2 * page_stride) % 128 == 0;
}
bool scales_ok(const CacheShape& S, const float* k, const float* v) {
  return S.e4m3 ? aligned(k, 4) && aligned(v, 4) : !k && !v;
}
bool table_ok(const moe_cache_config_t& cfg, int64_t stride) {
  return stride >= cfg.max_pages && stride < (int64_t)1 << 40;
}

// what each call refuses: MOE_OK or MOE_ERR_INVALID_ARG
int check_plan(const moe_cache_config_t& cfg, const moe_cache_plan_t& p) {
  if (p.n_requests < 0 || p.n_requests > cfg.max_requests || p.n_rows < 0 || p.n_rows > INT32_MAX)
    return MOE_ERR_INVALID_ARG;
  if (p.n_requests > 0 && (!aligned(p.lengths, 4) || !aligned(p.tables, 4) || !aligned(p.lengths_out, 4) ||
                           !table_ok(cfg, p.table_stride) || ((uintptr_t)p.new_tokens & 3)))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(p.free_pages, 4) || !aligned(p.free_state, 4) || !aligned(p.free_state_out, 4) || !aligned(p.starts, 4))
    return MOE_ERR_INVALID_ARG;
  if (p.n_rows > 0 && (!aligned(p.slots, 4) || !aligned(p.positions, 4))) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}
int check_write(const CacheShape& S, const moe_cache_write_t& w) {
  if (w.n_rows < 0 || w.n_rows > (int64_t)1 << 24) return MOE_ERR_INVALID_ARG;
  if (w.n_rows == 0) return MOE_OK;
  if ((w.q.p != nullptr) != (w.q_out.p != nullptr) ||
      (w.q.p && (!rows_ok(w.q, w.n_rows) || !rows_ok(w.q_out, w.n_rows))) || !rows_ok(w.k, w.n_rows) ||
      !rows_ok(w.v, w.n_rows) || ((uintptr_t)w.q_gamma & 15) || ((uintptr_t)w.k_gamma & 15) ||
      !aligned(w.positions, 4) || !aligned(w.slots, 4) || !pool_ok(S, w.k_cache, w.k_page_stride) ||
      !pool_ok(S, w.v_cache, w.v_page_stride) || !scales_ok(S, w.k_scale, w.v_scale))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}
int check_attend(const moe_cache_config_t& cfg, const CacheShape& S, const moe_cache_attend_t& a) {
  if (a.n_requests < 0 || a.n_requests > cfg.max_requests || !(fabs(a.scale) <= MAX_SCALE)) return MOE_ERR_INVALID_ARG;
  if (a.n_requests == 0) return MOE_OK;
  if (!rows_ok(a.q, a.n_requests) || (a.gate.p && !rows_ok(a.gate, a.n_requests)) || !rows_ok(a.out, a.n_requests) ||
      !aligned(a.tables, 4) || !table_ok(cfg, a.table_stride) || !aligned(a.lengths, 4) ||
      !pool_ok(S, a.k_cache, a.k_page_stride) || !pool_ok(S, a.v_cache, a.v_page_stride) ||
      !scales_ok(S, a.k_scale, a.v_scale))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

constexpr int64_t MAX_ROWS = (int64_t)1 << 24;
bool batch_ok(const moe_cache_config_t& cfg, int64_t n_requests, int64_t n_rows) {
  return n_requests >= 0 && n_requests <= cfg.max_requests && n_rows >= 0 && n_rows <= MAX_ROWS;
}
bool ring_ok(const void* pages, const void* state, const void* state_out) {
  return aligned(pages, 4) && aligned(state, 4) && aligned(state_out, 4);
}
bool pools_ok(const CacheShape& S, void* const* pools, const int64_t* strides, int64_t n) {
  if (n < 0 || n > 1024 || (n > 0 && (!pools || !strides))) return false;
  for (int64_t i = 0; i < n; ++i)
    if (!pool_ok(S, pools[i], strides[i])) return false;
  // rows that move in a pool named twice would move twice: the addresses go into a table, at most half full, by a
  // multiplicative hash (1024 pools 10 us, 464 where each was compared with each)
  constexpr int LOG2 = 11;
  uint16_t at[1 << LOG2] = {};                     // a pool's number and 1
  for (int64_t i = 0; i < n; ++i) {
    uint32_t h = (uint32_t)(((uint64_t)(uintptr_t)pools[i] >> 4) * 0x9E3779B97F4A7C15ull >> (64 - LOG2));
    for (; at[h]; h = (h + 1) & ((1 << LOG2) - 1))
      if (pools[at[h] - 1] == pools[i]) return false;
    at[h] = (uint16_t)(i + 1);
  }
  return true;
}
int check_tree(const moe_cache_config_t& cfg, const moe_cache_tree_t& t) {
  if (!batch_ok(cfg, t.n_requests, t.n_rows) || t.mask_words < 1 || t.mask_words > CACHE_MAX_NEW / 64)
    return MOE_ERR_INVALID_ARG;
  if (t.n_rows == 0) return MOE_OK;
  if (!aligned(t.masks, 8) || !aligned(t.positions, 4) || ((uintptr_t)t.slots & 3) ||
      (t.n_requests > 0 && (!aligned(t.parents, 4) || !aligned(t.starts, 4) || !aligned(t.lengths, 4))))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}
int check_attend_tree(const moe_cache_config_t& cfg, const CacheShape& S, const moe_cache_attend_tree_t& a) {
  if (!batch_ok(cfg, a.n_requests, a.n_rows) || !(fabs(a.scale) <= MAX_SCALE) ||
      (a.masks && (a.mask_words < 1 || a.mask_words > CACHE_MAX_NEW / 64)))
    return MOE_ERR_INVALID_ARG;
  if (a.n_requests == 0 || a.n_rows == 0) return MOE_OK;
  if (!rows_ok(a.q, a.n_rows) || (a.gate.p && !rows_ok(a.gate, a.n_rows)) || !rows_ok(a.out, a.n_rows) ||
      !aligned(a.starts, 4) || ((uintptr_t)a.slots & 3) || ((uintptr_t)a.masks & 7) || !aligned(a.tables, 4) ||
      !table_ok(cfg, a.table_stride) || !aligned(a.lengths, 4) || !pool_ok(S, a.k_cache, a.k_page_stride) ||
      !pool_ok(S, a.v_cache, a.v_page_stride) || !scales_ok(S, a.k_scale, a.v_scale))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}
int check_keep(const moe_cache_config_t& cfg, const CacheShape& S, const moe_cache_keep_t& k) {
  if (!batch_ok(cfg, k.n_requests, k.n_rows) || !ring_ok(k.free_pages, k.free_state, k.free_state_out) ||
      ((uintptr_t)k.starts & 3) || ((uintptr_t)k.slots & 3) || ((uintptr_t)k.path & 3) || ((uintptr_t)k.refs & 3) ||
      (!k.starts && (k.path || k.slots)) || !pools_ok(S, k.pools, k.page_strides, k.n_pools))
    return MOE_ERR_INVALID_ARG;
  if (k.n_requests == 0) return MOE_OK;
  if (!aligned(k.counts, 4) || !aligned(k.lengths, 4) || !aligned(k.lengths_out, 4) || !aligned(k.tables, 4) ||
      !table_ok(cfg, k.table_stride) || (k.path && (k.path_stride < 1 || k.path_stride >= (int64_t)1 << 40)))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}
int check_fork(const moe_cache_config_t& cfg, const CacheShape& S, const moe_cache_fork_t& f) {
  if (!batch_ok(cfg, f.n_requests, 0) || f.n_entries < 0 || f.n_entries > cfg.max_requests ||
      !ring_ok(f.free_pages, f.free_state, f.free_state_out) || !aligned(f.refs, 4) ||
      !pools_ok(S, f.pools, f.page_strides, f.n_pools))
    return MOE_ERR_INVALID_ARG;
  if (f.n_entries > 0 && (!aligned(f.src, 4) || !aligned(f.dst, 4))) return MOE_ERR_INVALID_ARG;
  if (f.n_requests > 0 && (!aligned(f.lengths, 4) || !aligned(f.lengths_out, 4) || !aligned(f.tables, 4) ||
                           !table_ok(cfg, f.table_stride)))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

}  // namespace

extern "C" int moe_cache_create(const moe_cache_config_t* cfg, moe_cache_t** out) {
  if (!cfg || !out) return MOE_ERR_INVALID_ARG;
  CacheShape S;
  const int cs = check_config(*cfg, &S);
  if (cs != MOE_OK) return cs;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_NO_DEVICE;
  cudaDeviceProp prop;
  if (cudaGetDeviceProperties(&prop, dev) != cudaSuccess) return MOE_ERR_NO_DEVICE;
  if (prop.major != 10 || prop.minor != 3) return MOE_ERR_NO_DEVICE;
  moe_cache* c = new (std::nothrow) moe_cache;
  if (!c) return MOE_ERR_CUDA;
  c->cfg = *cfg;
  c->S = S;
  c->dev = dev;
  c->num_sms = prop.multiProcessorCount;
  c->workspace_bytes = cache_attend_workspace(c->num_sms);
  const size_t bytes = CTL_WORDS * 4 + 1024 + c->workspace_bytes;
  uint64_t turns[128];
  for (int i = 0; i < S.rope / 2; ++i)
    turns[i] = (uint64_t)ldexp(pow(cfg->rope_theta, -2.0 * i / S.rope) / (2.0 * 3.14159265358979323846), 64);
  cudaError_t e = cache_plan_init();
  if (e == cudaSuccess) e = cudaMalloc(&c->mem, bytes);
  if (e == cudaSuccess) e = cudaMemset(c->mem, 0, bytes);
  if (e == cudaSuccess && S.rope)
    e = cudaMemcpy(c->mem + CTL_WORDS * 4, turns, (size_t)(S.rope / 2) * 8, cudaMemcpyHostToDevice);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    cudaFree(c->mem);
    delete c;
    return report_cuda(e, "moe_cache_create");
  }
  c->status = (uint32_t*)c->mem;
  c->arrivals = c->status + 1;
  c->turns = (uint64_t*)(c->mem + CTL_WORDS * 4);
  c->workspace = c->mem + CTL_WORDS * 4 + 1024;
  *out = c;
  return MOE_OK;
}

// a handle works on the device that was current when it was made
static bool on_device(const moe_cache* c) {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev == c->dev;
}
// makes a device current for as long as it lives
struct OnDevice {
  int before = -1;
  cudaError_t e;
  explicit OnDevice(int dev) {
    e = cudaGetDevice(&before);
    if (e == cudaSuccess && before == dev) before = -1;
    else if (e == cudaSuccess) e = cudaSetDevice(dev);
  }
  ~OnDevice() {
    if (before >= 0) cudaSetDevice(before);
  }
};

extern "C" void moe_cache_destroy(moe_cache_t* c) {
  if (!c) return;
  {
    const OnDevice on(c->dev);
    cudaDeviceSynchronize();
    cudaFree(c->mem);
    cudaFree(c->reserved);
  }
  delete c;
}

extern "C" int moe_debug_cache_check(const moe_cache_config_t* cfg, const moe_cache_plan_t* p,
                                     const moe_cache_write_t* w, const moe_cache_attend_t* a) {
  if (!cfg) return MOE_ERR_INVALID_ARG;
  CacheShape S;
  int st = check_config(*cfg, &S);
  if (st == MOE_OK && p) st = check_plan(*cfg, *p);
  if (st == MOE_OK && w) st = check_write(S, *w);
  if (st == MOE_OK && a) st = check_attend(*cfg, S, *a);
  return st;
}

extern "C" int moe_cache_plan(moe_cache_t* c, const moe_cache_plan_t* p, void* stream) {
  if (!c || !p) return MOE_ERR_INVALID_ARG;
  const int r = check_plan(c->cfg, *p);
  if (r != MOE_OK) return r;
  if (!on_device(c)) return MOE_ERR_INVALID_ARG;
  const cudaError_t e = cache_plan_launch(c->S, *p, c->arrivals, c->status, c->num_sms, (cudaStream_t)stream);
  return e == cudaSuccess ? MOE_OK : report_cuda(e, "moe_cache_plan");
}

extern "C" int moe_cache_write(moe_cache_t* c, const moe_cache_write_t* w, void* stream) {
  if (!c || !w) return MOE_ERR_INVALID_ARG;
  const int r = check_write(c->S, *w);
  if (r != MOE_OK || w->n_rows == 0) return r;
  if (!on_device(c)) return MOE_ERR_INVALID_ARG;
  const cudaError_t e = cache_write_launch(c->S, *w, c->turns, c->status, c->num_sms, (cudaStream_t)stream);
  return e == cudaSuccess ? MOE_OK : report_cuda(e, "moe_cache_write");
}

extern "C" int moe_cache_attend(moe_cache_t* c, const moe_cache_attend_t* a, void* stream) {
  if (!c || !a) return MOE_ERR_INVALID_ARG;
  const int r = check_attend(c->cfg, c->S, *a);
  if (r != MOE_OK || a->n_requests == 0) return r;
  if (!on_device(c)) return MOE_ERR_INVALID_ARG;
  const CacheAttendState w{c->workspace, c->status, c->num_sms, c->timeout_ns, c->skip_copy};
  c->skip_copy = 0;
  const cudaError_t e = cache_attend_launch(c->S, *a, w, (cudaStream_t)stream);
  return e == cudaSuccess ? MOE_OK : report_cuda(e, "moe_cache_attend");
}

// ---- several new tokens of a request ----
namespace {
size_t moves_bytes(const moe_cache* c) { return ((size_t)c->cfg.max_requests * sizeof(CacheMoves) + 255) & ~(size_t)255; }
// what the calls below check beside their arguments
int ready(const moe_cache* c) {
  if (!c->max_new) return MOE_ERR_NOT_LOADED;
  return on_device(c) ? MOE_OK : MOE_ERR_INVALID_ARG;
}
}  // namespace

extern "C" int moe_cache_reserve(moe_cache_t* c, int max_new) {
  if (!c || c->max_new || !on_device(c)) return MOE_ERR_INVALID_ARG;
  if (max_new < 1 || max_new > CACHE_MAX_NEW) return MOE_ERR_UNSUPPORTED;
  const size_t bytes = moves_bytes(c) + cache_attend_tree_workspace(c->num_sms, c->S.D);
  cudaError_t e = cache_pages_init();
  if (e == cudaSuccess) e = cudaMalloc(&c->reserved, bytes);
  if (e == cudaSuccess) e = cudaMemset(c->reserved, 0, bytes);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    cudaFree(c->reserved);
    c->reserved = nullptr;
    return report_cuda(e, "moe_cache_reserve");
  }
  c->max_new = max_new;
  return MOE_OK;
}

extern "C" int moe_cache_tree(moe_cache_t* c, const moe_cache_tree_t* t, void* stream) {
  if (!c || !t) return MOE_ERR_INVALID_ARG;
  int r = check_tree(c->cfg, *t);
  if (r == MOE_OK) r = ready(c);
  if (r != MOE_OK || t->n_rows == 0) return r;
  const cudaError_t e = cache_tree_launch(c->S, *t, c->max_new, c->status, (cudaStream_t)stream);
  return e == cudaSuccess ? MOE_OK : report_cuda(e, "moe_cache_tree");
}

extern "C" int moe_cache_attend_tree(moe_cache_t* c, const moe_cache_attend_tree_t* a, void* stream) {
  if (!c || !a) return MOE_ERR_INVALID_ARG;
  int r = check_attend_tree(c->cfg, c->S, *a);
  if (r == MOE_OK) r = ready(c);
  if (r != MOE_OK || a->n_requests == 0 || a->n_rows == 0) return r;
  const CacheTreeState w{c->reserved + moves_bytes(c), c->status, c->num_sms, c->max_new, c->timeout_ns,
                         c->skip_copy};
  c->skip_copy = 0;
  const cudaError_t e = cache_attend_tree_launch(c->S, *a, w, (cudaStream_t)stream);
  return e == cudaSuccess ? MOE_OK : report_cuda(e, "moe_cache_attend_tree");
}

extern "C" int moe_cache_keep(moe_cache_t* c, const moe_cache_keep_t* k, void* stream) {
  if (!c || !k) return MOE_ERR_INVALID_ARG;
  int r = check_keep(c->cfg, c->S, *k);
  if (r == MOE_OK) r = ready(c);
  if (r != MOE_OK) return r;
  const cudaError_t e = cache_keep_launch(c->S, *k, c->max_new, (CacheMoves*)c->reserved, c->status, c->num_sms,
                                          (cudaStream_t)stream);
  return e == cudaSuccess ? MOE_OK : report_cuda(e, "moe_cache_keep");
}

extern "C" int moe_cache_fork(moe_cache_t* c, const moe_cache_fork_t* f, void* stream) {
  if (!c || !f) return MOE_ERR_INVALID_ARG;
  int r = check_fork(c->cfg, c->S, *f);
  if (r == MOE_OK) r = ready(c);
  if (r != MOE_OK) return r;
  const cudaError_t e = cache_fork_launch(c->S, *f, (CacheMoves*)c->reserved, c->status, c->num_sms,
                                          (cudaStream_t)stream);
  return e == cudaSuccess ? MOE_OK : report_cuda(e, "moe_cache_fork");
}

extern "C" int moe_debug_cache_check_new(const moe_cache_config_t* cfg, int max_new, const moe_cache_tree_t* t,
                                         const moe_cache_attend_tree_t* a, const moe_cache_keep_t* k,
                                         const moe_cache_fork_t* f) {
  if (!cfg) return MOE_ERR_INVALID_ARG;
  CacheShape S;
  int st = check_config(*cfg, &S);
  if (st == MOE_OK && (max_new < 1 || max_new > CACHE_MAX_NEW)) st = MOE_ERR_UNSUPPORTED;
  if (st == MOE_OK && t) st = check_tree(*cfg, *t);
  if (st == MOE_OK && a) st = check_attend_tree(*cfg, S, *a);
  if (st == MOE_OK && k) st = check_keep(*cfg, S, *k);
  if (st == MOE_OK && f) st = check_fork(*cfg, S, *f);
  return st;
}

extern "C" int moe_cache_debug_set_wait(moe_cache_t* c, uint32_t timeout_us, int skip_copy) {
  if (!c) return MOE_ERR_INVALID_ARG;
  c->timeout_ns = timeout_us ? (uint64_t)timeout_us * 1000ull : 500ull * 1000 * 1000;
  c->skip_copy = skip_copy ? 1 : 0;
  return MOE_OK;
}

extern "C" int moe_cache_get_status(moe_cache_t* c, uint32_t* flags) {
  if (!c) return MOE_ERR_INVALID_ARG;
  const OnDevice on(c->dev);
  // the whole device: a captured call runs on whatever stream its graph is launched on, which the handle never sees
  cudaError_t e = on.e;
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  uint32_t st = 0;
  if (e == cudaSuccess) e = cudaMemcpy(&st, c->status, 4, cudaMemcpyDeviceToHost);
  if (e == cudaSuccess && st) e = cudaMemset(c->status, 0, 4);
  // the counts of parts too where a call gave up, which may have left some behind
  if (e == cudaSuccess && st & CACHE_BAD_WAIT) e = cudaMemset(c->mem, 0, CTL_WORDS * 4);
  if (e == cudaSuccess && st & CACHE_BAD_WAIT) e = cudaMemset(c->workspace, 0, c->workspace_bytes);
  if (e == cudaSuccess && st & CACHE_BAD_WAIT && c->reserved)
    e = cudaMemset(c->reserved + moves_bytes(c), 0, CACHE_TREE_COUNTS);
  if (e == cudaSuccess && st) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return report_cuda(e, "moe_cache_get_status");
  if (flags) *flags = st;
  return st & CACHE_BAD_WAIT ? MOE_ERR_DEVICE_TIMEOUT : st ? MOE_ERR_INVALID_ARG : MOE_OK;
}
