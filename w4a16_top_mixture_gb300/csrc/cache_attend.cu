// Attention of one new token of each request over the paged cache (moe_cache_attend).
//
// Every cached key and value is read once from HBM and meets only the query heads of its group, so the bytes of the
// cache bound the kernel; all else is arranged to keep them coming.
//   Work. The tokens of a request and key-value head (an item) are cut into tiles of TN. The tiles of all items, one
//   after another, are divided evenly over the CTAs, whatever the requests' lengths are: a CTA walks its range, and an
//   item that crosses a CTA's border is split. Nobody waits: every CTA of a split item leaves its partial sums in the
//   workspace, and the one that counts itself last joins them, in the order of the tiles.
//   Copies. One warp walks the block table ahead of the rest and brings 16 tokens x 128 bytes at a time with TMA into a
//   ring of stages, keys and values of a tile in stages of their own, across the borders of items.
//   Products. Heads are the narrow side of the tensor cores' m16n8k16: S^T[tokens x heads] = K Q^T and
//   O^T[d x heads] = V^T P^T, so that eight query heads fill a tile. Four warps share a tile: each takes 16 (32) tokens
//   of S and then a quarter of d of O. One maximum for the four, exchanged through shared memory, lets O be kept once.
#include <cuda.h>

#include "cache.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int MATH_WARPS = 4, THREADS = 32 * (MATH_WARPS + 1);
constexpr int COUNT_WORDS = 2048;                 // of the workspace; two CTAs to each of at most 1024 SMs
constexpr float LOG2E = 1.4426950408889634f;

struct AttendArgs {
  moe_cache_attend_t a;
  int B, Hq, Hkv, group, head_tiles, page_log2, n_pages, n_stages;
  long long max_len;
  float scale;
  float* parts;              // [CTA][2][part_floats]: the item a CTA began in the middle of, the one it left so
  uint32_t* counts;          // [CTA]: parts that have arrived of the item that crosses the CTA's end
  uint32_t* status;
  uint64_t timeout_ns;
  int skip_copy;             // test: the first copy of CTA 0 is left out, so that its wait runs out
};

template <int D_, bool BF16_, bool E4M3_, int NT_>
struct Shape {
  static constexpr int D = D_, NT = NT_, NH = 8 * NT_;      // query heads of an item
  static constexpr bool BF16 = BF16_, E4M3 = E4M3_;
  static constexpr bool MMA_BF16 = BF16_ && !E4M3_;         // e4m3 is exact in fp16
  static constexpr int RB = D * (E4M3 ? 1 : 2);             // bytes of a token's row
  static constexpr int CB = RB < 128 ? RB : 128, CH = RB / CB;
  static constexpr int TN = RB >= 512 ? 64 : 128;           // tokens of a tile: stages of 8 to 32 KB
  static constexpr int MT = TN / 64;                        // 16-token tiles of S per warp
  static constexpr int KT = TN / 16;
  static constexpr int STAGE = TN * RB, GROUP_BYTES = 16 * RB;
  static constexpr int MD = D / 64;                         // 16-row tiles of O per warp
  static constexpr int PP = TN + 8;                         // pitch of P: rows of 8 fall on different banks
  static constexpr int PART = NH * D + 2 * NH;              // floats of a partial result: O, maxima, sums
  static constexpr int JOIN = 64;                           // parts joined per step
  static constexpr int MISC = 1024 /* barriers */ + NH * PP * 2 + MATH_WARPS * NH * 8 + JOIN * NH * 4 + 2 * NH * 4;
};

// ---- instructions ----
__device__ __forceinline__ void ldsm4(uint32_t r[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t r[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void tma_rows(void* dst, const CUtensorMap* m, int x, int row, int page, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(smem_u32(dst)), "l"(m), "r"(x), "r"(row), "r"(page), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void math_barrier() { named_bar(1, 32 * MATH_WARPS); }

// ---- the division of the work ----
// Tiles are numbered request by request, within a request head by head; chunk of them go to a CTA.
struct Division {
  long long tiles, chunk;
};
__host__ __device__ inline Division divide(long long tiles, int ctas) {
  Division d;
  d.tiles = tiles;
  d.chunk = (tiles + ctas - 1) / ctas;
  if (d.chunk < 1) d.chunk = 1;
  return d;
}

// A place in the list of tiles: tile j of request b's head h (h: key-value head and its tile of query heads).
struct Place {
  int b, h, j, n;      // n: tiles of each head of request b
  __device__ void find(const int* upto, int B, int heads, long long tile) {
    int lo = 0, hi = B - 1;      // the request that holds the tile: the first whose tiles end past it
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if ((long long)upto[mid] * heads > tile) hi = mid; else lo = mid + 1;
    }
    b = lo;
    const int first = b ? upto[b - 1] : 0;
    n = upto[b] - first;
    const long long in = tile - (long long)first * heads;
    h = (int)(in / n);
    j = (int)(in - (long long)h * n);
  }
  // to the first tile of the next item (which exists)
  __device__ void next_item(const int* upto, int heads) {
    j = 0;
    if (++h < heads) return;
    h = 0;
    do {
      ++b;
      n = upto[b] - upto[b - 1];
    } while (n == 0);
  }
};

// o += V^T P^T over the first `groups` groups of 16 tokens of a tile, of which the first `left` tokens count (EDGE). from:
// the lane's address in the tile's values, pbase: in P.
template <class S, bool EDGE>
__device__ __forceinline__ void add_values(float (&o)[S::MD][S::NT][4], uint32_t from, uint32_t pbase, int groups, int left,
                                           int t4) {
#pragma unroll
  for (int kt = 0; kt < S::KT; kt += 2) {
    if (EDGE && kt >= groups) break;
    const bool both = !EDGE || kt + 1 < groups;
    uint32_t p[S::NT][4];                  // two steps of 16 tokens
#pragma unroll
    for (int nt = 0; nt < S::NT; ++nt) ldsm4(p[nt], pbase + (nt * 8 * S::PP + kt * 16) * 2);
    // tokens past the end hold whatever memory holds: their values become zeros (their weights are)
    uint32_t keep[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = kt * 16 + i * 8 + 2 * t4;
      keep[i] = EDGE ? (tok < left ? 0xFFFFu : 0u) | (tok + 1 < left ? 0xFFFF0000u : 0u) : ~0u;
    }
    if (S::E4M3) {
      // a 16-byte chunk of 8 tokens, transposed as 16-bit units: bytes (t0 d0, t0 d1, t1 d0, t1 d1)
#pragma unroll
      for (int md = 0; md < S::MD; ++md) {
        uint32_t v[4], x[4][2];
        ldsm4_t(v, (from ^ (md << 4)) + kt * S::GROUP_BYTES);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t y = __byte_perm(v[i], 0, 0x3120);
          x[i][0] = e4m3x2_to_f16x2((uint16_t)y) & keep[i];
          x[i][1] = e4m3x2_to_f16x2((uint16_t)(y >> 16)) & keep[i];
        }
#pragma unroll
        for (int nt = 0; nt < S::NT; ++nt) {
          mma16816<false>(o[md][nt], x[0][0], x[0][1], x[1][0], x[1][1], p[nt][0], p[nt][1]);
          if (both) mma16816<false>(o[md][nt], x[2][0], x[2][1], x[3][0], x[3][1], p[nt][2], p[nt][3]);
        }
      }
    } else {
#pragma unroll
      for (int k2 = 0; k2 < 2; ++k2) {
        if (k2 && !both) break;
#pragma unroll
        for (int md = 0; md < S::MD; ++md) {
          uint32_t v[4];
          ldsm4_t(v, (from ^ (md << 5)) + (kt + k2) * S::GROUP_BYTES);
          if (EDGE) {
            v[0] &= keep[2 * k2];
            v[1] &= keep[2 * k2];
            v[2] &= keep[2 * k2 + 1];
            v[3] &= keep[2 * k2 + 1];
          }
#pragma unroll
          for (int nt = 0; nt < S::NT; ++nt)
            mma16816<S::MMA_BF16>(o[md][nt], v[0], v[1], v[2], v[3], p[nt][2 * k2], p[nt][2 * k2 + 1]);
        }
      }
    }
  }
}

template <class S>
__global__ void __launch_bounds__(THREADS, 2)
    k_cache_attend(const __grid_constant__ AttendArgs A, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap) {
  constexpr int D = S::D, NT = S::NT, NH = S::NH, TN = S::TN, MT = S::MT, KT = S::KT, MD = S::MD, PP = S::PP;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const ring = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* const misc = ring + A.n_stages * S::STAGE;
  uint64_t* const full = (uint64_t*)misc;            // [n_stages <= 32]
  uint64_t* const empty = full + 32;
  volatile int* const s_flags = (int*)(empty + 32);  // 0: a wait ran out; 1: last to arrive
  int* const s_scan = (int*)(empty + 32) + 4;        // [THREADS / 32 + 1]
  uint16_t* const s_p = (uint16_t*)(misc + 1024);    // [NH][PP]
  float* const s_max = (float*)(s_p + NH * PP);      // [MATH_WARPS][NH]
  float* const s_sum = s_max + MATH_WARPS * NH;      // [MATH_WARPS][NH]
  float* const s_w = s_sum + MATH_WARPS * NH;        // [JOIN][NH]
  float* const s_top = s_w + S::JOIN * NH;           // [2][NH]
  int* const s_upto = (int*)(s_top + 2 * NH);        // [B]: tiles of a head, of the requests up to this one
  int* const s_len = s_upto + A.B;                   // [B]

  const moe_cache_attend_t& a = A.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int heads = A.Hkv * A.head_tiles;

  if (tid == 0) {
    for (int s = 0; s < A.n_stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], MATH_WARPS);
    }
    fence_mbar_init();
    s_flags[0] = 0;
  }
  // lengths and the running number of tiles
  int carry = 0;
  for (int b0 = 0; b0 < A.B; b0 += THREADS) {
    const int b = b0 + tid;
    int len = b < A.B ? a.lengths[b] : 0;
    if (len < 0 || len > A.max_len) {
      atomicOr(A.status, CACHE_BAD_LENGTH);
      len = len < 0 ? 0 : (int)A.max_len;
    }
    int x = (int)(((long long)len + TN - 1) / TN);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s_scan[warp] = x;
    __syncthreads();
    int before = carry;
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) before += s_scan[w];
      carry += s_scan[w];
    }
    if (b < A.B) {
      s_upto[b] = before + x;
      s_len[b] = len;
    }
  }
  __syncthreads();
  const Division dv = divide((long long)carry * heads, gridDim.x);
  const long long first = dv.chunk * blockIdx.x;
  const long long last = first + dv.chunk < dv.tiles ? first + dv.chunk : dv.tiles;

  if (warp == MATH_WARPS) {
    // ---------------------------------------------------------------- copies
    if (first >= last) return;
    Place at;
    at.find(s_upto, A.B, heads, first);
    const int grp = lane / S::CH, chunk = lane % S::CH;
    int stage = 0;
    uint32_t phase = 0;
    bool skip = A.skip_copy && blockIdx.x == 0;
    // the page of this lane's 16 tokens, one tile ahead of its copies
    auto page_of = [&](const Place& p) {
      const long long tok = (long long)p.j * TN + grp * 16;
      if (grp >= KT || tok >= s_len[p.b]) return -1;
      int page = __ldg(a.tables + (long long)p.b * a.table_stride + (tok >> A.page_log2));
      if (page < 0 || page >= A.n_pages) {
        atomicOr(A.status, CACHE_BAD_PAGE);
        page = A.n_pages;               // out of range: the copy reads zeros
      }
      return page;
    };
    int page = page_of(at);
    for (long long t = first; t < last; ++t) {
      Place nx = at;
      if (t + 1 < last) {
        if (++nx.j == nx.n) nx.next_item(s_upto, heads);
      }
      const int page_next = t + 1 < last ? page_of(nx) : -1;
      const int left = s_len[at.b] - at.j * TN;
      const int groups = left >= TN ? KT : (left + 15) >> 4;
      const int row = ((at.h / A.head_tiles) << A.page_log2) + (((at.j * TN) + grp * 16) & ((1 << A.page_log2) - 1));
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const bool ok = mbar_wait(&empty[stage], phase ^ 1, A.timeout_ns);
        if (!ok && lane == 0) {
          s_flags[0] = 1;
          atomicOr(A.status, CACHE_BAD_WAIT);
        }
        __syncwarp();
        if (s_flags[0]) {
          // a wait ran out, here or in a math warp, which then no longer waits: nothing more is copied, and what is on
          // its way is waited for (boundedly) before the CTA ends. Earlier stages of this lap, later ones of the last.
          int s = stage;
          uint32_t ph = phase;
          for (int i = 0; i < A.n_stages; ++i) {
            if (s == 0) { s = A.n_stages; ph ^= 1; }
            --s;
            mbar_wait(&full[s], ph, A.timeout_ns);
          }
          return;
        }
        uint8_t* const dst = ring + stage * S::STAGE;
        if (lane == 0) mbar_expect_tx(&full[stage], groups * S::GROUP_BYTES);
        __syncwarp();
        if (page >= 0 && !skip)
          tma_rows(dst + grp * S::GROUP_BYTES + chunk * 16 * S::CB, kv ? &vmap : &kmap, chunk * (D / S::CH), row, page,
                   &full[stage]);
        skip = false;
        if (++stage == A.n_stages) { stage = 0; phase ^= 1; }
      }
      at = nx;
      page = page_next;
    }
    return;
  }

  // ------------------------------------------------------------------ products
  const int g = lane >> 2, t4 = lane & 3;
  auto rows_at = [&](const moe_rows_t& r, int b, int h, int d) {
    return (uint16_t*)r.p + b * r.row_stride + h * r.head_stride + d;
  };
  // requests of length 0
  for (int b = blockIdx.x; b < A.B; b += gridDim.x)
    if (s_len[b] == 0)
      for (int i = tid; i < A.Hq * D / 8; i += 32 * MATH_WARPS)
        *reinterpret_cast<uint4*>(rows_at(a.out, b, i / (D / 8), i % (D / 8) * 8)) = make_uint4(0, 0, 0, 0);
  if (first >= last) return;

  // Where a lane's rows of a stage lie. 16-byte chunk c of row r of a group of 16 tokens is at
  //   c / PER * 16 * CB + r * CB + ((c % PER) ^ swizzle(r)) * 16,      PER = CB / 16,
  // so with chunks that differ in a constant's bits alone, the address differs by an exclusive or with 16 * constant.
  constexpr int PER = S::CB / 16;
  auto in_group = [](int r, int c) {
    const int sw = S::CB == 128 ? r & 7 : (r >> 1) & 3;
    return (uint32_t)((c / PER) * (16 * S::CB) + r * S::CB + (((c % PER) ^ sw) << 4));
  };
  const uint32_t ring0 = smem_u32(ring);
  const uint32_t k_lane = ring0 + in_group(lane & 15, lane >> 4);
  const uint32_t v_lane = ring0 + (S::E4M3 ? (lane >> 4) * S::GROUP_BYTES + in_group(lane & 15, warp * MD)
                                           : in_group((lane & 7) + ((lane >> 4) << 3), warp * MD * 2 + ((lane >> 3) & 1)));
  auto wait_full = [&](int stage, uint32_t phase) {
    // once a wait has run out the outputs are lost: run to the end without waiting
    if (!mbar_try_wait(&full[stage], phase) && !s_flags[0] && !mbar_wait(&full[stage], phase, A.timeout_ns)) {
      s_flags[0] = 1;
      atomicOr(A.status, CACHE_BAD_WAIT);
    }
    __syncwarp();
  };

  Place at;
  at.find(s_upto, A.B, heads, first);
  int stage = 0;
  uint32_t phase = 0;
  long long t = first;
  while (t < last) {
    const int kvh = at.h / A.head_tiles, h_in = (at.h % A.head_tiles) * NH;
    const int h0 = kvh * A.group + h_in;                       // first query head of the item
    const int nh = A.group - h_in < NH ? A.group - h_in : NH;
    const int len = s_len[at.b];
    const int j0 = at.j;
    const int j1 = last - t < at.n - j0 ? j0 + (int)(last - t) : at.n;

    // Q as B fragments; with an e4m3 cache the k index runs 4t..4t+3 within 16 bytes of a row, as the codes do
    uint32_t q[D / 16][NT][2];
    float sf[NT][2];                                           // what a product is multiplied by, for 2^x
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const bool in = nt * 8 + g < nh;
      const uint16_t* src = rows_at(a.q, at.b, h0 + (in ? nt * 8 + g : 0), 0);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        if (S::E4M3) {
          const uint2 v = *reinterpret_cast<const uint2*>(src + ks * 16 + 4 * t4);
          q[ks][nt][0] = in ? v.x : 0;
          q[ks][nt][1] = in ? v.y : 0;
        } else {
          q[ks][nt][0] = in ? *reinterpret_cast<const uint32_t*>(src + ks * 16 + 2 * t4) : 0;
          q[ks][nt][1] = in ? *reinterpret_cast<const uint32_t*>(src + ks * 16 + 2 * t4 + 8) : 0;
        }
      }
      float up = 1.f;
      if (S::E4M3 && S::BF16) {
        // bf16 queries in fp16: scaled by a power of two to a largest element in [1, 2), which keeps every bit but
        // those of elements 2^-16 below it
        float m = 0.f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 f = unpack2<true>(q[ks][nt][i]);
            m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        const int e = (__float_as_int(m) >> 23) - 127;
        const bool fine = e > -100 && e < 100;
        up = fine ? __int_as_float((127 + e) << 23) : 1.f;
        const float down = fine ? __int_as_float((127 - e) << 23) : 1.f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 f = unpack2<true>(q[ks][nt][i]);
            q[ks][nt][i] = pack2<false>(f.x * down, f.y * down);
          }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        sf[nt][i] = A.scale * (S::E4M3 ? a.k_scale[kvh] * __shfl_sync(0xFFFFFFFFu, up, (2 * t4 + i) * 4) : 1.f);
    }

    float o[MD][NT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m[nt][i] = -INFINITY;
        l[nt][i] = 0.f;
      }
#pragma unroll
      for (int md = 0; md < MD; ++md)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[md][nt][i] = 0.f;
    }

    for (int j = j0; j < j1; ++j) {
      const int left = len - j * TN;                           // tokens of the request from this tile on
      const int groups = left >= TN ? KT : (left + 15) >> 4;
      // ---- S^T = K Q^T for this warp's groups of 16 tokens
      float s[MT][NT][4];
      wait_full(stage, phase);
      {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const int gr = mt * MATH_WARPS + warp;
          // two chains of accumulators: one would wait for each product's latency
          float s2[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[mt][nt][i] = s2[nt][i] = 0.f;
          if (gr < groups) {
            const uint32_t from = k_lane + stage * S::STAGE + gr * S::GROUP_BYTES;
            if (S::E4M3) {
#pragma unroll
              for (int c = 0; c < S::RB / 16; c += 2) {
                uint32_t k[4];
                ldsm4(k, (from ^ (c % PER << 4)) + c / PER * (16 * S::CB));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  mma16816<false>(s[mt][nt], e4m3x2_to_f16x2((uint16_t)k[0]), e4m3x2_to_f16x2((uint16_t)k[1]),
                                  e4m3x2_to_f16x2((uint16_t)(k[0] >> 16)), e4m3x2_to_f16x2((uint16_t)(k[1] >> 16)),
                                  q[c][nt][0], q[c][nt][1]);
                  mma16816<false>(s2[nt], e4m3x2_to_f16x2((uint16_t)k[2]), e4m3x2_to_f16x2((uint16_t)k[3]),
                                  e4m3x2_to_f16x2((uint16_t)(k[2] >> 16)), e4m3x2_to_f16x2((uint16_t)(k[3] >> 16)),
                                  q[c + 1][nt][0], q[c + 1][nt][1]);
                }
              }
            } else {
#pragma unroll
              for (int ks = 0; ks < D / 16; ++ks) {
                uint32_t k[4];
                ldsm4(k, (from ^ (2 * ks % PER << 4)) + 2 * ks / PER * (16 * S::CB));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma16816<S::MMA_BF16>(ks & 1 ? s2[nt] : s[mt][nt], k[0], k[1], k[2], k[3], q[ks][nt][0], q[ks][nt][1]);
              }
            }
          }
          const bool edge = left < (gr + 1) * 16;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float x = (s[mt][nt][i] + s2[nt][i]) * sf[nt][i & 1];
              s[mt][nt][i] = edge && gr * 16 + g + (i >> 1) * 8 >= left ? -INFINITY : x;
            }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stage]);
      if (++stage == A.n_stages) { stage = 0; phase ^= 1; }

      // ---- the tile's maximum for each head
      float top[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x = -INFINITY;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) x = fmaxf(x, fmaxf(s[mt][nt][i], s[mt][nt][2 + i]));
          x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
          top[nt][i] = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
        }
      if (lane < 4)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          *reinterpret_cast<float2*>(&s_max[warp * NH + nt * 8 + 2 * t4]) = make_float2(top[nt][0], top[nt][1]);
      math_barrier();
      bool moved = false;
      float c[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float2 x = make_float2(m[nt][0], m[nt][1]);
#pragma unroll
        for (int w = 0; w < MATH_WARPS; ++w) {
          const float2 y = *reinterpret_cast<const float2*>(&s_max[w * NH + nt * 8 + 2 * t4]);
          x.x = fmaxf(x.x, y.x);
          x.y = fmaxf(x.y, y.y);
        }
        const float nm[2] = {x.x, x.y};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          moved |= nm[i] != m[nt][i];
          // while there are only scores of -inf, the base is 0: their weights are 2^-inf = 0, not NaN
          const float base = nm[i] == -INFINITY ? 0.f : nm[i];
          c[nt][i] = exp2_fast(m[nt][i] - base);
          m[nt][i] = nm[i];
          float sum = 0.f;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float p = exp2_fast(s[mt][nt][2 * r + i] - base);
              s[mt][nt][2 * r + i] = p;
              sum += p;
            }
          l[nt][i] = l[nt][i] * c[nt][i] + sum;
        }
        // P^T for the second product: 16 bits a weight, an error of half a step of the cache's own type
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            *reinterpret_cast<uint32_t*>(&s_p[(nt * 8 + g) * PP + (mt * MATH_WARPS + warp) * 16 + 8 * r + 2 * t4]) =
                transpose8x8(pack2<S::MMA_BF16>(s[mt][nt][2 * r], s[mt][nt][2 * r + 1]));
      }
      if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
        for (int md = 0; md < MD; ++md)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[md][nt][i] *= c[nt][i & 1];
      }
      math_barrier();

      // ---- O^T += V^T P^T for this warp's quarter of d
      wait_full(stage, phase);
      {
        const uint32_t from = v_lane + stage * S::STAGE;
        const uint32_t pbase = smem_u32(s_p) + ((lane & 7) * PP + (lane >> 3) * 8) * 2;
        if (left >= TN) add_values<S, false>(o, from, pbase, KT, TN, t4);
        else add_values<S, true>(o, from, pbase, groups, left, t4);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stage]);
      if (++stage == A.n_stages) { stage = 0; phase ^= 1; }
    }

    // ---- the end of the item, or of the CTA's share of it
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = l[nt][i];
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 4);
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 8);
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 16);
        if (lane < 4) s_sum[warp * NH + nt * 8 + 2 * t4 + i] = x;
      }
    math_barrier();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < MATH_WARPS; ++w) x += s_sum[w * NH + nt * 8 + 2 * t4 + i];
        l[nt][i] = x;
      }
    const float vs = S::E4M3 ? a.v_scale[kvh] : 1.f;
    // the rows of d that an accumulator's two halves hold
    auto d_of = [&](int md, int r) {
      return S::E4M3 ? (warp * MD + md) * 16 + 2 * g + r : (warp * MD + md) * 16 + g + 8 * r;
    };
    if (j0 == 0 && j1 == at.n) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int h = nt * 8 + 2 * t4 + i;
          if (h >= nh) continue;
          const float f = vs / l[nt][i];
#pragma unroll
          for (int md = 0; md < MD; ++md)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float y = o[md][nt][2 * r + i] * f;
              const int d = d_of(md, r);
              if (a.gate.p) {
                const float x = unpack2<S::BF16>(*rows_at(a.gate, at.b, h0 + h, d)).x;
                y = y / (1.f + __expf(-x));
              }
              *rows_at(a.out, at.b, h0 + h, d) = (uint16_t)pack2<S::BF16>(y, 0.f);
            }
        }
    } else {
      // a part: the item's tiles are those of CTAs c0 .. c1; c0 holds its part as the item it left, the others as the
      // item they began in the middle of
      const long long t0 = t - j0;
      const int c0 = (int)(t0 / dv.chunk), c1 = (int)((t0 + at.n - 1) / dv.chunk);
      float* part = A.parts + ((long long)blockIdx.x * 2 + (j0 == 0 ? 1 : 0)) * S::PART;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int h = nt * 8 + 2 * t4 + i;
#pragma unroll
          for (int md = 0; md < MD; ++md)
#pragma unroll
            for (int r = 0; r < 2; ++r) part[h * D + d_of(md, r)] = o[md][nt][2 * r + i];
          if (warp == 0 && g == 0) {
            part[NH * D + h] = m[nt][i];
            part[NH * D + NH + h] = l[nt][i];
          }
        }
      __threadfence();
      math_barrier();
      if (tid == 0) s_flags[1] = atomicAdd(&A.counts[c0], 1u) == (uint32_t)(c1 - c0);
      math_barrier();
      if (s_flags[1]) {
        __threadfence();
        if (tid == 0) A.counts[c0] = 0;
        const int n = c1 - c0 + 1;
        auto nth = [&](int i) { return A.parts + ((long long)(c0 + i) * 2 + (i == 0 ? 1 : 0)) * S::PART; };
        // the largest maximum of each head
        {
          const int h = tid % NH;
          float x = -INFINITY;
          for (int i = tid / NH; i < n; i += 32 * MATH_WARPS / NH) x = fmaxf(x, __ldcg(nth(i) + NH * D + h));
#pragma unroll
          for (int w = NH; w < 32; w <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, w));
          if (lane < NH) s_max[warp * NH + lane] = x;
          math_barrier();
          x = -INFINITY;
#pragma unroll
          for (int w = 0; w < MATH_WARPS; ++w) x = fmaxf(x, s_max[w * NH + h]);
          if (tid < NH) s_top[h] = x == -INFINITY ? 0.f : x;
          math_barrier();
        }
        constexpr int PER = NH * D / 4 / (32 * MATH_WARPS);     // groups of four d per thread
        float4 y[PER];
        float sum[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e) {
          y[e] = make_float4(0.f, 0.f, 0.f, 0.f);
          sum[e] = 0.f;
        }
        for (int i0 = 0; i0 < n; i0 += S::JOIN) {
          const int ni = n - i0 < S::JOIN ? n - i0 : S::JOIN;
          for (int i = tid; i < ni * NH; i += 32 * MATH_WARPS)
            s_w[i] = exp2_fast(__ldcg(nth(i0 + i / NH) + NH * D + i % NH) - s_top[i % NH]);
          math_barrier();
#pragma unroll 4
          for (int i = 0; i < ni; ++i) {
            const float* p = nth(i0 + i);
#pragma unroll
            for (int e = 0; e < PER; ++e) {
              const int at4 = (e * 32 * MATH_WARPS + tid) * 4, h = at4 / D;
              const float w = s_w[i * NH + h];
              const float4 v = __ldcg(reinterpret_cast<const float4*>(p + at4));
              y[e].x = fmaf(v.x, w, y[e].x);
              y[e].y = fmaf(v.y, w, y[e].y);
              y[e].z = fmaf(v.z, w, y[e].z);
              y[e].w = fmaf(v.w, w, y[e].w);
              sum[e] = fmaf(__ldcg(p + NH * D + NH + h), w, sum[e]);
            }
          }
          math_barrier();
        }
#pragma unroll
        for (int e = 0; e < PER; ++e) {
          const int at4 = (e * 32 * MATH_WARPS + tid) * 4, h = at4 / D, d = at4 % D;
          if (h >= nh) continue;
          const float f = vs / sum[e];
          float x[4] = {y[e].x * f, y[e].y * f, y[e].z * f, y[e].w * f};
          if (a.gate.p) {
            const uint2 gr = *reinterpret_cast<const uint2*>(rows_at(a.gate, at.b, h0 + h, d));
            const float2 g0 = unpack2<S::BF16>(gr.x), g1 = unpack2<S::BF16>(gr.y);
            x[0] /= 1.f + __expf(-g0.x);
            x[1] /= 1.f + __expf(-g0.y);
            x[2] /= 1.f + __expf(-g1.x);
            x[3] /= 1.f + __expf(-g1.y);
          }
          *reinterpret_cast<uint2*>(rows_at(a.out, at.b, h0 + h, d)) =
              make_uint2(pack2<S::BF16>(x[0], x[1]), pack2<S::BF16>(x[2], x[3]));
        }
      }
    }
    t += j1 - j0;
    if (t < last) at.next_item(s_upto, heads);
  }
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

cudaError_t encode_fn(EncodeFn* out) {
  static EncodeFn fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || !p) return cudaErrorNotSupported;
    fn = reinterpret_cast<EncodeFn>(p);
  }
  *out = fn;
  return cudaSuccess;
}

// a pool as rows of a head's D elements: [page][head, token][d], copied 16 tokens x CB bytes at a time
template <class S>
cudaError_t pool_map(const CacheShape& c, const void* pool, int64_t page_stride, CUtensorMap* m) {
  EncodeFn fn;
  const cudaError_t e = encode_fn(&fn);
  if (e != cudaSuccess) return e;
  const int es = S::E4M3 ? 1 : 2;
  const cuuint64_t dims[3] = {(cuuint64_t)S::D, (cuuint64_t)c.Hkv << c.page_log2, (cuuint64_t)c.n_pages};
  const cuuint64_t strides[2] = {(cuuint64_t)S::RB, (cuuint64_t)page_stride * es};
  const cuuint32_t box[3] = {(cuuint32_t)(S::CB / es), 16, 1}, ones[3] = {1, 1, 1};
  const CUresult r = fn(m, S::E4M3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, (void*)pool, dims,
                        strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        S::CB == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

constexpr int SMEM_PER_CTA = 113 * 1024;      // two CTAs to an SM's 228 KB, of which each costs one more

template <class S>
cudaError_t run(const CacheShape& c, AttendArgs& A, int ctas, cudaStream_t st) {
  static_assert(S::MISC + 1024 + CACHE_MAX_REQUESTS * 8 + 2 * S::STAGE <= SMEM_PER_CTA, "the ring needs two stages");
  CUtensorMap km, vm;
  cudaError_t e = pool_map<S>(c, A.a.k_cache, A.a.k_page_stride, &km);
  if (e == cudaSuccess) e = pool_map<S>(c, A.a.v_cache, A.a.v_page_stride, &vm);
  if (e != cudaSuccess) return e;
  A.head_tiles = (A.group + S::NH - 1) / S::NH;
  const int other = S::MISC + 1024 + A.B * 8;
  const int n = (SMEM_PER_CTA - other) / S::STAGE;
  A.n_stages = n > 32 ? 32 : n;
  static bool ready[64] = {};
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev < 0 || dev >= 64 || !ready[dev])) {
    e = cudaFuncSetAttribute(k_cache_attend<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_PER_CTA);
    if (e == cudaSuccess && dev >= 0 && dev < 64) ready[dev] = true;
  }
  if (e != cudaSuccess) return e;
  k_cache_attend<S><<<ctas, THREADS, other + A.n_stages * S::STAGE, st>>>(A, km, vm);
  return cudaGetLastError();
}

template <int D, bool BF16, bool E4M3>
cudaError_t run_heads(const CacheShape& c, AttendArgs& A, int ctas, cudaStream_t st) {
  return A.group <= 8 ? run<Shape<D, BF16, E4M3, 1>>(c, A, ctas, st) : run<Shape<D, BF16, E4M3, 2>>(c, A, ctas, st);
}
template <int D>
cudaError_t run_types(const CacheShape& c, AttendArgs& A, int ctas, cudaStream_t st) {
  if (c.bf16) return c.e4m3 ? run_heads<D, true, true>(c, A, ctas, st) : run_heads<D, true, false>(c, A, ctas, st);
  return c.e4m3 ? run_heads<D, false, true>(c, A, ctas, st) : run_heads<D, false, false>(c, A, ctas, st);
}

}  // namespace

size_t cache_attend_workspace(int num_sms) { return ((size_t)2 * num_sms * 2 * (16 * 256 + 32) + COUNT_WORDS) * 4; }

cudaError_t cache_attend_launch(const CacheShape& S, const moe_cache_attend_t& a, const CacheAttendState& w,
                                cudaStream_t st) {
  AttendArgs A;
  A.a = a;
  A.B = (int)a.n_requests;
  A.Hq = S.Hq;
  A.Hkv = S.Hkv;
  A.group = S.Hq / S.Hkv;
  A.page_log2 = S.page_log2;
  A.n_pages = S.n_pages;
  A.max_len = (long long)S.max_pages << S.page_log2;
  A.scale = (float)a.scale * LOG2E;
  const int ctas = 2 * w.num_sms;
  A.counts = (uint32_t*)w.workspace;
  A.parts = (float*)w.workspace + COUNT_WORDS;
  A.status = w.status;
  A.timeout_ns = w.timeout_ns;
  A.skip_copy = w.skip_copy;
  if (S.D == 64) return run_types<64>(S, A, ctas, st);
  if (S.D == 128) return run_types<128>(S, A, ctas, st);
  return run_types<256>(S, A, ctas, st);
}

}  // namespace moe
