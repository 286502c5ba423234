// Attention of one new token of each request over the paged cache (moe_cache_attend).
//
// Every cached key and value is read once from HBM and meets only the query heads of its group, so the bytes of the
// cache bound the kernel; all else is arranged to keep them coming. One CTA to an SM.
//   Work. The tokens of a request and key-value head (an item) are cut into tiles of TN. The tiles of all items, one
//   after another, are divided evenly over the CTAs, whatever the requests' lengths are: a CTA walks its range, and an
//   item that crosses a CTA's border is split. Nobody waits: every CTA of a split item leaves its partial sums in the
//   workspace, and the one that counts itself last joins them, in the order of the tiles (in two steps where they are
//   many). It does so when it has nothing else to do: joining between two items stalled the copies by 5 to 10 us.
//   Copies. For each of two teams of math warps a warp walks the block table ahead of it and brings 16 tokens x 128
//   bytes at a time (more tokens where their rows are short) with TMA into the team's ring of 16 KB stages, keys and
//   values in stages of their own, across the borders of items; queries and gates of the next item with it. One copying
//   warp for both teams issued too slowly (a first form of the kernel: 188 us where two take 183, and 114 against 101
//   with an e4m3 cache).
//   Products. Heads are the narrow side of the tensor cores' m16n8k16: S^T[tokens x heads] = K Q^T and
//   O^T[d x heads] = V^T P^T, so that eight query heads fill a tile (tcgen05's 128 rows would leave its results in
//   tensor memory, a round trip away from the softmax between the products; with eight heads mma.sync keeps the tensor
//   cores 10 % of the time over a 16-bit cache and 17 % over e4m3; 32 heads are four times the products for each byte).
//   The teams take the tiles in turn, so that one's softmax hides behind the other's products. The four
//   warps of a team share a tile: each takes 16 tokens (or 32, or 64) of S and then its share of the rows d of O. One
//   maximum for the four, exchanged through shared memory, lets O be kept once.
// Measured (16 query over 2 key-value heads of 256): 128 requests of 512 to 16000 tokens, 1.19 GB: 180 us, 6.6 TB/s (a
// plain copy runs at 6.8); 256 requests over an e4m3 cache, 445 MB: 74 us, where a tile's conversions and products
// leave less slack; one request of 130 tokens: 7.5 us, of which the chain lengths - table - keys takes 3, the launch 2.
// What is left in between: 5 us until the first keys arrive, up to 8 us of joining, and SMs that do not all get the
// same bandwidth (on equal shares 48 of them end 10 % later; smaller shares for whoever is done first cost more than
// they won).
#include <cuda.h>

#include <atomic>

#include "cache.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int SHORT = 5;                          // units of an item that is not split without need
// CTAs whose parts are joined first, from FLAT + 1 parts on. One request of 131072 tokens, 16 over 2 heads of 256, 76
// parts each: 51.4 us; groups of 5 53.2, of 20 52.3, none 57.7; 32 over 1 heads of 128, 147 parts: 34.6, 38.3, 35.6 and
// 79. Three of 65536, 8 over 2 heads of 128, some 25 parts: 39.4, 39.3, 38.3 and 38.4.
constexpr int GROUP = 10, FLAT = 20;
constexpr int MAX_CTAS = 1024, COUNT_WORDS = 2048;                               // of the workspace
static_assert(COUNT_WORDS >= MAX_CTAS + 2 * ((MAX_CTAS + GROUP - 1) / GROUP) && COUNT_WORDS % 4 == 0, "all counts");
constexpr int PART_MAX = 32 * 256 + 2 * 32;       // floats of the largest part
constexpr float LOG2E = 1.4426950408889634f;

struct AttendArgs {
  moe_cache_attend_t a;
  int B, Hq, Hkv, group, head_tiles, page_log2, n_pages, n_stages;
  int box;                   // groups of 16 tokens to a copy: a power of two
  long long max_len;
  float scale;
  float* parts;              // [CTA][2][part floats]: the item a CTA begins in the middle of, the one it leaves so
  uint32_t* counts;          // [CTA]: parts that have arrived of the item that crosses the CTA's end
  float* group_parts;        // [group of CTAs][2], as parts: the joined parts of a group
  uint32_t* group_counts;    // [group of CTAs][2]
  uint32_t* status;
  uint64_t timeout_ns;
  int skip_copy;             // test: the first copy of CTA 0 is left out, so that its wait runs out
};

template <int D_, bool BF16_, bool E4M3_, int NT_>
struct Shape {
  static constexpr int D = D_, NT = NT_, NH = 8 * NT_;      // query heads of an item
  static constexpr bool BF16 = BF16_, E4M3 = E4M3_;
  static constexpr bool MMA_BF16 = BF16_ && !E4M3_;         // e4m3 is exact in fp16
  static constexpr int WARPS = 4, TEAMS = 2;                // math warps: the teams take the tiles in turn
  static constexpr int MATH = 32 * WARPS, THREADS = TEAMS * (MATH + 32);   // and a warp to copy for each team
  static constexpr int RB = D * (E4M3 ? 1 : 2);             // bytes of a token's row
  // copies are of lines of 128 bytes: CH of them to a row, or LT tokens to a line
  static constexpr int CB = 128, CH = RB < CB ? 1 : RB / CB, LT = RB < CB ? CB / RB : 1;
  static constexpr int TN = RB >= 512 ? 64 : RB >= 128 || NT > 2 ? 128 : 256;   // tokens of a tile
  // queries as fragments in shared memory, a copy for each team, where registers do not hold them beside the rest (16
  // heads of 256 over an e4m3 cache of 400 MB: 81 us in registers, 73 us so; of 128: 81.7 and 82.9)
  static constexpr bool QS = NT > 2 || NT * D >= 512;
  static constexpr int ROWS = NT * D > 512 ? 1 : 2;         // rows of D copied for each head: q; the gate, if it fits
  static constexpr int QF = QS ? D / 16 * NT * 32 : 0;      // uint2 of a team's
  static constexpr int MT = TN / 16 / WARPS;                // 16-token tiles of S per warp
  static constexpr int KT = TN / 16;
  static constexpr int GPS = 16384 / (16 * RB) < KT ? 16384 / (16 * RB) : KT;   // 16-token groups of a stage
  static constexpr int GROUP_BYTES = 16 * RB, STAGE = GPS * GROUP_BYTES;
  static constexpr int MD = D / 16 / WARPS;                 // 16-row tiles of O per warp
  // the highest weight is 2^LIFT: fp16 loses bits below 2^-14, and a long flat tail under one high score can be most
  // of the output (131071 tokens 17.4 below one whose value is 0: 16 % off without). The factor is in O and the sums
  // alike.
  static constexpr float LIFT = MMA_BF16 ? 0.f : 15.f;
  static constexpr int EXTRA = 2;                           // units of an item, see the division of the work
  static constexpr int PP = TN + 8;                         // pitch of P: rows of 8 fall on different banks
  static constexpr int QP = D + 8;                          // pitch of queries and gates
  static constexpr int PART = NH * D + 2 * NH;              // floats of a partial result: O, maxima, sums
  // of shared memory besides the rings and the lengths: barriers; queries and gates, twice; for each team P, maxima and
  // sums; one's results on their way to the other
  static constexpr int MISC = 1024 + 2 * ROWS * NH * QP * 2 + TEAMS * QF * 8 +
                              TEAMS * (NH * PP * 2 + 2 * WARPS * NH * 4) + NH * D * 4 + (1 + WARPS) * NH * 4;
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
// The base of a tile's weights 2^(score - base): LIFT below its maximum, rounded up so that none passes 2^LIFT.
template <class S>
__device__ __forceinline__ float base_of(float top) { return __fsub_ru(top, S::LIFT); }
// y * sigmoid(x) from e = exp(-|x|), which cannot overflow: __expf is off by 2 + 1.17 |x| steps at most, 2^-16 at the
// smallest normal e, well under half a step of a 16-bit output; the quotient by 1 + e <= 2 by two.
__device__ __forceinline__ float gated(float y, float x) {
  const float e = __expf(-fabsf(x));
  return __fdividef(x < 0.f ? y * e : y, 1.f + e);
}
__device__ __forceinline__ void tma_rows(void* dst, const CUtensorMap* m, int x, int row, int page, uint64_t* bar,
                                         uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
      "l"(m), "r"(x), "r"(row), "r"(page), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ uint16_t* rows_at(const moe_rows_t& r, int b, int h, int d) {
  return (uint16_t*)r.p + b * r.row_stride + h * r.head_stride + d;
}
// named barriers: 1 and 2 of a team each, 3 and 4 of both
template <class S>
__device__ __forceinline__ void team_barrier(int team) { named_bar(1 + team, S::MATH); }
__device__ __forceinline__ void named_arrive(int id, int nthreads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}

// ---- the division of the work ----
// Items come request by request, within a request head by head. An item of n tiles is n + EXTRA units long, for what
// its beginning and end cost; CTA c takes units c * share .. (c + 1) * share - 1.
// An even share; but while no item is longer than SHORT, a CTA takes whole items: a split one's parts take longer to
// join than a few tiles to read (130 tokens of two 256-wide heads: 8.5 us whole, 10.5 us in six parts).
__host__ __device__ inline int even_share(int units, int longest, int ctas) {
  const int even = units > 0 ? (int)(((long long)units + ctas - 1) / ctas) : 1;
  return longest <= SHORT && even < longest ? longest : even;
}
template <class S>
__device__ __forceinline__ int tiles_of(int len) { return (int)(((unsigned)len + S::TN - 1) / S::TN); }

// A place among the units: tile j of request b's head h (h: key-value head and its tile of query heads).
struct Place {
  int b, h, j, n;      // n: tiles of each head of request b
  // to the first tile of the next item (which exists)
  template <class S>
  __device__ __forceinline__ void next_item(const int* len, int heads) {
    j = 0;
    if (++h < heads) return;
    h = 0;
    do n = tiles_of<S>(len[++b]);
    while (n == 0);
  }
};

// o += V^T P^T over the groups of 16 tokens of one stage, from group g0 of the tile on; the first `left` tokens of the
// tile count (EDGE). from: the lane's address in the stage, pbase: in P.
template <class S, bool EDGE>
__device__ __forceinline__ void add_values(float (&o)[S::MD][S::NT][4], uint32_t from, uint32_t pbase, int g0, int left,
                                           int t4) {
#pragma unroll
  for (int kt = 0; kt < S::GPS; kt += 2) {
    const int tok0 = (g0 + kt) * 16;
    if (EDGE && tok0 >= left) break;
    const bool both = !EDGE || tok0 + 16 < left;
    uint32_t p[S::NT][4];                  // two steps of 16 tokens
#pragma unroll
    for (int nt = 0; nt < S::NT; ++nt) ldsm4(p[nt], pbase + nt * 8 * S::PP * 2 + tok0 * 2);
    // tokens past the end hold whatever memory holds: their values become zeros (their weights are)
    uint32_t keep[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = tok0 + i * 8 + 2 * t4;
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
          e4m3x4_to_f16x4(__byte_perm(v[i], 0, 0x3120), x[i][0], x[i][1]);
          if (EDGE) {
            x[i][0] &= keep[i];
            x[i][1] &= keep[i];
          }
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

// An item of which a CTA holds a part: request, head, and the CTAs that hold parts. b < 0: none.
struct Split {
  int b, h, c0, c1;
};

// The parts of a split item, or of a group of CTAs where they are many, that have arrived when this CTA's does: their
// count is in arrive's word, complete when the last one is there (and then set back).
__device__ __forceinline__ uint32_t* count_of(const AttendArgs& A, const Split& sp, int* n) {
  const int gi = blockIdx.x / GROUP;
  if (sp.c1 - sp.c0 < FLAT) {
    *n = sp.c1 - sp.c0 + 1;
    return &A.counts[sp.c0];
  }
  const int from = sp.c0 > gi * GROUP ? sp.c0 : gi * GROUP;
  const int to = sp.c1 < gi * GROUP + GROUP ? sp.c1 : gi * GROUP + GROUP - 1;
  *n = to - from + 1;
  return &A.group_counts[2 * gi + (gi == sp.c0 / GROUP)];
}
__device__ __forceinline__ int arrive(const AttendArgs& A, const Split& sp) {
  int n;
  return (int)atomicAdd(count_of(A, sp, &n), 1u);
}
__device__ __forceinline__ bool complete(const AttendArgs& A, const Split& sp, int before) {
  int n;
  uint32_t* const count = count_of(A, sp, &n);
  if (before != n - 1) return false;
  *count = 0;
  return true;
}

// The joined parts of a split item: NH * D / 4 groups of four d, PER of them to each math thread.
template <class S>
struct Joined {
  static constexpr int NH = S::NH, D = S::D, VECS = NH * D / 4;
  static constexpr int STEP = S::TEAMS * S::MATH, PER = (VECS + STEP - 1) / STEP;
  static constexpr int FEW = 16 / PER < 8 ? 16 / PER : 8;
  static_assert(VECS % STEP == 0 || PER == 1, "whole vectors for each thread, or one for some");
  float4 y[PER];
  float sum[PER], top[PER];
  uint2 gate[PER];

  __device__ __forceinline__ static bool mine(int tid) { return VECS >= STEP || tid < VECS; }
  // Part i of ia .. ib lies in slot 2 i + (i == i0): i0 is where the item begins. Up to FEW of them come straight from
  // L2, every load on its way at once; the order of the sum is that of the parts.
  __device__ __forceinline__ void few(const float* parts, int ia, int ib, int i0, int tid) {
    if (!mine(tid)) return;
    float4 v[FEW][PER];
    float m[FEW][PER], l[FEW][PER];
#pragma unroll
    for (int k = 0; k < FEW; ++k) {
      const int i = ia + k < ib ? ia + k : ib;
      const float* p = parts + ((long long)i * 2 + (i == i0 ? 1 : 0)) * S::PART;
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        const int at4 = (e * STEP + tid) * 4, h = at4 / D;
        v[k][e] = __ldcg(reinterpret_cast<const float4*>(p + at4));
        m[k][e] = __ldcg(p + NH * D + h);
        l[k][e] = __ldcg(p + NH * D + NH + h);
      }
    }
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      float x = m[0][e];
#pragma unroll
      for (int k = 1; k < FEW; ++k) x = fmaxf(x, m[k][e]);     // the last part again does not matter
      const float base = x == -INFINITY ? 0.f : x;
      top[e] = x;
#pragma unroll
      for (int k = 0; k < FEW; ++k)
        if (ia + k <= ib) put(e, v[k][e], l[k][e], exp2_fast(m[k][e] - base));
    }
  }
  // n further parts, from shared memory. All math warps, in step.
  __device__ __forceinline__ void add(const float* parts, int n, int tid) {
    if (!mine(tid)) return;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const int at4 = (e * STEP + tid) * 4, h = at4 / D;
      float x = top[e];
#pragma unroll 8
      for (int k = 0; k < n; ++k) x = fmaxf(x, parts[k * S::PART + NH * D + h]);
      const float base = x == -INFINITY ? 0.f : x, c = exp2_fast(top[e] - base);
      top[e] = x;
      sum[e] *= c;
      y[e] = make_float4(y[e].x * c, y[e].y * c, y[e].z * c, y[e].w * c);
#pragma unroll 4
      for (int k = 0; k < n; ++k) {
        const float* p = parts + k * S::PART;
        put(e, *reinterpret_cast<const float4*>(p + at4), p[NH * D + NH + h], exp2_fast(p[NH * D + h] - base));
      }
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      y[e] = make_float4(0.f, 0.f, 0.f, 0.f);
      sum[e] = 0.f;
      top[e] = -INFINITY;
    }
  }
  __device__ __forceinline__ void put(int e, float4 v, float l, float w) {
    sum[e] = fmaf(l, w, sum[e]);
    y[e].x = fmaf(v.x, w, y[e].x);
    y[e].y = fmaf(v.y, w, y[e].y);
    y[e].z = fmaf(v.z, w, y[e].z);
    y[e].w = fmaf(v.w, w, y[e].w);
  }
  // as a part of its own
  __device__ __forceinline__ void keep(float* part, int tid) {
    if (!mine(tid)) return;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const int at4 = (e * STEP + tid) * 4;
      *reinterpret_cast<float4*>(part + at4) = y[e];
      if (at4 % D == 0) {
        part[NH * D + at4 / D] = top[e];
        part[NH * D + NH + at4 / D] = sum[e];
      }
    }
  }
  // the gates, on their way while the parts are joined
  __device__ __forceinline__ void fetch_gates(const AttendArgs& A, int b, int h0, int nh, int tid) {
    if (!A.a.gate.p || !mine(tid)) return;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const int at4 = (e * STEP + tid) * 4, h = at4 / D, d = at4 % D;
      gate[e] = h < nh ? __ldcg(reinterpret_cast<const uint2*>(rows_at(A.a.gate, b, h0 + h, d))) : make_uint2(0, 0);
    }
  }
  // as the output
  __device__ __forceinline__ void finish(const AttendArgs& A, int b, int h0, int nh, float vs, int tid) {
    if (!mine(tid)) return;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const int at4 = (e * STEP + tid) * 4, h = at4 / D, d = at4 % D;
      if (h >= nh) continue;
      const float f = vs / sum[e];
      float x[4] = {y[e].x * f, y[e].y * f, y[e].z * f, y[e].w * f};
      if (A.a.gate.p) {
        const float2 g0 = unpack2<S::BF16>(gate[e].x), g1 = unpack2<S::BF16>(gate[e].y);
        x[0] = gated(x[0], g0.x);
        x[1] = gated(x[1], g0.y);
        x[2] = gated(x[2], g1.x);
        x[3] = gated(x[3], g1.y);
      }
      *reinterpret_cast<uint2*>(rows_at(A.a.out, b, h0 + h, d)) =
          make_uint2(pack2<S::BF16>(x[0], x[1]), pack2<S::BF16>(x[2], x[3]));
    }
  }
};

template <class S>
__global__ void __launch_bounds__(S::THREADS, 1)
    k_cache_attend(const __grid_constant__ AttendArgs A, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap) {
  constexpr int D = S::D, NT = S::NT, NH = S::NH, TN = S::TN, MT = S::MT, KT = S::KT, MD = S::MD;
  constexpr int PP = S::PP, QP = S::QP;
  constexpr int GPS = S::GPS, WARPS = S::WARPS, TEAMS = S::TEAMS, MATH = S::MATH;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const ring = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* const misc = ring + TEAMS * A.n_stages * S::STAGE;
  uint64_t* const full0 = (uint64_t*)misc;           // [TEAMS][n_stages <= 16]: every team has a ring of its own
  uint64_t* const empty0 = full0 + 32;
  uint64_t* const rows_full = empty0 + 32;            // [2]: an item's queries and gates, by turns
  uint64_t* const rows_empty = rows_full + 2;
  uint64_t* const join_full = rows_empty + 2;        // parts, when the rings are done with
  volatile int* const s_flags = (int*)(join_full + 2);    // 0: a wait ran out; 1, 2: last to arrive; 3: the first has
  int* const s_scan = (int*)(join_full + 2) + 4;     // [THREADS / 32]
  int* const s_place = s_scan + 32;                  // [3]
  uint16_t* const s_q = (uint16_t*)(misc + 1024);    // [2][ROWS][NH][QP]: by turns, queries and gates
  uint2* const s_qf0 = (uint2*)(s_q + 2 * S::ROWS * NH * QP);  // [TEAMS][D / 16][NT / 2][lane][2], if QS
  uint16_t* const s_p0 = (uint16_t*)(s_qf0 + TEAMS * S::QF);   // [TEAMS][NH][PP]
  float* const s_max0 = (float*)(s_p0 + TEAMS * NH * PP);   // [TEAMS][WARPS][NH]
  float* const s_sum0 = s_max0 + TEAMS * WARPS * NH; // [TEAMS][WARPS][NH]
  float* const s_x = s_sum0 + TEAMS * WARPS * NH;    // [NH * D], [NH] maxima, [WARPS][NH] sums
  int* const s_len = (int*)(s_x + NH * D + NH + WARPS * NH);   // [B]

  const moe_cache_attend_t& a = A.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int heads = A.Hkv * A.head_tiles;

  if (tid < TEAMS * 16) {
    mbar_init(&full0[tid], 1);
    mbar_init(&empty0[tid], WARPS);
  } else if (tid == TEAMS * 16) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&rows_full[s], 1);
      mbar_init(&rows_empty[s], TEAMS * WARPS);
    }
    mbar_init(join_full, 1);
    s_flags[0] = s_flags[1] = s_flags[2] = s_flags[3] = 0;
  }
  if (tid <= TEAMS * 16) fence_mbar_init();
  follow_predecessor();
  // lengths and the running number of tiles: a thread's requests lie side by side, so that all its loads are on their
  // way at once
  const int each = (A.B + S::THREADS - 1) / S::THREADS, b_begin = tid * each < A.B ? tid * each : A.B;
  const int b_end = b_begin + each < A.B ? b_begin + each : A.B;
  int mine = 0, longest = 0;
#pragma unroll 4
  for (int b = b_begin; b < b_end; ++b) {
    int len = __ldcg(a.lengths + b);
    if (len < 0 || len > A.max_len) {
      atomicOr(A.status, CACHE_BAD_LENGTH);
      len = len < 0 ? 0 : (int)A.max_len;
    }
    s_len[b] = len;
    const int n = len ? tiles_of<S>(len) + S::EXTRA : 0;
    mine += n;
    longest = max(longest, n);
  }
  // a wait ran out in an earlier call, or has in this one: the counts are off until the status is read
  const bool dead = tid == 0 && (*(volatile uint32_t*)A.status & CACHE_BAD_WAIT);
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
    if (lane >= o) upto += y;
  }
  const int wlongest = __reduce_max_sync(0xFFFFFFFFu, longest);
  if (lane == 31) {
    s_scan[warp] = upto;
    s_scan[16 + warp] = wlongest;
  }
  if (__syncthreads_or(dead)) return;
  int carry = 0;
  for (int w = 0; w < S::THREADS / 32; ++w) {
    if (w < warp) upto += s_scan[w];
    carry += s_scan[w];
    longest = max(longest, s_scan[16 + w]);
  }
  const int units = carry * heads, share = even_share(units, longest, gridDim.x);
  const int first = (long long)share * blockIdx.x < units ? share * blockIdx.x : units;
  const int last = share < units - first ? first + share : units;
  // where the CTA begins: found by the thread that holds the request
  if (first < last && (upto - mine) * heads <= first && first < upto * heads) {
    int before = upto - mine, b = b_begin - 1, n;
    while (true) {
      const int len = s_len[++b];
      n = len ? tiles_of<S>(len) + S::EXTRA : 0;
      if ((before + n) * heads > first) break;
      before += n;
    }
    const int in = first - before * heads;
    s_place[0] = b;
    s_place[1] = in / n;
    s_place[2] = in % n;
  }
  __syncthreads();
  // begin: the first tile from unit `first` on, which is unit t0
  Place begin = {0, 0, 0, 0};
  int t0 = first;
  if (first < last) {
    begin = {s_place[0], s_place[1], s_place[2], tiles_of<S>(s_len[s_place[0]])};
    if (begin.j >= begin.n) {
      t0 += begin.n + S::EXTRA - begin.j;
      if (t0 < last) begin.template next_item<S>(s_len, heads);
    }
  }

  if (warp >= TEAMS * WARPS) {
    // ---------------------------------------------------------------- copies, for one team
    const int team = warp - TEAMS * WARPS;
    uint64_t* const full = full0 + team * 16;
    uint64_t* const empty = empty0 + team * 16;
    uint8_t* const my_ring = ring + team * A.n_stages * S::STAGE;
    int stage = 0;
    uint32_t phase = 0, n_rows = 0;                  // n_rows: copies of rows so far, by the first team's warp
    // keys and values are read once, so they leave L2 first (256 requests over an e4m3 cache: 74.9 us, 79.5 us
    // without); twice or more where a group's heads are several items
    const uint64_t policy = A.head_tiles == 1 ? policy_evict_first() : policy_evict_normal();
    bool skip = A.skip_copy && blockIdx.x == 0 && team == 0;
    // Waits until a buffer is free. False: a wait ran out, here or in a math warp, which then no longer waits. Nothing
    // more is copied then, and what is on its way is waited for (boundedly) before the CTA ends: the ring's stages,
    // earlier ones of this lap, later ones of the last, and the rows.
    auto free_to_fill = [&](uint64_t* bar, uint32_t parity) {
      if (!mbar_wait(bar, parity, A.timeout_ns)) {
        s_flags[0] = 1;
        atomicOr(A.status, CACHE_BAD_WAIT);
      }
      __syncwarp();
      if (!s_flags[0]) return true;
      for (int s = 0; s < A.n_stages; ++s) mbar_wait(&full[s], s < stage ? phase : phase ^ 1, A.timeout_ns);
      for (uint32_t i = n_rows > 2 ? n_rows - 2 : 0; i < n_rows; ++i)
        mbar_wait(&rows_full[i & 1], i >> 1 & 1, A.timeout_ns);
      return false;
    };
    // the item's queries, and its gates where the whole item is this CTA's: rows of D elements
    auto copy_rows = [&](const Place& p, bool gates) {
      const uint32_t buf = n_rows & 1;
      if (!free_to_fill(&rows_empty[buf], (n_rows >> 1 & 1) ^ 1)) return false;
      const int h_in = (p.h % A.head_tiles) * NH;
      const int h0 = (p.h / A.head_tiles) * A.group + h_in;
      const int nh = A.group - h_in < NH ? A.group - h_in : NH;
      if (lane == 0) mbar_expect_tx(&rows_full[buf], nh * D * 2 * (gates && S::ROWS == 2 ? 2 : 1));
      __syncwarp();
#pragma unroll
      for (int i = lane; i < S::ROWS * NH; i += 32) {
        const int which = i / NH, h = i % NH;
        if (h < nh && (which == 0 || gates))
          bulk_g2s(s_q + ((buf * S::ROWS + which) * NH + h) * QP, rows_at(which ? a.gate : a.q, p.b, h0 + h, 0), D * 2,
                   &rows_full[buf]);
      }
      ++n_rows;
      return true;
    };
    // the pages of 32 groups of 16 tokens from a tile on, one to a lane; looked at only when they are used, which is
    // while the next 32 are on their way
    auto pages_from = [&](const Place& p) {
      const long long tok = (long long)p.j * TN + lane * 16;
      return tok < s_len[p.b] ? __ldcg(a.tables + (long long)p.b * a.table_stride + (tok >> A.page_log2)) : 0;
    };
    if (t0 >= last) return;
    Place at = begin;
    int pages = pages_from(at), j_begin = at.j, turn = team;   // turn: odd when the next tile is the other team's
    for (int t = t0; t < last;) {
      constexpr int TILES = 32 / KT;
      int n_tiles = at.n - at.j < TILES ? at.n - at.j : TILES;
      n_tiles = last - t < n_tiles ? last - t : n_tiles;
      Place nx = at;
      nx.j += n_tiles;
      const bool ends = nx.j == nx.n;
      const int t_next = t + n_tiles + (ends ? S::EXTRA : 0);
      const bool more = t_next < last;
      if (more && ends) nx.template next_item<S>(s_len, heads);
      const int pages_next = more ? pages_from(nx) : 0;
      if (team == 0 && at.j == j_begin && !copy_rows(at, a.gate.p && at.j == 0 && at.n <= last - t)) return;
      if ((unsigned)pages >= (unsigned)A.n_pages) {
        atomicOr(A.status, CACHE_BAD_PAGE);
        pages = A.n_pages;                             // out of range: the copy reads zeros
      }
      const int row0 = (at.h / A.head_tiles) << A.page_log2;
      for (int i = turn & 1; i < n_tiles; i += TEAMS) {
        const int tok0 = (at.j + i) * TN, left = s_len[at.b] - tok0;
        const int groups = left >= TN ? KT : (left + 15) >> 4;
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
#pragma unroll 1
          for (int g0 = 0; g0 < groups; g0 += GPS) {
            if (!free_to_fill(&empty[stage], phase ^ 1)) return;
            const int n = groups - g0 < GPS ? groups - g0 : GPS;
            int page[GPS];
#pragma unroll
            for (int grp = 0; grp < GPS; ++grp) page[grp] = __shfl_sync(0xFFFFFFFFu, pages, (i * KT + g0 + grp) & 31);
            uint8_t* const dst = my_ring + stage * S::STAGE;
            const CUtensorMap* const map = kv ? &vmap : &kmap;
            const int tok = tok0 + g0 * 16, in_page = (1 << A.page_log2) - 1;
            if (elect_one()) {
              mbar_expect_tx(&full[stage], ((n + A.box - 1) & -A.box) * S::GROUP_BYTES);
#pragma unroll
              for (int grp = 0; grp < GPS; ++grp)
                if (grp < n && (grp & (A.box - 1)) == 0 && !skip)
#pragma unroll
                  for (int x = 0; x < S::CH; ++x)
                    tma_rows(dst + grp * S::GROUP_BYTES + x * 16 * S::CB, map, x * (D / S::CH),
                             (row0 + ((tok + grp * 16) & in_page)) / S::LT, page[grp], &full[stage], policy);
            }
            __syncwarp();
            skip = false;
            if (++stage == A.n_stages) { stage = 0; phase ^= 1; }
          }
        }
      }
      if (ends) j_begin = 0;
      t = t_next;
      turn += n_tiles;
      at = nx;
      pages = pages_next;
    }
    return;
  }

  // ------------------------------------------------------------------ products
  const int g = lane >> 2, t4 = lane & 3;
  const int team = warp / WARPS, wt = warp % WARPS, ttid = tid % MATH;    // a warp and a thread within their team
  uint16_t* const s_p = s_p0 + team * NH * PP;
  float* const s_max = s_max0 + team * WARPS * NH;
  uint2* const s_qf = s_qf0 + team * S::QF;
  float* const s_sum = s_sum0 + team * WARPS * NH;
  // requests of length 0
  for (int b = blockIdx.x; b < A.B; b += gridDim.x)
    if (s_len[b] == 0)
      for (int i = tid; i < A.Hq * D / 8; i += TEAMS * MATH)
        *reinterpret_cast<uint4*>(rows_at(a.out, b, i / (D / 8), i % (D / 8) * 8)) = make_uint4(0, 0, 0, 0);

  // Where a lane's rows of a stage lie. 16-byte chunk c of row r of a group of 16 tokens is at
  //   c / PER * 16 * CB + r * CB + ((c % PER) ^ (r % 8)) * 16,      PER = CB / 16,
  // and where a line holds LT rows, their chunks follow one another in it. With chunks that differ in a constant's bits
  // alone, the address differs by an exclusive or with 16 * constant.
  constexpr int PER = S::CB / 16;
  auto in_group = [](int r, int c) {
    const int line = r / S::LT, at = r % S::LT * (PER / S::LT) + c % PER;
    return (uint32_t)((c / PER) * (16 * S::CB) + line * S::CB + ((at ^ (line & 7)) << 4));
  };
  const uint32_t ring0 = smem_u32(ring) + team * A.n_stages * S::STAGE;
  uint64_t* const full = full0 + team * 16;
  uint64_t* const empty = empty0 + team * 16;
  const uint32_t k_lane = ring0 + in_group(lane & 15, lane >> 4);
  const uint32_t v_lane =
      ring0 + (S::E4M3 ? (lane >> 4) * S::GROUP_BYTES + in_group(lane & 15, wt * MD)
                       : in_group((lane & 7) + ((lane >> 4) << 3), wt * MD * 2 + ((lane >> 3) & 1)));
  const uint32_t p_lane = smem_u32(s_p) + ((lane & 7) * PP + (lane >> 3) * 8) * 2;
  auto wait_full = [&](uint64_t* bar, uint32_t parity) {
    // once a wait has run out the outputs are lost: run to the end without waiting
    if (!mbar_try_wait(bar, parity) && !s_flags[0] && !mbar_wait(bar, parity, A.timeout_ns)) {
      s_flags[0] = 1;
      atomicOr(A.status, CACHE_BAD_WAIT);
    }
    __syncwarp();
  };
  auto release = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };

  int stage = 0;
  uint32_t phase = 0, n_rows = 0;
  if (t0 >= last) return;
  int t = t0, done = 0;                                      // done: tiles of the CTA so far
  Place at = begin;
  Split split[2] = {{-1, 0, 0, 0}, {-1, 0, 0, 0}};           // of the first item and of the last
  // parts of the first item that had arrived before this CTA's
  int head_before = -1;
  while (t < last) {
    const int kvh = at.h / A.head_tiles, h_in = (at.h % A.head_tiles) * NH;
    const int h0 = kvh * A.group + h_in;                       // first query head of the item
    const int nh = A.group - h_in < NH ? A.group - h_in : NH;
    const int len = s_len[at.b];
    const int j0 = at.j;
    const int j1 = last - t < at.n - j0 ? j0 + last - t : at.n;

    // Q as B fragments; with an e4m3 cache the k index runs 4t..4t+3 within 16 bytes of a row, as the codes do. Heads
    // past nh hold whatever memory holds: no head's column reaches another's, and theirs are not written.
    uint32_t q[D / 16][NT][2];
    float sf[NT][2];                                           // what a product is multiplied by, for 2^x
    const float ks = S::E4M3 ? __ldcg(a.k_scale + kvh) : 1.f;
    wait_full(&rows_full[n_rows & 1], n_rows >> 1 & 1);
    const uint16_t* const q_rows = s_q + (n_rows & 1) * S::ROWS * NH * QP;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (S::E4M3) {
        const uint16_t* src = q_rows + (nt * 8 + g) * QP + 4 * t4;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint2 v = *reinterpret_cast<const uint2*>(src + ks * 16);
          q[ks][nt][0] = v.x;
          q[ks][nt][1] = v.y;
        }
      } else {
        const uint32_t src = smem_u32(q_rows + (nt * 8 + (lane & 7)) * QP + (lane >> 3) * 8);
#pragma unroll
        for (int ks = 0; ks < D / 16; ks += 2) {
          uint32_t r[4];
          ldsm4(r, src + ks * 32);
          q[ks][nt][0] = r[0];
          q[ks][nt][1] = r[1];
          q[ks + 1][nt][0] = r[2];
          q[ks + 1][nt][1] = r[3];
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
        // (0, infinities and NaN stay what they are at any power; past 2^126 its inverse would lose bits)
        const int e = min(max((__float_as_int(m) >> 23) - 127, -126), 126);
        up = __int_as_float((127 + e) << 23);
        const float down = __int_as_float((127 - e) << 23);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 f = unpack2<true>(q[ks][nt][i]);
            q[ks][nt][i] = pack2<false>(f.x * down, f.y * down);
          }
      }
      if (S::QS) {
        // the last tile's barriers are behind every reader of the item before
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          if (ks % WARPS == wt)
            s_qf[((ks * (NT / 2) + nt / 2) * 32 + lane) * 2 + nt % 2] = make_uint2(q[ks][nt][0], q[ks][nt][1]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        sf[nt][i] = A.scale * (S::E4M3 ? ks * __shfl_sync(0xFFFFFFFFu, up, (2 * t4 + i) * 4) : 1.f);
    }

    if (S::QS) team_barrier<S>(team);
    // the queries' fragments of step ks
    auto queries = [&](int ks, uint32_t (&f)[NT][2]) {
      if (S::QS) {
#pragma unroll
        for (int nt = 0; nt < NT; nt += 2) {
          const uint4 v = reinterpret_cast<const uint4*>(s_qf)[(ks * (NT / 2) + nt / 2) * 32 + lane];
          f[nt][0] = v.x;
          f[nt][1] = v.y;
          if (nt + 1 < NT) {
            f[nt + 1][0] = v.z;
            f[nt + 1][1] = v.w;
          }
        }
      } else {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          f[nt][0] = q[ks][nt][0];
          f[nt][1] = q[ks][nt][1];
        }
      }
    };

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

    for (int j = j0 + ((done + team) & 1); j < j1; j += TEAMS) {
      const int left = len - j * TN;                           // tokens of the request from this tile on
      const int groups = left >= TN ? KT : (left + 15) >> 4;
      // ---- S^T = K Q^T for this warp's groups of 16 tokens; two chains of accumulators for one or two tiles of heads,
      // as one would wait for each product's latency
      float s[MT][NT][4], s2[MT][NT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[mt][nt][i] = s2[mt][nt][i] = 0.f;
#pragma unroll 1
      for (int g0 = 0; g0 < groups; g0 += GPS) {
        // every warp of the team waits for every stage: one that went ahead could release a stage twice
        // before the others once
        wait_full(&full[stage], phase);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const int gr = mt * WARPS + wt - g0;
          if (gr < 0 || gr >= GPS || g0 + gr >= groups) continue;
          const uint32_t from = k_lane + stage * S::STAGE + gr * S::GROUP_BYTES;
          if (S::E4M3) {
#pragma unroll
            for (int c = 0; c < S::RB / 16; c += 2) {
              uint32_t k[4], lo[4], hi[4];
              ldsm4(k, (from ^ (c % PER << 4)) + c / PER * (16 * S::CB));
#pragma unroll
              for (int i = 0; i < 4; ++i) e4m3x4_to_f16x4(k[i], lo[i], hi[i]);
              uint32_t f0[NT][2], f1[NT][2];
              queries(c, f0);
              queries(c + 1, f1);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma16816<false>(s[mt][nt], lo[0], lo[1], hi[0], hi[1], f0[nt][0], f0[nt][1]);
                mma16816<false>(NT > 2 ? s[mt][nt] : s2[mt][nt], lo[2], lo[3], hi[2], hi[3], f1[nt][0], f1[nt][1]);
              }
            }
          } else {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              uint32_t k[4];
              ldsm4(k, (from ^ (2 * ks % PER << 4)) + 2 * ks / PER * (16 * S::CB));
              uint32_t f[NT][2];
              queries(ks, f);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma16816<S::MMA_BF16>(NT <= 2 && ks & 1 ? s2[mt][nt] : s[mt][nt], k[0], k[1], k[2], k[3], f[nt][0],
                                      f[nt][1]);
            }
          }
        }
        release(&empty[stage]);
        if (++stage == A.n_stages) { stage = 0; phase ^= 1; }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int tok = (mt * WARPS + wt) * 16;
        const bool edge = left < tok + 16;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = (NT > 2 ? s[mt][nt][i] : s[mt][nt][i] + s2[mt][nt][i]) * sf[nt][i & 1];
            s[mt][nt][i] = edge && tok + g + (i >> 1) * 8 >= left ? -INFINITY : x;
          }
      }

      // ---- the tile's maximum for each head, as the base of its weights: so are all maxima from here on
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
          *reinterpret_cast<float2*>(&s_max[wt * NH + nt * 8 + 2 * t4]) =
              make_float2(base_of<S>(top[nt][0]), base_of<S>(top[nt][1]));
      team_barrier<S>(team);
      bool moved = false;
      float c[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float2 x = make_float2(m[nt][0], m[nt][1]);
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
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
        // P^T for the second product: 16 bits a weight, an error of half a step of the products' type, which adds up
        // like the values' own rounding; fp16 keeps all its bits for weights down to 2^-29 of the highest
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            *reinterpret_cast<uint32_t*>(&s_p[(nt * 8 + g) * PP + (mt * WARPS + wt) * 16 + 8 * r + 2 * t4]) =
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
      team_barrier<S>(team);

      // ---- O^T += V^T P^T for this warp's rows of d
#pragma unroll 1
      for (int g0 = 0; g0 < groups; g0 += GPS) {
        wait_full(&full[stage], phase);
        const uint32_t from = v_lane + stage * S::STAGE;
        if (left >= (g0 + GPS) * 16) add_values<S, false>(o, from, p_lane, g0, left, t4);
        else add_values<S, true>(o, from, p_lane, g0, left, t4);
        release(&empty[stage]);
        if (++stage == A.n_stages) { stage = 0; phase ^= 1; }
      }
    }

    // ---- the end of the item, or of the CTA's share of it: the team with its last tile has the other's results added
    const bool owner = ((done + j1 - 1 - j0) & 1) == team, alone = j1 - j0 == 1;
    const bool whole = j0 == 0 && j1 == at.n;
    auto put_sums = [&](float* to) {             // [WARPS][NH]
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x = l[nt][i];
          x += __shfl_xor_sync(0xFFFFFFFFu, x, 4);
          x += __shfl_xor_sync(0xFFFFFFFFu, x, 8);
          x += __shfl_xor_sync(0xFFFFFFFFu, x, 16);
          if (lane < 4) to[wt * NH + nt * 8 + 2 * t4 + i] = x;
        }
    };
    if (!alone && !owner) {
      named_bar(3, TEAMS * MATH);                // what lay here has been read
      put_sums(s_x + NH * D + NH);
#pragma unroll
      for (int md = 0; md < MD; ++md)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          reinterpret_cast<float4*>(s_x)[(md * NT + nt) * MATH + ttid] =
              make_float4(o[md][nt][0], o[md][nt][1], o[md][nt][2], o[md][nt][3]);
      if (wt == 0 && g == 0)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) s_x[NH * D + nt * 8 + 2 * t4 + i] = m[nt][i];
      named_arrive(4, TEAMS * MATH);
    }
    if (owner) {
      put_sums(s_sum);
      if (alone) {
        team_barrier<S>(team);
      } else {
        named_arrive(3, TEAMS * MATH);
        named_bar(4, TEAMS * MATH);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int h = nt * 8 + 2 * t4 + i;
          float x = 0.f;
#pragma unroll
          for (int w = 0; w < WARPS; ++w) x += s_sum[w * NH + h];
          if (!alone) {
            const float m1 = s_x[NH * D + h], nm = fmaxf(m[nt][i], m1), base = nm == -INFINITY ? 0.f : nm;
            const float c0 = exp2_fast(m[nt][i] - base), c1 = exp2_fast(m1 - base);
            float x1 = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) x1 += s_x[NH * D + NH + w * NH + h];
            x = x * c0 + x1 * c1;
            m[nt][i] = nm;
#pragma unroll
            for (int md = 0; md < MD; ++md)
#pragma unroll
              for (int r = 0; r < 2; ++r)
                o[md][nt][2 * r + i] =
                    o[md][nt][2 * r + i] * c0 + s_x[((md * NT + nt) * MATH + ttid) * 4 + 2 * r + i] * c1;
          }
          l[nt][i] = x;
        }
    }
    const float vs = S::E4M3 ? __ldcg(a.v_scale + kvh) : 1.f;
    // the rows of d that an accumulator's two halves hold
    auto d_of = [&](int md, int r) {
      return S::E4M3 ? (wt * MD + md) * 16 + 2 * g + r : (wt * MD + md) * 16 + g + 8 * r;
    };
    // a part is joined with the others once this CTA has nothing else to do: the item's tiles are those of CTAs c0 ..
    // c1; c0 holds its part as the item it leaves, the others as the item they begin in the middle of
    const int which = j0 == 0 ? 1 : 0;
    if (!whole) {
      const Split sp = {at.b, at.h, (t - j0) / share, (t - j0 + at.n - 1) / share};
      if (which) split[1] = sp; else split[0] = sp;
    }
    if (!owner) {
      release(&rows_empty[n_rows & 1]);
    } else if (whole) {
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
                y = gated(y, unpack2<S::BF16>(S::ROWS == 2 ? q_rows[(NH + h) * QP + d]
                                                           : __ldcg(rows_at(a.gate, at.b, h0 + h, d))).x);
              }
              *rows_at(a.out, at.b, h0 + h, d) = (uint16_t)pack2<S::BF16>(y, 0.f);
            }
        }
    } else {
      float* part = A.parts + ((long long)blockIdx.x * 2 + which) * S::PART;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int h = nt * 8 + 2 * t4 + i;
#pragma unroll
          for (int md = 0; md < MD; ++md)
#pragma unroll
            for (int r = 0; r < 2; ++r) part[h * D + d_of(md, r)] = o[md][nt][2 * r + i];
          if (wt == 0 && g == 0) {
            part[NH * D + h] = m[nt][i];
            part[NH * D + NH + h] = l[nt][i];
          }
        }
    }
    if (owner) release(&rows_empty[n_rows & 1]);
    ++n_rows;
    if (owner && !whole && which == 0 && t + j1 - j0 < last) {
      // the first item's part arrives now, while there are tiles to come; whether it was the last is looked
      // at in the end
      team_barrier<S>(team);
      if (ttid == 0) {
        __threadfence();
        head_before = arrive(A, split[0]);
      }
    }
    done += j1 - j0;
    t += j1 - j0 + (j1 == at.n ? S::EXTRA : 0);
    if (t < last) at.template next_item<S>(s_len, heads);
  }

  // ---- joining the split items: the last of an item's parts to arrive joins them
  if (split[0].b < 0 && split[1].b < 0) return;
  if (head_before >= 0) {
    __threadfence();                 // the others' parts after the count that told of them
    s_flags[3] = 1;
    s_flags[1] = complete(A, split[0], head_before);
  }
  named_bar(3, TEAMS * MATH);
  if (lane == 0 && warp < 2) {
    const Split sp = warp ? split[1] : split[0];
    if (sp.b >= 0 && !(warp == 0 && s_flags[3])) {
      __threadfence();               // the barrier's threads' parts before the count, and the others' parts after it
      s_flags[1 + warp] = complete(A, sp, arrive(A, sp));
    }
    __threadfence();
  }
  named_bar(3, TEAMS * MATH);
  Joined<S> y;
  uint32_t join_phase = 0;
  auto join = [&](const float* parts, int ia, int ib, int i0) {
    y.clear();
    if (ib - ia < Joined<S>::FEW) {
      y.few(parts, ia, ib, i0, tid);
      return;
    }
    // more than FEW by bulk copies, to where the rings were
    static_assert(TEAMS * 2 * S::STAGE >= S::PART * 4, "the rings hold a part at least");
    const int at_once = TEAMS * A.n_stages * S::STAGE / (S::PART * 4);
    for (int k0 = ia; k0 <= ib; k0 += at_once) {
      const int n = ib - k0 + 1 < at_once ? ib - k0 + 1 : at_once;
      named_bar(3, TEAMS * MATH);                // what lay there has been read
      if (warp == 0) {
        if (lane == 0) mbar_expect_tx(join_full, n * S::PART * 4);
        __syncwarp();
        fence_proxy_async_global();
        for (int k = lane; k < n; k += 32)
          bulk_g2s(ring + k * S::PART * 4, parts + ((long long)(k0 + k) * 2 + (k0 + k == i0 ? 1 : 0)) * S::PART,
                   S::PART * 4, join_full);
      }
      wait_full(join_full, join_phase);
      if (s_flags[0]) mbar_wait(join_full, join_phase, A.timeout_ns);      // lost; the copies must not outlive the CTA
      join_phase ^= 1;
      y.add((const float*)ring, n, tid);
    }
  };
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    if (!s_flags[1 + i]) continue;
    const Split sp = i ? split[1] : split[0];
    const int kvh = sp.h / A.head_tiles, h_in = (sp.h % A.head_tiles) * NH, h0 = kvh * A.group + h_in;
    const int nh = A.group - h_in < NH ? A.group - h_in : NH;
    const float vs = S::E4M3 ? __ldcg(a.v_scale + kvh) : 1.f;
    y.fetch_gates(A, sp.b, h0, nh, tid);
    if (sp.c1 - sp.c0 < FLAT) {
      join(A.parts, sp.c0, sp.c1, sp.c0);
    } else {
      // many parts: each GROUP of CTAs joins its own, and the last group to do so the groups'
      const int g0 = sp.c0 / GROUP, g1 = sp.c1 / GROUP, gi = blockIdx.x / GROUP;
      join(A.parts, gi == g0 ? sp.c0 : gi * GROUP, gi == g1 ? sp.c1 : gi * GROUP + GROUP - 1, sp.c0);
      y.keep(A.group_parts + ((long long)gi * 2 + (gi == g0)) * S::PART, tid);
      named_bar(3, TEAMS * MATH);
      if (tid == 0) {
        __threadfence();
        const bool all = atomicAdd(&A.counts[sp.c0], 1u) == (uint32_t)(g1 - g0);
        if (all) A.counts[sp.c0] = 0;
        s_flags[1 + i] = all;
        __threadfence();
      }
      named_bar(3, TEAMS * MATH);
      if (!s_flags[1 + i]) continue;
      join(A.group_parts, g0, g1, g0);
    }
    y.finish(A, sp.b, h0, nh, vs, tid);
  }
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

using ReplaceFn = CUresult (*)(CUtensorMap*, void*);

template <class F>
cudaError_t driver_fn(const char* name, std::atomic<F>& known, F* out) {
  F f = known.load(std::memory_order_relaxed);
  if (!f) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion(name, &p, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || !p) return cudaErrorNotSupported;
    known.store(f = reinterpret_cast<F>(p), std::memory_order_relaxed);
  }
  *out = f;
  return cudaSuccess;
}
std::atomic<EncodeFn> g_encode{nullptr};
std::atomic<ReplaceFn> g_replace{nullptr};

// a pool as rows of a head's D elements, LT of them together: [page][head, token][d], copied `groups` of 16 tokens x
// CB bytes at a time
template <class S>
cudaError_t pool_map(const CacheShape& c, const void* pool, int64_t page_stride, int groups, CUtensorMap* m) {
  EncodeFn fn;
  const cudaError_t e = driver_fn("cuTensorMapEncodeTiled", g_encode, &fn);
  if (e != cudaSuccess) return e;
  const int es = S::E4M3 ? 1 : 2;
  const cuuint64_t rows = ((cuuint64_t)c.Hkv << c.page_log2) / S::LT;
  const cuuint64_t dims[3] = {(cuuint64_t)S::D * S::LT, rows, (cuuint64_t)c.n_pages};
  const cuuint64_t strides[2] = {(cuuint64_t)S::RB * S::LT, (cuuint64_t)page_stride * es};
  const cuuint32_t box[3] = {(cuuint32_t)(S::CB / es), (cuuint32_t)(16 * groups / S::LT), 1}, ones[3] = {1, 1, 1};
  const CUtensorMapDataType type = S::E4M3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16;
  const CUresult r = fn(m, type, 3, (void*)pool, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

constexpr int SMEM_PER_CTA = 227 * 1024;

template <class S>
cudaError_t run(const CacheShape& c, AttendArgs& A, int ctas, cudaStream_t st) {
  static_assert(S::MISC + 1024 + CACHE_MAX_REQUESTS * 4 + S::TEAMS * 2 * S::STAGE <= SMEM_PER_CTA,
                "a ring has two stages at least");
  // where a row is a line or less, a copy takes as much of a page as fits a stage (64 requests, 540 MB: rows of 64
  // bytes come at 3.7, 4.4, 4.7 and 5.1 TB/s from pages of 16, 32, 64 and 256 tokens, which are copies of 1, 2, 4 and
  // 16 KB; rows of 128 bytes at 5.6 to 6.2). Copies of longer rows are of 2 KB and more as they are: larger ones won
  // nothing (84.5 and 84.1 us for heads of 256)
  A.box = 1;
  while (S::CH == 1 && 2 * A.box <= S::GPS && 32 * A.box <= 1 << c.page_log2) A.box *= 2;
  CUtensorMap km, vm;
  cudaError_t e = pool_map<S>(c, A.a.k_cache, A.a.k_page_stride, A.box, &km);
  if (e == cudaSuccess && A.a.v_page_stride == A.a.k_page_stride) {
    // the same map at another address: half the host's time for two
    ReplaceFn replace;
    e = driver_fn("cuTensorMapReplaceAddress", g_replace, &replace);
    vm = km;
    if (e == cudaSuccess && replace(&vm, (void*)A.a.v_cache) != CUDA_SUCCESS) e = cudaErrorInvalidValue;
  } else if (e == cudaSuccess) {
    e = pool_map<S>(c, A.a.v_cache, A.a.v_page_stride, A.box, &vm);
  }
  if (e != cudaSuccess) return e;
  A.head_tiles = (A.group + S::NH - 1) / S::NH;
  const int other = S::MISC + 1024 + A.B * 4;
  const int n = (SMEM_PER_CTA - other) / (S::TEAMS * S::STAGE);
  A.n_stages = n > 16 ? 16 : n;
  // the kernel's shared-memory limit, once per device
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  e = cudaGetDevice(&dev);
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
  if (e == cudaSuccess && !(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(k_cache_attend<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_PER_CTA);
    if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_relaxed);
  }
  if (e != cudaSuccess) return e;
  return launch_following(k_cache_attend<S>, ctas, S::THREADS, other + S::TEAMS * A.n_stages * S::STAGE, st, A, km, vm);
}

template <int D, bool BF16, bool E4M3>
cudaError_t run_heads(const CacheShape& c, AttendArgs& A, int ctas, cudaStream_t st) {
  // the fewest heads to an item that keep a group in one, up to 32: an item more reads the cache once more, from L2 (32
  // over 1 heads of 128, 400 MB: 74 us as one item, 124 as two; of 256: 85 and 124, over an e4m3 cache 117 and 136)
  if (A.group <= 8) return run<Shape<D, BF16, E4M3, 1>>(c, A, ctas, st);
  if (A.group <= 16) return run<Shape<D, BF16, E4M3, 2>>(c, A, ctas, st);
  return run<Shape<D, BF16, E4M3, 4>>(c, A, ctas, st);
}
template <int D>
cudaError_t run_types(const CacheShape& c, AttendArgs& A, int ctas, cudaStream_t st) {
  if (c.bf16) return c.e4m3 ? run_heads<D, true, true>(c, A, ctas, st) : run_heads<D, true, false>(c, A, ctas, st);
  return c.e4m3 ? run_heads<D, false, true>(c, A, ctas, st) : run_heads<D, false, false>(c, A, ctas, st);
}

}  // namespace

size_t cache_attend_workspace(int num_sms) {
  const size_t ctas = num_sms < MAX_CTAS ? num_sms : MAX_CTAS;
  const size_t groups = (ctas + GROUP - 1) / GROUP;
  return ((ctas + groups) * 2 * PART_MAX + COUNT_WORDS) * 4;
}

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
  const int ctas = w.num_sms < MAX_CTAS ? w.num_sms : MAX_CTAS;       // one to an SM
  A.counts = (uint32_t*)w.workspace;
  A.group_counts = A.counts + MAX_CTAS;
  A.parts = (float*)w.workspace + COUNT_WORDS;
  A.group_parts = A.parts + (size_t)ctas * 2 * PART_MAX;
  A.status = w.status;
  A.timeout_ns = w.timeout_ns;
  A.skip_copy = w.skip_copy;
  if (S.D == 64) return run_types<64>(S, A, ctas, st);
  if (S.D == 128) return run_types<128>(S, A, ctas, st);
  return run_types<256>(S, A, ctas, st);
}

}  // namespace moe
