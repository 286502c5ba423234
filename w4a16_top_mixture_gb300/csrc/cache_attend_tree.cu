// Attention of several new tokens of each request over the paged cache (moe_cache_attend_tree).
//
// The new tokens of a request times the query heads of a group are rows that meet the same keys and values: 128 of them
// are a tile of the tensor cores, so that S[rows x tokens] = Q K^T and O[rows x d] += P V are tcgen05 products with the
// rows' statistics a thread's each. Up to 128 rows the bytes of the cache bound the kernel, above it the products.
//   Work. An item is a request, a key-value head and 128 rows. The tiles of TN tokens of all items, one after another, are
// divided evenly over the CTAs, one to an SM; an item that crosses a CTA's border is split. Nobody waits for another CTA:
// parts (O, the rows' bases and sums) go to the workspace, and the CTA that counts itself last joins them, in the order of
// the tiles; more than FLAT of them in groups first (one request of 131072 tokens has 76 for each head).
//   Roles. One warp finds the CTA's items, one copies (TMA, a ring of stages, keys one tile ahead of values), one issues
// the products, eight do the softmax, two threads to a row, and four prepare: the queries go to tensor memory, where they
// are the first operand; 8-bit tiles are converted to fp16 (two pairs of warps, every other stage each); and values of tiles
// with new tokens are looked through (below).
//   Tensor memory. O, Q and two S: the products of one tile run during the softmax of the other. P lies where S was. With
// Q there a product reads shared memory for its second operand alone (64 columns: 32.5 cycles, 48.5 with Q in shared
// memory), and all of it holds stages.
//   Layout. A stage holds [8 tokens][64 elements] blocks of 1 KB in the 128-byte swizzle, the blocks of 8 tokens side by
// side, whatever the pages: as K it is read along d, as V along the tokens, by the descriptors' strides alone.
//   Bases. P = 2^(score - base): the base is a row's first maximum and follows when one passes it by more than TAU, since
// that rescales O (2000 cycles; with TAU 2 some warp of the eight did at nearly every tile). fp16 weights are lifted by
// 2^LIFT, so that a long tail below the highest keeps its bits; bf16 weights are lowered to 1 at most, so that O stays in
// range as far as n times the largest value does.
//   Values that are not finite. A weight of 0 does not keep NaN out of a product. What lies past a request's end is zeroed
// in shared memory; a new token's value that some rows do not see is looked at, and where it is not finite, zeroed too and
// added at the item's end to the rows that see it.
//   Local memory. With 227 KB of shared memory there is next to no L1, so that spills and calls cost what a load from L2 does:
// nothing is called out of line (an item's end so was 30 to 50 % slower). At 128 registers the compiler spills 8 bytes a
// thread or none with heads of 256, 44 to 88 with smaller ones.
// Measured (16 query over 2 key-value heads of 256 unless said): 64 requests of 4096 tokens, 8 new ones each, 100 us, 5.5
// TB/s (a copy runs at 6.7); 16 new ones over an e4m3 cache 86 us, 3.4 TB/s; 32 over 8 heads of 128, 16 new ones, 178 us, 6.2
// TB/s; heads of 64, 8 new ones, 133 us in 16 bits and 138 over e4m3 (4.1 and 2.0 TB/s); one request of 131072 tokens, 5 new
// ones, 72 us, of which the tiles' bytes are 40; one of 130 tokens 13.7 us. Above 128 rows the tiles come from L2 once for
// each 128: 256 new tokens of 16 requests of 8192 tokens 584 us, 0.93 PFLOP/s.
// What is left is this design's: a tile's scores, maxima, weights and hand-over one after another in one set of warps, rows
// of the 128 that do not exist, 6 us until the first scores, an item's end on the warps that the next item waits for (5 to 12
// us for 128 gated rows), and the tiles' way from L2 for wide trees and chunks. One token of each request is moe_cache_attend's:
// its tiles have the heads as their narrow side, and it takes 7.7 us for 130 tokens, 50 us for the 64 requests over e4m3.
#include <cuda.h>

#include <atomic>

#include "cache.cuh"
#include "ptx.cuh"
#include "umma.cuh"

namespace moe {
namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr int THREADS = 512, MAX_CTAS = 1024, EXTRA = 7, SHORT = EXTRA + 3, ITEMS = 4, M = 128;
// Parts of a group, and parts that are joined without groups: 76 parts of one request of 131072 tokens take 72 us in groups of 8,
// 78 in groups of 4 and 75 of 16; four requests of 20000, 19 parts each, 50 us in groups and 58 without; 6 for FLAT changes
// nothing measured.
constexpr int GROUP_OF = 8, FLAT = 12;
constexpr int SMEM = 227 * 1024, MISC = 3 * 1024;
constexpr int W_PRODUCE = 0, W_MMA = 1, W_FIND = 2, W_SOFT = 4, W_PREP = 12, SOFT = 8;   // SOFT: warps of the softmax

struct TreeArgs {
  moe_cache_attend_tree_t a;
  int B, rows, Hkv, group, page_log2, n_pages, most;
  long long max_len;
  float scale;               // with log2(e)
  float* parts;              // [CTA][2][M * D + 2 * M]: the item a CTA begins in the middle of, the one it leaves so
  uint32_t* counts;          // [CTA][3]: parts that have arrived, of an item, of its group of parts that starts in the CTA
  uint32_t* status;
  uint64_t timeout_ns;
  int skip_copy;
};

template <int D_, bool BF16_, bool E4M3_>
struct Shape {
  static constexpr int D = D_;
  static constexpr bool BF16 = BF16_, E4M3 = E4M3_, MBF16 = BF16_ && !E4M3_;   // e4m3 is exact in fp16: both products' type
  static constexpr int TN = D == 256 ? 64 : 128;
  static constexpr int BLOCKS = D / 64, GROUP = BLOCKS * 1024;                 // of 8 tokens
  static constexpr int TILE = TN / 8 * GROUP, RAW = E4M3 ? TN * D : TILE;
  static constexpr int NC = E4M3 ? 4 : 0;                                      // converted tiles
  static constexpr int CTL = MISC + (E4M3 ? 2 * M * 4 : 0);
  static constexpr int NR0 = (SMEM - CTL - NC * TILE) / RAW, NR = NR0 > 12 ? 12 : NR0;
  static constexpr int DYN = NC * TILE + NR * RAW + CTL;
  static constexpr uint32_t O = 0, Q = D, S0 = D + D / 2;                      // columns of tensor memory
  static constexpr float TAU = 8.f, LIFT = MBF16 ? -TAU : 7.f;                 // weights: 1 or 2^15 at most
  static constexpr int NC1 = NC ? NC : 1;
  static constexpr int PART = M * D + 2 * M;
  static_assert(S0 + 2 * TN <= 512 && DYN <= SMEM && NR >= 4, "fits");
};

struct Item {
  int b, lo, n, older, len;  // b < 0: no more items. n: rows of the batch
  int g, m0, rows;           // key-value head; first row of the 128 and how many there are
  int t0, t1;                // tiles
  int c0, c1;                // the CTAs of its first and last tile
};

struct Control {
  // new_full, fixed: of the tiles that are looked through, or (c_full, c_empty) of the converted ones
  uint64_t full[12], empty[12], new_full[8], fixed[8], s_full[2], p_ready[2], pv_done, q_ready, q_free, o_free, o_full,
      drained, pair[4][2], soft;
  uint64_t item_full[ITEMS], item_empty[ITEMS];
  Item items[ITEMS];
  uint4 odd[ITEMS][CACHE_MAX_NEW / 128];   // bits of the new tokens whose values were not finite, in this CTA's tiles
  int last;                  // this CTA's part is the last to arrive
  union {
    struct {                 // of the warps' requests, read before the first item is given out
      long long sums[THREADS / 32];
      int longest[THREADS / 32];
    };
    float top[2][2][M];      // maxima of the halves of a row's tokens in a tile; their sums at an item's end
  };
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Control) <= MISC, "control words");

// ---- instructions ----
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// y sigmoid(x), four at a time: e = exp(-|x|) <= 1 cannot overflow, and one reciprocal of the product of the four 1 + e,
// at most 16, does for all. Of the special functions' rate five parts in four an element are left of two.
__device__ __forceinline__ void gated4(float (&y)[4], float2 g0, float2 g1) {
  const float x[4] = {g0.x, g0.y, g1.x, g1.y};
  float d[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float e = __expf(-fabsf(x[i]));
    y[i] = x[i] >= 0.f ? y[i] : y[i] * e;            // a NaN goes to its own element,
    d[i] = 1.f + fminf(e, 1.f);                     // and not into the product
  }
  const float a = d[0] * d[1], b = d[2] * d[3], r = __fdividef(1.f, a * b), ra = r * b, rb = r * a;
  y[0] *= ra * d[1];
  y[1] *= ra * d[0];
  y[2] *= rb * d[3];
  y[3] *= rb * d[2];
}
__device__ __forceinline__ void tma5(void* dst, const CUtensorMap* m, int group, int page, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1, {%2, %2, %2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
      "l"(m), "r"(0), "r"(group), "r"(page), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma3(void* dst, const CUtensorMap* m, int row, int page, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
      "l"(m), "r"(0), "r"(row), "r"(page), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// see tmem_wait_ld: the registers are valid from here on
__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
// 8 columns, valid on return; stored without a wait
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n tcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// a shared-memory descriptor of blocks in the 128-byte swizzle: bytes between blocks along the other dimension of the
// layout (lead, read where the operand runs across its rows) and between groups of 8 rows (stride)
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr, uint32_t lead, uint32_t stride) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(stride >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// 128 rows x n: 16-bit operands, fp32 sums, B across its rows where `across`
__device__ __forceinline__ uint32_t idesc(bool bf16, bool across, int n) {
  return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (across ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 |
         (uint32_t)(M >> 4) << 24;
}

// Rows of 16-bit elements lie apart, and a row is a lane's: 16 bytes of 32 rows are 32 half-used sectors (128 rows of 256
// elements took 8 us to load so, and 15 us to gate and store). So four lanes take 64 bytes of one row together, of four
// rows in turn, and change places in registers.
__device__ __forceinline__ void change_places(uint4 (&v)[4], int lane) {
#pragma unroll
  for (int b = 1; b < 4; b <<= 1) {
    const bool high = lane & b;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j & b) continue;
      uint4 t = high ? v[j] : v[j ^ b];
      t.x = __shfl_xor_sync(0xFFFFFFFFu, t.x, b);
      t.y = __shfl_xor_sync(0xFFFFFFFFu, t.y, b);
      t.z = __shfl_xor_sync(0xFFFFFFFFu, t.z, b);
      t.w = __shfl_xor_sync(0xFFFFFFFFu, t.w, b);
      if (high) v[j] = t; else v[j ^ b] = t;
    }
  }
}
// the lane's place in the rows of its four lanes: row k's 16 bytes are the lane & 3 rd, NULL where there is no row
struct FourRows {
  uint16_t* at[4];
  __device__ __forceinline__ FourRows(uint16_t* row, int lane) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint64_t p = __shfl_sync(0xFFFFFFFFu, (unsigned long long)row, (lane & ~3) + k);
      at[k] = p ? reinterpret_cast<uint16_t*>(p) + (lane & 3) * 8 : nullptr;
    }
  }
  // 32 elements from x on, as four lanes hold them together
  __device__ __forceinline__ void load(uint4 (&v)[4], int x) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = at[k] ? __ldcg(reinterpret_cast<const uint4*>(at[k] + x)) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void store(const uint4 (&v)[4], int x) const {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (at[k]) *reinterpret_cast<uint4*>(at[k] + x) = v[k];
  }
};

__device__ __forceinline__ uint16_t* rows_at(const moe_rows_t& r, int64_t row, int h) {
  return (uint16_t*)r.p + row * r.row_stride + h * r.head_stride;
}

// ---- the division of the work ----
// A request's items are of n_tiles tiles and EXTRA units for what an item's beginning and end cost. 16 requests with trees of
// 64, 80 to 8191 tokens, in us with 3, 5, 7, 10 of them: heads of 256 with a gate 88, 77, 70, 70, without 65, 62, 62, 63 (over
// e4m3 a few less); of 128 80, 66, 65, 70 and 64, 58, 61, 66; of 64 53, 52, 55, 59 and 46, 50, 53, 57. Long even batches and
// single requests do not depend on it. One number for all of them is a compromise: heads of 64 would have 5 or less.
// While no item is longer than SHORT units, a CTA's share is at least the longest item: 64 requests of 190 tokens take 18 us so
// and 30 with even shares, 8 of 130 tokens 14.3 and 16.4. Items are whole only where all are of one length: 40 requests of 20
// to 190 tokens are split at borders inside items all the same, and take 27 us so and 18 with even shares.
struct Request {
  int lo, n, older, len, tiles, m_tiles;
};
template <class S>
__device__ __forceinline__ Request request(const TreeArgs& A, int b, uint32_t* bad) {
  Request r = {};
  if (b >= A.B) return r;
  const NewTokens t = new_tokens_of(A.a.starts, A.a.slots, A.a.lengths, b, A.rows, A.max_len, A.most, bad);
  r.lo = t.lo;
  r.n = t.rows;
  const bool live = !t.left_out && t.n > 0;
  r.len = live ? t.len : 0;
  r.older = live ? t.len - t.n : 0;
  r.tiles = (int)(((unsigned)r.len + S::TN - 1) / S::TN);
  r.m_tiles = (int)(((long long)r.n * A.group + M - 1) / M);
  return r;
}
__device__ __forceinline__ long long units_of(const TreeArgs& A, const Request& r) {
  return (long long)A.Hkv * r.m_tiles * (r.tiles + EXTRA);
}

// An item's stages: keys are one tile ahead of values, K0 K1 V0 K2 V1 .. V(n-1)

// a place in a ring of N stages and the parity of its round, one after another
template <int N>
struct Place {
  int at = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next(int by = 1) {          // by <= N
    at += by;
    if (at >= N) {
      at -= N;
      parity ^= 1;
    }
  }
};

// a row's mask over its request's new tokens, as 32-bit words
struct Mask {
  uint32_t w[CACHE_MAX_NEW / 32];
  __device__ __forceinline__ uint32_t word(int k) const {
    uint32_t r = k < 0 ? 0xFFFFFFFFu : 0u;          // older tokens are seen, what lies past the end is not
#pragma unroll
    for (int i = 0; i < CACHE_MAX_NEW / 32; ++i) r = k == i ? w[i] : r;
    return r;
  }
  // the 32 tokens from place `from` among the new ones on (below 0: older ones)
  __device__ __forceinline__ uint32_t window(int from) const {
    const int k = from >> 5;
    return __funnelshift_r(word(k), word(k + 1), from & 31);
  }
  __device__ __forceinline__ void load(const TreeArgs& A, int row, int i, int n, bool some) {
#pragma unroll
    for (int k = 0; k < CACHE_MAX_NEW / 64; ++k) {
      uint64_t v = 0;
      if (some && A.a.masks) {
        if (k < A.a.mask_words) v = __ldcg((const unsigned long long*)A.a.masks + (size_t)row * A.a.mask_words + k);
      } else if (some) {
        const int upto = i - 64 * k;
        v = upto < 0 ? 0ull : upto >= 63 ? ~0ull : (2ull << upto) - 1;
      }
      const int left = n - 64 * k;
      v = left <= 0 ? 0ull : left >= 64 ? v : v & ((1ull << left) - 1);
      w[2 * k] = (uint32_t)v;
      w[2 * k + 1] = (uint32_t)(v >> 32);
    }
  }
};

// two elements in 16 bits with those that are not finite made 0
template <bool BF16>
__device__ __forceinline__ uint32_t finite2(uint32_t v) {
  const uint32_t e = BF16 ? 0x7F80u : 0x7C00u;
  if ((v & e) == e) v &= 0xFFFF0000u;
  if ((v >> 16 & e) == e) v &= 0xFFFFu;
  return v;
}

// What was taken out of the values of new tokens is added to the rows that see it: half of O's elements from x on, at `o`.
// Of the noted tokens 32 are looked at together, a lane's each and 8 elements at a time: whether a row gets an infinity or a
// NaN is a vote over the lanes and the row's mask, however many tokens hold one. 24 chunks of 256 tokens, 16 over 2 heads of
// 256, 307 us: 331 where one value of one request is infinite, 556 where all of its new ones are NaN, 622 infinite (an element
// of a token after the other: 64 to 69 ms).
template <class S>
__device__ __forceinline__ void add_odd(const TreeArgs& A, const Item& it, const uint4* odd, int t, int x, uint32_t o) {
  const moe_cache_attend_tree_t& a = A.a;
  const unsigned ALL = 0xFFFFFFFFu;
  const int lane = threadIdx.x & 31, i = (it.m0 + t) / A.group, ps = 1 << A.page_log2;
#pragma unroll 1
  for (int k = 0; k < CACHE_MAX_NEW / 32; ++k) {
    const uint32_t noted = *(volatile const uint32_t*)(reinterpret_cast<const uint32_t*>(odd) + k);
    if (!noted) continue;
    const bool own = noted >> lane & 1;
    const int p = it.older + (own ? 32 * k + lane : 0);
    const int page = own ? __ldcg(a.tables + (size_t)it.b * a.table_stride + (p >> A.page_log2)) : -1;
    const bool mine = page >= 0 && page < A.n_pages;
    const int64_t at = (mine ? page : 0) * a.v_page_stride + ((int64_t)it.g * ps + (p & (ps - 1))) * S::D + x;
    uint32_t sees = 0;                              // of these tokens, by the lane's row
    if (t < it.rows) {
      if (a.masks) sees = __ldcg(reinterpret_cast<const uint32_t*>(a.masks + (size_t)(it.lo + i) * a.mask_words) + k);
      else sees = i < 32 * k ? 0u : i >= 32 * k + 31 ? ~0u : (2u << (i & 31)) - 1;
    }
#pragma unroll 1
    for (int c = 0; c < S::D / 2; c += 8) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (mine && !S::E4M3) v = __ldcg(reinterpret_cast<const uint4*>((const uint16_t*)a.v_cache + at + c));
      if (mine && S::E4M3) {
        const uint2 w = __ldcg(reinterpret_cast<const uint2*>((const uint8_t*)a.v_cache + at + c));
        e4m3x4_to_f16x4(w.x, v.x, v.y);
        e4m3x4_to_f16x4(w.y, v.z, v.w);
      }
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t r[8];
      __syncwarp();
      tmem_ld8(o + c, r);
      bool nan = true;                              // in all rows: they stay so
#pragma unroll
      for (int e = 0; e < 8; ++e) nan = nan && (r[e] & 0x7FFFFFFFu) > 0x7F800000u;
      if (__all_sync(ALL, nan || t >= it.rows)) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 f = unpack2<S::BF16 && !S::E4M3>(w[e / 2]);
        const float y = e & 1 ? f.y : f.x;
        const bool up = !S::E4M3 && __ballot_sync(ALL, y == INFINITY) & sees;    // e4m3 has no infinities
        const bool down = !S::E4M3 && __ballot_sync(ALL, y == -INFINITY) & sees;
        if (up) r[e] = __float_as_uint(__uint_as_float(r[e]) + INFINITY);
        if (down) r[e] = __float_as_uint(__uint_as_float(r[e]) - INFINITY);
        if (__ballot_sync(ALL, y != y) & sees) r[e] = 0x7FFFFFFFu;
      }
      __syncwarp();
      tmem_st8(o + c, r);
    }
    tmem_wait_st();                                 // before these columns are read again
  }
}

// The sum of parts p0, p0 + by .. below p1 of a row, on their highest base, in the order of the parts.
template <class S>
struct Sum {
  float m = -INFINITY, l = 0.f;
  __device__ __forceinline__ float factor(float pm, float pl) const {
    return pm == -INFINITY ? (pl == pl ? 0.f : pl) : exp2_fast(pm - m);   // no base and a sum of NaN: all scores NaN
  }
  // base(p): a row's base, its sum M further on; four at a time
  template <class F>
  __device__ __forceinline__ void bases(F base, int p0, int p1, int by) {
#pragma unroll 1
    for (int p = p0; p < p1; p += 4 * by) {
      float pm[4], pl[4], top = m;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float* q = base(min(p + i * by, p1 - 1));       // the last one again adds nothing
        pm[i] = __ldcg(q);
        pl[i] = __ldcg(q + M);
        if (p + i * by >= p1) pm[i] = -INFINITY, pl[i] = 0.f;
        top = fmaxf(top, pm[i]);
      }
      l *= m == -INFINITY ? (l == l ? 0.f : l) : exp2_fast(m - top);
      m = top;
#pragma unroll
      for (int i = 0; i < 4; ++i) l = fmaf(pl[i], factor(pm[i], pl[i]), l);
    }
  }
  __device__ __forceinline__ static void load(float4 (&v)[8], const float* at) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __ldcg(reinterpret_cast<const float4*>(at) + e * M);
  }
  __device__ __forceinline__ static void put(float (&y)[32], const float4 (&v)[8], float f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[4 * e] = fmaf(v[e].x, f, y[4 * e]);
      y[4 * e + 1] = fmaf(v[e].y, f, y[4 * e + 1]);
      y[4 * e + 2] = fmaf(v[e].z, f, y[4 * e + 2]);
      y[4 * e + 3] = fmaf(v[e].w, f, y[4 * e + 3]);
    }
  }
  // 32 elements, at at(p)
  template <class F, class G>
  __device__ __forceinline__ void add(float (&y)[32], F at, G base, int p0, int p1, int by) const {
#pragma unroll 1
    for (int p = p0; p < p1; p += by) {
      float4 v[8];
      load(v, at(p));
      put(y, v, factor(__ldcg(base(p)), __ldcg(base(p) + M)));
    }
  }
};

// 32 elements of a row's output, y vs / l times the gate's sigmoid, from x on; 0 where l is 0, the row saw nothing or scores of
// -inf alone, whatever O (0 times an infinite value) and the gate hold
template <class S>
__device__ __forceinline__ void emit(const float (&y)[32], float l, float vs, uint16_t* gate, bool gated, uint16_t* out, int x,
                                     int lane) {
  uint4 g[4], z[4];
  if (gated) {
    FourRows(gate, lane).load(g, x);
    change_places(g, lane);
  }
  const float by = __fdividef(vs, l);
  const bool none = l == 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t w[4] = {g[e].x, g[e].y, g[e].z, g[e].w};
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      float q[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) q[k] = y[8 * e + 2 * i + k] * by;
      if (gated) gated4(q, unpack2<S::BF16>(w[i]), unpack2<S::BF16>(w[i + 1]));
      r[i] = pack2<S::BF16>(q[0], q[1]);
      r[i + 1] = pack2<S::BF16>(q[2], q[3]);
    }
    z[e] = none ? make_uint4(0, 0, 0, 0) : make_uint4(r[0], r[1], r[2], r[3]);
  }
  change_places(z, lane);
  FourRows(out, lane).store(z, x);
}

// By whole warps, and in line: a call would spill what is live. A wait that runs out ends its role's work, and so, as what
// it would have given is waited for, the CTA's.
__device__ __forceinline__ bool wait_for(const TreeArgs& A, Control& C, uint64_t* bar, uint32_t parity) {
  if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = globaltimer();
  do {
    if (__all_sync(0xFFFFFFFFu, mbar_try_wait_sleep(bar, parity, 20000u))) return true;
  } while (__any_sync(0xFFFFFFFFu, globaltimer() - t0 <= A.timeout_ns));
  if (!*(volatile int*)&C.abort) {
    *(volatile int*)&C.abort = 1;
    atomicOr(A.status, CACHE_BAD_WAIT);
  }
  return false;
}
// what is in flight lands, or 100 ms pass
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait_sleep(bar, parity, 20000u) && globaltimer() - t0 < 100000000) {
  }
}
// a barrier of the softmax's warps; n counts them
__device__ __forceinline__ bool soft_barrier(const TreeArgs& A, Control& C, int& n) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&C.soft);
  return wait_for(A, C, &C.soft, n++ & 1);
}

// What an item's rows get, from their O in tensor memory and the parts of other CTAs; called by the softmax's warps.
// False: a wait ran out.
template <class S>
__device__ __forceinline__ bool finish_item(const TreeArgs& A, Control& C, int slot, uint32_t lanes, float ref, float l, int& syncs) {
  constexpr int HD = S::D / 2;
  const moe_cache_attend_tree_t& a = A.a;
  const Item& it = C.items[slot];
  const int cta = blockIdx.x;
  const int lane = threadIdx.x & 31, sw = (threadIdx.x >> 5) - W_SOFT, half = sw >> 2, t = (sw & 3) * 32 + lane;
  const int n = it.t1 - it.t0, parts = it.c1 - it.c0 + 1, step = parts > FLAT ? GROUP_OF : 1, mine = cta - it.c0;
  const float vs = S::E4M3 ? __ldcg(a.v_scale + it.g) : 1.f;
  const bool gated = a.gate.p != nullptr;
  // a row of the batch and its head, NULL past the item's rows
  auto row_of = [&](const moe_rows_t& r, int t) -> uint16_t* {
    const int m = it.m0 + t, i = m / A.group;
    return t < it.rows ? rows_at(r, it.lo + i, it.g * A.group + m - i * A.group) : nullptr;
  };
  if (n) {
    const uint4 *odd = C.odd[slot], b0 = odd[0], b1 = odd[1];
    if (__builtin_expect(b0.x | b0.y | b0.z | b0.w | b1.x | b1.y | b1.z | b1.w, 0))
      add_odd<S>(A, it, odd, t, half * HD, lanes + S::O + half * HD);
  }
  if (parts == 1) {
    uint16_t *out = row_of(a.out, t), *gate = gated ? row_of(a.gate, t) : nullptr;
    if (t - lane < it.rows)                         // the warp has rows
#pragma unroll 1
      for (int x = half * HD; x < half * HD + HD; x += 32) {
        uint32_t r[32];
        float y[32];
        if (n) {
          tmem_ld32(lanes + S::O + x, r);
          tmem_wait_ld32(r);
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) y[e] = n ? __uint_as_float(r[e]) : 0.f;
        emit<S>(y, l, vs, gate, gated, out, x, lane);
      }
    __syncwarp();
  } else {
    float* part = A.parts + (size_t)(cta * 2 + (mine == 0)) * S::PART;
#pragma unroll 1
    for (int x = half * HD; x < half * HD + HD; x += 32) {   // [D / 4][rows] of four elements
      uint32_t r[32];
      __syncwarp();
      tmem_ld32(lanes + S::O + x, r);
      tmem_wait_ld32(r);
      if (t < it.rows) {
        float4* to = reinterpret_cast<float4*>(part) + x / 4 * M + t;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          __stcg(to + e * M, make_float4(__uint_as_float(r[4 * e]), __uint_as_float(r[4 * e + 1]),
                                         __uint_as_float(r[4 * e + 2]), __uint_as_float(r[4 * e + 3])));
      }
    }
    if (t < it.rows && half == 0) {
      __stcg(part + M * S::D + t, ref);
      __stcg(part + M * S::D + M + t, l);
    }
  }
  if (n) {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&C.o_free);
  }
  if (parts == 1) return true;

  // Whoever counts itself last joins: where there are many parts those of its group, and then the groups.
  bool last = false;
  auto arrive = [&](uint32_t* count, int of) {
    if (!soft_barrier(A, C, syncs)) return false;
    if (sw == 0 && lane == 0) {                     // its fences stand for all, on this side of each barrier
      __threadfence();
      C.last = atomicAdd(count, 1u) == (uint32_t)of - 1;
      if (C.last) {
        __threadfence();
        *count = 0;
      }
    }
    if (!soft_barrier(A, C, syncs)) return false;
    last = C.last;
    return true;
  };
  auto part_at = [&](int p) { return A.parts + (size_t)((it.c0 + p) * 2 + (p == 0)) * S::PART; };
  // 32 rows and 32 elements at a time, whichever warp: f(row, x, elements, sum)
  const int row_tiles = (it.rows + 31) / 32;
  auto join = [&](int p0, int p1, int by, auto f) {
#pragma unroll 1
    for (int q = sw; q < row_tiles * (S::D / 32); q += SOFT) {
      const int x = q / row_tiles * 32, t = q % row_tiles * 32 + lane, u = min(t, it.rows - 1);
      auto base = [&](int p) { return part_at(p) + M * S::D + u; };
      Sum<S> sum;
      float y[32] = {};
      sum.bases(base, p0, p1, by);
      sum.add(y, [&](int p) { return part_at(p) + (size_t)(x / 4 * M + u) * 4; }, base, p0, p1, by);
      f(t, x, y, sum);
    }
    __syncwarp();
  };
  if (step > 1) {
    const int p0 = mine / GROUP_OF * GROUP_OF, p1 = min(parts, p0 + GROUP_OF);
    if (!arrive(A.counts + 3 * (it.c0 + p0) + 1 + (p0 == 0), p1 - p0)) return false;
    if (!last) return true;
    float* to = part_at(p0);
    join(p0, p1, 1, [&](int t, int x, const float (&y)[32], const Sum<S>& sum) {
      if (t >= it.rows) return;
      float4* q = reinterpret_cast<float4*>(to) + x / 4 * M + t;
#pragma unroll
      for (int e = 0; e < 8; ++e) __stcg(q + e * M, make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]));
    });
    Sum<S> sum;
    if (t < it.rows) sum.bases([&](int p) { return part_at(p) + M * S::D + t; }, p0, p1, 1);
    if (!soft_barrier(A, C, syncs)) return false;   // all have read the group's bases
    if (t < it.rows && half == 0) {
      __stcg(to + M * S::D + t, sum.m);
      __stcg(to + M * S::D + M + t, sum.l);
    }
  }
  if (!arrive(A.counts + 3 * it.c0, (parts + step - 1) / step)) return false;
  if (last)
    join(0, parts, step, [&](int t, int x, const float (&y)[32], const Sum<S>& sum) {
      emit<S>(y, sum.l, vs, gated ? row_of(a.gate, t) : nullptr, gated, row_of(a.out, t), x, lane);
    });
  return true;
}

template <class S>
__global__ void __launch_bounds__(THREADS, 1)
    k_attend_tree(const __grid_constant__ TreeArgs A, const __grid_constant__ CUtensorMap km,
                  const __grid_constant__ CUtensorMap vm) {
  extern __shared__ __align__(1024) uint8_t sm[];
  if (smem_u32(sm) & 1023) {                        // the swizzle needs it, and the attribute gives it
    if (threadIdx.x == 0) atomicOr(A.status, CACHE_BAD_WAIT);
    return;
  }
  uint8_t* conv = sm;                               // converted tiles
  uint8_t* ring = sm + S::NC * S::TILE;
  Control& C = *reinterpret_cast<Control*>(ring + S::NR * S::RAW);
  const moe_cache_attend_tree_t& a = A.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x, ctas = gridDim.x;
  const unsigned ALL = 0xFFFFFFFFu;
  uint64_t *c_full = C.new_full, *c_empty = C.fixed;
  // [2][M], items in turn: undoes what bf16 queries over an 8-bit cache were multiplied by
  float* undo = reinterpret_cast<float*>(ring + S::NR * S::RAW + MISC);

  if (threadIdx.x == 0) {
    for (int i = 0; i < 12; ++i) {
      mbar_init(&C.full[i], 1);
      mbar_init(&C.empty[i], S::E4M3 ? 2 : 1);      // the converting warps, or the products that read it
    }
    for (int i = 0; i < 8; ++i) {
      mbar_init(&C.new_full[i], S::E4M3 ? 2 : 1);
      mbar_init(&C.fixed[i], S::E4M3 ? 1 : 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&C.s_full[i], 1);
      mbar_init(&C.p_ready[i], SOFT);
    }
    for (int i = 0; i < ITEMS; ++i) {
      mbar_init(&C.item_full[i], 1);
      mbar_init(&C.item_empty[i], 2 + SOFT + 4);
    }
    mbar_init(&C.pv_done, 1);
    mbar_init(&C.o_full, 1);
    mbar_init(&C.drained, 1);
    mbar_init(&C.q_ready, 4);
    mbar_init(&C.q_free, 1);
    mbar_init(&C.o_free, SOFT);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&C.pair[i][0], 2);
      mbar_init(&C.pair[i][1], 2);
    }
    mbar_init(&C.soft, SOFT);
    C.abort = 0;
    fence_mbar_init();
  }
  if (warp == W_MMA) {
    tmem_alloc(&C.tmem, 512);
    tmem_relinquish();
  }
  follow_predecessor();
  // an earlier call gave up and has not been reported: nothing is computed
  const bool dead = __ldcg(A.status) & CACHE_BAD_WAIT;
  // the units of all requests, a block of them to a warp
  const bool few = A.B <= 32;                       // the finding warp sees them all
  const int per = few ? 32 : (A.B + THREADS / 32 - 1) / (THREADS / 32);
  uint32_t bad = 0;
  if (!few) {
    long long sum = 0;
    int longest = 0;
    for (int i = lane; i < per && !dead; i += 32) {
      const Request r = request<S>(A, min(warp * per + i, A.B), &bad);
      sum += units_of(A, r);
      if (r.n > 0) longest = max(longest, r.tiles + EXTRA);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(ALL, sum, o);
    longest = __reduce_max_sync(ALL, longest);
    bad = __reduce_or_sync(ALL, bad);
    if (lane == 0) {
      C.sums[warp] = sum;
      C.longest[warp] = longest;
      if (bad && cta == 0) atomicOr(A.status, bad);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = C.tmem;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_for(A, C, bar, parity); };
  // the next item, from the ring of items; k counts them
  auto next_item = [&](int k, Item& it) {
    if (!wait(&C.item_full[k % ITEMS], (k / ITEMS) & 1)) return false;
    it = C.items[k % ITEMS];
    return it.b >= 0;
  };
  auto done_item = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&C.item_empty[k % ITEMS]);
  };

  if (warp == W_FIND) {
    uint32_t bad = 0;
    Request r = {};
    long long total = 0, upto = 0;
    int longest = 0;
    auto window = [&](int base) {                   // 32 requests and where their units end
      r = request<S>(A, dead ? A.B : min(base + lane, A.B), &bad);
      upto = units_of(A, r);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(ALL, upto, o);
        if (lane >= o) upto += y;
      }
    };
    if (few) {
      window(0);
      total = __shfl_sync(ALL, upto, 31);
      longest = __reduce_max_sync(ALL, r.n > 0 ? r.tiles + EXTRA : 0);
      bad = __reduce_or_sync(ALL, bad);
      if (bad && cta == 0 && lane == 0) atomicOr(A.status, bad);
    } else {
      for (int i = 0; i < THREADS / 32; ++i) {
        total += C.sums[i];
        longest = max(longest, C.longest[i]);
      }
    }
    auto quotient = [](long long x, long long y) {  // of numbers that mostly fit 32 bits
      return (x | y) >> 32 ? x / y : (long long)((uint32_t)x / (uint32_t)y);
    };
    const long long even = total > 0 ? quotient(total + ctas - 1, ctas) : 1;
    const long long share = longest <= SHORT && even < longest ? longest : even;
    long long u = share * cta;
    const long long end = min(total, u + share);
    int k = 0;
    if (u < end) {
      int base = 0;                                 // first request of the window, and its first unit
      long long at = 0;
      if (!few) {
        for (int i = 0; i < THREADS / 32 && at + C.sums[i] <= u; ++i) {
          at += C.sums[i];
          base += per;
        }
        window(base);
      }
      while (u < end) {
        const unsigned past = __ballot_sync(ALL, at + upto > u);
        if (!past) {                                // the next 32 requests
          at += __shfl_sync(ALL, upto, 31);
          base += 32;
          if (base >= A.B) break;
          window(base);
          continue;
        }
        const int l = __ffs(past) - 1;
        Request q;
        q.lo = __shfl_sync(ALL, r.lo, l);
        q.n = __shfl_sync(ALL, r.n, l);
        q.older = __shfl_sync(ALL, r.older, l);
        q.len = __shfl_sync(ALL, r.len, l);
        q.tiles = __shfl_sync(ALL, r.tiles, l);
        q.m_tiles = __shfl_sync(ALL, r.m_tiles, l);
        const long long before = __shfl_sync(ALL, upto, max(l - 1, 0)), start = at + (l ? before : 0);
        const int size = q.tiles + EXTRA;
        const long long index = quotient(u - start, size), first = start + index * size;   // the item, its first unit
        const int t0 = min((int)(u - first), q.tiles), t1 = (int)min((long long)q.tiles, end - first);
        if (q.tiles ? t0 < t1 : u == first) {
          if (!wait(&C.item_empty[k % ITEMS], ((k / ITEMS) & 1) ^ 1)) break;
          if (lane < CACHE_MAX_NEW / 128) C.odd[k % ITEMS][lane] = make_uint4(0, 0, 0, 0);
          __syncwarp();
          if (lane == 0) {
            Item it;
            it.b = base + l;
            it.lo = q.lo;
            it.n = q.n;
            it.older = q.older;
            it.len = q.len;
            it.g = (int)quotient(index, q.m_tiles);
            it.m0 = (int)(index - (long long)it.g * q.m_tiles) * M;
            it.rows = (int)min((long long)M, (long long)q.n * A.group - it.m0);
            it.t0 = t0;
            it.t1 = t1;
            it.c0 = t0 == 0 ? cta : (int)quotient(first, share);
            it.c1 = t1 == q.tiles ? cta : (int)quotient(first + q.tiles - 1, share);
            C.items[k % ITEMS] = it;
            mbar_arrive(&C.item_full[k % ITEMS]);
          }
          ++k;
          __syncwarp();
        }
        u = first + size;
      }
    }
    if (wait(&C.item_empty[k % ITEMS], ((k / ITEMS) & 1) ^ 1) && lane == 0) {
      C.items[k % ITEMS].b = -1;
      mbar_arrive(&C.item_full[k % ITEMS]);
    }
  } else if (warp == W_PRODUCE) {
    const uint64_t once = policy_evict_first(), again = policy_evict_normal();
    uint64_t policy = once;
    const int ps = 1 << A.page_log2;
    const int box = ps < S::TN ? ps : S::TN;        // tokens of a copy
    const uint32_t bytes = (uint32_t)box * S::D * (S::E4M3 ? 1 : 2);
    Place<S::NR> to;
    int at = 0, news = 0;                           // stages filled; those with values of new tokens, 16-bit
    bool ok = true, skip = A.skip_copy && cta == 0;
    Item it;
    for (int k = 0; ok && next_item(k, it); ++k) {
      done_item(k);
      policy = it.n * A.group <= M ? once : again;  // other rows of the request read the same tiles
      const int n = it.t1 - it.t0, held = (int)(((long long)it.len + ps - 1) >> A.page_log2);
      const int32_t* row = a.tables + (size_t)it.b * a.table_stride;
      auto entries = [&](int chunk) {               // 32 of the request's pages
        const int p = chunk * 32 + lane;
        if (p >= held) return -1;
        const int id = __ldcg(row + p);
        if (id >= 0 && id < A.n_pages) return id;
        atomicOr(A.status, CACHE_BAD_PAGE);
        return A.n_pages;                           // past the pool: copied as zeros
      };
      int chunk = ((int64_t)it.t0 * S::TN >> A.page_log2) >> 5;
      int ids = n ? entries(chunk) : 0, next = n ? entries(chunk + 1) : 0;
      auto ids_of = [&](int t) {
        const int p = (int)((int64_t)t * S::TN >> A.page_log2);
        if (p >> 5 != chunk) {
          chunk = p >> 5;
          ids = next;
          next = entries(chunk + 1);
        }
        return __shfl_sync(ALL, ids, (p & 31) + lane & 31);
      };
      auto copy = [&](const CUtensorMap* map, int t, int id, bool values) {
        const int st = to.at;
        // what is looked through first has barriers of its own: whoever looks waits for these alone, and would pass a
        // stage's barrier, by its parity, on an earlier use of the stage
        const bool fresh = !S::E4M3 && values && (int64_t)(t + 1) * S::TN > it.older;
        uint64_t* bar = fresh ? &C.new_full[news % 8] : &C.full[st];
        ok = ok && wait(&C.empty[st], to.parity ^ 1);
        if (!ok) return;
        const int64_t tok = (int64_t)t * S::TN;
        const int pages = min(S::TN / box, held - (int)(tok >> A.page_log2));
        if (lane == 0) {
          mbar_expect_tx(bar, bytes * pages);
          if (fresh) mbar_arrive(&C.full[st]);
        }
        __syncwarp();
        if (lane < pages && !skip) {
          const int off = it.g * ps + (int)(tok & (ps - 1));
          uint8_t* stage = ring + st * S::RAW + lane * bytes;
          if (S::E4M3) tma3(stage, map, off, id, bar, policy);
          else tma5(stage, map, off >> 3, id, bar, policy);
        }
        skip = false;
        ++at;
        to.next();
        news += fresh;
      };
      int kid = n ? ids_of(it.t0) : 0;
      if (n) copy(&km, it.t0, kid, false);
      for (int t = it.t0; t < it.t1 && ok; ++t) {
        const int vid = kid;
        if (t + 1 < it.t1) {
          kid = ids_of(t + 1);
          copy(&km, t + 1, kid, false);
        }
        copy(&vm, t, vid, true);
      }
    }
    // copies in flight land before the CTA ends
    if (!ok || *(volatile int*)&C.abort) {
      for (int i = max(0, at - S::NR); i < at; ++i) drain(&C.full[i % S::NR], (i / S::NR) & 1);
      for (int i = max(0, news - 8); i < news; ++i) drain(&C.new_full[i % 8], (i / 8) & 1);
    }
  } else if (warp == W_MMA) {
    Place<S::E4M3 ? S::NC1 : S::NR> from;           // in the order of the stages
    int tiles = 0, fixes = 0, items = 0;            // tiles, looked-through tiles, items with tiles so far
    bool ok = true;
    Item it;
    for (int k = 0; ok && next_item(k, it); ++k) {
      done_item(k);
      const int n = it.t1 - it.t0;
      if (n == 0) continue;
      ok = wait(&C.q_ready, items & 1);
      tc_fence_after();
      using At = Place<S::E4M3 ? S::NC1 : S::NR>;
      uint64_t *full = S::E4M3 ? c_full : C.full, *empty = S::E4M3 ? c_empty : C.empty;
      auto place = [&](const At& x) { return smem_u32(S::E4M3 ? conv + x.at * S::TILE : ring + x.at * S::RAW); };
      auto scores = [&](int j, const At& x0) {      // S = Q K^T of the item's tile j
        const uint64_t d = desc_sw128(place(x0), 0, S::GROUP);
        const int left = it.len - (it.t0 + j) * S::TN;
        const int cols = left < S::TN ? (left + 15) & ~15 : S::TN;
        const uint32_t id = idesc(S::MBF16, false, cols), s = tmem + S::S0 + (uint32_t)((tiles + j) & 1) * S::TN;
        if (elect_one()) {
#pragma unroll
          for (int x = 0; x < S::D / 16; ++x)
            umma_f16_ts(s, tmem + S::Q + x * 8, d + (x / 4) * 64 + (x % 4) * 2, id, x > 0);
          umma_commit(&C.s_full[(tiles + j) & 1]);
          umma_commit(&empty[x0.at]);
          if (j == n - 1) umma_commit(&C.q_free);
        }
        __syncwarp();
      };
      for (int j = 0; j < 2 && j < n && ok; ++j) {
        ok = wait(&full[from.at], from.parity);
        if (ok) scores(j, from);
        from.next();
      }
      for (int j = 0; j < n && ok; ++j) {
        const int g = tiles + j, left = it.len - (it.t0 + j) * S::TN;
        if (!S::E4M3 && (int64_t)(it.t0 + j + 1) * S::TN > it.older) {
          ok = wait(&C.fixed[fixes % 8], (fixes / 8) & 1);
          ++fixes;
        }
        // V of this tile, K of the one after the next; all three at once where they are ready
        const At v = from;
        from.next();
        const At x2 = from;
        const bool more = j + 2 < n;
        if (more) from.next();
        if (j == 0) ok = ok && wait(&C.o_free, (items & 1) ^ 1);
        if (!__all_sync(ALL, mbar_try_wait(&full[v.at], v.parity) && (!more || mbar_try_wait(&full[x2.at], x2.parity)) &&
                                 mbar_try_wait(&C.p_ready[g & 1], (g >> 1) & 1)))
          ok = ok && wait(&full[v.at], v.parity) && (!more || wait(&full[x2.at], x2.parity)) &&
               wait(&C.p_ready[g & 1], (g >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        const uint64_t d = desc_sw128(place(v), 1024, S::GROUP);
        const int steps = left < S::TN ? (left + 15) >> 4 : S::TN / 16;
        const uint32_t id = idesc(S::MBF16, true, S::D), p = tmem + S::S0 + (uint32_t)(g & 1) * S::TN;
        if (elect_one()) {
#pragma unroll
          for (int x = 0; x < S::TN / 16; ++x)
            if (x < steps) umma_f16_ts(tmem + S::O, p + x * 8, d + (uint64_t)(x * 2 * S::GROUP >> 4), id, j > 0 || x > 0);
          umma_commit(&empty[v.at]);
          umma_commit(&C.pv_done);
          if (j == n - 1) umma_commit(&C.o_full);
        }
        __syncwarp();
        if (more) scores(j + 2, x2);
      }
      tiles += n;
      ++items;
    }
    // what was issued ends before tensor memory is given back
    if (elect_one()) umma_commit(&C.drained);
    __syncwarp();
    drain(&C.drained, 0);
  } else if (warp >= W_PREP) {
    const int t = threadIdx.x - W_PREP * 32, wq = warp - W_PREP;   // a row's thread
    int at = 0, items = 0, news = 0;                // at: stages of the items before
    Place<S::NR> raw;                               // of an 8-bit cache: two warps take every other stage
    Place<S::NC1> cv;
    if (S::E4M3 && wq >> 1) {
      raw.next();
      cv.next();
    }
    bool ok = true;
    Item it;
    for (int k = 0; ok && next_item(k, it); ++k) {
      const int n = it.t1 - it.t0;
      if (n) {
        // the queries, turned where the scale is negative: the largest score is then the largest product
        const bool turn = A.scale * (S::E4M3 ? __ldcg(a.k_scale + it.g) : 1.f) < 0.f;
        const int m = it.m0 + t, i = m / A.group;
        const FourRows q(t < it.rows ? rows_at(a.q, it.lo + i, it.g * A.group + m - i * A.group) : nullptr, lane);
        constexpr int C0 = S::D / 2 < 64 ? S::D / 2 : 64;              // columns at a time
        // bf16 queries over an 8-bit cache, in fp16: times a power of two that brings the row's largest to 2^14 or above
        float by = 1.f;
        if (S::E4M3 && S::BF16) {
          uint32_t big = 0;
          // four lanes see parts of four rows; each row's maxima meet in its own lane
          uint32_t rows[4] = {};
#pragma unroll 2
          for (int x = 0; x < S::D; x += 32) {
            uint4 v[4];
            q.load(v, x);
#pragma unroll
            for (int z = 0; z < 4; ++z)
              rows[z] = __vmaxu2(rows[z], __vmaxu2(__vmaxu2(v[z].x & 0x7FFF7FFFu, v[z].y & 0x7FFF7FFFu),
                                                   __vmaxu2(v[z].z & 0x7FFF7FFFu, v[z].w & 0x7FFF7FFFu)));
          }
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            rows[z] = __vmaxu2(rows[z], __shfl_xor_sync(ALL, rows[z], 1));
            rows[z] = __vmaxu2(rows[z], __shfl_xor_sync(ALL, rows[z], 2));
            big = (lane & 3) == z ? rows[z] : big;
          }
          big = max(big & 0xFFFFu, big >> 16);
          // its exponent, 2^(e - 127): by 2^(141 - e), within fp32's normal range; infinities and NaN stay what they are
          const int e = (int)(big >> 7), f = e == 255 ? 127 : min(253, 268 - e);
          by = __uint_as_float((uint32_t)f << 23);
        }
#pragma unroll
        for (int c = 0; c < S::D / 2; c += C0) {
          uint4 v[C0 / 16][4];
#pragma unroll
          for (int x = 0; x < C0 / 16; ++x) q.load(v[x], 2 * c + 32 * x);
          if (c == 0) {
            ok = wait(&C.q_free, (items & 1) ^ 1);
            tc_fence_after();
            if (S::E4M3 && S::BF16) undo[(items & 1) * M + t] = __uint_as_float(0x7F000000u - __float_as_uint(by));
          }
#pragma unroll
          for (int x = 0; x < C0 / 16; ++x) {
            change_places(v[x], lane);
            uint32_t r[16];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              r[4 * z] = v[x][z].x;
              r[4 * z + 1] = v[x][z].y;
              r[4 * z + 2] = v[x][z].z;
              r[4 * z + 3] = v[x][z].w;
            }
#pragma unroll
            for (int z = 0; z < 16; ++z) {
              if (S::E4M3 && S::BF16) {
                const float2 f = unpack2<true>(r[z]);
                r[z] = pack2<false>(f.x * by, f.y * by);
              }
              if (turn) r[z] ^= 0x80008000u;
            }
            tmem_st16(tmem + ((uint32_t)(wq * 32) << 16) + S::Q + c + 16 * x, r);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&C.q_ready);
        ++items;
      }
      // a new token whose values are not finite
      auto note = [&](int j) { atomicOr(reinterpret_cast<uint32_t*>(C.odd[k % ITEMS]) + (j >> 5), 1u << (j & 31)); };
      if (S::E4M3) {
        // every tile, in the order of the stages; an item has an even number of them
        for (int x = wq >> 1; x < 2 * n && ok; x += 2, raw.next(2), cv.next(2)) {
          const bool key = x == 0 || (x % 2 == 1 && x < 2 * n - 1);
          const int j = x == 0 ? 0 : x == 2 * n - 1 ? n - 1 : key ? (x + 1) / 2 : x / 2 - 1;
          if (!__all_sync(ALL, mbar_try_wait(&C.full[raw.at], raw.parity) && mbar_try_wait(&c_empty[cv.at], cv.parity ^ 1)))
            ok = wait(&C.full[raw.at], raw.parity) && wait(&c_empty[cv.at], cv.parity ^ 1);
          if (!ok) break;
          // a thread's vectors lie 64 apart: the same 16 elements of rows a fixed number apart
          constexpr int VR = S::D / 16, ROWS = 64 / VR, STEPS = S::TN / ROWS;
          const int t = threadIdx.x & 63, tok = t / VR, c = t % VR;
          const uint8_t* from = ring + raw.at * S::RAW + t * 16;
          uint8_t* to = conv + cv.at * S::TILE + (c >> 2) * 1024;
          // lanes of neighbouring blocks store their halves in other orders: other banks
          const int turn = c >> 2 & 1;
          const int tok0 = (it.t0 + j) * S::TN, left = it.len - tok0, fresh = it.older - tok0;
          const bool look = !key && fresh < S::TN;
          // What is looked through is mended in the raw tile, a thread's own vectors before it converts them: within the
          // conversion the code of it cost every tile (128 requests over e4m3 caches 132 us, 165 so).
          if (look) {
            const int y1 = fresh > tok ? (fresh - tok + ROWS - 1) / ROWS : 0;
#pragma unroll 1
            for (int y = y1; y < STEPS; ++y) {
              const int at_tok = tok + y * ROWS;
              uint4* at_raw = reinterpret_cast<uint4*>(const_cast<uint8_t*>(from) + y * 1024);
              const uint4 w = *at_raw;
              const uint4 nan = make_uint4(__vcmpeq4(w.x & 0x7F7F7F7Fu, 0x7F7F7F7Fu), __vcmpeq4(w.y & 0x7F7F7F7Fu, 0x7F7F7F7Fu),
                                           __vcmpeq4(w.z & 0x7F7F7F7Fu, 0x7F7F7F7Fu), __vcmpeq4(w.w & 0x7F7F7F7Fu, 0x7F7F7F7Fu));
              if (at_tok >= left) {
                *at_raw = make_uint4(0, 0, 0, 0);
              } else if (nan.x | nan.y | nan.z | nan.w) {
                note(at_tok - fresh);
                *at_raw = make_uint4(w.x & ~nan.x, w.y & ~nan.y, w.z & ~nan.z, w.w & ~nan.w);
              }
            }
          }
#pragma unroll
          for (int y0 = 0; y0 < STEPS; y0 += 4) {
            uint4 v[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) v[y] = *reinterpret_cast<const uint4*>(from + (y0 + y) * 1024);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              uint4 lo, hi;
              e4m3x4_to_f16x4(v[y].x, lo.x, lo.y);
              e4m3x4_to_f16x4(v[y].y, lo.z, lo.w);
              e4m3x4_to_f16x4(v[y].z, hi.x, hi.y);
              e4m3x4_to_f16x4(v[y].w, hi.z, hi.w);
              const int at_tok = tok + (y0 + y) * ROWS, c0 = ((2 * (c & 3)) ^ (at_tok & 7)) ^ turn, c1 = c0 ^ 1;
              uint8_t* base = to + (at_tok >> 3) * S::GROUP + (at_tok & 7) * 128;
              *reinterpret_cast<uint4*>(base + c0 * 16) = turn ? hi : lo;
              *reinterpret_cast<uint4*>(base + c1 * 16) = turn ? lo : hi;
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&C.empty[raw.at]);
            mbar_arrive(&c_full[cv.at]);
          }
        }
      } else {
        // values of tiles with new tokens
        int j = it.older / S::TN - it.t0;
        for (j = j < 0 ? 0 : j; j < n && ok; ++j) {
          const int x = at + (j + 1 < n ? 2 * j + 2 : 2 * n - 1), st = x % S::NR;
          ok = wait(&C.new_full[news % 8], (news / 8) & 1);
          if (!ok) break;
          uint8_t* v = ring + st * S::RAW;
          const int tok0 = (it.t0 + j) * S::TN, left = it.len - tok0, fresh = max(0, it.older - tok0);
          const int rows = left < S::TN ? (left + 15) & ~15 : S::TN;
          constexpr int VR = S::D / 8;              // vectors of a row
          auto at_vector = [&](int e) {
            const int tok = e / VR, c = e % VR;
            return reinterpret_cast<uint4*>(v + (tok >> 3) * S::GROUP + (c >> 3) * 1024 + (tok & 7) * 128 +
                                            (((c & 7) ^ (tok & 7)) << 4));
          };
          // an exponent of ones overflows into the bit above it
          constexpr uint32_t EXP = S::BF16 ? 0x7F807F80u : 0x7C007C00u, ONE = S::BF16 ? 0x00800080u : 0x04000400u;
          uint32_t over = 0;
          const int e1 = min(left, S::TN) * VR;
#pragma unroll 8
          for (int e = fresh * VR + t; e < e1; e += 128) {
            const uint4 w = *at_vector(e);
            over |= ((w.x & EXP) + ONE) | ((w.y & EXP) + ONE) | ((w.z & EXP) + ONE) | ((w.w & EXP) + ONE);
          }
          if (over & 0x80008000u) {
            for (int e = fresh * VR + t; e < e1; e += 128) {
              const uint4 w = *at_vector(e);
              const uint4 f = make_uint4(finite2<S::BF16>(w.x), finite2<S::BF16>(w.y), finite2<S::BF16>(w.z),
                                         finite2<S::BF16>(w.w));
              if ((w.x ^ f.x) | (w.y ^ f.y) | (w.z ^ f.z) | (w.w ^ f.w)) {
                note(tok0 + e / VR - it.older);
                *at_vector(e) = f;
              }
            }
          }
          for (int e = max(fresh, left) * VR + t; e < rows * VR; e += 128) *at_vector(e) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&C.fixed[news % 8]);
          ++news;
        }
      }
      at += 2 * n;
      done_item(k);
    }
  } else if (warp >= W_SOFT) {
    // two threads to a row: the first four warps take the first half of a tile's tokens and of the output's elements
    constexpr int H = S::TN / 2, HD = S::D / 2;
    const int wq = warp & 3, half = (warp - W_SOFT) >> 2, t = wq * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(wq * 32) << 16);
    int tiles = 0, items = 0, syncs = 0;
    bool ok = true;
    auto all_arrive = [&] { return soft_barrier(A, C, syncs); };
    for (int k = 0; ok && wait(&C.item_full[k % ITEMS], (k / ITEMS) & 1); ++k) {
      const Item& it = C.items[k % ITEMS];          // in shared memory: registers are short
      if (it.b < 0) break;
      const int n = it.t1 - it.t0, m = it.m0 + t, i = m / A.group;
      const bool row = t < it.rows;
      if (a.gate.p && row) {
        const uint16_t* gate = rows_at(a.gate, it.lo + i, it.g * A.group + m - i * A.group) + half * HD;
#pragma unroll
        for (int x = 0; x < HD; x += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(gate + x));
      }
      Mask mask;
      mask.load(A, it.lo + i, i, it.len - it.older, row && n);
      float c = fabsf(A.scale * (S::E4M3 ? __ldcg(a.k_scale + it.g) : 1.f));
      float ref = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j, ++tiles) {
        ok = wait(&C.s_full[tiles & 1], (tiles >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        if (j == 0) {
          if (S::E4M3 && S::BF16) c *= undo[(items & 1) * M + t];
          c = c < 0x1p-149f ? 0x1p-149f : c;        // a score of -inf stays one when the scale is 0
        }
        const uint32_t s = lanes + S::S0 + (uint32_t)(tiles & 1) * S::TN;
        const int rel = (it.t0 + j) * S::TN - it.older;
        const bool edge = rel + S::TN > 0;
        uint32_t r[H / 32][32];
#pragma unroll
        for (int x = 0; x < H / 32; ++x) tmem_ld32(s + half * H + 32 * x, r[x]);
#pragma unroll
        for (int x = 0; x < H / 32; ++x) tmem_wait_ld32(r[x]);
        if (edge)
#pragma unroll
          for (int x = 0; x < H / 32; ++x) {
            const uint32_t w = mask.window(rel + half * H + 32 * x);
#pragma unroll
            for (int y = 0; y < 32; ++y)
              if (!(w >> y & 1)) r[x][y] = 0xFF800000u;
          }
        float top[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) top[y] = __uint_as_float(r[0][y]);
#pragma unroll
        for (int x = 0; x < H / 32; ++x)
#pragma unroll
          for (int y = 0; y < 32; ++y) top[y & 3] = fmaxf(top[y & 3], __uint_as_float(r[x][y]));
        top[0] = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        // the row's other half
        float* tops = C.top[tiles & 1][0];
        tops[half * M + t] = top[0];
        __syncwarp();
        if (lane == 0) mbar_arrive(&C.pair[wq][tiles & 1]);
        ok = wait(&C.pair[wq][tiles & 1], (tiles >> 1) & 1);
        if (!ok) break;
        const float high = fmaxf(top[0], tops[(half ^ 1) * M + t]) * c;
        // the base follows
        const bool up = high > ref + S::TAU;
        if (__any_sync(ALL, up)) {
          const float f = up ? exp2_fast(ref - high) : 1.f;
          if (up) ref = high;
          l *= f;
          if (j > 0) {                              // the product of the tile before; the one before that is done
            ok = wait(&C.pv_done, (tiles - 1) & 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int x = half * HD; x < half * HD + HD; x += 16) {
              uint32_t o[16];
              __syncwarp();
              tmem_ld16_nowait(lanes + S::O + x, o);
              tmem_wait_ld(o);
#pragma unroll
              for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
              tmem_st16(lanes + S::O + x, o);
            }
            tmem_wait_st();
          }
        }
        const float base = ref == -INFINITY ? 0.f : ref - S::LIFT;
        float sum0 = 0.f, sum1 = 0.f;
        __syncwarp();
#pragma unroll
        for (int x = 0; x < H / 32; ++x) {
          uint32_t p[16];
#pragma unroll
          for (int y = 0; y < 32; y += 2) {
            const float e0 = exp2_fast(fmaf(__uint_as_float(r[x][y]), c, -base));
            const float e1 = exp2_fast(fmaf(__uint_as_float(r[x][y + 1]), c, -base));
            sum0 += e0;
            sum1 += e1;
            p[y / 2] = pack2<S::MBF16>(e0, e1);
          }
          tmem_st16(s + half * (H / 2) + 16 * x, p);
        }
        l += sum0 + sum1;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&C.p_ready[tiles & 1]);
      }
      if (!ok) break;
      // the row's sum, and what the item's rows get
      float* sums = C.top[tiles & 1][0];            // read last two tiles ago
      sums[half * M + t] = l;
      ok = all_arrive();
      if (!ok) break;
      l = sums[t] + sums[M + t];
      ok = all_arrive();
      if (!ok) break;
      if (n) {
        ok = wait(&C.o_full, items++ & 1);
        if (!ok) break;
        tc_fence_after();
      }
      ok = finish_item<S>(A, C, k % ITEMS, lanes, ref, l, syncs);
      done_item(k);
    }
  }
  __syncthreads();
  if (warp == W_MMA) tmem_dealloc(tmem, 512);
}

// ---- launches ----
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
std::atomic<EncodeFn> g_encode{nullptr};

cudaError_t encode_fn(EncodeFn* out) {
  EncodeFn f = g_encode.load(std::memory_order_relaxed);
  if (!f) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || !p) return cudaErrorNotSupported;
    g_encode.store(f = reinterpret_cast<EncodeFn>(p), std::memory_order_relaxed);
  }
  *out = f;
  return cudaSuccess;
}

// a pool: 16-bit as blocks of 8 tokens x 64 elements, 8-bit as rows of a head's elements
template <class S>
cudaError_t pool_map(const CacheShape& c, const void* pool, int64_t page_stride, CUtensorMap* m) {
  EncodeFn fn;
  const cudaError_t e = encode_fn(&fn);
  if (e != cudaSuccess) return e;
  const int ps = 1 << c.page_log2, box_tokens = ps < S::TN ? ps : S::TN;
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  CUresult r;
  if (S::E4M3) {
    const cuuint64_t dims[3] = {(cuuint64_t)S::D, (cuuint64_t)c.Hkv * ps, (cuuint64_t)c.n_pages};
    const cuuint64_t strides[2] = {(cuuint64_t)S::D, (cuuint64_t)page_stride};
    const cuuint32_t box[3] = {(cuuint32_t)S::D, (cuuint32_t)box_tokens, 1};
    r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, (void*)pool, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
           CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  } else {
    const cuuint64_t dims[5] = {64, 8, (cuuint64_t)S::BLOCKS, (cuuint64_t)c.Hkv * ps / 8, (cuuint64_t)c.n_pages};
    const cuuint64_t strides[4] = {(cuuint64_t)S::D * 2, 128, (cuuint64_t)S::D * 16, (cuuint64_t)page_stride * 2};
    const cuuint32_t box[5] = {64, 8, (cuuint32_t)S::BLOCKS, (cuuint32_t)box_tokens / 8, 1};
    r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 5, (void*)pool, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  }
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <class S>
cudaError_t run(const CacheShape& c, const TreeArgs& A, int ctas, cudaStream_t st) {
  CUtensorMap km, vm;
  cudaError_t e = pool_map<S>(c, A.a.k_cache, A.a.k_page_stride, &km);
  if (e == cudaSuccess) e = pool_map<S>(c, A.a.v_cache, A.a.v_page_stride, &vm);
  // the kernel's shared-memory limit, once per device
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
  if (e == cudaSuccess && !(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(k_attend_tree<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::DYN);
    if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_relaxed);
  }
  if (e != cudaSuccess) return e;
  return launch_following(k_attend_tree<S>, ctas, THREADS, S::DYN, st, A, km, vm);
}
template <int D>
cudaError_t run_types(const CacheShape& c, const TreeArgs& A, int ctas, cudaStream_t st) {
  if (c.bf16) return c.e4m3 ? run<Shape<D, true, true>>(c, A, ctas, st) : run<Shape<D, true, false>>(c, A, ctas, st);
  return c.e4m3 ? run<Shape<D, false, true>>(c, A, ctas, st) : run<Shape<D, false, false>>(c, A, ctas, st);
}
static_assert(MAX_CTAS * 3 * 4 <= CACHE_TREE_COUNTS, "all counts");
int ctas_of(int num_sms) { return num_sms < MAX_CTAS ? num_sms : MAX_CTAS; }

}  // namespace

size_t cache_attend_tree_workspace(int num_sms, int head_dim) {
  return CACHE_TREE_COUNTS + (size_t)ctas_of(num_sms) * 2 * (size_t)(M * head_dim + 2 * M) * 4;
}

cudaError_t cache_attend_tree_launch(const CacheShape& S, const moe_cache_attend_tree_t& a, const CacheTreeState& w,
                                     cudaStream_t st) {
  TreeArgs A;
  A.a = a;
  A.B = (int)a.n_requests;
  A.rows = (int)a.n_rows;
  A.Hkv = S.Hkv;
  A.group = S.Hq / S.Hkv;
  A.page_log2 = S.page_log2;
  A.n_pages = S.n_pages;
  A.most = a.masks && 64 * (int)a.mask_words < w.max_new ? 64 * (int)a.mask_words : w.max_new;
  A.max_len = (long long)S.max_pages << S.page_log2;
  A.scale = (float)a.scale * LOG2E;
  const int ctas = ctas_of(w.num_sms);
  A.counts = (uint32_t*)w.workspace;
  A.parts = (float*)((uint8_t*)w.workspace + CACHE_TREE_COUNTS);
  A.status = w.status;
  A.timeout_ns = w.timeout_ns;
  A.skip_copy = w.skip_copy;
  return S.D == 64 ? run_types<64>(S, A, ctas, st) : S.D == 128 ? run_types<128>(S, A, ctas, st) : run_types<256>(S, A, ctas, st);
}

}  // namespace moe
