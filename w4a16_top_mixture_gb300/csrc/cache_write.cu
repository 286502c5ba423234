// The write into the paged cache (moe_cache_write): RMSNorm over each head of q and k, rotary embedding of the first
// R elements, and the append of k and v by slot.
#include "cache.cuh"

namespace moe {
namespace {

constexpr int WRITE_THREADS = 128, WRITE_AHEAD = 3, WRITE_CTAS = 6;   // CTAs to an SM
constexpr int WRITE_WARPS = 128;           // a row is cut into slices while there are fewer warps than these to an SM

struct WriteArgs {
  moe_cache_write_t w;
  int Hq, Hkv, rope, page_log2;
  int n_slots;
  const uint64_t* turns;     // [R / 2]: theta^(-2i/R) / (2 pi) in 2^-64 of a turn
  int slices, slice_steps;   // warps to a row, and the steps of each
  float gamma_offset, eps;
  uint32_t* status;
};

// Pairs of fp32, two to an instruction: the arithmetic of a row is most of what the kernel issues.
using pair = unsigned long long;
__device__ __forceinline__ pair make_pair2(float a, float b) {
  pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 split(pair p) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
  return f;
}
__device__ __forceinline__ pair mul2(pair a, pair b) {
  pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ pair fma2(pair a, pair b, pair c) {
  pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
template <bool BF16>
__device__ __forceinline__ void unpack4(uint2 v, pair x[2]) {
  const float2 f0 = unpack2<BF16>(v.x), f1 = unpack2<BF16>(v.y);
  x[0] = make_pair2(f0.x, f0.y);
  x[1] = make_pair2(f1.x, f1.y);
}
template <bool BF16>
__device__ __forceinline__ uint2 pack4(const pair x[2]) {
  const float2 f0 = split(x[0]), f1 = split(x[1]);
  return make_uint2(pack2<BF16>(f0.x, f0.y), pack2<BF16>(f1.x, f1.y));
}
// offset + gamma[e .. e + 3]
template <bool BF16>
__device__ __forceinline__ void weights(const void* gamma, int e, float offset, pair g[2]) {
  const uint2 r = gamma ? __ldcg(reinterpret_cast<const uint2*>((const uint16_t*)gamma + e)) : make_uint2(0, 0);
  const float2 f0 = unpack2<BF16>(r.x), f1 = unpack2<BF16>(r.y);
  g[0] = make_pair2(offset + f0.x, offset + f0.y);
  g[1] = make_pair2(offset + f1.x, offset + f1.y);
}
// A head's scale of e4m3 codes s, its reciprocal, and the power of two that it and what it divides are multiplied by
// first: beyond 2^-64 .. 2^64 the reciprocal, or the remainder below, could leave fp32's normal range.
struct CodeScale {
  float s, r, by;
  __device__ __forceinline__ explicit CodeScale(float scale) {
    by = fabsf(scale) < 0x1p-64f ? 0x1p100f : fabsf(scale) > 0x1p64f ? 0x1p-100f : 1.f;
    s = scale * by;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  }
  // x / s in three operations: Markstein's correction of a product with the reciprocal by its remainder. A reciprocal
  // good to one step does: the product is off by two, and the corrected one by 2^-21 of a step before its rounding.
  // Where the product is past what e4m3 holds the correction could only lose an infinity.
  __device__ __forceinline__ float quotient(float x) const {
    const float q = x * r;
    return fabsf(q) < 1e30f ? fmaf(fmaf(-q, s, x), r, q) : q;
  }
};
__device__ __forceinline__ uint32_t quantize4(pair x[2], const CodeScale& c) {
  if (c.by != 1.f) {
    const pair by = make_pair2(c.by, c.by);
    x[0] = mul2(x[0], by);
    x[1] = mul2(x[1], by);
  }
  const float2 f0 = split(x[0]), f1 = split(x[1]);
  const float2 a = make_float2(c.quotient(f0.x), c.quotient(f0.y));
  const float2 b = make_float2(c.quotient(f1.x), c.quotient(f1.y));
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

// A warp to a row, or to a slice of its heads where there are few rows. A head's D elements lie over D / 8 lanes, 8 to
// a lane, so a step of a warp is 256 / D heads of q, of k or of v. A lane among the first R / 8 holds elements 4l ..
// 4l+3 and their partners R/2 further on, so that the rotation needs no exchange; the others hold 8 in a row. Each lane
// makes its four cosines and sines once for all heads: the angle in turns is position times frequency modulo 1,
// exactly, as integers (fp32 loses its fraction), and its upper 32 bits are the argument. What bounds the kernel is the
// bytes, then the instructions and whole waves of warps: the loads of three steps are on their way while three others
// are worked on, nothing synchronises, and a row is cut in two where that fills the last wave. 8192 rows of 32 + 2 x 8
// heads of 128 (201 MB): 41 us, 4.9 TB/s; with four steps ahead and four CTAs to an SM 64 us, with whole rows 43 us;
// into an e4m3 cache (185 MB) 52 us. 80 registers are a cap that every variant spills at (20 to 40 bytes); the heads of
// a warp's step make the same sines, two or four times over.
template <int D, bool BF16, bool E4M3>
__global__ void __launch_bounds__(WRITE_THREADS, WRITE_CTAS) k_cache_write(const __grid_constant__ WriteArgs a) {
  constexpr int LANES = D / 8, PER_WARP = 32 / LANES;
  const moe_cache_write_t& w = a.w;
  const int lane = threadIdx.x & 31, l = lane % LANES, sub = lane / LANES;
  const int task = blockIdx.x * (WRITE_THREADS / 32) + (threadIdx.x >> 5);
  const int t = task / a.slices, slice = task - t * a.slices;
  follow_predecessor();
  if (t >= w.n_rows) return;
  const int half = a.rope / 2;
  const int q_steps = (a.Hq + PER_WARP - 1) / PER_WARP, kv_steps = (a.Hkv + PER_WARP - 1) / PER_WARP;
  const int first = slice * a.slice_steps, steps = q_steps + 2 * kv_steps;
  const int last = first + a.slice_steps < steps ? first + a.slice_steps : steps;
  const bool rot = 8 * l < a.rope;
  const int e0 = rot ? 4 * l : 8 * l, e1 = rot ? half + 4 * l : 8 * l + 4;
  // the lane's part of each kind's row, of the head it has in the kind's first step
  const uint16_t* const q0 = (const uint16_t*)w.q.p + t * w.q.row_stride + sub * w.q.head_stride + e0;
  const uint16_t* const k0 = (const uint16_t*)w.k.p + t * w.k.row_stride + sub * w.k.head_stride + e0;
  const uint16_t* const v0 = (const uint16_t*)w.v.p + t * w.v.row_stride + sub * w.v.head_stride + e0;
  const int64_t qs = PER_WARP * w.q.head_stride, ks = PER_WARP * w.k.head_stride, vs = PER_WARP * w.v.head_stride;
  auto load = [&](uint2 (&raw)[WRITE_AHEAD][2], int s0) {
#pragma unroll
    for (int i = 0; i < WRITE_AHEAD; ++i) {
      const int st = s0 + i;
      if (st >= last) break;
      const uint16_t* p;
      bool in;
      if (st < q_steps) {
        p = q0 + st * qs;
        in = st * PER_WARP + sub < a.Hq;
      } else if (st < q_steps + kv_steps) {
        p = k0 + (st - q_steps) * ks;
        in = (st - q_steps) * PER_WARP + sub < a.Hkv;
      } else {
        p = v0 + (st - q_steps - kv_steps) * vs;
        in = (st - q_steps - kv_steps) * PER_WARP + sub < a.Hkv;
      }
      if (in) {
        raw[i][0] = __ldcg(reinterpret_cast<const uint2*>(p));
        raw[i][1] = __ldcg(reinterpret_cast<const uint2*>(p + (e1 - e0)));
      }
    }
  };
  uint2 now[WRITE_AHEAD][2], then[WRITE_AHEAD][2];
  load(now, first);
  const int slot = __ldcg(w.slots + t), pos = __ldcg(w.positions + t);
  pair gq[2][2], gk[2][2];                 // the weights of q and of k
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    weights<BF16>(w.q_gamma, k ? e1 : e0, a.gamma_offset, gq[k]);
    weights<BF16>(w.k_gamma, k ? e1 : e0, a.gamma_offset, gk[k]);
  }
  const bool put = slot >= 0 && slot < a.n_slots;
  if (slot >= a.n_slots && lane == 0) atomicOr(a.status, CACHE_BAD_PAGE);
  // the lane's part of the token's row in its page; a head's rows are a page's tokens apart
  const long long in_page = (long long)(slot & ((1 << a.page_log2) - 1)) * D + ((long long)sub << a.page_log2) * D + e0;
  const long long k_at = (slot >> a.page_log2) * w.k_page_stride + in_page;
  const long long v_at = (slot >> a.page_log2) * w.v_page_stride + in_page;
  const int pool_step = PER_WARP * D << a.page_log2;
  uint16_t* const o0 = (uint16_t*)w.q_out.p + t * w.q_out.row_stride + sub * w.q_out.head_stride + e0;
  const int64_t os = PER_WARP * w.q_out.head_stride;
  pair c[2], s[2], ns[2];
  {
    float cf[4] = {1.f, 1.f, 1.f, 1.f}, sf[4] = {0.f, 0.f, 0.f, 0.f};
    if (rot && first < q_steps + kv_steps)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // 64-bit fractions of a turn: the product's overflow is whole turns
        const uint64_t turns = (uint64_t)(int64_t)pos * a.turns[4 * l + j];
        sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &sf[j], &cf[j]);
      }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      c[j] = make_pair2(cf[2 * j], cf[2 * j + 1]);
      s[j] = make_pair2(sf[2 * j], sf[2 * j + 1]);
      ns[j] = make_pair2(-sf[2 * j], -sf[2 * j + 1]);
    }
  }
  // RMSNorm and rotation of a head's part
  auto turned = [&](const uint2 (&raw)[2], bool norm, const pair (&g)[2][2], pair (&x)[2][2]) {
    unpack4<BF16>(raw[0], x[0]);
    unpack4<BF16>(raw[1], x[1]);
    if (norm) {
      const pair upper = fma2(x[1][0], x[1][0], mul2(x[1][1], x[1][1]));
      const float2 sum = split(fma2(x[0][0], x[0][0], fma2(x[0][1], x[0][1], upper)));
      float ss = sum.x + sum.y;
      // a head's lanes lie in one warp
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
      const float r = rsqrtf(ss * (1.f / D) + a.eps);
      const pair r2 = make_pair2(r, r);
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < 2; ++j) x[k][j] = mul2(x[k][j], mul2(r2, g[k][j]));
    }
    if (rot)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const pair lo = x[0][j], hi = x[1][j];
        x[0][j] = fma2(hi, ns[j], mul2(lo, c[j]));
        x[1][j] = fma2(lo, s[j], mul2(hi, c[j]));
      }
  };
  auto work = [&](const uint2 (&raw)[WRITE_AHEAD][2], int s0) {
#pragma unroll
    for (int i = 0; i < WRITE_AHEAD; ++i) {
      const int st = s0 + i;
      if (st >= last) break;
      pair x[2][2];
      if (st < q_steps) {
        turned(raw[i], w.q_gamma != nullptr, gq, x);
        if (st * PER_WARP + sub < a.Hq) {
          uint16_t* const p = o0 + st * os;
          *reinterpret_cast<uint2*>(p) = pack4<BF16>(x[0]);
          *reinterpret_cast<uint2*>(p + (e1 - e0)) = pack4<BF16>(x[1]);
        }
        continue;
      }
      const bool is_k = st < q_steps + kv_steps;
      const int n = st - q_steps - (is_k ? 0 : kv_steps), h = n * PER_WARP + sub;
      const bool in = put && h < a.Hkv;
      const long long at = (is_k ? k_at : v_at) + (long long)n * pool_step;
      void* const pool = is_k ? w.k_cache : w.v_cache;
      uint2 out[2] = {raw[i][0], raw[i][1]};                   // a value for a cache of its own type: as it is
      if (is_k) {
        turned(raw[i], w.k_gamma != nullptr, gk, x);
        out[0] = pack4<BF16>(x[0]);
        out[1] = pack4<BF16>(x[1]);
      } else if (E4M3) {
        unpack4<BF16>(raw[i][0], x[0]);
        unpack4<BF16>(raw[i][1], x[1]);
      }
      if (!in) continue;
      if (E4M3) {
        const CodeScale sc(__ldcg((is_k ? w.k_scale : w.v_scale) + h));
        *reinterpret_cast<uint32_t*>((uint8_t*)pool + at) = quantize4(x[0], sc);
        *reinterpret_cast<uint32_t*>((uint8_t*)pool + at + (e1 - e0)) = quantize4(x[1], sc);
      } else {
        *reinterpret_cast<uint2*>((uint16_t*)pool + at) = out[0];
        *reinterpret_cast<uint2*>((uint16_t*)pool + at + (e1 - e0)) = out[1];
      }
    }
  };
  for (int st = first; st < last; st += 2 * WRITE_AHEAD) {
    if (st + WRITE_AHEAD < last) load(then, st + WRITE_AHEAD);
    work(now, st);
    if (st + 2 * WRITE_AHEAD < last) load(now, st + 2 * WRITE_AHEAD);
    if (st + WRITE_AHEAD < last) work(then, st + WRITE_AHEAD);
  }
}

template <int D>
cudaError_t launch(const WriteArgs& a, bool bf16, bool e4m3, cudaStream_t st) {
  auto* kernel = bf16 ? (e4m3 ? k_cache_write<D, true, true> : k_cache_write<D, true, false>)
                      : (e4m3 ? k_cache_write<D, false, true> : k_cache_write<D, false, false>);
  return launch_following(kernel, (unsigned)((a.w.n_rows * a.slices + WRITE_THREADS / 32 - 1) / (WRITE_THREADS / 32)),
                          WRITE_THREADS, 0, st, a);
}

}  // namespace

cudaError_t cache_write_launch(const CacheShape& S, const moe_cache_write_t& w, const uint64_t* turns,
                               uint32_t* status, int num_sms, cudaStream_t st) {
  WriteArgs a;
  a.w = w;
  a.Hq = w.q.p ? S.Hq : 0;
  a.Hkv = S.Hkv;
  a.rope = S.rope;
  a.page_log2 = S.page_log2;
  a.n_slots = S.n_pages << S.page_log2;
  a.turns = turns;
  // a warp takes WRITE_AHEAD steps at least
  const int per = 256 / S.D, steps = (a.Hq + per - 1) / per + 2 * ((a.Hkv + per - 1) / per);
  const int most = (steps + WRITE_AHEAD - 1) / WRITE_AHEAD;
  const int64_t want = (int64_t)num_sms * WRITE_WARPS / w.n_rows;
  a.slices = want < 1 ? 1 : want < most ? (int)want : most;
  a.slice_steps = (steps + a.slices - 1) / a.slices;
  a.gamma_offset = S.gamma_offset;
  a.eps = S.eps;
  a.status = status;
  if (S.D == 64) return launch<64>(a, S.bf16, S.e4m3, st);
  if (S.D == 128) return launch<128>(a, S.bf16, S.e4m3, st);
  return launch<256>(a, S.bf16, S.e4m3, st);
}

}  // namespace moe
