// The write into the paged cache (moe_cache_write): RMSNorm over each head of q and k, rotary embedding of the first
// R elements, and the append of k and v by slot.
#include "cache.cuh"

namespace moe {
namespace {

struct WriteArgs {
  moe_cache_write_t w;
  int Hq, Hkv, rope, page_log2;
  int n_slots;
  const double* turns;       // [R / 2]: theta^(-2i/R) / (2 pi)
  float gamma_offset, eps;
  uint32_t* status;
};

// One CTA per row. A head's D elements lie over D / 8 lanes, 8 to a lane (one 16-byte access), so a warp holds
// 256 / D heads. The row's cosines and sines are made once, in shared memory: the angle in turns in fp64 (positions
// times frequency loses its fraction in fp32), its fractional part in fp32.
template <int D, bool BF16, bool E4M3>
__global__ void __launch_bounds__(256) k_cache_write(const __grid_constant__ WriteArgs a) {
  constexpr int LANES = D / 8, PER_WARP = 32 / LANES;
  __shared__ float2 s_cs[D / 2];
  const moe_cache_write_t& w = a.w;
  const long long t = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int half = a.rope / 2;
  follow_predecessor();
  for (int i = threadIdx.x; i < half; i += 256) {
    const double turns = (double)__ldcg(w.positions + t) * a.turns[i];
    float c, s;
    sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
    s_cs[i] = make_float2(c, s);
  }
  const int slot = __ldcg(w.slots + t);
  const bool put = slot >= 0 && slot < a.n_slots;
  if (slot >= a.n_slots && threadIdx.x == 0) atomicOr(a.status, CACHE_BAD_PAGE);
  const int page = slot >> a.page_log2, off = slot & ((1 << a.page_log2) - 1);
  __syncthreads();
  const int heads = a.Hq + 2 * a.Hkv;          // q, k and v heads one after another
  const int l = lane % LANES, sub = lane / LANES;
  for (int h0 = warp * PER_WARP; h0 < heads; h0 += 8 * PER_WARP) {
    const int hh = h0 + sub;
    const bool in = hh < heads;
    const int kind = hh < a.Hq ? 0 : hh < a.Hq + a.Hkv ? 1 : 2;
    const int h = kind == 0 ? hh : kind == 1 ? hh - a.Hq : hh - a.Hq - a.Hkv;
    const moe_rows_t& src = kind == 0 ? w.q : kind == 1 ? w.k : w.v;
    const bool live = in && src.p != nullptr;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (live)
      raw = __ldcg(reinterpret_cast<const uint4*>((const uint16_t*)src.p + t * src.row_stride + h * src.head_stride + 8 * l));
    float x[8];
    {
      const uint32_t r[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<BF16>(r[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    }
    const void* gamma = kind == 0 ? w.q_gamma : kind == 1 ? w.k_gamma : nullptr;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    if (gamma) {
      const float r = 1.f / sqrtf(ss * (1.f / D) + a.eps);
      const uint4 gr = __ldcg(reinterpret_cast<const uint4*>((const uint16_t*)gamma + 8 * l));
      const uint32_t g[4] = {gr.x, gr.y, gr.z, gr.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<BF16>(g[i]);
        x[2 * i] *= r * (a.gamma_offset + f.x);
        x[2 * i + 1] *= r * (a.gamma_offset + f.y);
      }
    }
    // the partner of element i < R/2 is i + R/2: R/16 lanes further on
    const int step = a.rope / 16, e = 8 * l;
    const bool rot = kind < 2 && e < a.rope, low = e < half;
    const int from = (lane - l) + (rot ? (low ? l + step : l - step) : l);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = __shfl_sync(0xFFFFFFFFu, x[i], from);
      if (rot) {
        const float2 cs = s_cs[(low ? e : e - half) + i];
        x[i] = low ? x[i] * cs.x - y * cs.y : x[i] * cs.x + y * cs.y;
      }
    }
    if (!live) continue;
    if (kind == 0) {
      *reinterpret_cast<uint4*>((uint16_t*)w.q_out.p + t * w.q_out.row_stride + h * w.q_out.head_stride + e) =
          make_uint4(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]), pack2<BF16>(x[4], x[5]), pack2<BF16>(x[6], x[7]));
    } else if (put) {
      const long long at = (long long)page * (kind == 1 ? w.k_page_stride : w.v_page_stride) +
                           ((long long)h << a.page_log2) * D + (long long)off * D + e;
      void* pool = kind == 1 ? w.k_cache : w.v_cache;
      if (E4M3) {
        const float s = __ldcg((kind == 1 ? w.k_scale : w.v_scale) + h);
        uint32_t c[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float* y = x + 4 * i;
          const uint32_t c0 = __nv_cvt_float2_to_fp8x2(make_float2(y[0] / s, y[1] / s), __NV_SATFINITE, __NV_E4M3);
          const uint32_t c1 = __nv_cvt_float2_to_fp8x2(make_float2(y[2] / s, y[3] / s), __NV_SATFINITE, __NV_E4M3);
          c[i] = c0 | c1 << 16;
        }
        *reinterpret_cast<uint2*>((uint8_t*)pool + at) = make_uint2(c[0], c[1]);
      } else {
        *reinterpret_cast<uint4*>((uint16_t*)pool + at) =
            make_uint4(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]), pack2<BF16>(x[4], x[5]), pack2<BF16>(x[6], x[7]));
      }
    }
  }
}

template <int D>
cudaError_t launch(const WriteArgs& a, bool bf16, bool e4m3, cudaStream_t st) {
  auto* kernel = bf16 ? (e4m3 ? k_cache_write<D, true, true> : k_cache_write<D, true, false>)
                      : (e4m3 ? k_cache_write<D, false, true> : k_cache_write<D, false, false>);
  return launch_following(kernel, (unsigned)a.w.n_rows, 256, 0, st, a);
}

}  // namespace

cudaError_t cache_write_launch(const CacheShape& S, const moe_cache_write_t& w, const double* turns,
                               uint32_t* status, cudaStream_t st) {
  WriteArgs a;
  a.w = w;
  a.Hq = w.q.p ? S.Hq : 0;
  a.Hkv = S.Hkv;
  a.rope = S.rope;
  a.page_log2 = S.page_log2;
  a.n_slots = S.n_pages << S.page_log2;
  a.turns = turns;
  a.gamma_offset = S.gamma_offset;
  a.eps = S.eps;
  a.status = status;
  if (S.D == 64) return launch<64>(a, S.bf16, S.e4m3, st);
  if (S.D == 128) return launch<128>(a, S.bf16, S.e4m3, st);
  return launch<256>(a, S.bf16, S.e4m3, st);
}

}  // namespace moe
