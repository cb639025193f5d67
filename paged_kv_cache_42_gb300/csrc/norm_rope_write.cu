// Per-head norm, position rotation and KV-cache write in one pass.
//
// The step before attention in a decoder layer: every query and key head is
// (optionally) normalised,
//   y_m = x_m * w_m / sqrt((1 / D) sum_n x_n^2 + eps),
// its first R = rotary_dim elements are turned by the token's position, pair
// (a, b) by the angle whose cosine and sine the table holds for pair i,
//   a' = a cos_i - b sin_i,   b' = b cos_i + a sin_i,
// with pairs (y_i, y_{i + R/2}), or (y_{2i}, y_{2i+1}) when interleaved; then
// the query goes to q_out and K and V to the token's cache slot, the scatter
// pa_write_kv does ("vLLM v1 Deep Dive: How LLM(...) and the Server Boot and
// Generate", Part 3, "Aside - KV cache and prefix caching"). Everything
// between the load and the store is binary32 and each result is rounded once
// (for an E4M3 cache straight from binary32: E4M3(y / scale), or with a
// row-scaled one E4M3(y 2^-e), rows.cuh, from the row's largest |y|).
//
// What bounds it: bytes, each element once in and once out, with arithmetic
// close behind; for a few tokens the launch and two dependent loads (position,
// then table row).
//
// Layout of the work. A lane holds 4 pairs of one head: elements 4i .. 4i + 3
// and their partners R / 2 further on (two 8-byte loads), or 8 consecutive
// elements when interleaved (one 16-byte load). A rotation is then arithmetic
// within the lane, on 4 cosines and 4 sines; elements past R go four and four
// the same way and are left alone. A head is D / 8 lanes, a warp 2 (D = 128) or 4
// (D = 64) heads, a norm's sum 4 or 3 shuffles. A warp takes ITER such groups
// of heads of ONE token and ONE kind (queries, K or V): their loads are all in
// flight together, before anything depends on the position; the token's
// cosines and sines and the kind's weight are loaded once for all of them, and
// V skips the arithmetic. 2048 tokens of 32 + 8 + 8 heads of 128 take 10.8 us,
// 4.8 TB/s (E4M3 12.9, row-scaled 12.3); 2, 6 or 8 groups a warp 12.3, 12.0 and 12.8 us (13.4, 14.3,
// 15.6). Units that mix the kinds were 9% slower: the choice is made per head.
#include <type_traits>

#include "pa_internal.h"
#include "ptx.cuh"
#include "rows.cuh"

namespace pa {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kThreads = 128;
constexpr int kManyIter = 4;  // head groups per warp when there are many tokens

// A lane's 8 values as 4 pairs {a, b}: x[0], x[1] the a's of pairs 0 1 and
// 2 3, x[2], x[3] the b's.
struct Pairs {
  float2 x[4];
};

// a's and b's in separate words (half split) or side by side (interleaved)
template <bool INTER>
__device__ __forceinline__ Pairs unpack(uint4 r) {
  Pairs v;
  if constexpr (INTER) {
    const float2 p0 = bf16x2_to_float2(r.x), p1 = bf16x2_to_float2(r.y);
    const float2 p2 = bf16x2_to_float2(r.z), p3 = bf16x2_to_float2(r.w);
    v.x[0] = make_float2(p0.x, p1.x);
    v.x[1] = make_float2(p2.x, p3.x);
    v.x[2] = make_float2(p0.y, p1.y);
    v.x[3] = make_float2(p2.y, p3.y);
  } else {
    v.x[0] = bf16x2_to_float2(r.x);
    v.x[1] = bf16x2_to_float2(r.y);
    v.x[2] = bf16x2_to_float2(r.z);
    v.x[3] = bf16x2_to_float2(r.w);
  }
  return v;
}

template <bool INTER>
__device__ __forceinline__ uint4 pack(const Pairs& v) {
  if constexpr (INTER)
    return make_uint4(
        float2_to_bf16x2(v.x[0].x, v.x[2].x), float2_to_bf16x2(v.x[0].y, v.x[2].y),
        float2_to_bf16x2(v.x[1].x, v.x[3].x), float2_to_bf16x2(v.x[1].y, v.x[3].y));
  return make_uint4(float2_to_bf16x2(v.x[0].x, v.x[0].y), float2_to_bf16x2(v.x[1].x, v.x[1].y),
                    float2_to_bf16x2(v.x[2].x, v.x[2].y), float2_to_bf16x2(v.x[3].x, v.x[3].y));
}

// The values over `scale` as E4M3 codes (correctly rounded quotient, then
// round-to-nearest-even with saturation, as pa_write_kv_fp8), in memory order.
template <bool INTER>
__device__ __forceinline__ uint2 pack_e4m3(const Pairs& v, float scale) {
  auto two = [&](float a, float b) -> uint32_t {
    return float2_to_e4m3x2(__fdiv_rn(a, scale), __fdiv_rn(b, scale));
  };
  if constexpr (INTER)
    return make_uint2(two(v.x[0].x, v.x[2].x) | two(v.x[0].y, v.x[2].y) << 16,
                      two(v.x[1].x, v.x[3].x) | two(v.x[1].y, v.x[3].y) << 16);
  return make_uint2(two(v.x[0].x, v.x[0].y) | two(v.x[1].x, v.x[1].y) << 16,
                    two(v.x[2].x, v.x[2].y) | two(v.x[3].x, v.x[3].y) << 16);
}

// The same for a row of a row-scaled cache; *b: its scale's byte.
template <bool INTER, int LPH>
__device__ __forceinline__ uint2 pack_row(const Pairs& v, int lane, int* b) {
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) top = row_top(row_top(top, v.x[e].x), v.x[e].y);
  *b = row_scale_byte(row_top_all<LPH>(top, lane));
  const float inv = row_inverse(*b);
  if constexpr (INTER)
    return make_uint2(
        row_codes(v.x[0].x, v.x[2].x, inv) | row_codes(v.x[0].y, v.x[2].y, inv) << 16,
        row_codes(v.x[1].x, v.x[3].x, inv) | row_codes(v.x[1].y, v.x[3].y, inv) << 16);
  return make_uint2(
      row_codes(v.x[0].x, v.x[0].y, inv) | row_codes(v.x[1].x, v.x[1].y, inv) << 16,
      row_codes(v.x[2].x, v.x[2].y, inv) | row_codes(v.x[3].x, v.x[3].y, inv) << 16);
}

// At least nine CTAs on an SM into a bf16 cache (56 registers): with 64 registers
// and eight of them 2048 tokens took 9% longer. The E4M3 forms do not fit 56.
// KV: what the caches hold, 0 bf16, 1 E4M3 with one scale per tensor, 2 row-scaled.
template <int D, int KV, bool INTER, int ITER>
__global__ void __launch_bounds__(kThreads, KV ? 8 : 9) pa_norm_rope_write_kernel(const NormRopeParams p) {
  constexpr bool F8 = KV != 0;
  constexpr int LPH = D / 8;     // lanes per head
  constexpr int HPG = 32 / LPH;  // heads per group
  const int lane = threadIdx.x & 31;
  const int sub = lane % LPH, hsub = lane / LPH;
  const int nq = p.num_q_heads, nk = p.num_kv_heads;
  // units of a token, each HPG x ITER heads of one kind: queries, then K, then V
  const unsigned uq = (unsigned)(nq + HPG * ITER - 1) / (HPG * ITER);
  const unsigned uk = (unsigned)(nk + HPG * ITER - 1) / (HPG * ITER);
  const unsigned chunks = uq + 2 * uk;
  const unsigned wid = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int t = (int)(wid / chunks);
  if (t >= p.num_tokens) return;
  const unsigned unit = wid - (unsigned)t * chunks;
  const int kind = unit < uq ? 0 : unit < uq + uk ? 1 : 2;
  const int rows = kind == 0 ? nq : nk;
  const unsigned first = kind == 0 ? 0u : kind == 1 ? uq : uq + uk;
  const int row0 = (int)(unit - first) * (HPG * ITER) + hsub;
  const uint16_t* const src = kind == 0   ? p.q + t * p.q_stride
                              : kind == 1 ? p.k + t * p.k_stride
                                          : p.v + t * p.v_stride;

  // first elements of this lane's two halves within a head
  const int half = p.rotary_dim >> 1;
  const bool turned = sub * 4 < half;  // interleaved: elements 8 sub .. 8 sub + 7 < 2 half alike
  int ea, eb;
  if constexpr (INTER) {
    ea = sub * 8;
    eb = ea + 4;
  } else {
    ea = turned ? sub * 4 : half + sub * 4;
    eb = turned ? ea + half : ea + (D - p.rotary_dim) / 2;
  }
  griddep_wait();  // a programmatic dependent of the grid before, which made q, k and v
  // every load that needs no position first
  const long long slot = __ldg(p.slot_mapping + t);
  const int pos = p.rotary_dim > 0 ? __ldg(p.positions + t) : 0;
  auto load8 = [&](const uint16_t* src) -> uint4 {
    if constexpr (INTER) return *reinterpret_cast<const uint4*>(src + ea);
    const uint2 a = *reinterpret_cast<const uint2*>(src + ea);
    const uint2 b = *reinterpret_cast<const uint2*>(src + eb);
    return make_uint4(a.x, a.y, b.x, b.y);
  };
  uint4 raw[ITER];
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int row = row0 + i * HPG;
    raw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (row < rows) raw[i] = load8(src + row * D);  // q_out may be q: no read-only path
  }
  const uint16_t* const w = kind == 0 ? p.q_weight : kind == 1 ? p.k_weight : nullptr;
  uint4 rw = make_uint4(0u, 0u, 0u, 0u);
  if (w != nullptr) rw = load8(w);
  if (slot < 0) return;  // a padding token: nothing of it is written
  if (slot >= p.num_slots) {
    if (lane == 0) report_error(p.err, PA_DEVERR_SLOT, t);
    return;
  }
  if (pos < 0 || pos >= p.max_position) {
    if (lane == 0) report_error(p.err, PA_DEVERR_POSITION, t);
    return;
  }
  // where a head's row goes
  const long long dst0 = kind == 0 ? (long long)t * nq * D
                                   : ((slot >> 4) * nk * kBlockSize + (slot & 15)) * D;
  const int step = kind == 0 ? D : kBlockSize * D;
  auto store = [&](void* base, int row, uint4 o) {
    uint16_t* const at = static_cast<uint16_t*>(base) + dst0 + row * step;
    if constexpr (INTER) {
      *reinterpret_cast<uint4*>(at + ea) = o;
    } else {
      *reinterpret_cast<uint2*>(at + ea) = make_uint2(o.x, o.y);
      *reinterpret_cast<uint2*>(at + eb) = make_uint2(o.z, o.w);
    }
  };
  auto store8 = [&](void* base, int row, uint2 o) {
    unsigned char* const at = static_cast<unsigned char*>(base) + dst0 + row * step;
    if constexpr (INTER) {
      *reinterpret_cast<uint2*>(at + ea) = o;
    } else {
      *reinterpret_cast<uint32_t*>(at + ea) = o.x;
      *reinterpret_cast<uint32_t*>(at + eb) = o.y;
    }
  };
  // a row-scaled cache's row: its codes, and one lane its scale
  auto store_row = [&](void* base, int row, const Pairs& v, int which) {
    int b;
    store8(base, row, pack_row<INTER, LPH>(v, lane, &b));
    if (sub == 0)
      p.scales[((slot >> 4) * nk + row) * kScaleBytes + which * kBlockSize + (slot & 15)] =
          (unsigned char)b;
  };
  if (kind == 2) {
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int row = row0 + i * HPG;
      if (row >= rows) break;
      if constexpr (KV == 2)
        store_row(p.v_cache, row, unpack<INTER>(raw[i]), 1);
      else if constexpr (F8)
        store8(p.v_cache, row, pack_e4m3<INTER>(unpack<INTER>(raw[i]), p.v_scale));
      else
        store(p.v_cache, row, raw[i]);
    }
    return;
  }
  float2 c[2] = {}, s[2] = {};  // of this lane's pairs
  if (turned) {
    const float* const cs = p.cos_sin + (long long)pos * p.rotary_dim + sub * 4;
    const float4 cv = __ldg(reinterpret_cast<const float4*>(cs));
    const float4 sv = __ldg(reinterpret_cast<const float4*>(cs + half));
    c[0] = make_float2(cv.x, cv.y);
    c[1] = make_float2(cv.z, cv.w);
    s[0] = make_float2(sv.x, sv.y);
    s[1] = make_float2(sv.z, sv.w);
  }
  auto heads = [&](auto normed) {
    constexpr bool NORM = decltype(normed)::value;
    const Pairs wv = unpack<INTER>(rw);
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int row = row0 + i * HPG;
      Pairs v = unpack<INTER>(raw[i]);
      if constexpr (NORM) {
        // the head's sum of squares (every lane of the warp takes the shuffles)
        float2 sq = fmul2(v.x[0], v.x[0]);
#pragma unroll
        for (int e = 1; e < 4; ++e) sq = ffma2(v.x[e], v.x[e], sq);
        float ss = sq.x + sq.y;
#pragma unroll
        for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor_sync(kAll, ss, o);
        const float r = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
        for (int e = 0; e < 4; ++e) v.x[e] = fmul2(fmul2(v.x[e], make_float2(r, r)), wv.x[e]);
      }
      if (row >= rows) continue;
      if (turned) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 a = v.x[e], b = v.x[2 + e];
          const float2 ns = make_float2(-s[e].x, -s[e].y);
          v.x[e] = ffma2(b, ns, fmul2(a, c[e]));
          v.x[2 + e] = ffma2(a, s[e], fmul2(b, c[e]));
        }
      }
      if (KV == 2 && kind == 1) {
        store_row(p.k_cache, row, v, 0);
      } else if (F8 && kind == 1) {
        store8(p.k_cache, row, pack_e4m3<INTER>(v, p.k_scale));
      } else {
        // neither normalised nor turned: the bits as they came, a NaN's too
        store(kind == 0 ? p.q_out : p.k_cache, row, NORM || turned ? pack<INTER>(v) : raw[i]);
      }
    }
  };
  if (w != nullptr)
    heads(std::true_type{});
  else
    heads(std::false_type{});
}

template <int D, int KV, bool INTER>
cudaError_t launch_nr(const NormRopeParams& p, int num_sms, cudaStream_t s) {
  constexpr int HPG = 32 / (D / 8);
  auto blocks = [&](int iter) {
    const int per = HPG * iter;
    const long long chunks = (p.num_q_heads + per - 1) / per + 2LL * ((p.num_kv_heads + per - 1) / per);
    return (p.num_tokens * chunks + kThreads / 32 - 1) / (kThreads / 32);
  };
  // Few tokens: one group of heads per warp, the shortest chain. Once that
  // would be more than eight CTAs (32 warps) per SM, kManyIter groups per warp.
  const bool small = blocks(1) <= 8LL * num_sms;
  const long long grid = small ? blocks(1) : blocks(kManyIter);
  if (grid > 0x3fffffffLL) return cudaErrorInvalidValue;  // warps are counted in 32 bits
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return small ? cudaLaunchKernelEx(&cfg, pa_norm_rope_write_kernel<D, KV, INTER, 1>, p)
               : cudaLaunchKernelEx(&cfg, pa_norm_rope_write_kernel<D, KV, INTER, kManyIter>, p);
}

template <int D>
cudaError_t launch_nr_d(const NormRopeParams& p, int num_sms, cudaStream_t s) {
  switch (p.kv_fp8) {
    case 2:
      return p.interleaved ? launch_nr<D, 2, true>(p, num_sms, s)
                           : launch_nr<D, 2, false>(p, num_sms, s);
    case 1:
      return p.interleaved ? launch_nr<D, 1, true>(p, num_sms, s)
                           : launch_nr<D, 1, false>(p, num_sms, s);
  }
  return p.interleaved ? launch_nr<D, 0, true>(p, num_sms, s)
                       : launch_nr<D, 0, false>(p, num_sms, s);
}

}  // namespace

cudaError_t launch_norm_rope_write(const NormRopeParams& p, int head_dim, int num_sms,
                                   cudaStream_t s) {
  return head_dim == 128 ? launch_nr_d<128>(p, num_sms, s) : launch_nr_d<64>(p, num_sms, s);
}

}  // namespace pa
