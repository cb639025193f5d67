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
// (for an E4M3 cache straight from binary32: E4M3(y / scale)).
//
// What bounds it: bytes, each element once in and once out; for a few tokens
// the launch and two dependent loads (position, then table row).
//
// Layout of the work. A lane holds 8 consecutive elements (one 16-byte load),
// a head is D / 8 lanes, so a warp holds 2 (D = 128) or 4 (D = 64) heads and a
// norm's sum is 3 or 4 shuffles. The partner of a rotation pair is in the same
// lane (interleaved) or R / 16 lanes away (one shuffle per element). A warp
// takes kIter such groups of heads of ONE token: their loads are all in flight
// together, before anything depends on the position, and the token's cosines
// and sines are loaded once into registers for all of them.
#include "pa_internal.h"
#include "ptx.cuh"

namespace pa {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kIter = 2;     // head groups per warp
constexpr int kThreads = 128;

__device__ __forceinline__ void unpack8(uint4 r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = bf16x2_to_float2(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(float2_to_bf16x2(x[0], x[1]), float2_to_bf16x2(x[2], x[3]),
                    float2_to_bf16x2(x[4], x[5]), float2_to_bf16x2(x[6], x[7]));
}

// 8 values over `scale` as E4M3 codes (correctly rounded quotient, then
// round-to-nearest-even with saturation, as pa_write_kv_fp8).
__device__ __forceinline__ uint2 pack8_e4m3(const float (&x)[8], float scale) {
  uint32_t o[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint16_t a = float2_to_e4m3x2(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale));
    const uint16_t b =
        float2_to_e4m3x2(__fdiv_rn(x[4 * i + 2], scale), __fdiv_rn(x[4 * i + 3], scale));
    o[i] = (uint32_t)a | ((uint32_t)b << 16);
  }
  return make_uint2(o[0], o[1]);
}

template <int D, bool F8>
__global__ void __launch_bounds__(kThreads) pa_norm_rope_write_kernel(const NormRopeParams p) {
  constexpr int LPH = D / 8;    // lanes per head
  constexpr int HPG = 32 / LPH;  // heads per group
  const int lane = threadIdx.x & 31;
  const int sub = lane % LPH, hsub = lane / LPH;
  const int rows = p.num_q_heads + 2 * p.num_kv_heads;
  const int chunks = (rows + HPG * kIter - 1) / (HPG * kIter);
  const long long wid = blockIdx.x * (long long)(kThreads / 32) + (threadIdx.x >> 5);
  const long long t = wid / chunks;
  if (t >= p.num_tokens) return;
  const int row0 = (int)(wid - t * chunks) * (HPG * kIter) + hsub;

  // every load that needs no position first
  const long long slot = __ldg(p.slot_mapping + t);
  const int pos = p.rotary_dim > 0 ? __ldg(p.positions + t) : 0;
  uint4 raw[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int row = row0 + i * HPG;
    raw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (row < rows) {
      const uint16_t* src;
      if (row < p.num_q_heads)
        src = p.q + t * p.q_stride + (long long)row * D;
      else if (row < p.num_q_heads + p.num_kv_heads)
        src = p.k + t * p.k_stride + (long long)(row - p.num_q_heads) * D;
      else
        src = p.v + t * p.v_stride + (long long)(row - p.num_q_heads - p.num_kv_heads) * D;
      raw[i] = *(reinterpret_cast<const uint4*>(src) + sub);  // q_out may be q: no read-only path
    }
  }
  if (slot < 0) return;  // a padding token: nothing of it is written
  if (slot >= p.num_slots) {
    if (lane == 0) report_error(p.err, PA_DEVERR_SLOT, t);
    return;
  }
  if (pos < 0 || pos >= p.max_position) {
    if (lane == 0) report_error(p.err, PA_DEVERR_POSITION, t);
    return;
  }

  // cosines and sines of this lane's elements: c[e], s[e] with the sign of
  // the partner's term in s (element a: -sin, element b: +sin)
  const int half = p.rotary_dim >> 1;
  const int e0 = sub * 8;
  const bool turned = e0 < p.rotary_dim;
  float c[8], s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    c[e] = 1.f;
    s[e] = 0.f;
  }
  if (turned) {
    const float* const cs = p.cos_sin + (long long)pos * p.rotary_dim;
    if (p.interleaved) {
      const float4 cv = __ldg(reinterpret_cast<const float4*>(cs + e0 / 2));
      const float4 sv = __ldg(reinterpret_cast<const float4*>(cs + half + e0 / 2));
      c[0] = c[1] = cv.x;
      c[2] = c[3] = cv.y;
      c[4] = c[5] = cv.z;
      c[6] = c[7] = cv.w;
      s[0] = -sv.x, s[1] = sv.x;
      s[2] = -sv.y, s[3] = sv.y;
      s[4] = -sv.z, s[5] = sv.z;
      s[6] = -sv.w, s[7] = sv.w;
    } else {
      const bool first = e0 < half;
      const int m = first ? e0 : e0 - half;
      const float sg = first ? -1.f : 1.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 cv = __ldg(reinterpret_cast<const float4*>(cs + m) + i);
        const float4 sv = __ldg(reinterpret_cast<const float4*>(cs + half + m) + i);
        c[4 * i] = cv.x, c[4 * i + 1] = cv.y, c[4 * i + 2] = cv.z, c[4 * i + 3] = cv.w;
        s[4 * i] = sg * sv.x, s[4 * i + 1] = sg * sv.y;
        s[4 * i + 2] = sg * sv.z, s[4 * i + 3] = sg * sv.w;
      }
    }
  }
  // the lane holding the other half of this lane's pairs (itself when untouched)
  const int hl = half / 8;
  const int partner = !turned || p.interleaved ? lane : (e0 < half ? lane + hl : lane - hl);

#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int row = row0 + i * HPG;
    const bool is_q = row < p.num_q_heads;
    const bool is_v = row >= p.num_q_heads + p.num_kv_heads;
    float x[8];
    unpack8(raw[i], x);
    const uint16_t* const w = is_q ? p.q_weight : p.k_weight;
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
    for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor_sync(kAll, ss, o);
    if (w != nullptr && !is_v) {
      const float r = rsqrtf(ss * (1.f / D) + p.eps);
      float wf[8];
      unpack8(__ldg(reinterpret_cast<const uint4*>(w) + sub), wf);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = x[e] * r * wf[e];
    }
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float far = __shfl_sync(kAll, x[e], partner);
      const float other = p.interleaved ? x[e ^ 1] : far;
      y[e] = is_v || !turned ? x[e] : fmaf(other, s[e], x[e] * c[e]);
    }
    if (row >= rows) continue;
    if (is_q) {
      *(reinterpret_cast<uint4*>(p.q_out + (t * p.num_q_heads + row) * D) + sub) = pack8(y);
    } else {
      const int h = row - p.num_q_heads - (is_v ? p.num_kv_heads : 0);
      const long long dst =
          (((slot >> 4) * p.num_kv_heads + h) * kBlockSize + (slot & 15)) * LPH + sub;
      void* const cache = is_v ? p.v_cache : p.k_cache;
      if constexpr (F8)
        static_cast<uint2*>(cache)[dst] = pack8_e4m3(y, is_v ? p.v_scale : p.k_scale);
      else
        static_cast<uint4*>(cache)[dst] = pack8(y);
    }
  }
  // The split-KV kernel that follows may be a programmatic dependent that
  // reads q without waiting for this grid's flush. This grid never releases a
  // dependent early (that happens when its last CTA ends), and the fence has
  // every store performed at the GPU's scope before its CTA ends.
  __threadfence();
}

}  // namespace

cudaError_t launch_norm_rope_write(const NormRopeParams& p, int head_dim, cudaStream_t s) {
  const int hpg = 32 / (head_dim / 8);
  const int rows = p.num_q_heads + 2 * p.num_kv_heads;
  const long long chunks = (rows + hpg * kIter - 1) / (hpg * kIter);
  const long long blocks = (p.num_tokens * chunks + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)blocks;
  if (head_dim == 128) {
    if (p.kv_fp8)
      pa_norm_rope_write_kernel<128, true><<<grid, kThreads, 0, s>>>(p);
    else
      pa_norm_rope_write_kernel<128, false><<<grid, kThreads, 0, s>>>(p);
  } else {
    if (p.kv_fp8)
      pa_norm_rope_write_kernel<64, true><<<grid, kThreads, 0, s>>>(p);
    else
      pa_norm_rope_write_kernel<64, false><<<grid, kThreads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace pa
