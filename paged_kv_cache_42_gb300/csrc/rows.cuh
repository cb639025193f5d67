// Row-scaled E4M3 caches: one power of two for every (token, KV head) row of K
// and of V, held as a byte b that stands for 2^(b - 127), in
// scales[block][kv head][K, V][16].
//
// With a = max |x| of a row, e is the smallest integer in [-100, 119] with
// a <= 448 x 2^e (448: E4M3's largest number), b = e + 127, and an element's
// code is E4M3(x 2^-e): an exact product, rounded once. A power of two loses
// nothing against a / 448: E4M3 is a floating format, whose steps are relative
// down to 2^-6, so where in (224, 448] a row's largest element lies moves only
// the place of its subnormals (below 2^-14 of that element). It makes the value
// code x 2^e a bf16 number, so the tensor cores take widened rows exactly and
// reading back rounds nothing, and it is a quarter of an fp32 scale's bytes.
// A row with an infinity or a NaN gets b = 255, which stands for NaN, and codes
// of zero (an E4M3 NaN among the codes of a tile would spread further than its
// row: 0 x NaN in the products of other rows).
#pragma once

#include "ptx.cuh"

namespace pa {

constexpr int kRowPoison = 255;
constexpr int kScaleBytes = 2 * 16;  // of a (block, KV head): K's 16 rows, then V's

// The byte of a row whose largest |x| has these binary32 bits. Unsigned
// comparison orders finite < infinity < NaN, so a maximum over bits keeps those.
__device__ __forceinline__ int row_scale_byte(uint32_t top) {
  if (top >= 0x7f800000u) return kRowPoison;
  // exponent + 127 - 8, and one more past 1.75 x 2^k: 448 is 1.75 x 2^8
  const int b = (int)((top + 0x1fffffu) >> 23) - 8;
  return b < 27 ? 27 : b > 246 ? 246 : b;
}
// 2^-e; 0 for a poisoned row (whose codes are not x 2^-e but zeros: see row_codes).
__device__ __forceinline__ float row_inverse(int b) {
  return b == kRowPoison ? 0.f : __uint_as_float((uint32_t)(254 - b) << 23);
}
// 2^e; NaN for a poisoned row.
__device__ __forceinline__ float row_size(int b) {
  return __uint_as_float(b == kRowPoison ? 0x7fc00000u : (uint32_t)b << 23);
}

// Largest |x| so far, as binary32 bits.
__device__ __forceinline__ uint32_t row_top(uint32_t top, float x) {
  const uint32_t a = __float_as_uint(x) & 0x7fffffffu;
  return a > top ? a : top;
}
// The maximum over the `lanes` (8 or 16, aligned) lanes of a row. Rows of a warp
// may come here apart from each other, a row's lanes not.
template <int LANES>
__device__ __forceinline__ uint32_t row_top_all(uint32_t top, int lane) {
  const unsigned mask = ((1u << LANES) - 1u) << (lane & ~(LANES - 1));
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) {
    const uint32_t y = __shfl_xor_sync(mask, top, o);
    top = y > top ? y : top;
  }
  return top;
}
// Two elements as codes. inv 0: zeros, whatever x is.
__device__ __forceinline__ uint32_t row_codes(float a, float b, float inv) {
  if (inv == 0.f) return 0u;
  return float2_to_e4m3x2(a * inv, b * inv);
}

}  // namespace pa
