// Row-scaled E4M3 caches: the write that finds each row's scale, and reading
// ranges of cached keys back as dense bf16 rows (from any cache format).
#include "pa_internal.h"
#include "ptx.cuh"
#include "rows.cuh"

namespace pa {

namespace {

constexpr int kWriteThreads = 256;

// ---------------------------------------------------------------------------------------
// Write: pa_write_kv's scatter ("vLLM v1 Deep Dive: How LLM(...) and the Server
// Boot and Generate", Part 3, "Aside - KV cache and prefix caching"), each row
// as codes and a scale (rows.cuh).
//
// A lane holds 8 elements of K and the matching 8 of V, a row is D / 8 lanes:
// its largest element is three or four shuffles away, and the row is never read
// twice. What bounds it: bytes for many tokens, for a few the launch and two
// dependent loads. 4 tokens 1.5 us, 2048 tokens of 8 heads at 128 dims 3.6 us (1.9 us
// of bytes), in a graph of calls.
// ---------------------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(kWriteThreads) pa_write_rows_kernel(const WriteRowsParams p) {
  constexpr int LPR = D / 8;  // lanes per row
  const int lane = threadIdx.x & 31;
  const long long i = blockIdx.x * (long long)kWriteThreads + threadIdx.x;
  const long long row = i / LPR;  // t * Hkv + h
  const int c = (int)(i % LPR);
  griddep_wait();  // a programmatic dependent of the grid before, which made k and v
  // The next grid may be placed now: it waits for this one, at its start or
  // (PA_OPT_WRITE_OVERLAP) before it reads what this one writes.
  griddep_launch_dependents();
  if (row >= (long long)p.num_tokens * p.num_kv_heads) return;  // a whole row's lanes
  const int t = (int)(row / p.num_kv_heads);
  const int h = (int)(row - (long long)t * p.num_kv_heads);
  const long long s = __ldg(p.slot_mapping + t);
  const uint4 kr = __ldg(reinterpret_cast<const uint4*>(p.k + t * p.k_stride + h * D) + c);
  const uint4 vr = __ldg(reinterpret_cast<const uint4*>(p.v + t * p.v_stride + h * D) + c);
  if (s < 0) return;  // a padding token
  if (s >= p.num_slots) {
    if (c == 0) report_error(p.err, PA_DEVERR_SLOT, t);
    return;
  }
  const long long tile = (s >> 4) * p.num_kv_heads + h;
  const int off = (int)(s & 15);
  auto half = [&](uint4 raw, unsigned char* cache, int which) {
    float2 x[4] = {bf16x2_to_float2(raw.x), bf16x2_to_float2(raw.y), bf16x2_to_float2(raw.z),
                   bf16x2_to_float2(raw.w)};
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) top = row_top(row_top(top, x[e].x), x[e].y);
    const int b = row_scale_byte(row_top_all<LPR>(top, lane));
    const float inv = row_inverse(b);
    const uint2 o = make_uint2(row_codes(x[0].x, x[0].y, inv) | row_codes(x[1].x, x[1].y, inv) << 16,
                               row_codes(x[2].x, x[2].y, inv) | row_codes(x[3].x, x[3].y, inv) << 16);
    *reinterpret_cast<uint2*>(cache + (tile * kBlockSize + off) * D + c * 8) = o;
    if (c == which) p.scales[tile * kScaleBytes + which * kBlockSize + off] = (unsigned char)b;
  };
  half(kr, p.k_cache, 0);
  half(vr, p.v_cache, 1);
}

// ---------------------------------------------------------------------------------------
// Read: out row read_start_loc[r] + i holds key first[r] + i of request r, as
// bf16: the element of a bf16 cache, code x k_scale (rounded) of an E4M3 one, or
// code x 2^e (exact) of a row-scaled one.
//
// What bounds it: bytes, codes in and bf16 out. A CTA takes `per` consecutive
// output rows (tokens). One thread of each finds its request (binary search over
// read_start_loc), checks the key and the block and leaves the row's place in
// shared memory: the dependent loads are paid once per CTA, and the copy that
// follows has all of its loads independent. A thread then moves 16 elements of K
// and of V at a time: one or two 16-byte loads and one 32-byte store each.
// 64 requests of 512 to 4096 keys, row-scaled: 145 us, 0.93 of the measured copy rate.
// ---------------------------------------------------------------------------------------
constexpr int kReadThreads = 256;
constexpr int kReadMost = 32;  // tokens of a CTA at most

__device__ __forceinline__ void store32(void* at, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// FMT: 0 bf16, 1 E4M3 with one scale per tensor, 2 row-scaled
template <int D, int FMT>
__global__ void __launch_bounds__(kReadThreads) pa_read_kernel(const ReadParams p) {
  constexpr int CPR = D / 16;  // 16-element chunks of a row
  __shared__ long long s_tile[kReadMost];  // (block * Hkv) of a token, -1: nothing to copy
  __shared__ int s_off[kReadMost];
  griddep_wait();
  const int per = p.tokens_per_cta;
  const long long t0 = blockIdx.x * (long long)per;
  if (threadIdx.x < (unsigned)per) {
    const long long t = t0 + threadIdx.x;
    long long tile = -1;
    int off = 0;
    if (t < p.num_tokens) {
      // the last request that starts at or before t
      int lo = 0, hi = p.num_reqs;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(p.read_start_loc + mid) <= t) lo = mid; else hi = mid;
      }
      const int a = __ldg(p.read_start_loc + lo), b = __ldg(p.read_start_loc + lo + 1);
      if (a < 0 || b < a || b > p.num_tokens) {
        report_error(p.err, PA_DEVERR_QSL, lo);
      } else if (t >= a && t < b) {  // rows before the first or past the last are nobody's
        const long long f = p.first ? __ldg(p.first + lo) : 0;
        if (f < 0 || (f + (b - a) + kBlockSize - 1) / kBlockSize > p.max_blocks_per_req) {
          report_error(p.err, PA_DEVERR_LENGTHS, lo);
        } else {
          const long long key = f + (t - a);
          const int pid = __ldg(p.block_tables + (long long)lo * p.max_blocks_per_req + key / kBlockSize);
          if (pid < 0 || pid >= p.num_blocks) {
            report_error(p.err, PA_DEVERR_BLOCK_ID, key / kBlockSize);
          } else {
            tile = (long long)pid * p.num_kv_heads;
            off = (int)(key % kBlockSize);
          }
        }
      }
    }
    s_tile[threadIdx.x] = tile;
    s_off[threadIdx.x] = off;
  }
  __syncthreads();
  const int hkv = p.num_kv_heads;
  const int per_token = hkv * CPR, n = per * per_token;
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += kReadThreads) {
    const int j = i / per_token, rest = i - j * per_token;
    const int h = rest / CPR, c = rest % CPR;
    const long long tile = s_tile[j];
    if (tile < 0) continue;
    const long long at = ((tile + h) * kBlockSize + s_off[j]) * D + c * 16;  // element
    const long long to = (t0 + j) * hkv * D + (long long)h * D + c * 16;
    if constexpr (FMT == 0) {
      const uint4* const ks = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.k_cache) + at);
      const uint4* const vs = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.v_cache) + at);
      const uint4 a = __ldg(ks), b = __ldg(ks + 1), x = __ldg(vs), y = __ldg(vs + 1);
      const uint32_t kw[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      const uint32_t vw[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
      store32(p.k_out + to, kw);
      store32(p.v_out + to, vw);
    } else {
      const uint4 a = __ldg(reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(p.k_cache) + at));
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(p.v_cache) + at));
      float ksz = p.k_scale, vsz = p.v_scale;
      if constexpr (FMT == 2) {
        const unsigned char* const sc = p.scales + (tile + h) * kScaleBytes + s_off[j];
        ksz = row_size(__ldg(sc));
        vsz = row_size(__ldg(sc + kBlockSize));
      }
      auto widen = [](uint4 r, float size, uint32_t (&w)[8]) {
        const uint32_t c4[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 lo = e4m3x2_to_float2((uint16_t)(c4[e] & 0xffffu));
          const float2 hi = e4m3x2_to_float2((uint16_t)(c4[e] >> 16));
          w[2 * e] = float2_to_bf16x2(lo.x * size, lo.y * size);
          w[2 * e + 1] = float2_to_bf16x2(hi.x * size, hi.y * size);
        }
      };
      uint32_t kw[8], vw[8];
      widen(a, ksz, kw);
      widen(x, vsz, vw);
      store32(p.k_out + to, kw);
      store32(p.v_out + to, vw);
    }
  }
}

template <typename K, typename P>
cudaError_t launch_dependent(K kern, long long grid, int threads, const P& p, cudaStream_t s) {
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_write_rows(const WriteRowsParams& p, int head_dim, cudaStream_t s) {
  const long long lanes = (long long)p.num_tokens * p.num_kv_heads * (head_dim / 8);
  const long long grid = (lanes + kWriteThreads - 1) / kWriteThreads;
  return head_dim == 128 ? launch_dependent(pa_write_rows_kernel<128>, grid, kWriteThreads, p, s)
                         : launch_dependent(pa_write_rows_kernel<64>, grid, kWriteThreads, p, s);
}

cudaError_t launch_read(ReadParams p, int head_dim, int format, int num_sms, cudaStream_t s) {
  // As many tokens per CTA as leave four CTAs per SM something to do.
  int per = kReadMost;
  while (per > 1 && (p.num_tokens + per - 1) / per < 4LL * num_sms) per >>= 1;
  p.tokens_per_cta = per;
  const long long grid = ((long long)p.num_tokens + per - 1) / per;
  if (head_dim == 128)
    return format == 0   ? launch_dependent(pa_read_kernel<128, 0>, grid, kReadThreads, p, s)
           : format == 1 ? launch_dependent(pa_read_kernel<128, 1>, grid, kReadThreads, p, s)
                         : launch_dependent(pa_read_kernel<128, 2>, grid, kReadThreads, p, s);
  return format == 0   ? launch_dependent(pa_read_kernel<64, 0>, grid, kReadThreads, p, s)
         : format == 1 ? launch_dependent(pa_read_kernel<64, 1>, grid, kReadThreads, p, s)
                       : launch_dependent(pa_read_kernel<64, 2>, grid, kReadThreads, p, s);
}

}  // namespace pa
