// Eviction from the paged KV cache by accumulated attention weight.
//
// For each (request, KV head) of a request with L > keep cached tokens, the
// tokens that stay are the first `sinks`, the last `recent`, and of the others,
// i in [sinks, L - recent), the keep - sinks - recent with the largest weight
// w[i] (ties to the lowest i). Their K and V rows move, in order, into the
// request's new blocks: kept token n of head h to row n % 16 of new block
// n / 16, head h. A KV head chooses its own tokens - a cache slot is one row
// per head, so the heads of a slot need not hold the same token. Rows are
// copied out of place: sources may be shared with other requests, and any
// number of CTAs can move rows with no order between them.
//
// Two kernels, chained by programmatic launch:
//   select  one CTA per (request, KV head): a radix select over the binary32
//           weights (11 + 11 + 10 bits, a 2048-bin histogram in shared memory),
//           then an order-preserving compaction: each warp counts the kept
//           tokens of its own contiguous part, one scan joins the counts.
//   move    the rows, bound by HBM: 2 x keep x D elements in, the same out.
#include "pa_internal.h"
#include "ptx.cuh"

namespace pa {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 64;  // rows of one move CTA

// A weight's place in the order: a larger key is a larger weight, -0 equals
// +0, and a NaN comes below every number (it is dropped first).
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The request's length when it is to be cut, else 0; `bad` for lengths that
// do not fit the tables (reported by the caller).
__device__ __forceinline__ int cut_length(const EvictParams& p, int r, bool& bad) {
  const int L = __ldg(p.seq_lens + r);
  bad = L < 0 || L > p.max_seq_len || L > p.weights_stride ||
        (L + kBlockSize - 1) / kBlockSize > p.max_blocks_per_req;
  return !bad && L > p.keep ? L : 0;
}

__global__ void __launch_bounds__(kSelThreads) pa_evict_select_kernel(const EvictParams p) {
  extern __shared__ uint32_t keys_sm[];  // the candidates' keys, when they fit
  __shared__ uint32_t hist[kBins];
  __shared__ int wsum[kSelWarps], wsum2[kSelWarps];
  __shared__ int s_bin, s_above;
  griddep_launch_dependents();  // the move grid may take its place; it waits for this one
  const int r = blockIdx.x / p.num_kv_heads, h = blockIdx.x - r * p.num_kv_heads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool bad;
  const int L = cut_length(p, r, bad);
  if (h == 0 && tid == 0) {
    if (bad)
      report_error(p.err, PA_DEVERR_LENGTHS, r);
    else
      p.new_seq_lens[r] = L ? p.keep : __ldg(p.seq_lens + r);
  }
  if (L == 0) return;
  const int a = p.sinks, n = L - p.recent - a, m = p.keep - p.sinks - p.recent;  // m of n stay
  const float* const w = p.weights + ((size_t)r * p.num_kv_heads + h) * p.weights_stride;
  const size_t orow = (size_t)r * p.num_kv_heads + h;
  int32_t* const kept = p.kept + orow * p.keep;
  float* const nw = p.new_weights ? p.new_weights + orow * p.new_weights_stride : nullptr;

  // the tokens that stay whatever they weigh
  for (int i = tid; i < a + p.recent; i += kSelThreads) {
    const int at = i < a ? i : p.keep - p.recent + (i - a);
    const int id = i < a ? i : L - p.recent + (i - a);
    kept[at] = id;
    if (nw) nw[at] = __ldg(w + id);
  }
  if (m == 0) return;

  const bool in_sm = n <= p.smem_keys;
  auto key_at = [&](int i) -> uint32_t { return in_sm ? keys_sm[i] : weight_key(__ldg(w + a + i)); };
  // radix select: after the passes, prefix is the m-th largest key and `need`
  // the number of tokens of exactly that key that stay (the lowest ones)
  uint32_t prefix = 0;
  int need = m;
  constexpr int kShift[3] = {21, 10, 0};
  constexpr int kWidth[3] = {11, 11, 10};
#pragma unroll
  for (int ps = 0; ps < 3; ++ps) {
    const int shift = kShift[ps], bins = 1 << kWidth[ps];
    for (int b = tid; b < bins; b += kSelThreads) hist[b] = 0u;
    __syncthreads();
    for (int i = tid; i < n; i += kSelThreads) {
      uint32_t k;
      if (ps == 0) {
        k = weight_key(__ldg(w + a + i));
        if (in_sm) keys_sm[i] = k;
      } else {
        k = key_at(i);
        if ((k >> (shift + kWidth[ps])) != prefix >> (shift + kWidth[ps])) continue;
      }
      atomicAdd(&hist[(k >> shift) & (uint32_t)(bins - 1)], 1u);  // a count: its order is nothing
    }
    __syncthreads();
    // the bin, from the top, in which the need-th token falls: thread t holds
    // bins-per-thread consecutive bins of the descending order
    constexpr int kPer = kBins / kSelThreads;
    const int per = bins / kSelThreads > 0 ? bins / kSelThreads : 1;
    int c[kPer], sum = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int b = bins - 1 - (tid * per + e);
      c[e] = e < per && b >= 0 ? (int)hist[b] : 0;
      sum += c[e];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kAll, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    int before = incl - sum;
    for (int v = 0; v < warp; ++v) before += wsum[v];
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      if (before < need && need <= before + c[e]) {
        s_bin = bins - 1 - (tid * per + e);
        s_above = before;
      }
      before += c[e];
    }
    __syncthreads();
    prefix |= (uint32_t)s_bin << shift;
    need -= s_above;
  }

  // compaction in order: warp v takes candidates [v seg, v seg + seg)
  const int seg = ((n + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int lo = min(n, warp * seg), hi = min(n, lo + seg);
  int gt = 0, eq = 0;
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const uint32_t k = i0 + lane < hi ? key_at(i0 + lane) : 0u;
    const bool in = i0 + lane < hi;
    gt += __popc(__ballot_sync(kAll, in && k > prefix));
    eq += __popc(__ballot_sync(kAll, in && k == prefix));
  }
  if (lane == 0) {
    wsum[warp] = gt;
    wsum2[warp] = eq;
  }
  __syncthreads();
  gt = eq = 0;
  for (int v = 0; v < warp; ++v) {
    gt += wsum[v];
    eq += wsum2[v];
  }
  const unsigned below = (1u << lane) - 1u;
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < hi ? key_at(i) : 0u;
    const unsigned bg = __ballot_sync(kAll, i < hi && k > prefix);
    const unsigned be = __ballot_sync(kAll, i < hi && k == prefix);
    const int eb = eq + __popc(be & below);  // equal ones before this one
    const bool stay = (bg >> lane & 1u) || ((be >> lane & 1u) && eb < need);
    if (stay) {
      const int at = a + gt + __popc(bg & below) + min(eb, need);
      kept[at] = a + i;
      if (nw) nw[at] = __ldg(w + a + i);
    }
    gt += __popc(bg);
    eq += __popc(be);
  }
}

// kMoveRows kept rows of one (request, KV head): the source and destination
// rows are looked up once per row, then every thread copies 16-byte vectors of
// K and V, all its loads in flight before its first store.
template <int RB>  // bytes of a row
__global__ void __launch_bounds__(kMoveThreads) pa_evict_move_kernel(const EvictParams p) {
  constexpr int VPR = RB / 16;                             // vectors per row
  constexpr int ITER = kMoveRows * VPR / kMoveThreads;     // vectors per thread and tensor
  static_assert(ITER >= 1, "every thread copies");
  __shared__ long long s_src[kMoveRows], s_dst[kMoveRows];  // row numbers in the caches; -1: none
  const int chunks = (p.keep + kMoveRows - 1) / kMoveRows;
  const long long g = blockIdx.x;
  const int c = (int)(g % chunks);
  const int rh = (int)(g / chunks);
  const int r = rh / p.num_kv_heads, h = rh - r * p.num_kv_heads;
  bool bad;
  const int L = cut_length(p, r, bad);
  griddep_wait();  // the select grid's lists
  if (L == 0) return;
  const int n0 = c * kMoveRows;
  if (threadIdx.x < kMoveRows) {
    const int n = n0 + threadIdx.x;
    long long src = -1, dst = -1;
    if (n < p.keep) {
      const int id = __ldcg(p.kept + (size_t)rh * p.keep + n);
      const int sb = __ldg(p.block_tables + (size_t)r * p.max_blocks_per_req + id / kBlockSize);
      const int db = __ldg(p.new_block_tables + (size_t)r * p.max_new_blocks + n / kBlockSize);
      if (sb < 0 || sb >= p.num_blocks)
        report_error(p.err, PA_DEVERR_BLOCK_ID, id / kBlockSize);
      else if (db < 0 || db >= p.num_blocks)
        report_error(p.err, PA_DEVERR_BLOCK_ID, n / kBlockSize);
      else {
        src = ((long long)sb * p.num_kv_heads + h) * kBlockSize + id % kBlockSize;
        dst = ((long long)db * p.num_kv_heads + h) * kBlockSize + n % kBlockSize;
      }
    }
    s_src[threadIdx.x] = src;
    s_dst[threadIdx.x] = dst;
  }
  __syncthreads();
  uint4 kv[ITER], vv[ITER];
  uint4* const kc = static_cast<uint4*>(p.k_cache);
  uint4* const vc = static_cast<uint4*>(p.v_cache);
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int e = i * kMoveThreads + threadIdx.x;
    const long long src = s_src[e / VPR];
    kv[i] = vv[i] = make_uint4(0u, 0u, 0u, 0u);
    if (src >= 0) {
      kv[i] = __ldcs(kc + src * VPR + e % VPR);  // read once: no use keeping it in a cache
      vv[i] = __ldcs(vc + src * VPR + e % VPR);
    }
  }
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int e = i * kMoveThreads + threadIdx.x;
    const long long dst = s_dst[e / VPR];
    if (dst >= 0) {
      kc[dst * VPR + e % VPR] = kv[i];
      vc[dst * VPR + e % VPR] = vv[i];
    }
  }
  __threadfence();  // performed before the CTA ends: the next grid may be a programmatic one
}

}  // namespace

cudaError_t launch_evict(EvictParams p, int row_bytes, cudaStream_t s) {
  const long long rows = (long long)p.num_reqs * p.num_kv_heads;
  const long long chunks = (p.keep + kMoveRows - 1) / kMoveRows;
  if (rows > 0x7fffffffLL || rows * chunks > 0x7fffffffLL) return cudaErrorInvalidValue;
  // candidates' keys in shared memory up to 40960 of them; longer caches read
  // their weights again in every pass (from L2)
  constexpr int kMaxKeys = 40960;
  static bool attr_set[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(pa_evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMaxKeys * 4);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  const int most = p.max_seq_len - p.sinks - p.recent;
  p.smem_keys = most < 1 ? 1 : (most < kMaxKeys ? most : kMaxKeys);
  pa_evict_select_kernel<<<(unsigned)rows, kSelThreads, (size_t)p.smem_keys * 4, s>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * chunks));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  switch (row_bytes) {
    case 64: return cudaLaunchKernelEx(&cfg, pa_evict_move_kernel<64>, p);
    case 128: return cudaLaunchKernelEx(&cfg, pa_evict_move_kernel<128>, p);
    case 256: return cudaLaunchKernelEx(&cfg, pa_evict_move_kernel<256>, p);
  }
  return cudaErrorInvalidValue;
}

}  // namespace pa
