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
//   select  a cluster of 1 to 4 CTAs per (request, KV head), each with its own
//           contiguous part of the candidates, a key or more per thread in
//           registers: a radix select over the binary32 weights (11 + 11 + 10
//           bits; each CTA counts its keys' digits in shared memory and adds
//           the few bins in use to every CTA's total, so that each picks the
//           digit by itself after one cluster barrier), then an
//           order-preserving compaction by ballots, with the counts of the
//           warps and CTAs before. Bound by its chain of barriers.
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

__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// Every CTA of a cluster reaches every cluster barrier: the paths depend on the
// request alone. KPT: keys per thread, in registers; 0: parts longer than that, whose weights
// are read again (from L2) in every pass.
template <int KPT>
__global__ void __launch_bounds__(kSelThreads) pa_evict_select_kernel(const EvictParams p) {
  __shared__ uint32_t hist[kBins];      // digits of this CTA's keys
  __shared__ uint32_t total[3][kBins];  // of the cluster's, one per pass
  __shared__ int wsum[kSelWarps], wsum2[kSelWarps];
  __shared__ uint32_t s_pick[2];        // a pass's bin, and the tokens in the bins above it
  __shared__ uint32_t s_count[2];       // this CTA's tokens above the threshold, and at it
  griddep_wait();  // a programmatic dependent of the grid before
  griddep_launch_dependents();  // the move grid may take its place; it waits for this one
  const int C = p.cluster, rank = (int)(blockIdx.x % (unsigned)C);
  const int rh = (int)(blockIdx.x / (unsigned)C);
  const int r = rh / p.num_kv_heads, h = rh - r * p.num_kv_heads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool bad;
  const int L = cut_length(p, r, bad);
  if (h == 0 && rank == 0 && tid == 0) {
    if (bad)
      report_error(p.err, PA_DEVERR_LENGTHS, r);
    else
      p.new_seq_lens[r] = L ? p.keep : __ldg(p.seq_lens + r);
  }
  if (L == 0) return;
  const int a = p.sinks, n = L - p.recent - a, m = p.keep - p.sinks - p.recent;  // m of n stay
  const float* const w = p.weights + (size_t)rh * p.weights_stride;
  int32_t* const kept = p.kept + (size_t)rh * p.keep;
  float* const nw = p.new_weights ? p.new_weights + (size_t)rh * p.new_weights_stride : nullptr;
  // this CTA's candidates: c0 .. c0 + nc - 1 of the n; this warp's: lo .. hi - 1 of those
  const int part = ((n + C - 1) / C + 31) & ~31;
  const int c0 = min(n, rank * part), nc = min(n, c0 + part) - c0;
  const int seg = ((nc + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int lo = min(nc, warp * seg), hi = min(nc, lo + seg);
  const float* const wc = w + a + c0;
  uint32_t key[KPT > 0 ? KPT : 1];
  if (m > 0 && KPT > 0) {  // on their way while the totals are cleared
#pragma unroll
    for (int e = 0; e < KPT; ++e) {
      const int i = lo + e * 32 + lane;
      key[e] = i < hi ? __float_as_uint(__ldg(wc + i)) : 0u;
    }
  }
  // fn(i, key, in): the warp's candidates 32 at a time, in order
  auto each = [&](auto fn) {
    if constexpr (KPT > 0) {
#pragma unroll
      for (int e = 0; e < KPT; ++e) {
        const int i = lo + e * 32 + lane;
        fn(i, key[e], i < hi);
      }
    } else {
      for (int i0 = lo; i0 < hi; i0 += 32) {
        const int i = i0 + lane;
        fn(i, i < hi ? weight_key(__ldg(wc + i)) : 0u, i < hi);
      }
    }
  };

  // the tokens that stay whatever they weigh
  for (int i = rank * kSelThreads + tid; i < a + p.recent; i += C * kSelThreads) {
    const int at = i < a ? i : p.keep - p.recent + (i - a);
    const int id = i < a ? i : L - p.recent + (i - a);
    kept[at] = id;
    if (nw) nw[at] = __ldg(w + id);
  }
  if (m == 0) return;

  // radix select: after the passes, prefix is the m-th largest key and `need`
  // the number of tokens of exactly that key that stay (the lowest ones)
  uint32_t prefix = 0;
  int need = m;
  constexpr int kShift[3] = {21, 10, 0};
  constexpr int kWidth[3] = {11, 11, 10};
  for (int b = tid; b < kBins; b += kSelThreads) hist[b] = total[0][b] = total[1][b] = total[2][b] = 0u;
  if constexpr (KPT > 0) {
#pragma unroll
    for (int e = 0; e < KPT; ++e) key[e] = weight_key(__uint_as_float(key[e]));
  }
  if (C > 1) cluster_sync(); else __syncthreads();
#pragma unroll
  for (int ps = 0; ps < 3; ++ps) {
    const int shift = kShift[ps], bins = 1 << kWidth[ps];
    uint32_t* const own = C > 1 ? hist : total[ps];
    each([&](int, uint32_t k, bool in) {
      if (in && (ps == 0 || (k >> (shift + kWidth[ps])) == prefix >> (shift + kWidth[ps])))
        atomicAdd(&own[(k >> shift) & (uint32_t)(bins - 1)], 1u);  // a count: its order is nothing
    });
    __syncthreads();
    if (C > 1) {
      for (int b = tid; b < bins; b += kSelThreads) {
        const uint32_t v = hist[b];
        if (v) {
          hist[b] = 0u;
          for (int k = 0; k < C; ++k) add_cluster(cluster_addr(&total[ps][b], k), v);
        }
      }
      cluster_sync();
    }
    // the bin, from the top, in which the need-th token falls: thread t holds
    // `per` consecutive bins of the descending order
    constexpr int kPer = kBins / kSelThreads;
    const int per = bins / kSelThreads;
    int c[kPer], sum = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      c[e] = e < per ? (int)total[ps][bins - 1 - (tid * per + e)] : 0;
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
    int before = incl - sum + warp_sum(lane < warp ? wsum[lane & (kSelWarps - 1)] : 0);
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      if (before < need && need <= before + c[e]) {
        s_pick[0] = (uint32_t)(bins - 1 - (tid * per + e));
        s_pick[1] = (uint32_t)before;
      }
      before += c[e];
    }
    __syncthreads();
    prefix |= s_pick[0] << shift;
    need -= (int)s_pick[1];
  }

  // compaction in order
  int gt = 0, eq = 0;
  each([&](int, uint32_t k, bool in) {
    gt += __popc(__ballot_sync(kAll, in && k > prefix));
    eq += __popc(__ballot_sync(kAll, in && k == prefix));
  });
  if (lane == 0) {
    wsum[warp] = gt;
    wsum2[warp] = eq;
  }
  __syncthreads();
  if (C > 1) {
    const int all_gt = warp_sum(lane < kSelWarps ? wsum[lane] : 0);
    const int all_eq = warp_sum(lane < kSelWarps ? wsum2[lane] : 0);
    if (tid == 0) {
      s_count[0] = (uint32_t)all_gt;
      s_count[1] = (uint32_t)all_eq;
    }
    cluster_sync();
  }
  // the warps and the parts before this one
  const bool part_before = C > 1 && lane < rank;
  gt = warp_sum((lane < warp ? wsum[lane & (kSelWarps - 1)] : 0) +
                (part_before ? (int)ld_cluster(cluster_addr(&s_count[0], lane)) : 0));
  eq = warp_sum((lane < warp ? wsum2[lane & (kSelWarps - 1)] : 0) +
                (part_before ? (int)ld_cluster(cluster_addr(&s_count[1], lane)) : 0));
  const unsigned below = (1u << lane) - 1u;
  each([&](int i, uint32_t k, bool in) {
    const unsigned bg = __ballot_sync(kAll, in && k > prefix);
    const unsigned be = __ballot_sync(kAll, in && k == prefix);
    const int eb = eq + __popc(be & below);  // equal ones before this one
    const bool stay = (bg >> lane & 1u) || ((be >> lane & 1u) && eb < need);
    if (stay) {
      const int at = a + gt + __popc(bg & below) + min(eb, need);
      kept[at] = a + c0 + i;
      if (nw) nw[at] = __ldg(wc + i);
    }
    gt += __popc(bg);
    eq += __popc(be);
  });
  if (C > 1) cluster_sync();  // no CTA ends while another may still read its shared memory
}

template <int KPT>
cudaError_t launch_select(const EvictParams& p, unsigned rows, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(rows * (unsigned)p.cluster);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, pa_evict_select_kernel<KPT>, p);
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
  const int chunks = (p.keep - 1) / kMoveRows + 1;
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
}

}  // namespace

cudaError_t launch_evict(EvictParams p, int row_bytes, int num_sms, cudaStream_t s) {
  const long long rows = (long long)p.num_reqs * p.num_kv_heads;
  const long long chunks = (p.keep - 1) / kMoveRows + 1;
  if (rows > 0x7fffffffLL || rows * chunks > 0x7fffffffLL) return cudaErrorInvalidValue;
  // CTAs per (request, KV head): parts of at most 8192 keys, sixteen per thread,
  // as long as the grid leaves SMs idle (64 rows of 32768 keys, whole call: 41.2
  // us with four CTAs each, 42.6 with two of 32 keys per thread, 51.4 with eight
  // of eight, whose barriers cost more than the shorter parts give, 106 with one,
  // whose keys no longer fit registers; 512 rows of up to 4096 keys: one CTA each).
  const long long most = (long long)p.max_seq_len - p.sinks - p.recent;
  p.cluster = 1;
  while (p.cluster < 4 && most > 8192LL * p.cluster && rows * p.cluster < 4LL * num_sms) p.cluster *= 2;
  if (rows * p.cluster > 0x7fffffffLL) return cudaErrorInvalidValue;
  const long long part = (((most > 0 ? most : 1) + p.cluster - 1) / p.cluster + 31) / 32 * 32;
  cudaError_t e = part <= 4 * kSelThreads    ? launch_select<4>(p, (unsigned)rows, s)
                  : part <= 8 * kSelThreads  ? launch_select<8>(p, (unsigned)rows, s)
                  : part <= 16 * kSelThreads ? launch_select<16>(p, (unsigned)rows, s)
                  : part <= 32 * kSelThreads ? launch_select<32>(p, (unsigned)rows, s)
                                             : launch_select<0>(p, (unsigned)rows, s);
  if (e != cudaSuccess) return e;
  if (p.max_seq_len <= p.keep) return cudaSuccess;  // no request is cut: the lengths were all
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
