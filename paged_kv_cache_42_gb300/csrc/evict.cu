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
//   select  a cluster of 1 to 8 CTAs per (request, KV head), each with its own
//           contiguous part of the candidates: a radix select over the binary32
//           weights (11 + 11 + 10 bits; a 2048-bin histogram per CTA, summed
//           into the first one's shared memory), then an order-preserving
//           compaction: each warp counts the kept tokens of its own contiguous
//           part, one scan joins the counts. Bound by its chain of about ten
//           barriers, so the cluster is sized for a few keys per thread.
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

// Cluster-wide barrier and reads of another CTA's shared memory. Every CTA of
// a cluster reaches every barrier: the paths depend on the request alone.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::
                   : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster(const void* mine, int rank) {
  uint32_t at, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(mine)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

__device__ __forceinline__ void add_cluster(const void* mine, int rank, uint32_t v) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(mine)), "r"(rank));
  asm volatile("red.shared::cluster.add.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

__global__ void __launch_bounds__(kSelThreads) pa_evict_select_kernel(const EvictParams p) {
  extern __shared__ uint32_t keys_sm[];  // this CTA's candidates' keys, when they fit
  __shared__ uint32_t hist[2][kBins];    // counts of this CTA; of the cluster (in its first CTA)
  __shared__ int wsum[kSelWarps], wsum2[kSelWarps];
  __shared__ uint32_t s_pick[2];         // a pass's bin, and the tokens in the bins above it
  __shared__ uint32_t s_count[2];        // kept tokens above the threshold, tokens at it
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
  // this CTA's candidates: c0 .. c0 + nc - 1 of the n
  const int part = ((n + C - 1) / C + 31) & ~31;
  const int c0 = min(n, rank * part), nc = min(n, c0 + part) - c0;
  const float* const wc = w + a + c0;

  // the tokens that stay whatever they weigh
  for (int i = rank * kSelThreads + tid; i < a + p.recent; i += C * kSelThreads) {
    const int at = i < a ? i : p.keep - p.recent + (i - a);
    const int id = i < a ? i : L - p.recent + (i - a);
    kept[at] = id;
    if (nw) nw[at] = __ldg(w + id);
  }
  if (m == 0) return;

  const bool in_sm = nc <= p.smem_keys;
  auto key_at = [&](int i) -> uint32_t { return in_sm ? keys_sm[i] : weight_key(__ldg(wc + i)); };
  // radix select: after the passes, prefix is the m-th largest key and `need`
  // the number of tokens of exactly that key that stay (the lowest ones)
  uint32_t prefix = 0;
  int need = m;
  constexpr int kShift[3] = {21, 10, 0};
  constexpr int kWidth[3] = {11, 11, 10};
  for (int b = tid; b < kBins; b += kSelThreads) hist[0][b] = hist[1][b] = 0u;
  cluster_sync();
#pragma unroll
  for (int ps = 0; ps < 3; ++ps) {
    const int shift = kShift[ps], bins = 1 << kWidth[ps];
    for (int i = tid; i < nc; i += kSelThreads) {
      uint32_t k;
      if (ps == 0) {
        k = weight_key(__ldg(wc + i));
        if (in_sm) keys_sm[i] = k;
      } else {
        k = key_at(i);
        if ((k >> (shift + kWidth[ps])) != prefix >> (shift + kWidth[ps])) continue;
      }
      atomicAdd(&hist[0][(k >> shift) & (uint32_t)(bins - 1)], 1u);  // a count: its order is nothing
    }
    __syncthreads();
    // into the first CTA's total: few bins are in use, whatever the pass
    if (C > 1) {
      for (int b = tid; b < bins; b += kSelThreads) {
        const uint32_t v = hist[0][b];
        if (v) add_cluster(&hist[1][b], 0, v);
        hist[0][b] = 0u;
      }
      cluster_sync();
    }
    if (rank == 0) {
      // the bin, from the top, in which the need-th token falls: thread t
      // holds `per` consecutive bins of the descending order
      uint32_t* const hs = hist[C > 1 ? 1 : 0];
      constexpr int kPer = kBins / kSelThreads;
      const int per = bins / kSelThreads;
      int c[kPer], sum = 0;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int b = bins - 1 - (tid * per + e);
        c[e] = 0;
        if (e < per) {
          c[e] = (int)hs[b];
          hs[b] = 0u;  // for the next pass
        }
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
    }
    if (C > 1) {
      cluster_sync();
      prefix |= ld_cluster(&s_pick[0], 0) << shift;
      need -= (int)ld_cluster(&s_pick[1], 0);
    } else {
      __syncthreads();
      prefix |= s_pick[0] << shift;
      need -= (int)s_pick[1];
    }
  }

  // compaction in order: warp v takes candidates [v seg, v seg + seg) of the part
  const int seg = ((nc + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int lo = min(nc, warp * seg), hi = min(nc, lo + seg);
  int gt = 0, eq = 0;
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const bool in = i0 + lane < hi;
    const uint32_t k = in ? key_at(i0 + lane) : 0u;
    gt += __popc(__ballot_sync(kAll, in && k > prefix));
    eq += __popc(__ballot_sync(kAll, in && k == prefix));
  }
  if (lane == 0) {
    wsum[warp] = gt;
    wsum2[warp] = eq;
  }
  __syncthreads();
  const int all_gt = warp_sum(lane < kSelWarps ? wsum[lane] : 0);
  const int all_eq = warp_sum(lane < kSelWarps ? wsum2[lane] : 0);
  gt = warp_sum(lane < warp ? wsum[lane & (kSelWarps - 1)] : 0);
  eq = warp_sum(lane < warp ? wsum2[lane & (kSelWarps - 1)] : 0);
  if (tid == 0) {
    s_count[0] = (uint32_t)all_gt;
    s_count[1] = (uint32_t)all_eq;
  }
  cluster_sync();
  for (int k = 0; k < rank; ++k) {  // the parts before this one
    gt += (int)ld_cluster(&s_count[0], k);
    eq += (int)ld_cluster(&s_count[1], k);
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
      kept[at] = a + c0 + i;
      if (nw) nw[at] = __ldg(wc + i);
    }
    gt += __popc(bg);
    eq += __popc(be);
  }
  cluster_sync();  // no CTA ends while another may still read its shared memory
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

cudaError_t launch_evict(EvictParams p, int row_bytes, int num_sms, cudaStream_t s) {
  const long long rows = (long long)p.num_reqs * p.num_kv_heads;
  const long long chunks = (p.keep + kMoveRows - 1) / kMoveRows;
  if (rows > 0x7fffffffLL || rows * chunks > 0x7fffffffLL) return cudaErrorInvalidValue;
  // a part's keys stay in shared memory up to this many; longer ones are read
  // again in every pass (from L2)
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
  // CTAs per (request, KV head): parts of about 4096 keys, eight per thread,
  // as long as the grid leaves SMs idle; beyond that a larger cluster only
  // repeats the barriers (64 rows of 32768: SELLONG us with eight CTAs, 40 us
  // with one; 512 rows of up to 4096: one CTA each)
  const long long most = (long long)p.max_seq_len - p.sinks - p.recent;
  p.cluster = 1;
  while (p.cluster < 8 && most > 4096LL * p.cluster && rows * p.cluster < 4LL * num_sms) p.cluster *= 2;
  const long long part = (most + p.cluster - 1) / p.cluster + 31;
  p.smem_keys = part < 1 ? 1 : (part < kMaxKeys ? (int)part : kMaxKeys);
  if (rows * p.cluster > 0x7fffffffLL) return cudaErrorInvalidValue;
  {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * p.cluster));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = (size_t)p.smem_keys * 4;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, pa_evict_select_kernel, p);
    if (e != cudaSuccess) return e;
  }
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
