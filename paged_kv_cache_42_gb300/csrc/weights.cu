// Accumulated attention weight of every cached key.
//
// For request r with qlen new tokens on ctx cached ones, KV head h and key i,
//   out[r][h][i] = (i < ctx ? w[r][h][i] : 0)
//                + sum_{j < qlen} sum_{g < G} p_{j,g}[i],
//   p_{j,g}[i] = exp(s_{j,g}[i] - lse_{j,g}),  s = scale q . k,  i <= ctx + j,
// the softmax weights attention gives the key, summed over the step's queries
// and the query heads of the KV head (a heavy-hitter score; the eviction in
// evict.cu goes by it). Keys that are new in this step start from zero, so a
// fresh row needs no clearing. K is read; V plays no part. Two forms, chosen
// for each request by its rows = qlen G:
//
// Few rows (<= 8: decodes, and spans of a token or two): bound by the bytes of
// K, which are read once. pa_weights_score_kernel computes S = K Q^T on 16 keys
// x 8 rows x head_dim with mma.sync - here the tensor pipe is idle most of the
// time whatever form is used, and the warp-level form takes K straight from
// global memory into fragments, with no shared memory, no barrier and no wait -
// stores the scaled scores (4 bytes a row, against 256 or 128 of K) and each
// 256-key chunk's softmax maximum and sum. pa_weights_finish_kernel joins the
// chunks and turns the scores, which are still in L2, into weights. A dot
// product may take its terms in any order, so a lane loads 16 consecutive
// bytes of a row and both operands read the same elements in the same order.
// E4M3 codes are exact in f16, and so is a query row scaled by the power of two
// that brings its largest element into [2^13, 2^14).
//
// Many rows (prompt chunks): bound by arithmetic, 2 x 2 head_dim flops and two
// exponentials per (row, key). Two passes of one tcgen05 kernel: a stationary
// 128-row operand X against a stream of 128-row operands Y, S = X Y^T into
// TMEM, one thread per row of X with no exchange between threads:
//   pass 1  X = 128 query rows (G heads x 128 / G tokens), Y = key tiles: the
//           thread keeps its query's running maximum and sum -> lse. Keys are
//           cut into parts of 16 tiles, joined by a small kernel.
//   pass 2  X = 128 keys, Y = the query row tiles that see them: the thread
//           sums exp2(s - lse) over its key's columns, in a fixed order, and
//           writes the key's weight. No atomics and no partial sums.
// The softmax warpgroups take the Y tiles in turn; four S buffers in TMEM let
// the MMAs run ahead of them. A pass's pace is the exponentials: 128 x 128 of
// them are 1024 cycles of an SM's special-function unit, the MMA about half.
#include <cuda.h>

#include "pa_internal.h"
#include "ptx.cuh"

namespace pa {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kFewRows = 8;          // rows the bandwidth-bound form takes (the MMA's N)
constexpr int kChunkBlocks = 16;     // 16-key blocks per warp
constexpr int kScoreWarps = 4;
constexpr int kClusterWarps = 8;
constexpr int kClusterSmem = 64 * 1024;  // scores of one CTA of a cluster, at most: three CTAs on an SM
constexpr int kFinishThreads = 256;

constexpr int kFinishRound = 1024;   // keys of one round of a finish CTA
constexpr int kFinishKeys = 4 * kFinishRound;  // keys of one finish CTA (joining the chunks costs
                                                 // each CTA the same, whatever its keys)
constexpr int kSplitTiles = 32;      // key tiles of one part in pass 1
constexpr int kPlanThreads = 1024;
constexpr int kBuckets = 1024;
constexpr float kNone = -1e30f;      // a running maximum before the first key

struct Span {
  int q0, qlen, L;
  bool ok;
};

// Request r's span; `report`: record what is wrong with it on the error word.
__device__ __forceinline__ Span get_span(const WeightsParams& p, int r, bool report) {
  Span s;
  s.q0 = __ldg(p.qsl + r);
  const int q1 = __ldg(p.qsl + r + 1);
  s.L = __ldg(p.seq_lens + r);
  s.qlen = q1 - s.q0;
  s.ok = true;
  if (s.q0 < 0 || q1 < s.q0 || q1 > p.num_tokens) {
    if (report) report_error(p.err, PA_DEVERR_QSL, r);
    s.ok = false;
  } else if (s.L < s.qlen || (s.L + kBlockSize - 1) / kBlockSize > p.bt_stride ||
             s.qlen > p.max_query_len || s.L > p.max_seq_len || s.L > p.weights_stride) {
    if (report) report_error(p.err, PA_DEVERR_LENGTHS, r);
    s.ok = false;
  }
  return s;
}

// ---------------------------------------------------------------------------------------
// few rows
// ---------------------------------------------------------------------------------------
// K passes through once.
__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Cluster-wide barrier, and a read of another CTA's shared memory.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ float2 ld_cluster_f2(const void* mine, int rank) {
  uint32_t at;
  float2 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(mine)), "r"(rank));
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
  return v;
}

template <bool F16>
__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t w) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(w));
  return h;
}
__device__ __forceinline__ uint32_t float2_to_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The query operand of up to 8 rows (row g: token g / G, head g % G of KV head
// h) as B fragments, this lane's elements; unscale: of row g (E4M3 form).
template <int D, bool F8>
struct QFrag {
  uint32_t b[D / 16][2];
  float unscale;
};
template <int D, bool F8>
__device__ __forceinline__ void load_query(const WeightsParams& p, const Span& sp, int h, int rows,
                                           int lane, QFrag<D, F8>& q) {
  constexpr int NK = D / 16, NJ = D * (F8 ? 1 : 2) / 64;
  const int g = lane >> 2, t = lane & 3, G = p.group;
  q.unscale = 1.f;
#pragma unroll
  for (int i = 0; i < NK; ++i) q.b[i][0] = q.b[i][1] = 0u;
  const uint4* const qrow = reinterpret_cast<const uint4*>(
      p.q + ((size_t)(sp.q0 + g / G) * p.num_q_heads + (size_t)h * G + g % G) * D);
  if constexpr (F8) {
    uint4 raw[NJ][2];
    float mx = 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        raw[j][e] = g < rows ? __ldg(qrow + (j * 4 + t) * 2 + e) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t w[4] = {raw[j][e].x, raw[j][e].y, raw[j][e].z, raw[j][e].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = bf16x2_to_float2(w[i]);
          mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
    mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 2));
    int ex = 0;  // 13 - floor(log2 mx), from the exponent field
    if (mx > 0.f) {
      ex = 13 - (((int)(__float_as_uint(mx) >> 23) & 0xff) - 127);
      ex = ex < -120 ? -120 : (ex > 120 ? 120 : ex);
    }
    const float sc = __uint_as_float((uint32_t)(127 + ex) << 23);
    q.unscale = __uint_as_float((uint32_t)(127 - ex) << 23);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const uint32_t w[8] = {raw[j][0].x, raw[j][0].y, raw[j][0].z, raw[j][0].w,
                             raw[j][1].x, raw[j][1].y, raw[j][1].z, raw[j][1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 f = bf16x2_to_float2(w[i]);
        q.b[4 * j + i / 2][i & 1] = float2_to_f16x2(f.x * sc, f.y * sc);
      }
    }
  } else if (g < rows) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const uint4 v = __ldg(qrow + j * 4 + t);
      q.b[2 * j][0] = v.x;
      q.b[2 * j][1] = v.y;
      q.b[2 * j + 1][0] = v.z;
      q.b[2 * j + 1][1] = v.w;
    }
  }
}

// A 16-key block of K as A fragments: keys g and g + 8, this lane's elements.
template <int D, bool F8>
struct KFrag {
  uint4 a[D * (F8 ? 1 : 2) / 64][2];
};
template <int D, bool F8>
__device__ __forceinline__ void load_block(const WeightsParams& p, int h, int id, int lane,
                                           KFrag<D, F8>& f) {
  constexpr int VPR = D * (F8 ? 1 : 2) / 16, NJ = VPR / 4;  // vectors of a row, of a lane
  const uint4* const src = static_cast<const uint4*>(p.k_cache) +
                           (((size_t)(id < 0 ? 0 : id) * p.num_kv_heads + h) * kBlockSize +
                            (lane >> 2)) * VPR + (lane & 3);
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    f.a[j][0] = f.a[j][1] = make_uint4(0u, 0u, 0u, 0u);
    if (id >= 0) {
      f.a[j][0] = ld_stream(src + 4 * j);
      f.a[j][1] = ld_stream(src + 8 * VPR + 4 * j);
    }
  }
}

// Scores n >= 1 blocks: id(j) and take(j, fragment) for block j, the next
// block's loads issued before a block is scored (deeper rings of three and four
// blocks measured slower: their registers cost more warps than they add loads).
template <int D, bool F8, typename ID, typename TAKE>
__device__ __forceinline__ void stream_blocks(const WeightsParams& p, int h, int lane, int n, ID id,
                                              TAKE take) {
  KFrag<D, F8> fa, fb;
  load_block<D, F8>(p, h, id(0), lane, fa);
#pragma unroll 1
  for (int j = 0; j < n; j += 2) {
    if (j + 1 < n) load_block<D, F8>(p, h, id(j + 1), lane, fb);
    take(j, fa);
    if (j + 1 >= n) break;
    if (j + 2 < n) load_block<D, F8>(p, h, id(j + 2), lane, fa);
    take(j + 1, fb);
  }
}

// The running softmax maximum and sum of the two rows a lane holds.
struct Run2 {
  float m0, m1, l0, l1;
  __device__ __forceinline__ void clear() {
    m0 = m1 = kNone;
    l0 = l1 = 0.f;
  }
  __device__ __forceinline__ void add(float x0, float y0, float x1, float y1) {
    const float k0 = fmaxf(m0, fmaxf(x0, y0)), k1 = fmaxf(m1, fmaxf(x1, y1));
    l0 = l0 * ex2_approx(m0 - k0) + (ex2_approx(x0 - k0) + ex2_approx(y0 - k0));
    l1 = l1 * ex2_approx(m1 - k1) + (ex2_approx(x1 - k1) + ex2_approx(y1 - k1));
    m0 = k0;
    m1 = k1;
  }
  __device__ __forceinline__ void over_lanes() {  // the lanes of a row are those of equal lane % 4
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      const float a = __shfl_xor_sync(kAll, m0, o), b = __shfl_xor_sync(kAll, m1, o);
      const float la = __shfl_xor_sync(kAll, l0, o), lb = __shfl_xor_sync(kAll, l1, o);
      const float k0 = fmaxf(m0, a), k1 = fmaxf(m1, b);
      l0 = l0 * ex2_approx(m0 - k0) + la * ex2_approx(a - k0);
      l1 = l1 * ex2_approx(m1 - k1) + lb * ex2_approx(b - k1);
      m0 = k0;
      m1 = k1;
    }
  }
};

// Scores of a block: x0, x1 of key `key` (the lane's first) for rows n0, n1, y0,
// y1 of key + 8, scaled; -inf where the row does not see the key or the block
// is missing. They go to `at` (+ 8 NR: of key + 8), NR values per key, and into
// the running maxima and sums.
template <int D, bool F8, int NR>
__device__ __forceinline__ void score_block(const KFrag<D, F8>& f, const QFrag<D, F8>& q, int t,
                                            bool have, int key, int lim0, int lim1, float sc0,
                                            float sc1, float* at, Run2& run) {
  constexpr int NJ = D * (F8 ? 1 : 2) / 64;
  float c[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};  // two chains of MMAs
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const uint4 u = f.a[j][0], v = f.a[j][1];
    if constexpr (F8) {
      const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        mma_16x8x16<true>(c[e & 1], e4m3x2_to_f16x2((uint16_t)(uw[e] & 0xffffu)),
                          e4m3x2_to_f16x2((uint16_t)(vw[e] & 0xffffu)),
                          e4m3x2_to_f16x2((uint16_t)(uw[e] >> 16)),
                          e4m3x2_to_f16x2((uint16_t)(vw[e] >> 16)), q.b[4 * j + e][0],
                          q.b[4 * j + e][1]);
    } else {
      mma_16x8x16<false>(c[0], u.x, v.x, u.y, v.y, q.b[2 * j][0], q.b[2 * j][1]);
      mma_16x8x16<false>(c[1], u.z, v.z, u.w, v.w, q.b[2 * j + 1][0], q.b[2 * j + 1][1]);
    }
  }
  const float x0 = have && key <= lim0 ? (c[0][0] + c[1][0]) * sc0 : -INFINITY;
  const float x1 = have && key <= lim1 ? (c[0][1] + c[1][1]) * sc1 : -INFINITY;
  const float y0 = have && key + 8 <= lim0 ? (c[0][2] + c[1][2]) * sc0 : -INFINITY;
  const float y1 = have && key + 8 <= lim1 ? (c[0][3] + c[1][3]) * sc1 : -INFINITY;
  if constexpr (NR == 1) {
    if (t == 0) {
      at[0] = x0;
      at[8] = y0;
    }
  } else if (2 * t < NR) {
    *reinterpret_cast<float2*>(at) = make_float2(x0, x1);
    *reinterpret_cast<float2*>(at + 8 * NR) = make_float2(y0, y1);
  }
  run.add(x0, y0, x1, y1);
}

// Few rows, all of a (request, KV head)'s scores in shared memory: a cluster of
// 1 to 8 CTAs shares its blocks, a warp takes every kClusterWarps-th block of
// its CTA's part, the maxima and sums are exchanged over distributed shared
// memory, and each CTA turns its own scores into weights. NR: rows stored per
// key (the batch's largest count: G for decodes, else 8).
template <int D, bool F8, int NR>
__global__ void __launch_bounds__(32 * kClusterWarps, 2) pa_weights_cluster_kernel(const WeightsParams p) {
  extern __shared__ __align__(16) float score_sm[];  // [keys of the part][NR]
  __shared__ float2 s_run[kClusterWarps][kFewRows];
  __shared__ float2 s_cta[kFewRows];                 // this CTA's {max, sum} of each row
  __shared__ float2 s_row[kFewRows];                 // the request's {max, 1 / sum}
  if (p.num_slots > 0) griddep_launch_dependents();  // prompt chunks' passes need nothing of this
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int C = p.cluster, rank = (int)(blockIdx.x % (unsigned)C);
  const int rh = (int)(blockIdx.x / (unsigned)C);
  const int r = rh / p.num_kv_heads, h = rh - r * p.num_kv_heads;
  const Span sp = get_span(p, r, rank == 0 && h == 0 && threadIdx.x == 0);
  const int G = p.group, rows = sp.qlen * G;
  if (!sp.ok || rows == 0 || rows > kFewRows) {  // the whole cluster alike
    if (p.num_slots > 0) griddep_wait();  // completes after the plan before it
    return;
  }
  const int nb = (sp.L + kBlockSize - 1) / kBlockSize;
  const int part = (nb + C - 1) / C;
  const int b0 = min(nb, rank * part), n = min(nb, b0 + part) - b0;  // this CTA's blocks
  const int g = lane >> 2, t = lane & 3;
  QFrag<D, F8> q;
  load_query<D, F8>(p, sp, h, rows, lane, q);
  // the two rows whose scores this lane holds, their scales and last keys
  const int n0 = 2 * t, n1 = 2 * t + 1;
  float sc0 = p.scale_log2, sc1 = p.scale_log2;
  if constexpr (F8) {
    sc0 *= __shfl_sync(kAll, q.unscale, n0 * 4);
    sc1 *= __shfl_sync(kAll, q.unscale, n1 * 4);
  }
  const int ctx = sp.L - sp.qlen;
  const int lim0 = n0 < rows ? ctx + n0 / G : -1, lim1 = n1 < rows ? ctx + n1 / G : -1;
  Run2 run;
  run.clear();
  // this warp's blocks: warp, warp + kClusterWarps, ... of the part; 32 ids at
  // a time, the next block on its way while one is scored
  const int mine = n > warp ? (n - warp + kClusterWarps - 1) / kClusterWarps : 0;
  const int32_t* const table = p.block_tables + (size_t)r * p.bt_stride + b0 + warp;
  for (int j0 = 0; j0 < mine; j0 += 32) {
    int pid = -1;
    if (j0 + lane < mine) {
      pid = __ldg(table + (j0 + lane) * kClusterWarps);
      if (pid < 0 || pid >= p.num_blocks) {
        report_error(p.err, PA_DEVERR_BLOCK_ID, b0 + warp + (j0 + lane) * kClusterWarps);
        pid = -1;
      }
    }
    const int nj = min(32, mine - j0);
    auto take = [&](int j, const KFrag<D, F8>& f) {
      const int b = warp + (j0 + j) * kClusterWarps;  // block of the part
      score_block<D, F8, NR>(f, q, t, __shfl_sync(kAll, pid, j) >= 0, (b0 + b) * kBlockSize + g, lim0,
                             lim1, sc0, sc1, score_sm + (size_t)(b * kBlockSize + g) * NR + n0, run);
    };
    stream_blocks<D, F8>(p, h, lane, nj, [&](int j) { return __shfl_sync(kAll, pid, j); }, take);
  }
  run.over_lanes();
  if (g == 0) {
    s_run[warp][n0] = make_float2(run.m0, run.l0);
    s_run[warp][n1] = make_float2(run.m1, run.l1);
  }
  __syncthreads();
  if (threadIdx.x < kFewRows) {
    float m = kNone, l = 0.f;
#pragma unroll
    for (int w = 0; w < kClusterWarps; ++w) m = fmaxf(m, s_run[w][threadIdx.x].x);
#pragma unroll
    for (int w = 0; w < kClusterWarps; ++w)
      l += s_run[w][threadIdx.x].y * ex2_approx(s_run[w][threadIdx.x].x - m);
    s_cta[threadIdx.x] = make_float2(m, l);
  }
  cluster_sync();
  if (threadIdx.x < kFewRows) {
    float m = kNone, l = 0.f;
    for (int k = 0; k < C; ++k) {
      const float2 v = ld_cluster_f2(&s_cta[threadIdx.x], k);
      const float top = fmaxf(m, v.x);
      l = l * ex2_approx(m - top) + v.y * ex2_approx(v.x - top);
      m = top;
    }
    s_row[threadIdx.x] = make_float2(m, threadIdx.x < rows ? 1.f / l : 0.f);
  }
  cluster_sync();  // (no CTA ends while another may still read its shared memory)
  float rm[NR], rl[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    rm[i] = s_row[i].x;
    rl[i] = s_row[i].y;
  }
  const float* const old = p.weights + (size_t)rh * p.weights_stride;
  float* const out = p.out + (size_t)rh * p.weights_stride;
  const int k0 = b0 * kBlockSize, k1 = min(sp.L, (b0 + n) * kBlockSize);
#pragma unroll 2
  for (int key = k0 + (int)threadIdx.x; key < k1; key += 32 * kClusterWarps) {
    const float was = key < ctx ? old[key] : 0.f;
    const float* const s = score_sm + (size_t)(key - k0) * NR;
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < NR; ++i)
      if (i < rows) a += ex2_approx(s[i] - rm[i]) * rl[i];
    out[key] = was + a;
  }
  if (p.num_slots > 0) griddep_wait();
  __threadfence();  // performed before the CTA ends: the next grid may be a programmatic one
}

// Few rows of sequences whose scores outgrow a cluster's shared memory: scores
// and each 256-key chunk's maximum and sum go through global memory to the
// finish kernel.
template <int D, bool F8, int NR>
__global__ void __launch_bounds__(32 * kScoreWarps) pa_weights_score_kernel(const WeightsParams p) {
  griddep_launch_dependents();      // the finish grid waits for this one
  // (the plan, if any, comes before: this grid completes after it)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (p.num_chunks + kScoreWarps - 1) / kScoreWarps;
  const int rh = (int)(blockIdx.x / (unsigned)per), cc = (int)(blockIdx.x - (unsigned)(rh * per));
  const int r = rh / p.num_kv_heads, h = rh - r * p.num_kv_heads;
  const Span sp = get_span(p, r, cc == 0 && h == 0 && threadIdx.x == 0);
  const int G = p.group, rows = sp.qlen * G;
  const int nb = (sp.L + kBlockSize - 1) / kBlockSize;
  const int chunk = cc * kScoreWarps + warp;
  const int b0 = chunk * kChunkBlocks;
  if (!sp.ok || rows == 0 || rows > kFewRows || b0 >= nb) {
    if (p.num_slots > 0) griddep_wait();
    return;
  }
  const int n = min(kChunkBlocks, nb - b0);
  int pid = -1;
  if (lane < n) {
    pid = __ldg(p.block_tables + (size_t)r * p.bt_stride + b0 + lane);
    if (pid < 0 || pid >= p.num_blocks) {
      report_error(p.err, PA_DEVERR_BLOCK_ID, b0 + lane);
      pid = -1;
    }
  }
  const int g = lane >> 2, t = lane & 3;
  QFrag<D, F8> q;
  load_query<D, F8>(p, sp, h, rows, lane, q);
  const int n0 = 2 * t, n1 = 2 * t + 1;  // as in the cluster form
  float sc0 = p.scale_log2, sc1 = p.scale_log2;
  if constexpr (F8) {
    sc0 *= __shfl_sync(kAll, q.unscale, n0 * 4);
    sc1 *= __shfl_sync(kAll, q.unscale, n1 * 4);
  }
  const int ctx = sp.L - sp.qlen;
  const int lim0 = n0 < rows ? ctx + n0 / G : -1, lim1 = n1 < rows ? ctx + n1 / G : -1;
  float* const score = p.scores + ((size_t)rh * p.padded_len + (size_t)b0 * kBlockSize) * NR;
  Run2 run;
  run.clear();
  auto take = [&](int i, const KFrag<D, F8>& f) {
    score_block<D, F8, NR>(f, q, t, __shfl_sync(kAll, pid, i) >= 0, (b0 + i) * kBlockSize + g, lim0,
                           lim1, sc0, sc1, score + (size_t)(i * kBlockSize + g) * NR + n0, run);
  };
  stream_blocks<D, F8>(p, h, lane, n, [&](int j) { return __shfl_sync(kAll, pid, j); }, take);
  run.over_lanes();
  if (g == 0) {  // [row][chunk]: the finish kernel reads a row's chunks side by side
    float2* const st = reinterpret_cast<float2*>(p.stats) + (size_t)rh * kFewRows * p.num_chunks + chunk;
    st[(size_t)n0 * p.num_chunks] = make_float2(run.m0, run.l0);
    st[(size_t)n1 * p.num_chunks] = make_float2(run.m1, run.l1);
  }
  if (p.num_slots > 0) griddep_wait();
}

template <int NR>
__global__ void __launch_bounds__(kFinishThreads) pa_weights_finish_kernel(const WeightsParams p) {
  __shared__ float s_m[kFewRows], s_inv[kFewRows];
  const int per = (p.padded_len + kFinishKeys - 1) / kFinishKeys;
  const int rh = (int)(blockIdx.x / (unsigned)per), cc = (int)(blockIdx.x - (unsigned)(rh * per));
  const int r = rh / p.num_kv_heads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Span sp = get_span(p, r, false);
  const int rows = sp.qlen * p.group;
  // with prompt chunks in the batch their passes follow; they need nothing of
  // this grid and wait for it before they complete
  if (p.num_slots > 0) griddep_launch_dependents();
  griddep_wait();  // the score grid (and, through it, what came before)
  if (!sp.ok || rows == 0 || rows > kFewRows || cc * kFinishKeys >= sp.L) return;
  const int ctx = sp.L - sp.qlen;
  const float* const old = p.weights + (size_t)rh * p.weights_stride;
  float* const out = p.out + (size_t)rh * p.weights_stride;
  // A thread takes up to four rows of a key (two threads a key of eight rows:
  // a warp's loads are then one contiguous run). The next round's scores and
  // sums so far are always on their way: the first round's while the chunks
  // are joined.
  constexpr int LPK = NR == 8 ? 2 : 1, RPL = NR / LPK;
  constexpr int SLOTS = kFinishRound * LPK / kFinishThreads;
  const int half = LPK == 2 ? (tid & 1) : 0;
  const int first = cc * kFinishKeys, last = min(sp.L, first + kFinishKeys);
  struct Round {
    float x[SLOTS][RPL], was[SLOTS];
  };
  auto load = [&](int k0, Round& q) {
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      const int key = k0 + (i * kFinishThreads + tid) / LPK;
      const float* const s = p.scores + ((size_t)rh * p.padded_len + key) * NR + half * RPL;
      q.was[i] = 0.f;
      if (key < last) {
        if constexpr (RPL == 4) {
          const float4 v = __ldcg(reinterpret_cast<const float4*>(s));
          q.x[i][0] = v.x, q.x[i][1] = v.y, q.x[i][2] = v.z, q.x[i][3] = v.w;
        } else {
#pragma unroll
          for (int n = 0; n < RPL; ++n) q.x[i][n] = __ldcg(s + n);
        }
        if (key < ctx && half == 0) q.was[i] = old[key];
      }
    }
  };
  Round ra, rb;
  load(first, ra);
  // warp n joins row n's chunks
  {
    static_assert(kFinishThreads / 32 == kFewRows, "a warp per row");
    const int chunks = (sp.L + kChunkBlocks * kBlockSize - 1) / (kChunkBlocks * kBlockSize);
    const float2* const st = reinterpret_cast<const float2*>(p.stats) +
                             ((size_t)rh * kFewRows + warp) * p.num_chunks;
    float m = kNone, l = 0.f;
    for (int c0 = 0; c0 < chunks; c0 += 128) {  // four chunks per lane and round trip
      float2 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int c = c0 + u * 32 + lane;
        v[u] = c < chunks ? __ldcg(st + c) : make_float2(kNone, 0.f);
      }
      const float k = fmaxf(fmaxf(m, fmaxf(v[0].x, v[1].x)), fmaxf(v[2].x, v[3].x));
      l *= ex2_approx(m - k);
#pragma unroll
      for (int u = 0; u < 4; ++u) l += v[u].y * ex2_approx(v[u].x - k);
      m = k;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float a = __shfl_xor_sync(kAll, m, o), b = __shfl_xor_sync(kAll, l, o);
      const float k = fmaxf(m, a);
      l = l * ex2_approx(m - k) + b * ex2_approx(a - k);
      m = k;
    }
    if (lane == 0) {
      s_m[warp] = m;
      s_inv[warp] = warp < rows ? 1.f / l : 0.f;
    }
  }
  __syncthreads();
  float m[RPL], inv[RPL];
#pragma unroll
  for (int n = 0; n < RPL; ++n) {
    m[n] = s_m[half * RPL + n];
    inv[n] = s_inv[half * RPL + n];
  }
  auto finish = [&](int k0, const Round& q) {
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      const int key = k0 + (i * kFinishThreads + tid) / LPK;
      float a = 0.f;
#pragma unroll
      for (int n = 0; n < RPL; ++n)
        if (half * RPL + n < rows && key < last) a += ex2_approx(q.x[i][n] - m[n]) * inv[n];
      if constexpr (LPK == 2) a += __shfl_xor_sync(kAll, a, 1);
      if (key < last && half == 0) out[key] = q.was[i] + a;
    }
  };
#pragma unroll 1
  for (int k0 = first; k0 < last; k0 += 2 * kFinishRound) {
    if (k0 + kFinishRound < last) load(k0 + kFinishRound, rb);
    finish(k0, ra);
    if (k0 + kFinishRound >= last) break;
    if (k0 + 2 * kFinishRound < last) load(k0 + 2 * kFinishRound, ra);
    finish(k0 + kFinishRound, rb);
  }
  __threadfence();  // performed before the CTA ends: the next grid may be a programmatic one
}

// ---------------------------------------------------------------------------------------
// many rows
// ---------------------------------------------------------------------------------------
// One work item, all its roles need in 32 bytes.
struct WItem {
  int r, h, q0, qlen;
  int ctx;
  int x;      // row tile (pass 1) or key tile (pass 2) of X
  int y0, n;  // Y tiles y0 .. y0 + n - 1
};
static_assert(sizeof(WItem) == 32, "two 16-byte loads");

// The work lists of both passes, longest items first (bucket counts), and the
// number of key parts of every row tile. Row tile rt of request r has slot
// q0 / TOK + r + rt: consecutive requests' slots never meet, since a span of
// qlen tokens has at most (q0 + qlen) / TOK - q0 / TOK + 1 tiles. A warp takes
// a request, its lanes the request's tiles.
__global__ void __launch_bounds__(kPlanThreads) pa_weights_plan_kernel(const WeightsParams p) {
  __shared__ int cnt[2][kBuckets];
  __shared__ int wsum[kPlanThreads / 32], s_fits;
  griddep_launch_dependents();  // the decodes' grids need no plan and wait for this one at their end
  bool none = false;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int TOK = 128 / p.group;
  for (int b = tid; b < kBuckets; b += kPlanThreads) cnt[0][b] = cnt[1][b] = 0;
  for (int i = tid; i < p.num_slots; i += kPlanThreads) p.parts[i] = 0;
  __syncthreads();
  auto put = [&](int k, const WItem& w) -> int {  // a place in the list for every KV head
    return atomicAdd(&cnt[k][min(w.n, kBuckets - 1)], p.num_kv_heads);
  };
  auto write = [&](int k, int at, WItem w) {
    int4* const dst = p.items[k] + 2 * (size_t)at;
    for (int h = 0; h < p.num_kv_heads; ++h) {
      dst[2 * h] = make_int4(w.r, h, w.q0, w.qlen);
      dst[2 * h + 1] = make_int4(w.ctx, w.x, w.y0, w.n);
    }
  };
  // what: 0 counts the items per bucket, 1 writes them
  auto walk = [&](int what) {
    for (int r0 = warp * 32; r0 < p.num_reqs; r0 += kPlanThreads) {
      // 32 requests' spans in one round trip; then those with many rows in turn
      Span mine{0, 0, 0, false};
      if (r0 + lane < p.num_reqs) mine = get_span(p, r0 + lane, what == 0);
      unsigned todo = __ballot_sync(kAll, mine.ok && mine.qlen * p.group > kFewRows);
      while (todo) {
        const int src = __ffs((int)todo) - 1, r = r0 + src;
        todo &= todo - 1;
        const int q0 = __shfl_sync(kAll, mine.q0, src), qlen = __shfl_sync(kAll, mine.qlen, src);
        const int L = __shfl_sync(kAll, mine.L, src), ctx = L - qlen;
        const int nrt = (qlen + TOK - 1) / TOK;
        for (int rt = lane; rt < nrt; rt += 32) {
          const int nkt = (ctx + min(qlen, (rt + 1) * TOK) - 1) / 128 + 1;
          if (what) p.parts[q0 / TOK + r + rt] = (nkt + kSplitTiles - 1) / kSplitTiles;
          for (int i0 = 0; i0 < nkt; i0 += kSplitTiles) {
            const WItem w{r, 0, q0, qlen, ctx, rt, i0, min(kSplitTiles, nkt - i0)};
            const int at = put(0, w);
            if (what) write(0, at, w);
          }
        }
        const int nkt = (L + 127) / 128;
        for (int kt = lane; kt < nkt; kt += 32) {
          const int rt0 = max(0, kt * 128 - ctx) / TOK;  // the first row tile that sees the keys
          const WItem w{r, 0, q0, qlen, ctx, kt, rt0, nrt - rt0};
          const int at = put(1, w);
          if (what) write(1, at, w);
        }
      }
    }
  };
  walk(0);
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {  // first places, longest bucket first
    const int b = kBuckets - 1 - tid;
    const int v = cnt[k][b];
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kAll, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    int below = lane < warp ? wsum[lane] : 0;  // the warps before this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) below += __shfl_xor_sync(kAll, below, o);
    const int before = below + incl - v;
    cnt[k][b] = before;
    // spans that overlap (a query_start_loc that falls) could outgrow the list
    if (tid == kPlanThreads - 1) {
      const bool fits = before + v <= p.max_items[k];
      if (!fits) report_error(p.err, PA_DEVERR_QSL, p.num_reqs);
      p.counts[k] = s_fits = fits ? before + v : 0;
    }
    __syncthreads();
    none = none || s_fits == 0;
    __syncthreads();
  }
  if (none) {  // no such request, or spans that cannot be
    if (tid < 2) p.counts[tid] = 0;
  } else {
    walk(1);
  }
}
static_assert(kBuckets == kPlanThreads, "one bucket per thread");

// Joins the key parts of the row tiles that have more than one.
__global__ void __launch_bounds__(128) pa_weights_join_kernel(const WeightsParams p) {
  griddep_wait();
  const int slot = (int)(blockIdx.x % (unsigned)p.num_slots);
  const int h = (int)(blockIdx.x / (unsigned)p.num_slots);
  const int n = __ldcg(p.parts + slot);
  if (n <= 1) return;
  const size_t at = ((size_t)h * p.num_slots + slot) * 128 + threadIdx.x;
  const size_t step = (size_t)p.num_kv_heads * p.num_slots * 128;
  float m = kNone, l = 0.f;
  for (int i = 0; i < n; ++i) {
    const float2 v = __ldcg(p.partial + (size_t)i * step + at);
    const float k = fmaxf(m, v.x);
    l = l * ex2_approx(m - k) + v.y * ex2_approx(v.x - k);
    m = k;
  }
  p.neg_lse[at] = l > 0.f ? -(m + log2f(l)) : -INFINITY;  // rows past the span: a weight of zero
  __threadfence();
}

template <int D, bool F8>
struct WCfg {
  // Softmax warpgroups. A tile is a chain of TMEM loads, exponentials and sums
  // in one thread; four tiles in work at once hide it (two: 34 us and 30 us for
  // the passes over three 512-token chunks, against PASS1 and PASS2). The E4M3
  // form has converter warps besides, and registers for three.
  static constexpr int NWG = F8 ? 3 : 4;
  static constexpr int THREADS = 64 + 128 * NWG;      // producer, MMA issuer, softmax
  static constexpr int ALL_THREADS = THREADS + (F8 ? 128 : 0);  // + 4 converter warps
  static constexpr int NCH = D / 64;           // 64-element (128-byte) parts of a row
  static constexpr int CHUNK = 128 * 128;
  static constexpr int TILE = NCH * CHUNK;     // a 128-row operand
  static constexpr int NY = 4, NS = 4;         // Y stages, S buffers
  static constexpr int NLSE = NY + NS;         // row statistics: a slot is refilled NY + NS tiles
                                               // later, after the S buffer before it was read
  static constexpr int OFF_X = 0;              // two X operands
  static constexpr int OFF_Y = 2 * TILE;
  static constexpr int OFF_LSE = OFF_Y + NY * TILE;
  static constexpr int OFF_XCH = OFF_LSE + NLSE * 512;
  static constexpr int OFF_BAR = OFF_XCH + (NWG - 1) * 128 * 8;
  static constexpr int B_XF = 0, B_XE = 2, B_YF = 4, B_YE = B_YF + NY, B_SF = B_YE + NY,
                       B_SE = B_SF + NS, B_XCHF = B_SE + NS, B_XCHE = B_XCHF + 1,
                       B_DRAIN = B_XCHE + 1, B_COUNT = B_DRAIN + 1;
  static constexpr int SMEM = OFF_BAR + 8 * B_COUNT + 16 + 1024;
  static_assert(SMEM <= 227 * 1024, "one CTA per SM");
};
}  // namespace

struct WeightsTcParams {
  CUtensorMap tm_q;  // q as [T][Hq][D], box {64, G, 128 / G}, 128B swizzle
  CUtensorMap tm_k;  // k_cache as [blocks * Hkv * 16][D], box {64, 16} (bf16 caches)
  WeightsParams w;
};

namespace {

template <int PASS>
__device__ __forceinline__ WItem get_witem(const WeightsParams& p, int t) {
  const int4 a = __ldcg(p.items[PASS - 1] + 2 * (size_t)t);
  const int4 b = __ldcg(p.items[PASS - 1] + 2 * (size_t)t + 1);
  return WItem{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

__device__ __forceinline__ int snake(int i) {  // rounds of items in alternating direction
  const int g = (int)gridDim.x, b = (int)blockIdx.x;
  return i * g + ((i & 1) ? g - 1 - b : b);
}

template <int D, int PASS, bool F8>
__global__ void __launch_bounds__(WCfg<D, F8>::ALL_THREADS, 1)
    pa_weights_tc_kernel(const __grid_constant__ WeightsTcParams tp) {
  using C = WCfg<D, F8>;
  const WeightsParams& p = tp.w;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;  // swizzled operand tiles
  unsigned char* const gb = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto BAR = [&](int i) -> uint32_t { return base + C::OFF_BAR + 8u * (uint32_t)i; };
  auto wait = [&](int i, int parity) -> bool {
    if (mbar_wait_bounded(BAR(i), (uint32_t)parity & 1u)) return true;
    report_error(p.err, PA_DEVERR_WAIT_TIMEOUT, 3000 + i);
    return false;
  };
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(gb + C::OFF_BAR + 8 * C::B_COUNT);
  constexpr bool kConvY = F8 && PASS == 1, kConvX = F8 && PASS == 2;  // who fills the key operand

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::B_COUNT; ++i) {
      int n = 1;
      if (i >= C::B_SE && i < C::B_SE + C::NS) n = 128;  // a softmax warpgroup
      if (i == C::B_XCHF) n = 128 * (C::NWG - 1);
      if (i == C::B_XCHE) n = 128;
      if (kConvY && i >= C::B_YF && i < C::B_YF + C::NY) n = 4;  // the converter warps
      if (kConvX && i >= C::B_XF && i < C::B_XF + 2) n = 4;
      mbar_init(BAR(i), n);
    }
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  griddep_wait();  // the plan; in pass 2 the row statistics too
  // pass 2 releases nothing early: what follows the call may read its output
  if (PASS == 1) griddep_launch_dependents();
  const int nitems = __ldcg(p.counts + (PASS - 1));
  const int TOK = 128 / p.group;

  // a request's key tile: 16-key blocks by lanes 0 .. 7, one copy per 64 dims
  auto load_keys = [&](const WItem& it, int kt, uint32_t dst, uint32_t bar) {
    const int b = kt * 8 + lane, nb = (it.ctx + it.qlen + kBlockSize - 1) / kBlockSize;
    int pid = -1;
    if (lane < 8 && b < nb) {
      pid = __ldg(p.block_tables + (size_t)it.r * p.bt_stride + b);
      if (pid < 0 || pid >= p.num_blocks) {
        report_error(p.err, PA_DEVERR_BLOCK_ID, b);
        pid = -1;
      }
    }
    const int nload = __popc(__ballot_sync(kAll, pid >= 0));
    if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(nload * C::NCH) * 2048u);
    __syncwarp();
    if (pid >= 0) {
      const int row = (pid * p.num_kv_heads + it.h) * kBlockSize;
#pragma unroll
      for (int c = 0; c < C::NCH; ++c)
        tma_load_2d(dst + c * C::CHUNK + lane * 2048, &tp.tm_k, c * 64, row, bar);
    }
  };
  auto load_rows = [&](const WItem& it, int rt, uint32_t dst, uint32_t bar, int lse_slot) {
    if (lane == 0) {
      mbar_arrive_expect_tx(bar, C::TILE + (PASS == 2 ? 512u : 0u));
#pragma unroll
      for (int c = 0; c < C::NCH; ++c)
        tma_load_3d(dst + c * C::CHUNK, &tp.tm_q, c * 64, it.h * p.group, it.q0 + rt * TOK, bar);
      if (PASS == 2) {
        const int slot = it.q0 / TOK + it.r + rt;
        bulk_g2s(base + C::OFF_LSE + lse_slot * 512,
                 p.neg_lse + ((size_t)it.h * p.num_slots + slot) * 128, 512, bar);
      }
    }
    __syncwarp();
  };

  if (warp == 0) {
    // ======================= TMA producer =======================
    int g = 0, it = 0, nx = 0;  // Y and X operands copied
    bool ok = true;
    for (int t = snake(it); ok && t < nitems; t = snake(++it)) {
      const WItem w = get_witem<PASS>(p, t);
      const int xs = it & 1;
      const uint32_t xdst = base + C::OFF_X + xs * C::TILE;
      if (!kConvX) {
        if (it >= 2 && !wait(C::B_XE + xs, it / 2 - 1)) break;
        ++nx;
        if (PASS == 1)
          load_rows(w, w.x, xdst, BAR(C::B_XF + xs), 0);
        else
          load_keys(w, w.x, xdst, BAR(C::B_XF + xs));
      }
      for (int i = 0; !kConvY && i < w.n; ++i, ++g) {
        const int ys = g % C::NY;
        if (g >= C::NY && !wait(C::B_YE + ys, g / C::NY - 1)) { ok = false; break; }
        const uint32_t ydst = base + C::OFF_Y + ys * C::TILE;
        if (PASS == 1)
          load_keys(w, w.y0 + i, ydst, BAR(C::B_YF + ys));
        else
          load_rows(w, w.y0 + i, ydst, BAR(C::B_YF + ys), g % C::NLSE);
      }
    }
    // every copy issued has landed before the CTA may exit
    for (int j = nx > 2 ? nx - 2 : 0; j < nx; ++j)
      mbar_wait_bounded(BAR(C::B_XF + (j & 1)), (uint32_t)(j / 2) & 1u);
    for (int j = g > C::NY ? g - C::NY : 0; j < g; ++j)
      mbar_wait_bounded(BAR(C::B_YF + j % C::NY), (uint32_t)(j / C::NY) & 1u);
  } else if (warp == 1) {
    // ======================= MMA issuer =======================
    constexpr uint32_t idesc = idesc_bf16_f32(128, 128, false);
    const uint64_t desc = smem_desc_sw128(base, 16, 1024);  // K-major, 8-row groups 1 KB apart
    int g = 0, it = 0;
    bool ok = true;
    for (int t = snake(it); ok && t < nitems; t = snake(++it)) {
      const WItem w = get_witem<PASS>(p, t);
      const int xs = it & 1;
      if (!wait(C::B_XF + xs, it / 2)) break;
      for (int i = 0; i < w.n; ++i, ++g) {
        const int ys = g % C::NY, sb = g % C::NS;
        if (!wait(C::B_YF + ys, g / C::NY)) { ok = false; break; }
        if (g >= C::NS && !wait(C::B_SE + sb, g / C::NS - 1)) { ok = false; break; }
        tc_fence_after();
        if (lane == 0) {
          const uint64_t a0 = desc + ((uint64_t)(C::OFF_X + xs * C::TILE) >> 4);
          const uint64_t b0 = desc + ((uint64_t)(C::OFF_Y + ys * C::TILE) >> 4);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint64_t off = (uint64_t)((ks / 4) * C::CHUNK + (ks % 4) * 32) >> 4;
            umma_bf16(tmem + 128 * sb, a0 + off, b0 + off, idesc, ks > 0 ? 1u : 0u);
          }
          umma_commit(BAR(C::B_SF + sb));
          umma_commit(BAR(C::B_YE + ys));
          if (i + 1 == w.n) umma_commit(BAR(C::B_XE + xs));
        }
        __syncwarp();
      }
    }
    // every MMA issued above has completed before TMEM is released
    if (lane == 0) umma_commit(BAR(C::B_DRAIN));
    __syncwarp();
    mbar_wait_bounded(BAR(C::B_DRAIN), 0);
  } else if (warp < 2 + 4 * C::NWG) {
    // ======================= softmax =======================
    const int wg = (warp - 2) / 4;
    const int q4 = warp & 3;             // the TMEM lane quarter this warp may access
    const int m = q4 * 32 + lane;        // row of X
    const uint32_t trow = ((uint32_t)(q4 * 32) << 16) + tmem;
    float2* const xch = reinterpret_cast<float2*>(gb + C::OFF_XCH);
    const float sc = p.scale_log2;
    const float2 sc2 = make_float2(sc, sc), one2 = make_float2(1.f, 1.f);
    int g = 0, it = 0;
    bool ok = true;
    for (int t = snake(it); ok && t < nitems; t = snake(++it)) {
      const WItem w = get_witem<PASS>(p, t);
      const int L = w.ctx + w.qlen;
      // pass 1: this thread's query row; pass 2: its key
      const int j = w.x * TOK + m / p.group;
      const int lim = PASS == 1 ? (j < w.qlen ? w.ctx + j : -1) : L - 1;
      const int key = w.x * 128 + m;
      float mx = kNone, l = 0.f;
      // pass 2: the key's sum so far, needed at the end
      const size_t okey = ((size_t)w.r * p.num_kv_heads + w.h) * p.weights_stride + key;
      const float was = PASS == 2 && wg == 0 && key < w.ctx ? p.weights[okey] : 0.f;
      for (int i = 0; i < w.n; ++i, ++g) {
        if (g % C::NWG != wg) continue;
        const int sb = g % C::NS;
        if (!wait(C::B_SF + sb, g / C::NS)) { ok = false; break; }
        tc_fence_after();
        const uint32_t s0 = trow + 128 * sb;
        // this thread's columns: lo .. hi - 1
        int lo, hi;
        if (PASS == 1) {
          lo = 0;
          hi = lim - (w.y0 + i) * 128 + 1;
        } else {
          const int j0 = (w.y0 + i) * TOK;  // the tile's first token
          lo = (key - w.ctx - j0) * p.group;
          hi = (w.qlen - j0) * p.group;
        }
        const float4* const nlse =
            reinterpret_cast<const float4*>(gb + C::OFF_LSE + (g % C::NLSE) * 512);
        // 32 columns, the next 32 on their way from TMEM meanwhile
        auto take = [&](int c, uint32_t (&rr)[32]) {
          const int lc = lo - c * 32, hc = hi - c * 32;
          if (__all_sync(kAll, hc <= 0 || lc >= 32)) return;  // no thread sees any of them
          const bool full = __all_sync(kAll, lc <= 0 && hc >= 32);
          float2 acc[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[e] = make_float2(0.f, 0.f);
          if (PASS == 1) {
            float2 x[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
              x[e] = fmul2(make_float2(__uint_as_float(rr[2 * e]), __uint_as_float(rr[2 * e + 1])),
                           sc2);
            if (!full) {
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                x[e].x = 2 * e < hc ? x[e].x : -INFINITY;
                x[e].y = 2 * e + 1 < hc ? x[e].y : -INFINITY;
              }
            }
            float top[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) top[e] = fmaxf(x[e].x, x[e].y);
#pragma unroll
            for (int e = 4; e < 16; ++e) top[e & 3] = fmaxf(top[e & 3], fmaxf(x[e].x, x[e].y));
            const float k = fmaxf(mx, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
            const float2 nk = make_float2(-k, -k);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 d = ffma2(x[e], one2, nk);
              acc[e & 3] = ffma2(make_float2(ex2_approx(d.x), ex2_approx(d.y)), one2, acc[e & 3]);
            }
            l *= ex2_approx(mx - k);
            mx = k;
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 v = nlse[c * 8 + e];
              float2 d0 = ffma2(make_float2(__uint_as_float(rr[4 * e]), __uint_as_float(rr[4 * e + 1])),
                                sc2, make_float2(v.x, v.y));
              float2 d1 =
                  ffma2(make_float2(__uint_as_float(rr[4 * e + 2]), __uint_as_float(rr[4 * e + 3])),
                        sc2, make_float2(v.z, v.w));
              if (!full) {
                d0.x = 4 * e >= lc && 4 * e < hc ? d0.x : -INFINITY;
                d0.y = 4 * e + 1 >= lc && 4 * e + 1 < hc ? d0.y : -INFINITY;
                d1.x = 4 * e + 2 >= lc && 4 * e + 2 < hc ? d1.x : -INFINITY;
                d1.y = 4 * e + 3 >= lc && 4 * e + 3 < hc ? d1.y : -INFINITY;
              }
              const int q = (2 * e) & 3;
              acc[q] = ffma2(make_float2(ex2_approx(d0.x), ex2_approx(d0.y)), one2, acc[q]);
              acc[q + 1] = ffma2(make_float2(ex2_approx(d1.x), ex2_approx(d1.y)), one2, acc[q + 1]);
            }
          }
          l += ((acc[0].x + acc[0].y) + (acc[1].x + acc[1].y)) +
               ((acc[2].x + acc[2].y) + (acc[3].x + acc[3].y));
        };
        uint32_t ra[32], rb[32];
        tmem_ld32(s0, ra);
        tmem_wait_ld();
        tmem_ld32(s0 + 32, rb);
        take(0, ra);
        tmem_wait_ld();
        tmem_ld32(s0 + 64, ra);
        take(1, rb);
        tmem_wait_ld();
        tmem_ld32(s0 + 96, rb);
        take(2, ra);
        tmem_wait_ld();
        // the whole buffer is in registers: the MMAs may have it back
        tc_fence_before();
        if (PASS == 1) mbar_arrive(BAR(C::B_SE + sb));
        take(3, rb);
        if (PASS == 2) mbar_arrive(BAR(C::B_SE + sb));  // the row statistics are read too
      }
      if (!ok) break;
      // the other warpgroups' parts join warpgroup 0's
      if (wg > 0) {
        if (it > 0 && !wait(C::B_XCHE, it - 1)) break;
        xch[(wg - 1) * 128 + m] = make_float2(mx, l);
        mbar_arrive(BAR(C::B_XCHF));
        continue;
      }
      if (!wait(C::B_XCHF, it)) break;
      float2 o[C::NWG - 1];
#pragma unroll
      for (int e = 0; e < C::NWG - 1; ++e) o[e] = xch[e * 128 + m];
      mbar_arrive(BAR(C::B_XCHE));
      if (PASS == 1) {
        float k = mx;
#pragma unroll
        for (int e = 0; e < C::NWG - 1; ++e) k = fmaxf(k, o[e].x);
        l *= ex2_approx(mx - k);
#pragma unroll
        for (int e = 0; e < C::NWG - 1; ++e) l += o[e].y * ex2_approx(o[e].x - k);
        const int slot = w.q0 / TOK + w.r + w.x;
        const size_t at = ((size_t)w.h * p.num_slots + slot) * 128 + m;
        const int nkt = (w.ctx + min(w.qlen, (w.x + 1) * TOK) - 1) / 128 + 1;
        if (nkt <= kSplitTiles)
          p.neg_lse[at] = l > 0.f ? -(k + log2f(l)) : -INFINITY;
        else
          __stcg(p.partial + (size_t)(w.y0 / kSplitTiles) * p.num_kv_heads * p.num_slots * 128 + at,
                 make_float2(k, l));
      } else if (key < L) {
#pragma unroll
        for (int e = 0; e < C::NWG - 1; ++e) l += o[e].y;
        p.out[okey] = was + l;
      }
    }
  } else if constexpr (F8) {
    // ======================= E4M3 converters: the key operand =======================
    const int row = threadIdx.x - C::THREADS;
    int g = 0, it = 0;
    bool ok = true;
    for (int t = snake(it); ok && t < nitems; t = snake(++it)) {
      const WItem w = get_witem<PASS>(p, t);
      auto convert = [&](int kt, unsigned char* dst) {
        const int key = kt * 128 + row;
        bool valid = key < w.ctx + w.qlen;
        size_t src = 0;
        if (valid) {
          const int pid = __ldg(p.block_tables + (size_t)w.r * p.bt_stride + key / kBlockSize);
          if (pid < 0 || pid >= p.num_blocks) {
            report_error(p.err, PA_DEVERR_BLOCK_ID, key / kBlockSize);
            valid = false;
          } else {
            src = (((size_t)pid * p.num_kv_heads + w.h) * kBlockSize + key % kBlockSize) * D;
          }
        }
        widen_e4m3_row<D>(static_cast<const unsigned char*>(p.k_cache) + src, valid, dst, row);
        fence_proxy_async_smem();  // generic-proxy stores -> visible to the tensor core
        __syncwarp();
      };
      if (PASS == 2) {
        const int xs = it & 1;
        if (it >= 2 && !wait(C::B_XE + xs, it / 2 - 1)) break;
        convert(w.x, gb + C::OFF_X + xs * C::TILE);
        if (lane == 0) mbar_arrive(BAR(C::B_XF + xs));
      } else {
        for (int i = 0; i < w.n; ++i, ++g) {
          const int ys = g % C::NY;
          if (g >= C::NY && !wait(C::B_YE + ys, g / C::NY - 1)) { ok = false; break; }
          convert(w.y0 + i, gb + C::OFF_Y + ys * C::TILE);
          if (lane == 0) mbar_arrive(BAR(C::B_YF + ys));
        }
      }
    }
  }
  __threadfence();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------------------
template <typename K, typename P>
cudaError_t launch_chained(K kern, const P& p, long long grid, int threads, int smem,
                           cudaStream_t s) {
  if (grid <= 0 || grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

// Bytes of scores of one CTA of a cluster of C over sequences of padded_len keys.
long long cluster_smem(int padded_len, int C, int rows) {
  const long long blocks = padded_len / kBlockSize;
  return (blocks + C - 1) / C * kBlockSize * rows * 4;
}

template <int D, bool F8, int NR>
cudaError_t launch_few(const WeightsParams& p, cudaStream_t s) {
  const long long rh = (long long)p.num_reqs * p.num_kv_heads;
  if (p.cluster > 0) {
    auto kern = pa_weights_cluster_kernel<D, F8, NR>;
    static bool attr_set[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kClusterSmem);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    if (rh * p.cluster > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rh * p.cluster));
    cfg.blockDim = dim3(32 * kClusterWarps);
    cfg.dynamicSmemBytes = (size_t)cluster_smem(p.padded_len, p.cluster, NR);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    // behind the plan, beside it; without one this is the first grid of the
    // call and no programmatic dependent
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.num_slots > 0 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
  }
  const long long g1 = rh * ((p.num_chunks + kScoreWarps - 1) / kScoreWarps);
  if (g1 > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaError_t e;
  if (p.num_slots > 0) {  // behind the plan, beside it
    e = launch_chained(pa_weights_score_kernel<D, F8, NR>, p, g1, 32 * kScoreWarps, 0, s);
  } else {
    // the first grid of the call is no programmatic dependent: everything the
    // stream did before is complete and visible
    pa_weights_score_kernel<D, F8, NR><<<(unsigned)g1, 32 * kScoreWarps, 0, s>>>(p);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  return launch_chained(pa_weights_finish_kernel<NR>, p,
                        rh * ((p.padded_len + kFinishKeys - 1) / kFinishKeys), kFinishThreads, 0, s);
}

template <int D, bool F8>
cudaError_t launch_few_rows(const WeightsParams& p, cudaStream_t s) {
  switch (p.stored_rows) {
    case 1: return launch_few<D, F8, 1>(p, s);
    case 2: return launch_few<D, F8, 2>(p, s);
    case 4: return launch_few<D, F8, 4>(p, s);
    case 8: return launch_few<D, F8, 8>(p, s);
  }
  return cudaErrorInvalidValue;
}

template <int D, int PASS, bool F8>
cudaError_t launch_pass(const WeightsTcParams& tp, int num_sms, cudaStream_t s) {
  auto kern = pa_weights_tc_kernel<D, PASS, F8>;
  static bool attr_set[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             WCfg<D, F8>::SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  return launch_chained(kern, tp, num_sms, WCfg<D, F8>::ALL_THREADS, WCfg<D, F8>::SMEM, s);
}

template <int D, bool F8>
cudaError_t launch_many(const WeightsParams& p, int num_sms, cudaStream_t s) {
  WeightsTcParams tp;
  tp.w = p;
  {
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)p.num_q_heads, (uint64_t)p.num_tokens};
    const uint64_t str[2] = {(uint64_t)D * 2, (uint64_t)p.num_q_heads * D * 2};
    const uint32_t box[3] = {64, (uint32_t)p.group, (uint32_t)(128 / p.group)};
    if (!encode_tmap_bf16(&tp.tm_q, 3, p.q, dims, str, box)) return cudaErrorInvalidValue;
  }
  if (F8) {
    tp.tm_k = tp.tm_q;  // not used: the converter warps load the codes
  } else {
    const uint64_t rows = (uint64_t)p.num_blocks * p.num_kv_heads * kBlockSize;
    if (!encode_tmap_bf16_2d(&tp.tm_k, p.k_cache, D, rows, (uint64_t)D * 2, 64, kBlockSize))
      return cudaErrorInvalidValue;
  }
  cudaError_t e = launch_pass<D, 1, F8>(tp, num_sms, s);
  if (e == cudaSuccess && p.max_seq_len > 128 * kSplitTiles)
    e = launch_chained(pa_weights_join_kernel, p, (long long)p.num_slots * p.num_kv_heads, 128, 0, s);
  if (e == cudaSuccess) e = launch_pass<D, 2, F8>(tp, num_sms, s);
  return e;
}

template <int D, bool F8>
cudaError_t launch_weights_t(const WeightsParams& p, int num_sms, cudaStream_t s, int* launches) {
  // decodes: score, finish. With chunks: plan, score, finish, pass 1, (join,)
  // pass 2 - the first two need nothing of one another and run together
  *launches = p.cluster > 0 ? 1 : 2;
  cudaError_t e = cudaSuccess;
  if (p.num_slots > 0) {
    *launches += p.max_seq_len > 128 * kSplitTiles ? 4 : 3;
    pa_weights_plan_kernel<<<1, kPlanThreads, 0, s>>>(p);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) e = launch_few_rows<D, F8>(p, s);
  if (e != cudaSuccess || p.num_slots == 0) return e;
  return launch_many<D, F8>(p, num_sms, s);
}

}  // namespace

WeightsLayout weights_layout(int num_reqs, int num_tokens, int num_q_heads, int num_kv_heads,
                             int max_query_len, int max_seq_len) {
  WeightsLayout l;
  const int G = num_q_heads / num_kv_heads;
  const bool many = (long long)max_query_len * G > kFewRows;
  l.stored_rows = max_query_len <= 1 ? G : kFewRows;
  const size_t rh = (size_t)num_reqs * num_kv_heads;
  const size_t blocks = ((size_t)max_seq_len + kBlockSize - 1) / kBlockSize;
  l.num_chunks = (int)((blocks + kChunkBlocks - 1) / kChunkBlocks);
  l.padded_len = (int)(blocks * kBlockSize);
  l.stats_off = 0;
  l.scores_off = pa_align256(sizeof(float) * 2 * kFewRows * rh * (size_t)l.num_chunks);
  l.total = l.scores_off + pa_align256(sizeof(float) * rh * blocks * kBlockSize * l.stored_rows);
  l.counts_off = l.parts_off = l.items1_off = l.items2_off = l.lse_off = l.partial_off = l.total;
  l.num_slots = l.max_items[0] = l.max_items[1] = 0;
  if (!many) return l;
  const size_t tok = (size_t)(128 / G);
  const size_t slots = (size_t)num_tokens / tok + (size_t)num_reqs + 1;
  const size_t tiles = ((size_t)max_seq_len + 127) / 128;
  const size_t parts = (tiles + kSplitTiles - 1) / kSplitTiles;
  l.num_slots = (int)slots;
  l.max_items[0] = (int)(slots * parts * num_kv_heads);
  l.max_items[1] = (int)(rh * tiles);
  l.parts_off = l.counts_off + 256;
  l.items1_off = l.parts_off + pa_align256(sizeof(int) * slots);
  l.items2_off = l.items1_off + pa_align256(2 * sizeof(int4) * slots * parts * num_kv_heads);
  l.lse_off = l.items2_off + pa_align256(2 * sizeof(int4) * rh * tiles);
  l.partial_off = l.lse_off + pa_align256(sizeof(float) * 128 * slots * num_kv_heads);
  l.total = l.partial_off +
            (parts > 1 ? pa_align256(sizeof(float2) * 128 * slots * num_kv_heads * parts) : 0);
  return l;
}

cudaError_t launch_weights(WeightsParams p, int head_dim, bool f8, int num_sms, cudaStream_t s,
                           int* launches) {
  // CTAs per (request, KV head) of the few-rows form: enough that a CTA's
  // scores leave room for three CTAs on an SM and the grid has at least two
  // waves of them; 0: they do not fit even eight CTAs (kClusterSmem each)
  const long long rh = (long long)p.num_reqs * p.num_kv_heads;
  p.cluster = 1;
  while (p.cluster < 8 && (cluster_smem(p.padded_len, p.cluster, p.stored_rows) > kClusterSmem ||
                           (rh * p.cluster < 6LL * num_sms && p.padded_len > 1024 * p.cluster)))
    p.cluster *= 2;
  if (cluster_smem(p.padded_len, p.cluster, p.stored_rows) > kClusterSmem) p.cluster = 0;
  if (head_dim == 128)
    return f8 ? launch_weights_t<128, true>(p, num_sms, s, launches)
              : launch_weights_t<128, false>(p, num_sms, s, launches);
  return f8 ? launch_weights_t<64, true>(p, num_sms, s, launches)
            : launch_weights_t<64, false>(p, num_sms, s, launches);
}

}  // namespace pa
