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
// exponentials per (row, key). Two passes of one tcgen05 kernel: a pair of
// stationary 128-row operands X against a stream of 128-row operands Y, S = X
// Y^T into TMEM, one thread per row of X with no exchange between threads:
//   pass 1  X = 2 x 128 query rows (G heads x 128 / G tokens), Y = key tiles:
//           the thread keeps its query's running maximum and sum -> lse.
//   pass 2  X = 2 x 128 keys, Y = the query row tiles that see them: the
//           thread sums exp2(s - lse) over its key's columns and writes the
//           key's weight.
// A pair's Y tiles are cut into parts where that evens out the CTAs' shares (a
// planner kernel decides). A part leaves its 32 rows' results per warp in the
// workspace and counts itself done; the warp that counts last joins all parts,
// in their order, so the result does not depend on which that is.
// X comes in pairs because a Y tile costs more to bring (its copies take the
// TMA unit some 40 ns each, whatever their size, and a stage about 2 us to turn
// around) than one 128 x 128 product on it takes. Two warps issue the MMAs:
// between the products of a step one warp's waits, fences and commits take as
// long as the products. Warpgroup w takes X tile w % 2 and half w / 2 of the
// columns; it copies its 64 columns to registers, gives the S buffer back and
// only then takes exponentials, so that the next steps' MMAs run meanwhile.
// Three 512-token chunks on 0, 1024 and 2048 keys, 32 / 8 heads: single X tiles
// and one issuer 63 us per call, pairs 55.5, two issuers 54, halves of the
// columns 53. A step (two products) then takes about 1900 cycles against 1024 of
// the tensor pipe and of the special-function units each (per-step clock probe;
// leaving out every exponential gains 4 us of the 53, so it is neither alone):
// the products' operands and the copies load shared memory for about 1250.
#include <cuda.h>

#include <cfloat>

#include "pa_internal.h"
#include "ptx.cuh"

namespace pa {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kFewRows = 8;          // rows the bandwidth-bound form takes (the MMA's N)
constexpr int kChunkBlocks = 16;     // 16-key blocks per warp
constexpr int kScoreWarps = 4;
constexpr int kClusterWarps = 8;
// Scores of one CTA of a cluster, at most. Two CTAs share an SM (their registers),
// but what 112 KB each would keep on the SM are few CTAs with long parts: 8 x 24576
// keys at G = 8 59.1 -> 56.1 us, 1 x 28672 18.6 -> 38.4, 8 x 49152 at G = 4 145 ->
// 163, against the form through global memory.
constexpr int kClusterSmem = 64 * 1024;
constexpr int kFinishThreads = 256;

constexpr int kFinishRound = 1024;   // keys of one round of a finish CTA
constexpr int kFinishKeys = 4 * kFinishRound;  // keys of one finish CTA (joining the chunks costs
                                                 // each CTA the same, whatever its keys)
constexpr int kMaxParts = 16;        // parts of a pair's Y tiles
constexpr int kMinPart = 8;          // Y tiles of a part in pass 1, at least (pass 2: 2)
constexpr int kMaxUnits = 512;       // pairs of pass 2 that may be cut: only few of them are
constexpr int kPlanThreads = 1024;
constexpr int kBuckets = 1024;
constexpr float kNone = -FLT_MAX;    // a running maximum before the first key

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
  // The first grid of the call waits for the grid before it; behind a plan,
  // which has waited, this one does so only to complete after it, and lets the
  // chunks' passes, which need nothing of it, take their places.
  if (p.num_slots == 0)
    griddep_wait();
  else
    griddep_launch_dependents();
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
      const float2 v = ld_cluster_f2(cluster_addr(&s_cta[threadIdx.x], k));
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
}

// Few rows of sequences whose scores outgrow a cluster's shared memory: scores
// and each 256-key chunk's maximum and sum go through global memory to the
// finish kernel.
template <int D, bool F8, int NR>
__global__ void __launch_bounds__(32 * kScoreWarps) pa_weights_score_kernel(const WeightsParams p) {
  // the first grid of the call waits for the grid before it; behind a plan,
  // which has waited, this one does so only to complete after it
  if (p.num_slots == 0) griddep_wait();
  griddep_launch_dependents();  // the finish grid waits for this one
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
}

// ---------------------------------------------------------------------------------------
// many rows
// ---------------------------------------------------------------------------------------
// One work item, all its roles need in 48 bytes.
struct WItem {
  int r, h, q0, qlen;
  int ctx;
  int x;            // first row tile (pass 1) or key tile (pass 2) of the X pair
  int y0, n;        // Y tiles y0 .. y0 + n - 1
  int part, parts;  // which part of the pair's Y tiles, of how many
  int unit;         // pass 2, parts > 1: the pair's place in the partial sums
  int pad;
};
static_assert(sizeof(WItem) == 48, "three 16-byte loads");

// The work lists of both passes, longest items first (bucket counts). Row tile
// rt of request r has slot q0 / TOK + r + rt: consecutive requests' slots never
// meet, since a span of qlen tokens has at most (q0 + qlen) / TOK - q0 / TOK + 1
// tiles. Request r belongs to warp r % 32, whose lanes take its pairs if it has
// many rows: chunks stand side by side in a batch, and so go to different
// warps. Pairs are cut into parts (of half a CTA's even share) only where there
// are fewer of them than half the CTAs: joining costs a warpgroup about 3000
// cycles per part, two steps' time, and on three 512-token chunks (192 and 144
// pairs) it took more than the evener shares gave (65.7 us against 52.9).
__global__ void __launch_bounds__(kPlanThreads) pa_weights_plan_kernel(const WeightsParams p) {
  __shared__ int cnt[2][kBuckets];
  __shared__ int wsum[kPlanThreads / 32], s_fits;
  __shared__ int s_steps[2], s_pairs[2], s_unit;
  griddep_wait();               // the first grid of the call waits for the grid before it
  griddep_launch_dependents();  // the decodes' grids need no plan and wait for this one at their end
  bool none = false;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int TOK = 128 / p.group, tsh = __ffs(TOK) - 1;  // a power of two
  for (int b = tid; b < kBuckets; b += kPlanThreads) cnt[0][b] = cnt[1][b] = 0;
  for (int i = tid; i < p.num_counters; i += kPlanThreads) p.counters[i] = 0;
  if (tid < 2) s_steps[tid] = s_pairs[tid] = 0;
  if (tid == 2) s_unit = 0;
  __syncthreads();
  // the spans; a batch of up to 1024 requests keeps them in registers
  Span kept{0, 0, 0, false};
  auto span_of = [&](int r, bool first) {
    if (r >= p.num_reqs) return Span{0, 0, 0, false};
    return first || r >= kPlanThreads ? get_span(p, r, first) : kept;
  };
  static_assert(kPlanThreads == 1024, "32 warps of 32 lanes");
  const int r_of = warp + 32 * lane;  // of each 1024 requests
  for (int r = r_of; r < p.num_reqs; r += kPlanThreads) {
    const Span s = span_of(r, true);
    if (r < kPlanThreads) kept = s;
    if (!s.ok || s.qlen * p.group <= kFewRows) continue;
    // pairs, and their Y tiles as if these grew evenly from the first to the last
    const int ctx = s.L - s.qlen, nrt = (s.qlen + TOK - 1) >> tsh, nkt = (s.L + 127) / 128;
    const int pairs1 = (nrt + 1) / 2 * p.num_kv_heads, pairs2 = (nkt + 1) / 2 * p.num_kv_heads;
    const int nk0 = (ctx + min(s.qlen, 2 * TOK) - 1) / 128 + 1;
    const int rt0 = max(0, (nkt - 1) * 128 - ctx) >> tsh;
    atomicAdd(&s_pairs[0], pairs1);
    atomicAdd(&s_pairs[1], pairs2);
    atomicAdd(&s_steps[0], pairs1 * (nk0 + nkt) / 2);
    atomicAdd(&s_steps[1], pairs2 * (2 * nrt - rt0) / 2);
  }
  __syncthreads();
  int len1 = 0, len2 = 0;  // Y tiles of a part
  auto item = [&](int k, bool fill, WItem w) {
    const int at = atomicAdd(&cnt[k][min(w.n, kBuckets - 1)], p.num_kv_heads);  // every KV head's
    if (!fill) return;
    int4* const dst = p.items[k] + 3 * (size_t)at;
    for (int h = 0; h < p.num_kv_heads; ++h) {
      dst[3 * h] = make_int4(w.r, h, w.q0, w.qlen);
      dst[3 * h + 1] = make_int4(w.ctx, w.x, w.y0, w.n);
      dst[3 * h + 2] = make_int4(w.part, w.parts, w.unit + h, 0);
    }
  };
  // fill: write the items, else count them per bucket
  auto walk = [&](bool fill) {
    for (int r0 = 0; r0 < p.num_reqs; r0 += kPlanThreads) {
      const Span mine = span_of(r0 + r_of, false);
      unsigned todo = __ballot_sync(kAll, mine.ok && mine.qlen * p.group > kFewRows);
      while (todo) {
        const int src = __ffs((int)todo) - 1, r = r0 + warp + 32 * src;
        todo &= todo - 1;
        const int q0 = __shfl_sync(kAll, mine.q0, src), qlen = __shfl_sync(kAll, mine.qlen, src);
        const int L = __shfl_sync(kAll, mine.L, src), ctx = L - qlen;
        const int nrt = (qlen + TOK - 1) >> tsh;
        for (int rt = 2 * lane; rt < nrt; rt += 64) {  // pairs of row tiles
          const int nkt = (ctx + min(qlen, (rt + 2) * TOK) - 1) / 128 + 1;
          const int parts = (nkt - 1) / len1 + 1, per = (nkt + parts - 1) / parts;
          for (int i = 0; i < parts; ++i)
            item(0, fill,
                 WItem{r, 0, q0, qlen, ctx, rt, i * per, min(per, nkt - i * per), i, parts, 0, 0});
        }
        const int nkt = (L + 127) / 128;
        for (int kt = 2 * lane; kt < nkt; kt += 64) {  // pairs of key tiles
          const int rt0 = max(0, kt * 128 - ctx) >> tsh;  // the first row tile that sees the keys
          const int n = nrt - rt0, parts = (n - 1) / len2 + 1, per = (n + parts - 1) / parts;
          const int unit = parts > 1 && fill ? atomicAdd(&s_unit, p.num_kv_heads) : 0;
          for (int i = 0; i < parts; ++i)
            item(1, fill,
                 WItem{r, 0, q0, qlen, ctx, kt, rt0 + i * per, min(per, n - i * per), i, parts, unit, 0});
        }
      }
    }
  };
  {
    const int most1 = (p.max_seq_len + 127) / 128, most2 = (p.max_query_len + TOK - 1) >> tsh;
    len1 = s_pairs[0] >= p.num_sms / 2
               ? 0x40000000
               : max(max(kMinPart, s_steps[0] / (2 * p.num_sms) + 1), (most1 + kMaxParts - 1) / kMaxParts);
    // (fewer pairs than SMs: the units fit)
    len2 = s_pairs[1] >= p.num_sms / 2 || s_pairs[1] > kMaxUnits
               ? 0x40000000
               : max(max(2, s_steps[1] / (2 * p.num_sms) + 1), (most2 + kMaxParts - 1) / kMaxParts);
  }
  walk(false);
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
    walk(true);
  }
}
static_assert(kBuckets == kPlanThreads, "one bucket per thread");

template <int D, bool F8>
struct WCfg {
  // Softmax warpgroups: warpgroup w works on X tile w % 2 of the pair and on part
  // w / 2 of the SPLIT its columns are in. The E4M3 form has converter warps
  // besides.
  static constexpr int NWG = F8 ? 2 : 4;
  static constexpr int SPLIT = NWG / 2;
  static constexpr int SOFT0 = 3;                     // first softmax warp: after the producer
                                                      // and two MMA issuers
  static constexpr int THREADS = 32 * SOFT0 + 128 * NWG;
  static constexpr int ALL_THREADS = THREADS + (F8 ? 128 : 0);  // + 4 converter warps
  static constexpr int NCH = D / 64;           // 64-element (128-byte) parts of a row
  static constexpr int CHUNK = 128 * 128;
  static constexpr int TILE = NCH * CHUNK;     // a 128-row operand
  static constexpr int NY = 4, NS = 4;         // Y stages, S buffers
  // Row statistics (pass 2): slot g % NLSE is refilled for Y tile g + 8, once
  // every softmax warp has taken the scores of tile g + 4, hence finished tile
  // g + 3.
  static constexpr int NLSE = 8;
  static_assert(NY == 4 && NS == 4, "what the slots' reuse relies on");
  static constexpr int OFF_X = 0;              // the pair of X operands
  // layout of the key operand: 8-row groups KSBO apart, 64-element parts KHALF
  // apart. A 128-dim bf16 block of 16 keys lands by one 4 KB copy as [group]
  // [part][8 rows][128 B]; otherwise whole parts lie one after the other.
  static constexpr bool ONE_COPY = D == 128 && !F8;
  static constexpr int KSBO = ONE_COPY ? 2048 : 1024, KHALF = ONE_COPY ? 1024 : CHUNK;
  static constexpr int OFF_Y = 2 * TILE;
  static constexpr int OFF_LSE = OFF_Y + NY * TILE;
  static constexpr int OFF_XCH = OFF_LSE + NLSE * 512;
  static constexpr int OFF_BAR = OFF_XCH + 2 * 128 * 8;
  static constexpr int B_XF = 0, B_XE = 1, B_YF = 2, B_YE = B_YF + NY, B_SF = B_YE + NY,
                       B_SE = B_SF + NS, B_XCHF = B_SE + NS, B_XCHE = B_XCHF + 2,
                       B_DRAIN = B_XCHE + 2, B_COUNT = B_DRAIN + 1;
  static constexpr int SMEM = OFF_BAR + 8 * B_COUNT + 16 + 1024;
  static_assert(SMEM <= 227 * 1024, "one CTA per SM");
};
}  // namespace

struct WeightsTcParams {
  CUtensorMap tm_q;  // q as [T][Hq][D], box {64, G, 128 / G}, 128B swizzle
  // bf16 caches: k_cache as [blocks * Hkv * 16][64], box {64, 16}; of head_dim
  // 128 as {64, 8 rows, 2 parts, 8-row groups}, box {64, 8, 2, 2}
  CUtensorMap tm_k;
  WeightsParams w;
};

namespace {

template <int PASS>
__device__ __forceinline__ WItem get_witem(const WeightsParams& p, int t) {
  const int4* const src = p.items[PASS - 1] + 3 * (size_t)t;
  const int4 a = __ldcg(src), b = __ldcg(src + 1), c = __ldcg(src + 2);
  return WItem{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, 0};
}

// Counts a part of `parts` as done for the 32 rows of this warp, whose results
// are stored; true for the one that counts last, which then sees all of them.
__device__ __forceinline__ bool last_part(int* counter, int parts, int lane) {
  __threadfence();
  __syncwarp();
  int n = 0;
  if (lane == 0) n = atomicAdd(counter, 1);
  n = __shfl_sync(kAll, n, 0);
  if (n != parts - 1) return false;
  __threadfence();
  return true;
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
      if (i >= C::B_SE && i < C::B_SE + C::NS) n = 4 * C::SPLIT;  // the warps that share it
      if (i >= C::B_XCHF && i < C::B_XCHE + 2) n = 128;
      if (kConvY && i >= C::B_YF && i < C::B_YF + C::NY) n = 4;  // the converter warps
      if (kConvX && i == C::B_XF) n = 4;
      // every softmax warp has its scores of a Y tile, whose products are done then
      if (i >= C::B_YE && i < C::B_YE + C::NY) n = 8 * C::SPLIT;
      if (i == C::B_XE || i == C::B_DRAIN) n = 2;  // the MMA issuers
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

  // the block id of this lane's block of a key tile (lanes 0 .. 7), -1: none
  auto key_block = [&](const WItem& it, int kt) -> int {
    const int b = kt * 8 + lane, nb = (it.ctx + it.qlen + kBlockSize - 1) / kBlockSize;
    int pid = -1;
    if (lane < 8 && b < nb) {
      pid = __ldg(p.block_tables + (size_t)it.r * p.bt_stride + b);
      if (pid < 0 || pid >= p.num_blocks) {
        report_error(p.err, PA_DEVERR_BLOCK_ID, b);
        pid = -1;
      }
    }
    return pid;
  };
  auto copy_block = [&](const WItem& it, int pid, uint32_t dst, uint32_t bar) {
    if (pid < 0) return;
    if constexpr (C::ONE_COPY) {
      const int grp = (pid * p.num_kv_heads + it.h) * (kBlockSize / 8);  // the block's first group
      tma_load_4d(dst + lane * 2 * C::KSBO, &tp.tm_k, 0, 0, 0, grp, bar);
    } else {
      const int row = (pid * p.num_kv_heads + it.h) * kBlockSize;
#pragma unroll
      for (int c = 0; c < C::NCH; ++c)
        tma_load_2d(dst + c * C::CHUNK + lane * 2048, &tp.tm_k, c * 64, row, bar);
    }
  };
  auto copy_rows = [&](const WItem& it, int rt, uint32_t dst, uint32_t bar) {  // one thread
#pragma unroll
    for (int c = 0; c < C::NCH; ++c)
      tma_load_3d(dst + c * C::CHUNK, &tp.tm_q, c * 64, it.h * p.group, it.q0 + rt * TOK, bar);
  };
  constexpr uint32_t kBlockBytes = (uint32_t)C::NCH * 2048u;

  if (warp == 0) {
    // ======================= TMA producer =======================
    int g = 0, it = 0, nx = 0;  // Y operands and X pairs copied
    bool ok = true;
    for (int t = snake(it); ok && t < nitems; t = snake(++it)) {
      const WItem w = get_witem<PASS>(p, t);
      const uint32_t xdst = base + C::OFF_X, xbar = BAR(C::B_XF);
      if (!kConvX) {
        int id0 = -1, id1 = -1;
        if (PASS == 2) {
          id0 = key_block(w, w.x);
          id1 = key_block(w, w.x + 1);
        }
        if (it >= 1 && !wait(C::B_XE, it - 1)) break;
        ++nx;
        if (PASS == 1) {
          // a second tile past the span reads rows of other spans (zeros past
          // the batch): nothing of it is used
          if (lane == 0) {
            mbar_arrive_expect_tx(xbar, 2u * C::TILE);
            copy_rows(w, w.x, xdst, xbar);
            copy_rows(w, w.x + 1, xdst + C::TILE, xbar);
          }
        } else {
          const int nload = __popc(__ballot_sync(kAll, id0 >= 0)) + __popc(__ballot_sync(kAll, id1 >= 0));
          if (lane == 0) mbar_arrive_expect_tx(xbar, (uint32_t)nload * kBlockBytes);
          __syncwarp();
          copy_block(w, id0, xdst, xbar);
          copy_block(w, id1, xdst + C::TILE, xbar);
        }
        __syncwarp();
      }
      int id = !kConvY && PASS == 1 ? key_block(w, w.y0) : -1;
      for (int i = 0; !kConvY && i < w.n; ++i, ++g) {
        const int ys = g % C::NY;
        // the next tile's block ids are on their way while this one waits
        const int next = PASS == 1 && i + 1 < w.n ? key_block(w, w.y0 + i + 1) : -1;
        if (g >= C::NY && !wait(C::B_YE + ys, g / C::NY - 1)) { ok = false; break; }
        const uint32_t ydst = base + C::OFF_Y + ys * C::TILE, ybar = BAR(C::B_YF + ys);
        if (PASS == 1) {
          const int nload = __popc(__ballot_sync(kAll, id >= 0));
          if (lane == 0) mbar_arrive_expect_tx(ybar, (uint32_t)nload * kBlockBytes);
          __syncwarp();
          copy_block(w, id, ydst, ybar);
          id = next;
        } else if (lane == 0) {
          const int rt = w.y0 + i, slot = w.q0 / TOK + w.r + rt;
          mbar_arrive_expect_tx(ybar, C::TILE + 512u);
          copy_rows(w, rt, ydst, ybar);
          bulk_g2s(base + C::OFF_LSE + (g % C::NLSE) * 512,
                   p.neg_lse + ((size_t)w.h * p.num_slots + slot) * 128, 512, ybar);
        }
        __syncwarp();
      }
    }
    // every copy issued has landed before the CTA may exit
    if (nx > 0) mbar_wait_bounded(BAR(C::B_XF), (uint32_t)(nx - 1) & 1u);
    for (int j = g > C::NY ? g - C::NY : 0; j < g; ++j)
      mbar_wait_bounded(BAR(C::B_YF + j % C::NY), (uint32_t)(j / C::NY) & 1u);
  } else if (warp < C::SOFT0) {
    // ======================= MMA issuers =======================
    // Warp 1 + xi issues the products on X tile xi: one warp's waits, fences and
    // commits between the products take as long as the products, two overlap them.
    const int xi = warp - 1;
    constexpr uint32_t idesc = idesc_bf16_f32(128, 128, false);
    // K-major operands: rows as TMA lands them, and the key operand
    const uint64_t qdesc = smem_desc_sw128(base, 16, 1024), kdesc = smem_desc_sw128(base, 16, C::KSBO);
    const uint64_t a0 = (PASS == 1 ? qdesc : kdesc) + ((uint64_t)(C::OFF_X + xi * C::TILE) >> 4);
    int g = 0, it = 0;
    bool ok = true;
    for (int t = snake(it); ok && t < nitems; t = snake(++it)) {
      const int n = get_witem<PASS>(p, t).n;
      if (!wait(C::B_XF, it)) break;
      for (int i = 0; i < n; ++i, ++g) {
        const int ys = g % C::NY, gs = 2 * g + xi, sb = gs % C::NS;
        if (!wait(C::B_YF + ys, g / C::NY)) { ok = false; break; }
        if (gs >= C::NS && !wait(C::B_SE + sb, gs / C::NS - 1)) { ok = false; break; }
        tc_fence_after();
        if (lane == 0) {
          const uint64_t b0 = (PASS == 1 ? kdesc : qdesc) + ((uint64_t)(C::OFF_Y + ys * C::TILE) >> 4);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint64_t qo = (uint64_t)((ks / 4) * C::CHUNK + (ks % 4) * 32) >> 4;
            const uint64_t ko = (uint64_t)((ks / 4) * C::KHALF + (ks % 4) * 32) >> 4;
            umma_bf16(tmem + 128 * sb, a0 + (PASS == 1 ? qo : ko), b0 + (PASS == 1 ? ko : qo), idesc,
                      ks > 0 ? 1u : 0u);
          }
          umma_commit(BAR(C::B_SF + sb));
        }
        __syncwarp();
      }
      if (!ok) break;
      if (lane == 0) umma_commit(BAR(C::B_XE));  // once this issuer's products on the pair are done
      __syncwarp();
    }
    // every MMA issued above has completed before TMEM is released
    if (lane == 0) umma_commit(BAR(C::B_DRAIN));
    __syncwarp();
    mbar_wait_bounded(BAR(C::B_DRAIN), 0);
  } else if (warp < C::SOFT0 + 4 * C::NWG) {
    // ======================= softmax =======================
    const int wg = (warp - C::SOFT0) / 4;
    const int xi = wg & 1;               // its X tile of the pair
    const int q4 = warp & 3;             // the TMEM lane quarter this warp may access
    const int m = q4 * 32 + lane;        // row of X
    const uint32_t trow = ((uint32_t)(q4 * 32) << 16) + tmem;
    float2* const xch = reinterpret_cast<float2*>(gb + C::OFF_XCH) + xi * 128;
    const float sc = p.scale_log2;
    const float2 sc2 = make_float2(sc, sc), one2 = make_float2(1.f, 1.f);
    const bool ordered = sc > 0.f;  // the largest raw score is the largest scaled one
    const float2 msc = ordered ? sc2 : one2;
    int g = 0, it = 0;
    bool ok = true;
    for (int t = snake(it); ok && t < nitems; t = snake(++it)) {
      const WItem w = get_witem<PASS>(p, t);
      const int L = w.ctx + w.qlen;
      // pass 1: this thread's query row; pass 2: its key
      const int xt = w.x + xi;
      const int j = xt * TOK + m / p.group;
      const int lim = PASS == 1 ? (j < w.qlen ? w.ctx + j : -1) : L - 1;
      const int key = xt * 128 + m;
      float mx = kNone, l = 0.f;
      // pass 2: the key's sum so far, needed at the end
      const size_t okey = ((size_t)w.r * p.num_kv_heads + w.h) * p.weights_stride + key;
      const float was = PASS == 2 && wg < 2 && key < w.ctx ? p.weights[okey] : 0.f;
      for (int i = 0; i < w.n; ++i, ++g) {
        const int gs = 2 * g + xi, sb = gs % C::NS;
        if (!wait(C::B_SF + sb, gs / C::NS)) { ok = false; break; }
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
        const bool whole = __all_sync(kAll, lo <= 0 && hi >= 128);
        const float4* const nlse =
            reinterpret_cast<const float4*>(gb + C::OFF_LSE + (g % C::NLSE) * 512);
        // 32 columns
        auto take = [&](int c, uint32_t (&rr)[32]) {
          const int lc = lo - c * 32, hc = hi - c * 32;
          if (!whole && __all_sync(kAll, hc <= 0 || lc >= 32)) return;  // no thread sees any
          const bool full = whole || __all_sync(kAll, lc <= 0 && hc >= 32);
          float2 acc[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[e] = make_float2(0.f, 0.f);
          if (PASS == 1) {
            float2 x[16];  // raw scores; scaled ones where the scale does not keep their order
#pragma unroll
            for (int e = 0; e < 16; ++e)
              x[e] = make_float2(__uint_as_float(rr[2 * e]), __uint_as_float(rr[2 * e + 1]));
            if (!ordered) {
#pragma unroll
              for (int e = 0; e < 16; ++e) x[e] = fmul2(x[e], sc2);
            }
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
            const float k =
                fmaxf(mx, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * msc.x);
            const float2 nk = make_float2(-k, -k);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 d = ffma2(x[e], msc, nk);
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
        if constexpr (C::SPLIT == 2) {
          const int c0 = wg >= 2 ? 2 : 0;
          tmem_ld32(s0 + c0 * 32, ra);
          tmem_ld32(s0 + c0 * 32 + 32, rb);
          tmem_wait_ld();
          // the columns are in registers: the MMAs may have the buffer back
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(BAR(C::B_SE + sb));
            mbar_arrive(BAR(C::B_YE + g % C::NY));
          }
          take(c0, ra);
          take(c0 + 1, rb);
        } else {
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
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(BAR(C::B_SE + sb));
            mbar_arrive(BAR(C::B_YE + g % C::NY));
          }
          take(3, rb);
        }
      }
      if (!ok) break;
      // the part of the warpgroup that took the other columns
      float2 o = make_float2(kNone, 0.f);
      if (C::SPLIT == 2) {
        if (wg >= 2) {
          if (it > 0 && !wait(C::B_XCHE + xi, it - 1)) break;
          xch[m] = make_float2(mx, l);
          mbar_arrive(BAR(C::B_XCHF + xi));
          continue;
        }
        if (!wait(C::B_XCHF + xi, it)) break;
        o = xch[m];
        mbar_arrive(BAR(C::B_XCHE + xi));
      }
      if (PASS == 1) {
        const float k = fmaxf(mx, o.x);
        l = l * ex2_approx(mx - k) + o.y * ex2_approx(o.x - k);
        // A row past the span leaves anything (no key takes it); one with a NaN or an
        // infinity among its scores a NaN, which reaches every key that it sees.
        if (xt * TOK >= w.qlen) continue;  // the pair's second tile is past the span
        const int slot = w.q0 / TOK + w.r + xt;
        const size_t at = ((size_t)w.h * p.num_slots + slot) * 128 + m;
        if (w.parts > 1) {
          const size_t step = (size_t)p.num_kv_heads * p.num_slots * 128;
          __stcg(p.partial + (size_t)w.part * step + at, make_float2(k, l));
          if (!last_part(p.counters + ((size_t)w.h * p.num_slots + slot) * 4 + q4, w.parts, lane)) continue;
          float top = kNone, sum = 0.f;
          for (int i = 0; i < w.parts; ++i) {
            const float2 v = __ldcg(p.partial + (size_t)i * step + at);
            const float t2 = fmaxf(top, v.x);
            sum = sum * ex2_approx(top - t2) + v.y * ex2_approx(v.x - t2);
            top = t2;
          }
          p.neg_lse[at] = -(top + log2f(sum));
        } else {
          p.neg_lse[at] = -(k + log2f(l));
        }
      } else {
        l += o.y;
        if (w.parts > 1) {
          float* const sums = p.sums + (size_t)w.unit * (kMaxParts * 256) + xi * 128 + m;
          __stcg(sums + w.part * 256, l);
          if (!last_part(p.counters + (size_t)p.num_kv_heads * p.num_slots * 4 + w.unit * 8 + xi * 4 + q4,
                         w.parts, lane))
            continue;
          l = 0.f;
          for (int i = 0; i < w.parts; ++i) l += __ldcg(sums + i * 256);
        }
        if (key < L) p.out[okey] = was + l;
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
        if (it >= 1 && !wait(C::B_XE, it - 1)) break;
        convert(w.x, gb + C::OFF_X);
        convert(w.x + 1, gb + C::OFF_X + C::TILE);
        if (lane == 0) mbar_arrive(BAR(C::B_XF));
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
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p);
  }
  const long long g1 = rh * ((p.num_chunks + kScoreWarps - 1) / kScoreWarps);
  if (g1 > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaError_t e = launch_chained(pa_weights_score_kernel<D, F8, NR>, p, g1, 32 * kScoreWarps, 0, s);
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
    if (D == 128) {
      const uint64_t cd[4] = {64, 8, 2, rows / 8}, cs[3] = {D * 2, 128, 8 * D * 2};
      const uint32_t cb[4] = {64, 8, 2, kBlockSize / 8};
      if (!encode_tmap_bf16(&tp.tm_k, 4, p.k_cache, cd, cs, cb)) return cudaErrorInvalidValue;
    } else if (!encode_tmap_bf16_2d(&tp.tm_k, p.k_cache, D, rows, (uint64_t)D * 2, 64, kBlockSize))
      return cudaErrorInvalidValue;
  }
  cudaError_t e = launch_pass<D, 1, F8>(tp, num_sms, s);
  if (e == cudaSuccess) e = launch_pass<D, 2, F8>(tp, num_sms, s);
  return e;
}

template <int D, bool F8>
cudaError_t launch_weights_t(const WeightsParams& p, int num_sms, cudaStream_t s, int* launches) {
  // decodes: one grid, or score and finish. With chunks: the plan before them -
  // they need nothing of one another and run together - and the passes after
  *launches = p.cluster > 0 ? 1 : 2;
  cudaError_t e = cudaSuccess;
  if (p.num_slots > 0) {
    *launches += 3;
    e = launch_chained(pa_weights_plan_kernel, p, 1, kPlanThreads, 0, s);
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
  l.counts_off = l.counters_off = l.items1_off = l.items2_off = l.lse_off = l.partial_off =
      l.sums_off = l.total;
  l.num_slots = l.max_items[0] = l.max_items[1] = l.num_counters = 0;
  if (!many) return l;
  const size_t tok = (size_t)(128 / G);
  const size_t slots = (size_t)num_tokens / tok + (size_t)num_reqs + 1;
  const size_t tiles = ((size_t)max_seq_len + 127) / 128;
  size_t parts = (tiles + kMinPart - 1) / kMinPart;
  if (parts > kMaxParts) parts = kMaxParts;
  l.num_slots = (int)slots;
  l.num_counters = (int)(4 * slots * num_kv_heads + 8 * kMaxUnits);
  l.max_items[0] = (int)(slots * parts * num_kv_heads);
  l.max_items[1] = (int)(rh * tiles) + kMaxUnits * kMaxParts;
  l.counters_off = l.counts_off + 256;
  l.items1_off = l.counters_off + pa_align256(sizeof(int) * (size_t)l.num_counters);
  l.items2_off = l.items1_off + pa_align256(sizeof(WItem) * (size_t)l.max_items[0]);
  l.lse_off = l.items2_off + pa_align256(sizeof(WItem) * (size_t)l.max_items[1]);
  l.partial_off = l.lse_off + pa_align256(sizeof(float) * 128 * slots * num_kv_heads);
  l.sums_off = l.partial_off +
               (parts > 1 ? pa_align256(sizeof(float2) * 128 * slots * num_kv_heads * parts) : 0);
  l.total = l.sums_off + sizeof(float) * 256 * kMaxParts * (size_t)kMaxUnits;
  return l;
}

cudaError_t launch_weights(WeightsParams p, int head_dim, bool f8, int num_sms, cudaStream_t s,
                           int* launches) {
  // CTAs per (request, KV head) of the few-rows form: enough that a CTA's scores
  // fit kClusterSmem and, while parts are longer than 1024 keys, that the grid has
  // three waves of two CTAs per SM (two waves measure the same over 1 to 256
  // requests); 0: they do not fit even eight CTAs
  const long long rh = (long long)p.num_reqs * p.num_kv_heads;
  p.num_sms = num_sms;
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
