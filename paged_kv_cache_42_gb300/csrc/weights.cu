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
// Two softmax warpgroups take the Y tiles in turn; four S buffers in TMEM let
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
constexpr int kFinishThreads = 256;
constexpr int kFinishKeys = 1024;    // keys of one finish CTA
constexpr int kSplitTiles = 16;      // key tiles of one part in pass 1
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

// NR: rows stored per key (the batch's largest count: G for decodes, else 8).
template <int D, bool F8, int NR>
__global__ void __launch_bounds__(32 * kScoreWarps) pa_weights_score_kernel(const WeightsParams p) {
  constexpr int EB = F8 ? 1 : 2;
  constexpr int VPR = D * EB / 16;  // 16-byte vectors of a key row
  constexpr int NJ = VPR / 4;       // vectors a lane takes of a row
  constexpr int NK = D / 16;        // MMAs per block
  griddep_launch_dependents();      // the finish grid waits for this one
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (p.num_chunks + kScoreWarps - 1) / kScoreWarps;
  const int rh = (int)(blockIdx.x / (unsigned)per), cc = (int)(blockIdx.x - (unsigned)(rh * per));
  const int r = rh / p.num_kv_heads, h = rh - r * p.num_kv_heads;
  const Span sp = get_span(p, r, cc == 0 && h == 0 && threadIdx.x == 0);
  const int G = p.group, rows = sp.qlen * G;
  if (!sp.ok || rows == 0 || rows > kFewRows) return;
  const int nb = (sp.L + kBlockSize - 1) / kBlockSize;
  const int chunk = cc * kScoreWarps + warp;
  const int b0 = chunk * kChunkBlocks;
  if (b0 >= nb) return;
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

  // the query operand: row g (token g / G, head g % G), this lane's elements
  uint32_t bq[NK][2];
  float unscale = 1.f;  // of row g
#pragma unroll
  for (int i = 0; i < NK; ++i) bq[i][0] = bq[i][1] = 0u;
  {
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
      unscale = __uint_as_float((uint32_t)(127 - ex) << 23);
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const uint32_t w[8] = {raw[j][0].x, raw[j][0].y, raw[j][0].z, raw[j][0].w,
                               raw[j][1].x, raw[j][1].y, raw[j][1].z, raw[j][1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = bf16x2_to_float2(w[i]);
          bq[4 * j + i / 2][i & 1] = float2_to_f16x2(f.x * sc, f.y * sc);
        }
      }
    } else if (g < rows) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const uint4 v = __ldg(qrow + j * 4 + t);
        bq[2 * j][0] = v.x;
        bq[2 * j][1] = v.y;
        bq[2 * j + 1][0] = v.z;
        bq[2 * j + 1][1] = v.w;
      }
    }
  }
  // the two rows whose scores this lane holds, their scales and last keys
  const int n0 = 2 * t, n1 = 2 * t + 1;
  float sc0 = p.scale_log2, sc1 = p.scale_log2;
  if constexpr (F8) {
    sc0 *= __shfl_sync(kAll, unscale, n0 * 4);
    sc1 *= __shfl_sync(kAll, unscale, n1 * 4);
  }
  const int ctx = sp.L - sp.qlen;
  const int lim0 = n0 < rows ? ctx + n0 / G : -1, lim1 = n1 < rows ? ctx + n1 / G : -1;

  struct Frag {
    uint4 a[NJ][2];
  };
  const uint4* const kc = static_cast<const uint4*>(p.k_cache);
  auto load = [&](int i, Frag& f) {
    const int id = __shfl_sync(kAll, pid, i);
    const uint4* const src =
        kc + (((size_t)(id < 0 ? 0 : id) * p.num_kv_heads + h) * kBlockSize + g) * VPR + t;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      f.a[j][0] = f.a[j][1] = make_uint4(0u, 0u, 0u, 0u);
      if (id >= 0) {
        f.a[j][0] = ld_stream(src + 4 * j);
        f.a[j][1] = ld_stream(src + 8 * VPR + 4 * j);
      }
    }
  };
  float m0 = kNone, m1 = kNone, l0 = 0.f, l1 = 0.f;
  float* const score = p.scores + ((size_t)rh * p.padded_len + (size_t)b0 * kBlockSize) * NR;
  auto take = [&](int i, const Frag& f) {
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
                            e4m3x2_to_f16x2((uint16_t)(vw[e] >> 16)), bq[4 * j + e][0],
                            bq[4 * j + e][1]);
      } else {
        mma_16x8x16<false>(c[0], u.x, v.x, u.y, v.y, bq[2 * j][0], bq[2 * j][1]);
        mma_16x8x16<false>(c[1], u.z, v.z, u.w, v.w, bq[2 * j + 1][0], bq[2 * j + 1][1]);
      }
    }
    const bool have = __shfl_sync(kAll, pid, i) >= 0;
    const int key = (b0 + i) * kBlockSize + g;
    const float x0 = have && key <= lim0 ? (c[0][0] + c[1][0]) * sc0 : -INFINITY;
    const float x1 = have && key <= lim1 ? (c[0][1] + c[1][1]) * sc1 : -INFINITY;
    const float y0 = have && key + 8 <= lim0 ? (c[0][2] + c[1][2]) * sc0 : -INFINITY;
    const float y1 = have && key + 8 <= lim1 ? (c[0][3] + c[1][3]) * sc1 : -INFINITY;
    float* const at = score + (size_t)(i * kBlockSize + g) * NR + n0;
    if constexpr (NR == 1) {
      if (t == 0) {
        at[0] = x0;
        at[8] = y0;
      }
    } else if (n0 < NR) {
      *reinterpret_cast<float2*>(at) = make_float2(x0, x1);
      *reinterpret_cast<float2*>(at + 8 * NR) = make_float2(y0, y1);
    }
    const float k0 = fmaxf(m0, fmaxf(x0, y0)), k1 = fmaxf(m1, fmaxf(x1, y1));
    l0 = l0 * ex2_approx(m0 - k0) + (ex2_approx(x0 - k0) + ex2_approx(y0 - k0));
    l1 = l1 * ex2_approx(m1 - k1) + (ex2_approx(x1 - k1) + ex2_approx(y1 - k1));
    m0 = k0;
    m1 = k1;
  };
  Frag fa, fb;
  load(0, fa);
#pragma unroll 1
  for (int i = 0; i < n; i += 2) {
    if (i + 1 < n) load(i + 1, fb);
    take(i, fa);
    if (i + 1 >= n) break;
    if (i + 2 < n) load(i + 2, fa);
    take(i + 1, fb);
  }
  // over the lanes of a row (those of equal t)
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
  if (g == 0)
    *reinterpret_cast<float4*>(p.stats + ((size_t)rh * p.num_chunks + chunk) * (2 * kFewRows) +
                               4 * t) = make_float4(m0, l0, m1, l1);
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
  griddep_wait();  // the score grid (and, through it, what came before)
  if (!sp.ok || rows == 0 || rows > kFewRows || cc * kFinishKeys >= sp.L) return;
  // warp n joins row n's chunks
  {
    static_assert(kFinishThreads / 32 == kFewRows, "a warp per row");
    const int chunks = (sp.L + kChunkBlocks * kBlockSize - 1) / (kChunkBlocks * kBlockSize);
    const float2* const st = reinterpret_cast<const float2*>(p.stats) +
                             (size_t)rh * p.num_chunks * kFewRows + warp;
    float m = kNone, l = 0.f;
    for (int c = lane; c < chunks; c += 32) {
      const float2 v = __ldcg(st + (size_t)c * kFewRows);
      const float k = fmaxf(m, v.x);
      l = l * ex2_approx(m - k) + v.y * ex2_approx(v.x - k);
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
  float m[NR], inv[NR];
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    m[n] = s_m[n];
    inv[n] = s_inv[n];
  }
  const int ctx = sp.L - sp.qlen;
  const float* const old = p.weights + (size_t)rh * p.weights_stride;
  float* const out = p.out + (size_t)rh * p.weights_stride;
#pragma unroll
  for (int i = 0; i < kFinishKeys / kFinishThreads; ++i) {
    const int key = cc * kFinishKeys + i * kFinishThreads + tid;
    if (key >= sp.L) break;
    const float* const s = p.scores + ((size_t)rh * p.padded_len + key) * NR;
    float x[NR];
    if constexpr (NR >= 4) {
#pragma unroll
      for (int n = 0; n < NR; n += 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(s + n));
        x[n] = v.x, x[n + 1] = v.y, x[n + 2] = v.z, x[n + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int n = 0; n < NR; ++n) x[n] = __ldcg(s + n);
    }
    float a = 0.f;
#pragma unroll
    for (int n = 0; n < NR; ++n)
      if (n < rows) a += ex2_approx(x[n] - m[n]) * inv[n];
    out[key] = key < ctx ? old[key] + a : a;
  }
  __threadfence();  // performed before the CTA ends: the next grid may be a programmatic one
}

// ---------------------------------------------------------------------------------------
// many rows
// ---------------------------------------------------------------------------------------
// The work lists of both passes, longest items first (bucket counts), and the
// number of key parts of every row tile. Row tile rt of request r has slot
// q0 / TOK + r + rt: consecutive requests' slots never meet, since a span of
// qlen tokens has at most (q0 + qlen) / TOK - q0 / TOK + 1 tiles.
__global__ void __launch_bounds__(kPlanThreads) pa_weights_plan_kernel(const WeightsParams p) {
  __shared__ int cnt[2][kBuckets];
  __shared__ int wsum[kPlanThreads / 32], s_fits;
  bool none = false;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int TOK = 128 / p.group;
  for (int b = tid; b < kBuckets; b += kPlanThreads) cnt[0][b] = cnt[1][b] = 0;
  __syncthreads();
  // what: 0 counts the items per bucket, 1 writes them
  auto walk = [&](int what) {
    for (int r = tid; r < p.num_reqs; r += kPlanThreads) {
      const Span s = get_span(p, r, what == 0);
      if (!s.ok || s.qlen * p.group <= kFewRows) continue;
      const int ctx = s.L - s.qlen, nrt = (s.qlen + TOK - 1) / TOK;
      for (int rt = 0; rt < nrt; ++rt) {
        const int last = ctx + min(s.qlen, (rt + 1) * TOK) - 1;
        const int nkt = last / 128 + 1;
        const int slot = s.q0 / TOK + r + rt;
        if (what) p.parts[slot] = (nkt + kSplitTiles - 1) / kSplitTiles;
        for (int i0 = 0; i0 < nkt; i0 += kSplitTiles) {
          const int len = min(kSplitTiles, nkt - i0);
          const int at = atomicAdd(&cnt[0][min(len, kBuckets - 1)], p.num_kv_heads);
          if (what)
            for (int h = 0; h < p.num_kv_heads; ++h) p.items[0][at + h] = make_int4(r, h, rt, i0);
        }
      }
      const int nkt = (s.L + 127) / 128;
      for (int kt = 0; kt < nkt; ++kt) {
        const int rt0 = max(0, kt * 128 - ctx) / TOK;  // the first row tile that sees the keys
        const int at = atomicAdd(&cnt[1][min(nrt - rt0, kBuckets - 1)], p.num_kv_heads);
        if (what)
          for (int h = 0; h < p.num_kv_heads; ++h) p.items[1][at + h] = make_int4(r, h, kt, rt0);
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
    int before = incl - v;
    for (int w = 0; w < warp; ++w) before += wsum[w];
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
  for (int i = tid; i < p.num_slots; i += kPlanThreads) p.parts[i] = 0;
  __syncthreads();
  if (none) {  // no such request, or spans that cannot be
    if (tid < 2) p.counts[tid] = 0;
  } else {
    walk(1);
  }
  griddep_launch_dependents();
  griddep_wait();  // complete only after the grid before: later waits see its work too
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
  p.lse[at] = l > 0.f ? m + log2f(l) : INFINITY;  // rows past the span: +inf, a weight of zero
  __threadfence();
}

template <int D>
struct WCfg {
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
  static constexpr int OFF_BAR = OFF_XCH + 128 * 8;
  static constexpr int B_XF = 0, B_XE = 2, B_YF = 4, B_YE = B_YF + NY, B_SF = B_YE + NY,
                       B_SE = B_SF + NS, B_XCHF = B_SE + NS, B_XCHE = B_XCHF + 1,
                       B_DRAIN = B_XCHE + 1, B_COUNT = B_DRAIN + 1;
  static constexpr int SMEM = OFF_BAR + 8 * B_COUNT + 16 + 1024;
  static_assert(SMEM <= 227 * 1024, "one CTA per SM");
};
constexpr int kTcThreads = 320;             // producer, MMA issuer, 2 x 4 softmax warps
constexpr int kTcThreadsF8 = kTcThreads + 128;  // + 4 converter warps

}  // namespace

struct WeightsTcParams {
  CUtensorMap tm_q;  // q as [T][Hq][D], box {64, G, 128 / G}, 128B swizzle
  CUtensorMap tm_k;  // k_cache as [blocks * Hkv * 16][D], box {64, 16} (bf16 caches)
  WeightsParams w;
};

namespace {

struct WItem {
  int r, h, q0, qlen, ctx, L;
  int x;         // row tile (pass 1) or key tile (pass 2) of X
  int y0, n;     // Y tiles y0 .. y0 + n - 1
};

template <int PASS>
__device__ __forceinline__ WItem get_witem(const WeightsParams& p, int t) {
  const int4 v = __ldcg(p.items[PASS - 1] + t);
  const int TOK = 128 / p.group;
  WItem it;
  it.r = v.x;
  it.h = v.y;
  it.x = v.z;
  it.y0 = v.w;
  it.q0 = __ldg(p.qsl + it.r);
  it.qlen = __ldg(p.qsl + it.r + 1) - it.q0;
  it.L = __ldg(p.seq_lens + it.r);
  it.ctx = it.L - it.qlen;
  if (PASS == 1) {
    const int last = it.ctx + min(it.qlen, (it.x + 1) * TOK) - 1;
    it.n = min(kSplitTiles, last / 128 + 1 - it.y0);
  } else {
    it.n = (it.qlen + TOK - 1) / TOK - it.y0;
  }
  return it;
}

__device__ __forceinline__ int snake(int i) {  // rounds of items in alternating direction
  const int g = (int)gridDim.x, b = (int)blockIdx.x;
  return i * g + ((i & 1) ? g - 1 - b : b);
}

template <int D, int PASS, bool F8>
__global__ void __launch_bounds__(F8 ? kTcThreadsF8 : kTcThreads, 1)
    pa_weights_tc_kernel(const __grid_constant__ WeightsTcParams tp) {
  using C = WCfg<D>;
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
      if (i == C::B_XCHF || i == C::B_XCHE) n = 128;
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
    const int b = kt * 8 + lane, nb = (it.L + kBlockSize - 1) / kBlockSize;
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
                 p.lse + ((size_t)it.h * p.num_slots + slot) * 128, 512, bar);
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
  } else if (warp < 10) {
    // ======================= softmax (two warpgroups) =======================
    const int wg = (warp - 2) / 4;
    const int q4 = warp & 3;             // the TMEM lane quarter this warp may access
    const int m = q4 * 32 + lane;        // row of X
    const uint32_t trow = ((uint32_t)(q4 * 32) << 16) + tmem;
    float2* const xch = reinterpret_cast<float2*>(gb + C::OFF_XCH);
    const float sc = p.scale_log2;
    int g = 0, it = 0;
    bool ok = true;
    for (int t = snake(it); ok && t < nitems; t = snake(++it)) {
      const WItem w = get_witem<PASS>(p, t);
      // pass 1: this thread's query row; pass 2: its key
      const int j = w.x * TOK + m / p.group;
      const int lim = PASS == 1 ? (j < w.qlen ? w.ctx + j : -1) : w.L - 1;
      const int key = w.x * 128 + m;
      float mx = kNone, l = 0.f;
      for (int i = 0; i < w.n; ++i, ++g) {
        if ((g & 1) != wg) continue;
        const int sb = g % C::NS;
        if (!wait(C::B_SF + sb, g / C::NS)) { ok = false; break; }
        tc_fence_after();
        const uint32_t s0 = trow + 128 * sb;
        // columns lo .. hi - 1 of this row count
        int lo, hi;
        if (PASS == 1) {
          lo = 0;
          hi = lim - (w.y0 + i) * 128 + 1;
        } else {
          const int j0 = (w.y0 + i) * TOK;  // the tile's first token
          lo = (key - w.ctx - j0) * p.group;
          hi = (w.qlen - j0) * p.group;
        }
        const bool full = __all_sync(kAll, lo <= 0 && hi >= 128);
        const float4* const lse =
            reinterpret_cast<const float4*>(gb + C::OFF_LSE + (g % C::NLSE) * 512);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t rr[32];
          tmem_ld32(s0 + c * 32, rr);
          tmem_wait_ld();
          float x[32];
          if (PASS == 1) {
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(rr[e]);
            if (!full) {
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] = c * 32 + e < hi ? x[e] : -INFINITY;
            }
            float top = x[0];
#pragma unroll
            for (int e = 1; e < 32; ++e) top = fmaxf(top, x[e]);
            // scale > 0 keeps the order; another one looks at the scaled scores
            if (!(sc > 0.f)) {
              top = -INFINITY;
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (full || c * 32 + e < hi) top = fmaxf(top, x[e] * sc);
            } else {
              top *= sc;
            }
            const float k = fmaxf(mx, top);
            float a0 = 0.f, a1 = 0.f;
            if (full) {
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                a0 += ex2_approx(fmaf(x[e], sc, -k));
                a1 += ex2_approx(fmaf(x[e + 1], sc, -k));
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (c * 32 + e < hi) a0 += ex2_approx(fmaf(x[e], sc, -k));
            }
            l = l * ex2_approx(mx - k) + (a0 + a1);
            mx = k;
          } else {
            float a0 = 0.f, a1 = 0.f;
            if (full) {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float4 v = lse[c * 8 + e];
                a0 += ex2_approx(fmaf(__uint_as_float(rr[4 * e]), sc, -v.x));
                a1 += ex2_approx(fmaf(__uint_as_float(rr[4 * e + 1]), sc, -v.y));
                a0 += ex2_approx(fmaf(__uint_as_float(rr[4 * e + 2]), sc, -v.z));
                a1 += ex2_approx(fmaf(__uint_as_float(rr[4 * e + 3]), sc, -v.w));
              }
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float4 v = lse[c * 8 + e];
                const float ls[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                  const int col = c * 32 + 4 * e + f;
                  if (col >= lo && col < hi)
                    a0 += ex2_approx(fmaf(__uint_as_float(rr[4 * e + f]), sc, -ls[f]));
                }
              }
            }
            l += a0 + a1;
          }
        }
        tc_fence_before();
        mbar_arrive(BAR(C::B_SE + sb));
      }
      if (!ok) break;
      // warpgroup 1's part joins warpgroup 0's
      if (wg == 1) {
        if (it > 0 && !wait(C::B_XCHE, it - 1)) break;
        xch[m] = make_float2(mx, l);
        mbar_arrive(BAR(C::B_XCHF));
        continue;
      }
      if (!wait(C::B_XCHF, it)) break;
      const float2 o = xch[m];
      mbar_arrive(BAR(C::B_XCHE));
      if (PASS == 1) {
        const float k = fmaxf(mx, o.x);
        l = l * ex2_approx(mx - k) + o.y * ex2_approx(o.x - k);
        const int slot = w.q0 / TOK + w.r + w.x;
        const size_t at = ((size_t)w.h * p.num_slots + slot) * 128 + m;
        const int nkt = (w.ctx + min(w.qlen, (w.x + 1) * TOK) - 1) / 128 + 1;
        if (nkt <= kSplitTiles)
          p.lse[at] = l > 0.f ? k + log2f(l) : INFINITY;
        else
          __stcg(p.partial + (size_t)(w.y0 / kSplitTiles) * p.num_kv_heads * p.num_slots * 128 + at,
                 make_float2(k, l));
      } else if (key < w.L) {
        const size_t at = ((size_t)w.r * p.num_kv_heads + w.h) * p.weights_stride + key;
        l += o.y;
        p.out[at] = key < w.ctx ? p.weights[at] + l : l;
      }
    }
  } else if constexpr (F8) {
    // ======================= E4M3 converters: the key operand =======================
    const int row = threadIdx.x - kTcThreads;
    int g = 0, it = 0;
    bool ok = true;
    for (int t = snake(it); ok && t < nitems; t = snake(++it)) {
      const WItem w = get_witem<PASS>(p, t);
      auto convert = [&](int kt, unsigned char* dst) {
        const int key = kt * 128 + row;
        bool valid = key < w.L;
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

template <int D, bool F8, int NR>
cudaError_t launch_few(const WeightsParams& p, cudaStream_t s) {
  const long long rh = (long long)p.num_reqs * p.num_kv_heads;
  const long long g1 = rh * ((p.num_chunks + kScoreWarps - 1) / kScoreWarps);
  if (g1 > 0x7fffffffLL) return cudaErrorInvalidValue;
  // the first grid of the call is no programmatic dependent: everything the
  // stream did before is complete and visible
  pa_weights_score_kernel<D, F8, NR><<<(unsigned)g1, 32 * kScoreWarps, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
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
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, WCfg<D>::SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  return launch_chained(kern, tp, num_sms, F8 ? kTcThreadsF8 : kTcThreads, WCfg<D>::SMEM, s);
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
  cudaError_t e = launch_chained(pa_weights_plan_kernel, p, 1, kPlanThreads, 0, s);
  if (e == cudaSuccess) e = launch_pass<D, 1, F8>(tp, num_sms, s);
  if (e == cudaSuccess && p.max_seq_len > 128 * kSplitTiles)
    e = launch_chained(pa_weights_join_kernel, p, (long long)p.num_slots * p.num_kv_heads, 128, 0, s);
  if (e == cudaSuccess) e = launch_pass<D, 2, F8>(tp, num_sms, s);
  return e;
}

template <int D, bool F8>
cudaError_t launch_weights_t(const WeightsParams& p, int num_sms, cudaStream_t s, int* launches) {
  *launches = 2;
  cudaError_t e = launch_few_rows<D, F8>(p, s);
  if (e != cudaSuccess || p.max_query_len * (long long)p.group <= kFewRows) return e;
  *launches += p.max_seq_len > 128 * kSplitTiles ? 4 : 3;
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
  l.items2_off = l.items1_off + pa_align256(sizeof(int4) * slots * parts * num_kv_heads);
  l.lse_off = l.items2_off + pa_align256(sizeof(int4) * rh * tiles);
  l.partial_off = l.lse_off + pa_align256(sizeof(float) * 128 * slots * num_kv_heads);
  l.total = l.partial_off +
            (parts > 1 ? pa_align256(sizeof(float2) * 128 * slots * num_kv_heads * parts) : 0);
  return l;
}

cudaError_t launch_weights(const WeightsParams& p, int head_dim, bool f8, int num_sms,
                           cudaStream_t s, int* launches) {
  if (head_dim == 128)
    return f8 ? launch_weights_t<128, true>(p, num_sms, s, launches)
              : launch_weights_t<128, false>(p, num_sms, s, launches);
  return f8 ? launch_weights_t<64, true>(p, num_sms, s, launches)
            : launch_weights_t<64, false>(p, num_sms, s, launches);
}

}  // namespace pa
