// Prefill-chunk attention on the tensor cores (tcgen05 + TMEM + TMA).
//
// What is computed ("vLLM v1 Deep Dive: How LLM(...) and the Server Boot and
// Generate", Part 3, "Aside - KV cache and prefix caching": a prefill query
// attends causally over [its already-cached prefix blocks] + [its new
// tokens]): for a request with ctx cached tokens and a chunk of qlen new
// tokens, new token j attends to keys 0 .. ctx + j, K/V read through the
// request's block table.
//
// Tiling (ours). A row tile is 128 query rows of one (request, kv head): the G
// query heads of the kv head times 128/G consecutive chunk tokens, row
// m = token * G + head - the GQA "Q block" packing ("vLLM: An Exhaustive
// Technical Study for Kernel Engineers", 2.4, Triton unified attention), so a
// row tile shares one K/V stream. A CTA work item is a PAIR of adjacent row
// tiles (256 rows) over the same keys; keys come in tiles of 128 = eight
// 16-key cache blocks, loaded once for both row tiles.
//
//   S_t = Q_t K^T   tcgen05.mma kind::f16, M=128 N=128, A=Q_t and B=K from
//                   128B-swizzled shared memory, fp32 into TMEM.
//   softmax         one thread per row (one TMEM lane): mask, scale, running
//                   max, exp2; P_t rounded to bf16 and written back into TMEM
//                   over the S_t it came from.
//   O_t += P_t V    tcgen05.mma with A=P_t from TMEM, B=V (M/N-major) from
//                   shared memory, O_t in TMEM.
// The two row tiles ping-pong: while one warpgroup runs the softmax of its
// tile, the tensor core runs the other tile's P*V and next S.
//
// The running max is only moved (and O rescaled through TMEM) when it grows
// by more than 2^8; otherwise P is formed against the stale max, which keeps
// every P <= 256 and the result exact up to rounding.
//
// Cascade prefix pass (the PREFIX instantiation; "vLLM: An Exhaustive
// Technical Study for Kernel Engineers", 2.3, cascade attention): the same
// pipeline over the common prefix shared by every request of the batch. A
// work item is (pair of row tiles of consecutive batch tokens, kv head, chunk
// of prefix key tiles); every row sees every prefix key (the prefix lies in
// each request's context), and the epilogue writes an fp32 partial (running
// max, sum, unnormalised output) per (chunk, token, kv head) for the split-KV
// kernel to merge, instead of bf16 rows. Groups of requests with a prefix each
// (MODE kGroups, pa_attention_shared) run the same pass over the planner's list of
// items. A group of few requests has few rows: those that fit one tile are given to
// both, one warpgroup taking the even key tiles and the other the odd ones, each
// into a partial of its own. That keeps the two-tile pipeline as it is - per tile
// of keys, half the products - where an empty second tile would double the work
// and a lone first one would leave nothing to run beside its softmax.
//
// FP8 caches (the F8 instantiation; "vLLM: An Exhaustive Technical Study for
// Kernel Engineers", 2.8: E4M3 codes with per-tensor k_scale / v_scale): a block's
// codes are copied into the stage that their bf16 values will fill - over the
// rows of their own (a block's 16 rows, at head dim 128 their second halves) - and
// eight more warps (576 threads), four for K and four for V, widen them in place:
// a warp takes 32 key rows into registers and writes them back as the
// 128B-swizzled operand that the MMA reads - exactly, every E4M3 value being a
// bf16 - and arrives on the stage's full barrier. So a ring of E4M3 tiles has all of
// its stages in flight, as one of bf16 tiles has. (Loads into registers, two tiles
// ahead, were limited to what the SM's remaining 28 KB of L1 can await: 4.3 us per
// key tile of a long prefix against 1.9.) k_scale is
// folded into the softmax scale and v_scale into the epilogue. Over row-scaled
// caches (KV 2, rows.cuh) the converters multiply each row by its 2^e, which is
// exact in bf16 too, and nothing else differs.
//
// Warp roles (320 threads over bf16 caches): warp 0 issues TMA loads (both Q tiles per work
// item, K into a 3-stage ring released right after both S MMAs of a key tile,
// V into a 2-stage ring released after both P*V), warp 1 allocates TMEM and
// one thread issues the MMAs in order
//   S0(0) S1(0) | PV0(i) S0(i+1) PV1(i) S1(i+1) | ...
// and warps 2-5 / 6-9 (warpgroup t; warp w reads TMEM lanes 32*(w%4)..) run
// the softmax and epilogue of row tile t. Every wait is bounded; a wait that
// gives up sets the device error word and the CTA winds down.
#pragma once

#include <cuda.h>

#include <cfloat>

#include "pa_internal.h"
#include "ptx.cuh"
#include "rows.cuh"

namespace pa {

// What a prefill launch computes: chunks of prompts, a cascade's prefix pass over
// one prefix, or the prefix pass over the groups of a shared call.
enum PrefillMode { kChunks = 0, kOnePrefix = 1, kGroups = 2 };

namespace {

constexpr unsigned kAll = 0xffffffffu;
// A softmax reference of more than this (base-2 units) is subtracted before the
// scale: below it the rounding of its product moves P by a factor of at most 2^(2^-15).
constexpr float kFar = 1024.f;

// Threads per S row in the softmax (1 or 2). With 2, the two threads of a row
// take 64 score columns each and combine their row maxima through shared
// memory (a bounded mbarrier exchange). It shortens the softmax but not the
// kernel: in steady state the tensor pipe, not the softmax, sets the pace of
// a key tile (measured 52.6 us with 2 vs 51.4 us with 1 on the mixed batch),
// so the default is 1.
#ifndef PA_PREFILL_SPLIT
#define PA_PREFILL_SPLIT 1
#endif
constexpr int kSplit = PA_PREFILL_SPLIT;
static_assert(kSplit == 1 || kSplit == 2, "one or two threads per row");

template <int D, int G>
struct PCfg {
  static constexpr int TOK = 128 / G;         // chunk tokens per 128-row tile
  static constexpr int NCH = D / 64;          // 64-element (128-byte) d chunks
  static constexpr int CHUNK = 128 * 128;     // one [128 rows][128 B] operand chunk
  static constexpr int Q_BYTES = NCH * CHUNK; // one row tile of Q
  static constexpr int KV_BYTES = NCH * CHUNK;  // one 128-key tile of K or of V
  // a third K stage does not fit beside the row-max exchange buffer
#ifdef PA_PREFILL_KSTAGES
  static constexpr int KSTAGES = PA_PREFILL_KSTAGES;
#else
  static constexpr int KSTAGES = kSplit == 2 ? 2 : 3;
#endif
#ifndef PA_PREFILL_VSTAGES
#define PA_PREFILL_VSTAGES 2
#endif
  static constexpr int VSTAGES = PA_PREFILL_VSTAGES;
  // E4M3: where in a stage block b's codes land (+ 2048 b), within the block's own rows
  static constexpr int OFF_RAW = (NCH - 1) * CHUNK;
  static constexpr int OFF_Q = 0;  // two row tiles
  static constexpr int OFF_K = OFF_Q + 2 * Q_BYTES;
  static constexpr int OFF_V = OFF_K + KSTAGES * KV_BYTES;
  static constexpr int OFF_BAR = OFF_V + VSTAGES * KV_BYTES;
  // E4M3: a byte for each of K's stages, then V's: which of its tile's blocks were copied
  static constexpr int OFF_GOOD = OFF_BAR + 272;
  // row-max / row-sum exchange of the split softmax: [row tile][parity][half][128 rows]
  static constexpr int OFF_XCH = OFF_BAR + 320;
  static constexpr int XCH_BYTES = kSplit == 2 ? 2 * 2 * 2 * 128 * 4 : 0;
  // KV 2: the scale bytes of each stage's rows, K's stages, then V's
  static constexpr int OFF_SC = OFF_XCH + XCH_BYTES;
  static constexpr int SMEM = OFF_SC + (KSTAGES + VSTAGES) * 128 + 1024;  // + 1 KB alignment slack
  static constexpr uint32_t TMEM_COLS = 512;
  // S_t (fp32, 128 columns) at 128*t; P_t (bf16 pairs, 64 columns) is written
  // over S_t, each thread's part over its own S columns (P column of key k:
  // pcol(k / 32) + (k % 32) / 2); O_t at 256 + 128*t.
  static constexpr uint32_t TM_S = 0;
  static constexpr uint32_t TM_O = 256;
  static constexpr int CPH = 4 / kSplit;  // 32-column S chunks per softmax thread
  // first P column of S chunk c: chunk c's 32 scores become 16 bf16 pairs
  __host__ __device__ static constexpr uint32_t pcol(int c) {
    return 64u * (uint32_t)(c / CPH) + 16u * (uint32_t)(c % CPH);
  }
};

// barrier slots
enum : int {
  B_Q_FULL = 0, B_Q_EMPTY = 1, B_K_FULL = 2 /* x3 */, B_K_EMPTY = 5 /* x3 */,
  B_V_FULL = 8 /* x3 */, B_V_EMPTY = 11 /* x3 */, B_S_FULL = 14 /* x2: per row tile */,
  B_P_FULL = 16 /* x2 */, B_PV_DONE = 18 /* x2 */, B_O_EMPTY = 20 /* x2 */, B_DRAIN = 22,
  B_XCH = 23 /* x4: [row tile][parity], the split softmax's row exchange */,
  B_K_RAW = 27 /* x3 */, B_V_RAW = 30 /* x3 */, /* E4M3: the codes have landed */
  B_COUNT = 33
};

constexpr int kSoftWarps = 8 * kSplit;            // 4 * split per row tile
constexpr int kThreads = 32 * (2 + kSoftWarps);   // bf16 caches
constexpr int kThreadsF8 = kThreads + 256;        // E4M3 caches: + 4 converter warps each for K, V

}  // namespace

struct PrefillParams {
  CUtensorMap tm_q;  // q as [T][Hq][D], box {64, G, 128/G}, 128B swizzle
  CUtensorMap tm_k;  // k_cache as [(blocks * Hkv * 16)][D], box {64, 16}
  CUtensorMap tm_v;
  const int32_t* qsl;
  const int32_t* seq_lens;
  const int32_t* block_tables;
  uint16_t* out;
  const WsHeader* header;
  const PrefillTile* tiles;
  int bt_stride, num_q_heads, num_kv_heads, num_blocks;
  // A negative scale: S = -Q K^T (idesc_qk) under its absolute value, so that the
  // largest raw score is the largest scaled one. A scale of zero becomes the
  // smallest number: -inf times it stays -inf.
  float scale_log2;
  uint32_t idesc_qk;
  // cascade prefix pass
  int num_tokens, prefix_len, prefix_chunks, prefix_pairs, slot_floats;
  float* prefix_partials;
  // E4M3 caches (F8): raw codes and the output multiplier (1 for bf16)
  const unsigned char* k_cache8;
  const unsigned char* v_cache8;
  const unsigned char* scales;  // KV 2
  float v_scale;
  const SharedItem* shared_items;  // kGroups
  int overlap;  // PrefillLaunch::overlap
  int window, sinks;  // WIN
  unsigned long long* err;
};

// One work item as every role sees it.
struct Item {
  int req;    // block-table row (request 0 for the prefix pass)
  int kv;     // kv head
  int j0;     // first chunk token of the pair (prefill)
  int i0, n;  // key tiles i0 .. i0 + n - 1
  int L;      // keys that exist (sequence length; prefix length)
  int tok0;   // batch token of the pair's first row
  int chunk;  // which of its tokens' partials it makes (prefix pass)
  bool split; // kGroups: both row tiles hold the same rows, one takes the even key tiles
  int tok_end;  // batch tokens from here on are not the item's (prefix pass)
  WinTiles wt;  // WIN: the key tiles of the item's rows
};

// Key tile i of an item as a tile of the sequence.
template <bool WIN>
__device__ __forceinline__ int key_tile(const Item& it, int i) {
  if constexpr (WIN) return i < it.wt.st ? i : i - it.wt.st + it.wt.wt;
  return it.i0 + i;
}
// WIN: whether any row of the item may see a key of [key, key + n).
__device__ __forceinline__ bool item_sees(const Item& it, int key, int n, int sinks) {
  return key < it.L && (key + n > it.wt.lo || key < sinks);
}

template <int D, int G, int MODE, bool WIN = false>
__device__ __forceinline__ Item get_item(const PrefillParams& p, int t) {
  using C = PCfg<D, G>;
  Item it;
  if constexpr (MODE == kGroups) {
    const int4* const at = reinterpret_cast<const int4*>(p.shared_items + t);
    const int4 a = __ldcg(at), b = __ldcg(at + 1);
    it.req = a.x;
    it.kv = a.y & ~kSharedSplit;
    it.split = (a.y & kSharedSplit) != 0;
    it.j0 = 0;
    it.tok0 = a.z;
    it.tok_end = a.w;
    it.chunk = b.x;
    it.i0 = b.y;
    it.n = b.z;
    it.L = b.w;
  } else if constexpr (MODE == kOnePrefix) {
    const int nkt = (p.prefix_len + 127) / 128;
    const int per = (nkt + p.prefix_chunks - 1) / p.prefix_chunks;
    it.kv = t % p.num_kv_heads;
    const int rest = t / p.num_kv_heads;
    it.chunk = rest % p.prefix_chunks;
    it.req = 0;
    it.j0 = 0;
    it.i0 = it.chunk * per;
    it.n = min(per, nkt - it.i0);  // >= 1: the host picks chunks that are all non-empty
    it.L = p.prefix_len;
    it.tok0 = (rest / p.prefix_chunks) * 2 * C::TOK;
    it.tok_end = p.num_tokens;
  } else {
    const PrefillTile tl = p.tiles[t];
    it.req = tl.req;
    it.kv = tl.kv;
    it.j0 = tl.j0;
    it.i0 = 0;
    it.n = tl.nkv;
    it.L = __ldg(p.seq_lens + tl.req);
    it.tok0 = __ldg(p.qsl + tl.req) + tl.j0;
    it.chunk = 0;
    if constexpr (WIN) {
      const int first = it.L - (__ldg(p.qsl + tl.req + 1) - (it.tok0 - tl.j0)) + tl.j0;
      it.wt = win_tiles(first, min(it.L - 1, first + 2 * C::TOK - 1), p.window, p.sinks);
    }
  }
  return it;
}

// A converter warp's 32 key rows of a stage (rows 32 cw ..): E4M3 codes at raw, a
// block's 16 rows 2048 bytes from the next's, widened in place to bf16 in the
// swizzled operand layout. Rows that are no keys (bit n of `rows`: the lane's n-th,
// row n RPI + lane / LPR of the 32) become zeros. SCALED: times 2^e, sc the rows'
// bytes. (By conversion instructions: moving the bits of four codes to two bf16
// pairs with a byte permute, a shift and two masks and multiplying by 2^120 takes
// as many instructions, on the pipe that the softmax needs most.)
template <int D, bool SCALED>
__device__ __forceinline__ void widen_rows(unsigned char* stage, const unsigned char* raw,
                                           const unsigned char* sc, uint32_t rows, int cw, int lane) {
  constexpr int LPR = D / 16, RPI = 32 / LPR, NI = LPR;
  constexpr int CHUNK = 128 * 128;
  const int sub = lane % LPR, rsub = lane / LPR;
  uint4 in[NI];
#pragma unroll
  for (int n = 0; n < NI; ++n) {
    const int r = n * RPI + rsub;
    in[n] = rows >> n & 1u ? *reinterpret_cast<const uint4*>(
                                 raw + (2 * cw + r / kBlockSize) * 2048 + (r % kBlockSize) * D + sub * 16)
                           : make_uint4(0u, 0u, 0u, 0u);
  }
  __syncwarp();  // every code of the 32 rows is read before the first value is written
#pragma unroll
  for (int n = 0; n < NI; ++n) {
    const int r = cw * 32 + n * RPI + rsub;
    uint32_t size = 0;
    if constexpr (SCALED) {
      const uint32_t b = rows >> n & 1u ? sc[r] : 127u;
      size = b == kRowPoison ? 0x7fc07fc0u : b << 7 | b << 23;  // 2^e as a pair of bf16
    }
    const uint32_t w4[4] = {in[n].x, in[n].y, in[n].z, in[n].w};
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 a = e4m3x2_to_float2((uint16_t)(w4[e / 2] >> (16 * (e & 1))));
      o[e] = float2_to_bf16x2(a.x, a.y);
      if constexpr (SCALED) o[e] = bf16x2_mul(o[e], size);
    }
    // elements 16 sub .. + 15: chunk sub / 4, units 2 (sub % 4) and the next. The
    // chunks are a multiple of all banks apart, so lanes of the second one store
    // their second unit first.
    unsigned char* const rowp = stage + (sub / 4) * CHUNK + r * 128;
    const int u = 2 * (sub % 4), f = sub / 4;
    const uint4 lo = make_uint4(o[0], o[1], o[2], o[3]), hi = make_uint4(o[4], o[5], o[6], o[7]);
    *reinterpret_cast<uint4*>(rowp + (((u + f) ^ (r & 7)) << 4)) = f ? hi : lo;
    *reinterpret_cast<uint4*>(rowp + (((u + 1 - f) ^ (r & 7)) << 4)) = f ? lo : hi;
  }
  fence_proxy_async_smem();  // generic-proxy stores -> visible to the tensor core
  __syncwarp();
}

// The r-th work item of CTA blockIdx.x among the g CTAs that take items.
// Items come sorted longest first; rounds of g items alternate direction (CTA b takes b, then 2g-1-b, then
// 2g+b, ...), so a CTA that drew a long item in one round draws a short one
// in the next instead of the next-longest.
__device__ __forceinline__ int snake_item(int r, int g) {
  const int b = (int)blockIdx.x;
  return r * g + ((r & 1) ? g - 1 - b : b);
}

// WIN: windowed attention. An item reads the key tiles that some row of it
// sees (win_tiles: the sinks', then the windows'), every row masks its own
// keys, and a block that no row sees is not read at all - its table entry may
// be stale - and counts as zeros in V. A row may see no key of its item's
// first tiles: it has no reference then, and the first tile it does see
// rescales a zero O by zero.
// KV: the caches, 0 bf16, 1 E4M3 with one scale per tensor, 2 row-scaled E4M3.
template <int D, int G, int MODE, int KV, bool WIN>
__global__ void __launch_bounds__(KV ? kThreadsF8 : kThreads, 1)
    pa_prefill_kernel(const __grid_constant__ PrefillParams p) {
  constexpr bool F8 = KV != 0, PREFIX = MODE != kChunks;
  using C = PCfg<D, G>;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;  // operand tiles need 1024-byte alignment
  unsigned char* const gbase = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bar0 = base + C::OFF_BAR;
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::OFF_BAR + 8 * B_COUNT);

  if (threadIdx.x == 0) {
    for (int i = 0; i < B_COUNT; ++i) {
      // P_FULL and O_EMPTY are arrived at by the 128 threads of one warpgroup;
      // every other slot once, by an expect_tx arrive or an MMA commit.
      const bool by_threads = (i == B_P_FULL || i == B_P_FULL + 1 || i == B_O_EMPTY ||
                               i == B_O_EMPTY + 1 || (i >= B_XCH && i < B_XCH + 4));
      // E4M3 caches: the K / V stages are filled by the 4 converter warps
      const bool by_converters =
          F8 && ((i >= B_K_FULL && i < B_K_FULL + C::KSTAGES) ||
                 (i >= B_V_FULL && i < B_V_FULL + C::VSTAGES));
      mbar_init(bar0 + 8 * i, by_threads ? 128 * kSplit : (by_converters ? 4 : 1));
    }
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // The work list comes from the preceding (planner) grid. The prefix pass
  // of a cascade needs none of it and waits only before it completes (see the end).
  if constexpr (MODE != kOnePrefix) griddep_wait();
  // (A shared call's grids release their dependents on completion only: with the plan
  // or this one doing so at the top, the next grid's CTAs take their places too early;
  // documents 133 -> 139 and 151 us.)
  int ntiles = MODE == kGroups      ? p.header->num_prefix_items
               : MODE == kOnePrefix ? p.prefix_pairs * p.num_kv_heads * p.prefix_chunks
                                    : p.header->num_tiles;
  // CTAs taking items: all, or (overlapped mixed batch) the planner's share;
  // the others retire at once and leave their SMs to the split-KV grid,
  // which every CTA releases here rather than on completion
  int ctas = (int)gridDim.x;
  // Overlapped cascade: the prefix pass runs on a few SMs beside the suffix
  // split-KV grid, which needs the plan. One warp (the last softmax warp,
  // idle until the first scores) waits for the planner and then releases it.
  if (MODE == kOnePrefix && p.overlap && warp == 1 + kSoftWarps) {
    griddep_wait();
    griddep_launch_dependents();
  }
  if (!PREFIX && p.overlap) {
    const int c = __ldcg(&p.header->prefill_ctas);
    if (c > 0 && c < ctas) {
      ctas = c;
      griddep_launch_dependents();
    }
    if ((int)blockIdx.x >= ctas) ntiles = 0;
  }

  auto BAR = [&](int i) -> uint32_t { return bar0 + 8 * i; };
  auto wait = [&](int i, uint32_t parity) -> bool {
    if (mbar_wait_bounded(BAR(i), parity)) return true;
    report_error(p.err, PA_DEVERR_WAIT_TIMEOUT, 1000 + i);
    return false;
  };

  if (warp == 0) {
    // ======================= TMA producer =======================
    // Block ids are fetched 32 at a time (four key tiles), one group ahead;
    // lanes 0..7 each copy one 16-key block.
    int g = 0, it = 0;
    bool ok = true;
    for (int t = snake_item(it, ctas); ok && t < ntiles; t = snake_item(++it, ctas)) {
      const Item tl = get_item<D, G, MODE, WIN>(p, t);
      const int nb = (tl.L + kBlockSize - 1) / kBlockSize;
      const int32_t* const bt_row = p.block_tables + (size_t)tl.req * p.bt_stride;
      auto load_group = [&](int grp) -> int {  // blocks of key tiles i0 + 4 grp .. + 3
        int b = tl.i0 * 8 + grp * 32 + lane;
        if constexpr (WIN) {
          const int i = grp * 4 + (lane >> 3);
          if (i >= tl.n) return -1;
          b = key_tile<WIN>(tl, i) * 8 + (lane & 7);
          if (!item_sees(tl, b * kBlockSize, kBlockSize, p.sinks)) return -1;
        }
        if (b >= nb) return -1;
        const int pid = __ldg(bt_row + b);
        if (pid < 0 || pid >= p.num_blocks) {
          report_error(p.err, PA_DEVERR_BLOCK_ID, b);
          return -1;
        }
        return pid;
      };
      int pid_cur = load_group(0);
      int pid_nxt = tl.n > 4 ? load_group(1) : -1;
      if (it > 0 && !wait(B_Q_EMPTY, (it - 1) & 1)) { ok = false; break; }
      if (lane == 0) {
        const int tiles = MODE == kGroups && tl.split ? 1 : 2;
        mbar_arrive_expect_tx(BAR(B_Q_FULL), tiles * C::Q_BYTES);
#pragma unroll
        for (int rt = 0; rt < 2; ++rt)
          if (rt < tiles) {
#pragma unroll
            for (int c = 0; c < C::NCH; ++c)
              tma_load_3d(base + C::OFF_Q + rt * C::Q_BYTES + c * C::CHUNK, &p.tm_q, c * 64,
                          tl.kv * G, tl.tok0 + rt * C::TOK, BAR(B_Q_FULL));
          }
      }
      // copies this lane's block of key tile gt into stage st: bf16 as the operand, E4M3
      // codes (and scales) to be widened there
      auto copy = [&](int pid, bool is_v, int st) {
        const bool mine = lane < 8 && pid >= 0;
        const uint32_t good = __ballot_sync(kAll, mine);
        const int nload = __popc(good);
        const uint32_t stage = base + (is_v ? C::OFF_V : C::OFF_K) + st * C::KV_BYTES;
        const uint32_t bar = BAR((F8 ? (is_v ? B_V_RAW : B_K_RAW) : (is_v ? B_V_FULL : B_K_FULL)) + st);
        constexpr int kBytes = F8 ? kBlockSize * D + (KV == 2 ? kBlockSize : 0) : C::NCH * 2048;
        if (lane == 0) {
          if constexpr (F8) gbase[C::OFF_GOOD + (is_v ? C::KSTAGES : 0) + st] = (unsigned char)good;
          mbar_arrive_expect_tx(bar, nload * kBytes);
        }
        __syncwarp();
        if (!mine) return;
        if constexpr (F8) {  // a block's rows of one head, one behind the other
          const size_t tile = (size_t)pid * p.num_kv_heads + tl.kv;
          bulk_g2s(stage + C::OFF_RAW + lane * 2048,
                   (is_v ? p.v_cache8 : p.k_cache8) + tile * (kBlockSize * D), kBlockSize * D, bar);
          if constexpr (KV == 2)
            bulk_g2s(base + C::OFF_SC + ((is_v ? C::KSTAGES : 0) + st) * 128 + lane * kBlockSize,
                     p.scales + tile * kScaleBytes + (is_v ? kBlockSize : 0), kBlockSize, bar);
        } else {
          const int row = (pid * p.num_kv_heads + tl.kv) * kBlockSize;
#pragma unroll
          for (int c = 0; c < C::NCH; ++c)
            tma_load_2d(stage + c * C::CHUNK + lane * 2048, is_v ? &p.tm_v : &p.tm_k, c * 64, row, bar);
        }
      };
      // K a tile ahead of V: its stages are free once S is done, V's only behind P V
      int before = -1;  // the block of the tile before
      for (int i = 0; i <= tl.n; ++i) {
        int pid = -1;
        if (i < tl.n) {
          if (i > 0 && (i & 3) == 0) {
            pid_cur = pid_nxt;
            pid_nxt = (i + 4 < tl.n) ? load_group((i >> 2) + 1) : -1;
          }
          pid = __shfl_sync(kAll, pid_cur, ((i & 3) << 3) + (lane & 7));
          const int gk = g + i, ks = gk % C::KSTAGES;
          if (gk >= C::KSTAGES && !wait(B_K_EMPTY + ks, ((gk / C::KSTAGES) - 1) & 1)) { ok = false; break; }
          copy(pid, false, ks);
        }
        if (i > 0) {
          const int gv = g + i - 1, vs = gv % C::VSTAGES;
          if (gv >= C::VSTAGES && !wait(B_V_EMPTY + vs, ((gv / C::VSTAGES) - 1) & 1)) { ok = false; break; }
          copy(before, true, vs);
        }
        before = pid;
      }
      g += tl.n;
    }
  } else if (warp == 1) {
    // ======================= MMA issuer =======================
    constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, true);
    // Shared-memory descriptors differ only in their start address field
    // (address >> 4), so each MMA takes a base descriptor plus a constant.
    const uint64_t kmaj_base = smem_desc_sw128(base, 16, 1024);        // K-major (Q, K)
    const uint64_t vmaj_base = smem_desc_sw128(base, C::CHUNK, 1024);  // M/N-major (V)
    int gk = 0;   // key tiles whose S MMAs were issued
    int gv = 0;   // key tiles whose P*V MMAs were issued
    int np[2] = {0, 0};  // P_t events consumed
    int it = 0;
    bool ok = true;
    for (int t = snake_item(it, ctas); ok && t < ntiles; t = snake_item(++it, ctas)) {
      const Item tl = get_item<D, G, MODE, WIN>(p, t);
      const int L = tl.L;
      if (!wait(B_Q_FULL, it & 1)) { ok = false; break; }

      const bool split = MODE == kGroups && tl.split;
      // S_rt(key tile of counter gk) for row tile rt
      auto issue_s = [&](int rt, bool last_of_item) -> bool {
        const int kst = gk % C::KSTAGES;
        if ((rt == 0 || split) && !wait(B_K_FULL + kst, (gk / C::KSTAGES) & 1)) return false;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t d = tmem + C::TM_S + 128 * rt;
          const uint64_t a0 = kmaj_base + ((C::OFF_Q + (split ? 0 : rt * C::Q_BYTES)) >> 4);
          const uint64_t b0 = kmaj_base + ((C::OFF_K + kst * C::KV_BYTES) >> 4);
#pragma unroll
          for (int c = 0; c < C::NCH; ++c)
            umma_bf16_x4<2>(d, a0 + c * (C::CHUNK >> 4), b0 + c * (C::CHUNK >> 4), p.idesc_qk,
                            c > 0 ? 1u : 0u);
          umma_commit(BAR(B_S_FULL + rt));
          if (rt == 1 || split) {
            umma_commit(BAR(B_K_EMPTY + kst));
            if (last_of_item) umma_commit(BAR(B_Q_EMPTY));
          }
        }
        __syncwarp();
        if (rt == 1 || split) ++gk;
        return true;
      };
      // P_rt(key tile i) * V for row tile rt (split: key tile 2 i + rt)
      auto issue_pv = [&](int rt, int i) -> bool {
        const int vst = gv % C::VSTAGES;
        if (!wait(B_P_FULL + rt, np[rt] & 1)) return false;
        ++np[rt];
        if (rt == 0 || split) {
          if (!wait(B_V_FULL + vst, (gv / C::VSTAGES) & 1)) return false;
          const int kv0 = key_tile<WIN>(tl, split ? 2 * i + rt : i) * 128;
          if (WIN && !F8 && (kv0 + 128 > L || (kv0 < tl.wt.lo && kv0 + 128 > p.sinks))) {
            // rows of keys no row of the item sees, whose blocks were not read
            for (int idx = lane; idx < 128 * 8 * C::NCH; idx += 32) {
              const int c = idx >> 10, row = (idx >> 3) & 127, u = idx & 7;
              if (!item_sees(tl, kv0 + row, 1, p.sinks))
                *reinterpret_cast<uint4*>(gbase + C::OFF_V + vst * C::KV_BYTES + c * C::CHUNK +
                                          row * 128 + u * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
          } else if (!WIN && !F8 && kv0 + 128 > L) {  // (the converters write such rows as zeros)
            // Rows of keys past the sequence end may hold anything (NaN too);
            // their P is 0, but 0 * NaN would poison O, so clear them.
            const int r0 = L - kv0;
            const int per_chunk = (128 - r0) * 8;  // 16-byte units
            for (int idx = lane; idx < per_chunk * C::NCH; idx += 32) {
              const int c = idx / per_chunk, rem = idx - c * per_chunk;
              const int row = r0 + (rem >> 3), u = rem & 7;
              *reinterpret_cast<uint4*>(gbase + C::OFF_V + vst * C::KV_BYTES + c * C::CHUNK +
                                        row * 128 + u * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
        }
        if (i == 0 && it > 0 && !wait(B_O_EMPTY + rt, (it - 1) & 1)) return false;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t d = tmem + C::TM_O + 128 * rt;
          const uint32_t a_tm = tmem + C::TM_S + 128 * rt;  // P_rt: 64 columns of bf16 pairs
          const uint64_t b0 = vmaj_base + ((C::OFF_V + vst * C::KV_BYTES) >> 4);
#pragma unroll
          for (int c = 0; c < 4; ++c)  // keys 32 c .. 32 c + 31: 16 P columns
            umma_bf16_ta_x2<(2048 >> 4)>(d, a_tm + C::pcol(c), b0 + ((c * 4096) >> 4), idesc_pv,
                                         (i > 0 || c > 0) ? 1u : 0u);
          umma_commit(BAR(B_PV_DONE + rt));
          if (rt == 1 || split) umma_commit(BAR(B_V_EMPTY + vst));
        }
        __syncwarp();
        if (rt == 1 || split) ++gv;
        return true;
      };

      if (split) {  // the same order, each row tile over its own half of the key tiles
        const int n0 = (tl.n + 1) / 2, n1 = tl.n / 2;  // n1 >= 1
        ok = issue_s(0, false) && issue_s(1, tl.n == 2);
        for (int i = 0; ok && i < n0; ++i) {
          ok = issue_pv(0, i);
          if (ok && i + 1 < n0) ok = issue_s(0, 2 * i + 3 == tl.n);
          if (ok && i < n1) ok = issue_pv(1, i);
          if (ok && i + 1 < n1) ok = issue_s(1, 2 * i + 4 == tl.n);
        }
        continue;
      }
      ok = issue_s(0, tl.n == 1) && issue_s(1, tl.n == 1);
      for (int i = 0; ok && i < tl.n; ++i) {
        const bool more = i + 1 < tl.n;
        const bool last_next = i + 2 == tl.n;
        ok = issue_pv(0, i);
        if (ok && more) ok = issue_s(0, last_next);
        if (ok) ok = issue_pv(1, i);
        if (ok && more) ok = issue_s(1, last_next);
      }
    }
    // every MMA issued above has completed before TMEM is released
    if (elect_one()) umma_commit(BAR(B_DRAIN));
    __syncwarp();
    mbar_wait_bounded(BAR(B_DRAIN), 0);
  } else if (warp < 2 + kSoftWarps) {
    // ======================= softmax + epilogue ==========================================
    // Row tile rt has warps 2 + 4*split*rt ...; within it, 4 warps per column
    // half hf (warp w reads TMEM lanes 32*(w%4) .. 32*(w%4)+31).
    const int sw = warp - 2;
    const int rt = sw / (4 * kSplit);     // row tile of this warp
    const int hf = (sw / 4) % kSplit;     // column half (0 without the split)
    const int q4 = warp & 3;              // TMEM lane quarter this warp may access
    const int m = q4 * 32 + lane;         // row == TMEM lane
    const uint32_t trow = ((uint32_t)(q4 * 32) << 16) + tmem;
    const uint32_t s_addr = trow + C::TM_S + 128 * rt;
    const uint32_t o_addr = trow + C::TM_O + 128 * rt;
    constexpr int OCH = D / 32 / kSplit;  // 32-column O chunks per thread
    float* const xch = reinterpret_cast<float*>(gbase + C::OFF_XCH);
    int nx = 0;  // exchanges done
    // Combine a per-thread row value with the other half's (max or sum). The
    // two halves meet on an mbarrier with a bounded wait (a half that gives up
    // cannot strand the other); exchange k uses barrier and buffer k % 2, so
    // a barrier is reused only after every thread has passed the other one.
    auto exchange = [&](float v, bool take_max, bool& good) -> float {
      if constexpr (kSplit == 1) {
        return v;
      } else {
        const int k = nx++;
        float* const xb = xch + ((rt * 2 + (k & 1)) * 2) * 128;
        xb[hf * 128 + m] = v;
        mbar_arrive(BAR(B_XCH + rt * 2 + (k & 1)));  // release: the store above is visible
        if (!wait(B_XCH + rt * 2 + (k & 1), (k >> 1) & 1)) {
          good = false;
          return v;
        }
        const float o = xb[(1 - hf) * 128 + m];
        return take_max ? fmaxf(v, o) : v + o;
      }
    };
    int ns = 0, it = 0;  // S_rt events consumed; work items done
    bool ok = true;
    for (int t = snake_item(it, ctas); ok && t < ntiles; t = snake_item(++it, ctas)) {
      const Item tl = get_item<D, G, MODE, WIN>(p, t);
      const int L = tl.L;
      int qlen = 0, j = 0, lim;
      if constexpr (PREFIX) {
        lim = L - 1;  // the whole prefix, for every row
      } else {
        qlen = __ldg(p.qsl + tl.req + 1) - __ldg(p.qsl + tl.req);
        const int ctx = L - qlen;
        j = tl.j0 + rt * C::TOK + m / G;  // chunk token of this row
        lim = min(ctx + j, L - 1);        // last key this row may see
      }
      // m_raw is the largest raw score so far, m_used that times the scale (-inf:
      // no key seen). P = exp2(score x scale - m_used) takes one FMA, exact but for
      // the rounding of m_used: a factor common to all of a row's P. `far`: it
      // could overflow P (kFar) in some row of the warp; the raw differences are
      // then taken first, and the largest P is 1 whatever the scores' size.
      float m_used = -INFINITY, m_raw = -INFINITY, l = 0.f;
      bool far = false;
      const bool split = MODE == kGroups && tl.split;
      const int n = split ? (tl.n + 1 - rt) / 2 : tl.n;
      for (int i = 0; i < n; ++i) {
        // S_rt(i) complete implies every earlier MMA is too: O_rt is stable
        // and P_rt(i-1) has been consumed.
        if (!wait(B_S_FULL + rt, ns & 1)) { ok = false; break; }
        ++ns;
        tc_fence_after();
        const int kv0 = key_tile<WIN>(tl, split ? 2 * i + rt : i) * 128;
        const bool unmasked = __all_sync(kAll, kv0 + 127 <= lim);
        // WIN: the row sees lo .. lim and the sinks; whole and empty runs of 32
        // columns are told apart, since a window has two edges to every item
        const int lo = WIN ? max(0, lim - p.window + 1) : 0;
        uint32_t whole = unmasked ? 15u : 0u, empty = 0u;  // bit c: columns 32 c .. 32 c + 31
        if constexpr (WIN) {
          whole = 0u;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int k0 = kv0 + c * 32;
            if (__all_sync(kAll, k0 + 31 <= lim && (k0 >= lo || k0 + 31 < p.sinks))) whole |= 1u << c;
            if (__all_sync(kAll, k0 > lim || (k0 + 31 < lo && k0 >= p.sinks))) empty |= 1u << c;
          }
        }
        // pass 1: row max of the raw scores over visible keys
        float mx = -INFINITY;
#pragma unroll 1
        for (int cc = 0; cc < C::CPH; ++cc) {
          const int c = hf * C::CPH + cc;
          if (WIN && (empty >> c & 1u)) continue;
          uint32_t r[32];
          tmem_ld32(s_addr + c * 32, r);
          tmem_wait_ld();
          if (whole >> c & 1u) {
#pragma unroll
            for (int e = 0; e < 32; ++e) mx = fmaxf(mx, __uint_as_float(r[e]));
          } else {
            const int lim_c = lim - kv0 - c * 32;  // columns e <= lim_c are visible
            const int lo_c = lo - kv0 - c * 32, s_c = WIN ? p.sinks - kv0 - c * 32 : 0;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              mx = fmaxf(mx, e <= lim_c && (!WIN || e >= lo_c || e < s_c) ? __uint_as_float(r[e])
                                                                          : -INFINITY);
          }
        }
        mx = exchange(mx, true, ok);         // the whole row's max
        if (!ok) break;
        // A tile of which the row sees no key (mx = -inf) changes nothing.
        const float mt = mx * p.scale_log2;
        const float was = m_used, was_raw = m_raw;
        float alpha = 1.f;
        bool resc = false;
        if (i == 0) {
          m_used = mt;
          m_raw = mx;
        } else if (mt > m_used + 8.f) {
          alpha = exp2f(m_used - mt);
          m_used = mt;
          m_raw = mx;
          resc = true;
        }
        if (__any_sync(kAll, resc || fabsf(mt) > kFar)) {
          const bool blind = mx == -INFINITY;
          far = far || __any_sync(kAll, fabsf(mt) > kFar && !blind);
          if (far && i > 0) {  // the same by the raw scores, whose products may round alike
            const bool none = was == -INFINITY;
            resc = !blind && (none || (mx - was_raw) * p.scale_log2 > 8.f);
            alpha = !resc ? 1.f : none ? 0.f : exp2f((was_raw - mx) * p.scale_log2);
            m_used = resc ? mt : was;
            m_raw = resc ? mx : was_raw;
          }
          if (__any_sync(kAll, resc)) {
#pragma unroll 1
            for (int oc = 0; oc < OCH; ++oc) {
              const int c = hf * OCH + oc;
              uint32_t o[32];
              tmem_ld32(o_addr + c * 32, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(o_addr + c * 32, o);
            }
            tmem_wait_st();
          }
        }
        l *= alpha;
        if (far) {  // S - m_raw in the place of S
#pragma unroll 1
          for (int cc = 0; cc < C::CPH; ++cc) {
            const uint32_t at = s_addr + (hf * C::CPH + cc) * 32;
            uint32_t r[32];
            tmem_ld32(at, r);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) - m_raw);
            tmem_st32(at, r);
          }
          tmem_wait_st();
        }
        // pass 2: P = exp2(s * scale - m) as bf16 pairs, written over this
        // thread's own S columns: chunk c's 16 P columns start at pcol(c),
        // which only covers S columns this thread has already read.
        const float nm = far ? 0.f : -m_used;
        const float sc = p.scale_log2;
        float l2[2] = {0.f, 0.f};  // two partial sums: shorter dependency chains
#pragma unroll 1
        for (int cc = 0; cc < C::CPH; ++cc) {
          const int c = hf * C::CPH + cc;
          uint32_t w[16];
          if (WIN && (empty >> c & 1u)) {
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = 0u;
            tmem_st16(s_addr + C::pcol(c), w);
            continue;
          }
          uint32_t r[32];
          tmem_ld32(s_addr + c * 32, r);
          tmem_wait_ld();
          if (whole >> c & 1u) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float p0 = ex2_approx(fmaf(__uint_as_float(r[2 * e]), sc, nm));
              const float p1 = ex2_approx(fmaf(__uint_as_float(r[2 * e + 1]), sc, nm));
              l2[e & 1] += p0 + p1;
              w[e] = float2_to_bf16x2(p0, p1);
            }
          } else {
            const int lim_c = lim - kv0 - c * 32;
            const int lo_c = lo - kv0 - c * 32, s_c = WIN ? p.sinks - kv0 - c * 32 : 0;
            auto sees = [&](int e) { return e <= lim_c && (!WIN || e >= lo_c || e < s_c); };
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float p0 = sees(2 * e) ? ex2_approx(fmaf(__uint_as_float(r[2 * e]), sc, nm)) : 0.f;
              const float p1 =
                  sees(2 * e + 1) ? ex2_approx(fmaf(__uint_as_float(r[2 * e + 1]), sc, nm)) : 0.f;
              l2[e & 1] += p0 + p1;
              w[e] = float2_to_bf16x2(p0, p1);
            }
          }
          tmem_st16(s_addr + C::pcol(c), w);
        }
        l += l2[0] + l2[1];
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(BAR(B_P_FULL + rt));
      }
      if (!ok) break;
      // ---- epilogue: O / l -> bf16 rows of out ----
      if (!wait(B_PV_DONE + rt, (ns - 1) & 1)) { ok = false; break; }
      tc_fence_after();
      l = exchange(l, false, ok);  // the whole row's sum
      if (!ok) break;
      if constexpr (PREFIX) {
        // fp32 partial of (chunk, token, kv head), head m % G of the slot
        const int tok = tl.tok0 + (split ? 0 : rt * C::TOK) + m / G;
        const int h = m % G;
        const bool store = tok < tl.tok_end;
        float* const slot = p.prefix_partials +
                            (((size_t)(tl.chunk + (split ? rt : 0)) * p.num_tokens +
                              (store ? tok : 0)) *
                                 p.num_kv_heads + tl.kv) * p.slot_floats;
        if (store && hf == 0) {
          __stcg(slot + h, m_used);
          __stcg(slot + G + h, l);
        }
#pragma unroll 1
        for (int oc = 0; oc < OCH; ++oc) {
          const int c = hf * OCH + oc;
          uint32_t o[32];
          tmem_ld32(o_addr + c * 32, o);
          tmem_wait_ld();
          if (store) {
            float* const dst = slot + 16 + h * D + c * 32;
#pragma unroll
            for (int v = 0; v < 8; ++v)
              __stcg(reinterpret_cast<float4*>(dst + 4 * v),
                     make_float4(__uint_as_float(o[4 * v]), __uint_as_float(o[4 * v + 1]),
                                 __uint_as_float(o[4 * v + 2]), __uint_as_float(o[4 * v + 3])));
          }
        }
        tc_fence_before();
        mbar_arrive(BAR(B_O_EMPTY + rt));
        continue;
      }
      const float inv = p.v_scale / l;
      const bool store = j < qlen;
      uint16_t* const orow =
          p.out + ((size_t)(tl.tok0 - tl.j0 + j) * p.num_q_heads + (size_t)tl.kv * G + (m % G)) * D;
#pragma unroll 1
      for (int oc = 0; oc < OCH; ++oc) {
        const int c = hf * OCH + oc;
        uint32_t o[32];
        tmem_ld32(o_addr + c * 32, o);
        tmem_wait_ld();
        if (store) {
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint4 pk;
            pk.x = float2_to_bf16x2(__uint_as_float(o[8 * v + 0]) * inv, __uint_as_float(o[8 * v + 1]) * inv);
            pk.y = float2_to_bf16x2(__uint_as_float(o[8 * v + 2]) * inv, __uint_as_float(o[8 * v + 3]) * inv);
            pk.z = float2_to_bf16x2(__uint_as_float(o[8 * v + 4]) * inv, __uint_as_float(o[8 * v + 5]) * inv);
            pk.w = float2_to_bf16x2(__uint_as_float(o[8 * v + 6]) * inv, __uint_as_float(o[8 * v + 7]) * inv);
            *reinterpret_cast<uint4*>(orow + c * 32 + 8 * v) = pk;
          }
        }
      }
      tc_fence_before();
      mbar_arrive(BAR(B_O_EMPTY + rt));
    }
  } else if constexpr (F8) {
    // ======================= E4M3 converters (warps 10-13: K, 14-17: V) ==================
    constexpr int LPR = D / 16, RPI = 32 / LPR, NI = LPR;  // lanes a row, rows and parts a warp
    const bool is_v = warp >= 2 + kSoftWarps + 4;
    const int cw = (warp - (2 + kSoftWarps)) & 3;  // key rows 32 cw .. + 31 of a tile: two blocks
    const int nst = is_v ? C::VSTAGES : C::KSTAGES;
    const int full = is_v ? B_V_FULL : B_K_FULL, landed = is_v ? B_V_RAW : B_K_RAW;
    unsigned char* const ring = gbase + (is_v ? C::OFF_V : C::OFF_K);
    const unsigned char* const scs = gbase + C::OFF_SC + (is_v ? C::KSTAGES * 128 : 0);
    const volatile unsigned char* const copied = gbase + C::OFF_GOOD + (is_v ? C::KSTAGES : 0);
    int st = 0, parity = 0, it = 0;
    bool ok = true;
    for (int t = snake_item(it, ctas); ok && t < ntiles; t = snake_item(++it, ctas)) {
      const Item tl = get_item<D, G, MODE, WIN>(p, t);
      for (int i = 0; i < tl.n; ++i) {
        const int key0 = key_tile<WIN>(tl, i) * 128 + cw * 32 + lane / LPR;
        uint32_t rows = 0;  // which of this lane's rows are keys
#pragma unroll
        for (int n = 0; n < NI; ++n) {
          const int key = key0 + n * RPI;
          if (WIN ? item_sees(tl, key, 1, p.sinks) : key < tl.L) rows |= 1u << n;
        }
        if (!wait(landed + st, parity)) { ok = false; break; }
        // the rows of a block outside the pool (reported) are zeros
        const int good = copied[st] >> (2 * cw);
        constexpr uint32_t kFirst = (1u << NI / 2) - 1u;
        rows &= (good & 1 ? kFirst : 0u) | (good & 2 ? kFirst << NI / 2 : 0u);
        unsigned char* const stage = ring + st * C::KV_BYTES;
        widen_rows<D, KV == 2>(stage, stage + C::OFF_RAW, scs + st * 128, rows, cw, lane);
        if (lane == 0) mbar_arrive(BAR(full + st));
        if (++st == nst) {
          st = 0;
          parity ^= 1;
        }
      }
    }
  }

  if constexpr (MODE == kOnePrefix) {
    // The split-KV grid launched after this one may start now; this grid does
    // not complete before the planner (and the KV write before it) has, so a
    // dependent that waits for this grid sees the plan too. (The prefill-chunk
    // grid releases its dependent only by completing: triggering here too
    // measured 0.53 vs 0.435 ms per mixed step.) Overlapped, it did both at
    // the top.
    if (!p.overlap) {
      griddep_launch_dependents();
      griddep_wait();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

namespace {

template <int D, int G, int MODE, int KV, bool WIN>
cudaError_t launch_prefill_t(const PrefillLaunch& a, int num_sms, cudaStream_t s) {
  using C = PCfg<D, G>;
  constexpr bool F8 = KV != 0;
  PrefillParams p;
  {
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)a.num_q_heads, (uint64_t)a.num_tokens};
    const uint64_t str[2] = {(uint64_t)D * 2, (uint64_t)a.num_q_heads * D * 2};
    const uint32_t box[3] = {64, (uint32_t)G, (uint32_t)C::TOK};
    if (!encode_tmap_bf16(&p.tm_q, 3, a.q, dims, str, box)) return cudaErrorInvalidValue;
  }
  if (!F8) {  // E4M3 K/V are loaded by the converter warps, not by TMA
    const uint64_t rows = (uint64_t)a.num_blocks * a.num_kv_heads * kBlockSize;
    const uint64_t dims[2] = {(uint64_t)D, rows};
    const uint64_t str[1] = {(uint64_t)D * 2};
    const uint32_t box[2] = {64, (uint32_t)kBlockSize};
    if (!encode_tmap_bf16(&p.tm_k, 2, a.k_cache, dims, str, box)) return cudaErrorInvalidValue;
    if (!encode_tmap_bf16(&p.tm_v, 2, a.v_cache, dims, str, box)) return cudaErrorInvalidValue;
  }
  p.qsl = a.qsl;
  p.seq_lens = a.seq_lens;
  p.block_tables = a.block_tables;
  p.out = a.out;
  p.header = a.header;
  p.tiles = a.tiles;
  p.bt_stride = a.bt_stride;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.num_blocks = a.num_blocks;
  p.scale_log2 = fmaxf(fabsf(a.scale_log2), FLT_TRUE_MIN);
  p.idesc_qk = idesc_bf16_f32(128, 128, false) | (a.scale_log2 < 0.f ? kIdescNegateA : 0u);
  p.err = a.err;
  p.num_tokens = a.num_tokens;
  p.prefix_len = a.prefix_len;
  p.prefix_chunks = a.prefix_chunks;
  p.prefix_pairs = prefix_pairs(a.num_tokens, G);
  p.slot_floats = a.slot_floats;
  p.prefix_partials = a.prefix_partials;
  p.k_cache8 = F8 ? static_cast<const unsigned char*>(a.k_cache) : nullptr;
  p.v_cache8 = F8 ? static_cast<const unsigned char*>(a.v_cache) : nullptr;
  p.scales = a.scales;
  p.v_scale = F8 ? a.v_scale : 1.f;
  p.shared_items = a.shared_items;
  p.overlap = a.overlap;
  p.window = a.window;
  p.sinks = a.sinks;
  int grid = num_sms;
  if (MODE == kOnePrefix) {
    const int items = p.prefix_pairs * a.num_kv_heads * a.prefix_chunks;
    grid = items < num_sms ? items : num_sms;
    // overlapped cascade: the pass keeps to its share of the SMs
    if (a.overlap && a.prefix_ctas > 0 && a.prefix_ctas < grid) grid = a.prefix_ctas;
  }

  auto kern = pa_prefill_kernel<D, G, MODE, KV, WIN>;
  static bool attr_set[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(F8 ? kThreadsF8 : kThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

template <int MODE, int KV, bool WIN>
cudaError_t launch_prefill_mode(const PrefillLaunch& a, int num_sms, cudaStream_t s) {
  const int G = a.num_q_heads / a.num_kv_heads;
  if (a.head_dim == 128) {
    switch (G) {
      case 1: return launch_prefill_t<128, 1, MODE, KV, WIN>(a, num_sms, s);
      case 2: return launch_prefill_t<128, 2, MODE, KV, WIN>(a, num_sms, s);
      case 4: return launch_prefill_t<128, 4, MODE, KV, WIN>(a, num_sms, s);
      case 8: return launch_prefill_t<128, 8, MODE, KV, WIN>(a, num_sms, s);
    }
  } else if (a.head_dim == 64) {
    switch (G) {
      case 1: return launch_prefill_t<64, 1, MODE, KV, WIN>(a, num_sms, s);
      case 2: return launch_prefill_t<64, 2, MODE, KV, WIN>(a, num_sms, s);
      case 4: return launch_prefill_t<64, 4, MODE, KV, WIN>(a, num_sms, s);
      case 8: return launch_prefill_t<64, 8, MODE, KV, WIN>(a, num_sms, s);
    }
  }
  return cudaErrorInvalidValue;
}

}  // namespace pa
