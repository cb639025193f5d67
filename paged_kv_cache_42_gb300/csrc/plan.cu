// Planner: turns the batch metadata into the work lists of the two
// attention kernels, on the device, once per pa_attention call.
//
//  - Requests with at least kPrefillMinQlen new tokens become tensor-core
//    work items (two 128-row tiles of one kv head each), bucket-sorted by the
//    number of 64-key tiles they read, longest first.
//  - Every other new token becomes a split-KV unit: the compacted list
//    {token, request, keys to attend, first flattened position} with the
//    prefix sum of Hkv * ceil(keys / 16) positions, which the split-KV
//    kernel's workers slice into equal parts.
//  - Cascade calls (common prefix of prefix_blocks blocks): every span goes
//    to the split-KV path with the prefix blocks left out of its positions;
//    requests must see the whole prefix and start with request 0's prefix
//    blocks, which is checked here.
//  - Shared calls (groups of requests, each with its own prefix): the tokens of a
//    group that share its prefix become units over their own keys only - the
//    unit's `req` is then the offset of its first own block in the tables (the
//    split-KV kernels run with a row stride of 1), its `len` the keys from there
//    on - and every (pair of row tiles, kv head, key chunk) of a prefix a work
//    item of the prefix pass. More CTAs check the tables' prefix blocks, a group
//    each.
// Invalid spans or lengths are skipped and reported on the device error word.
//  - Windowed calls count only the blocks (tiles) that hold a key the token
//    (an item's rows) attends to.
// A decode-only batch needs no planner: the split-KV kernel builds its own
// unit list.
#include "pa_internal.h"
#include "ptx.cuh"

namespace pa {

constexpr unsigned kFull = 0xffffffffu;

constexpr int kPlanThreads = 1024;

__device__ __forceinline__ long long block_exclusive_scan(long long v, long long* total,
                                                          long long* sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sm[warp] = x;
  __syncthreads();
  if (warp == 0) {
    long long s = lane < nw ? sm[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(kFull, s, o);
      if (lane >= o) s += y;
    }
    sm[lane] = s;
  }
  __syncthreads();
  const long long before = warp ? sm[warp - 1] : 0;
  *total = sm[nw - 1];
  __syncthreads();
  return before + x - v;
}

constexpr int kSharedCandidates = 256;  // lengths of a shared call's key chunks looked at
constexpr int kTileBuckets = 512;  // tiles sorted by key-tile count, longest first

// ---- shared calls -----------------------------------------------------------------
// The group of request r, or -1: its prefix in blocks goes to *blocks (0: none, or
// not one that this call takes). start, lens: group_start_loc and prefix_lens.
__device__ __forceinline__ int shared_group(const PlanParams& p, const int* start, const int* lens,
                                            int r, int* blocks) {
  int lo = 0, hi = p.num_groups;  // the last group that starts at or before r
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= r) lo = mid; else hi = mid;
  }
  const int a = start[lo], b = start[lo + 1], len = lens[lo];
  *blocks = 0;
  if (r < a || r >= b || a < 0 || b > p.num_reqs) return -1;
  if (len > 0 && len % kBlockSize == 0 && len <= p.max_prefix_len) *blocks = len / kBlockSize;
  return lo;
}

// Request r's span and length, false if they do not agree (reported if asked).
__device__ __forceinline__ bool check_request(const PlanParams& p, int r, int& q0, int& qlen, int& L,
                                              bool report) {
  // the three loads are issued together: one DRAM round trip, not two
  q0 = __ldg(p.qsl + r);
  const int q1 = __ldg(p.qsl + r + 1);
  L = __ldg(p.seq_lens + r);
  if (q0 < 0 || q1 < q0 || q1 > p.num_tokens) {
    if (report) report_error(p.err, PA_DEVERR_QSL, r);
    return false;
  }
  qlen = q1 - q0;
  if (L < qlen || (L + kBlockSize - 1) / kBlockSize > p.max_blocks_per_req ||
      qlen > p.max_query_len || L > p.max_seq_len || L - qlen < p.prefix_blocks * kBlockSize) {
    if (report) report_error(p.err, PA_DEVERR_LENGTHS, r);
    return false;
  }
  return true;
}

// Whether request r shares a prefix of `blocks` blocks: it has tokens on the
// split-KV path, and they see all of it.
__device__ __forceinline__ bool shares(const PlanParams& p, int qlen, int L, int blocks) {
  return blocks > 0 && qlen > 0 && !(p.use_prefill && qlen >= kPrefillMinQlen) &&
         L - qlen >= blocks * kBlockSize;
}

// A pair of row tiles with `left` tokens (its own and the group's behind it): rows
// that fit one tile are split over the two by key tiles (SharedItem). Two tiles of
// keys take them 4/3 of the time that one takes a pair of full tiles (1.6 and 2.4 us
// a tile of a long prefix), so that their key chunks are half as long again (ct tiles
// otherwise).
__device__ __forceinline__ bool shared_split(int left, int group) { return left * group <= 128; }
__device__ __forceinline__ int shared_len(int ct, bool split) { return split ? ct + (ct + 1) / 2 : ct; }
__device__ __forceinline__ int shared_chunks(int tiles, int ct, bool split) {
  const int len = shared_len(ct, split);
  return (tiles + len - 1) / len;
}
// The partials that such a pair leaves of a prefix: two of a split chunk, unless it has
// one tile only.
__device__ __forceinline__ int shared_parts(int tiles, int ct, bool split) {
  const int chunks = shared_chunks(tiles, ct, split);
  return split ? 2 * chunks - (tiles - (chunks - 1) * shared_len(ct, true) == 1 ? 1 : 0) : chunks;
}

// CTAs 1 .. of a shared call's plan: every request that shares its group's prefix
// starts with the same blocks as the first one that does. A few groups are taken by
// four CTAs each, a share of the requests per CTA; many by one, in turn.
__host__ __device__ inline int check_parts(int num_groups) { return num_groups > 32 ? 1 : 4; }
__device__ void check_shared_tables(const PlanParams& p) {
  __shared__ int s_leader;
  const int warps = blockDim.x >> 5, parts = check_parts(p.num_groups);
  const int part = ((int)blockIdx.x - 1) % parts;
  for (int g = ((int)blockIdx.x - 1) / parts; g < p.num_groups;
       g += ((int)gridDim.x - 1) / parts) {
    const int a = __ldg(p.group_start + g), b = __ldg(p.group_start + g + 1);
    const int len = __ldg(p.prefix_lens + g);
    if (threadIdx.x == 0) {
      if (a < 0 || b < a || b > p.num_reqs) report_error(p.err, PA_DEVERR_QSL, g);
      else if (len < 0 || len % kBlockSize != 0 || len > p.max_prefix_len)
        report_error(p.err, PA_DEVERR_PREFIX, g);
      s_leader = 0x7fffffff;
    }
    if (a < 0 || b <= a || b > p.num_reqs || len <= 0 || len % kBlockSize != 0 ||
        len > p.max_prefix_len)
      continue;  // the same for every thread
    const int blocks = len / kBlockSize;
    __syncthreads();
    int q0, qlen, L;
    for (int r = a + (int)threadIdx.x; r < b; r += blockDim.x)
      if (check_request(p, r, q0, qlen, L, false) && shares(p, qlen, L, blocks)) {
        atomicMin(&s_leader, r);
        break;  // a thread's later requests have larger numbers
      }
    __syncthreads();
    const int leader = s_leader;
    if (leader < b) {
      const int32_t* const want = p.block_tables + (size_t)leader * p.max_blocks_per_req;
      // a warp takes a request at a time, with several loads in flight per lane
      for (int r = leader + 1 + part * warps + (int)(threadIdx.x >> 5); r < b;
           r += parts * warps) {
        if (!check_request(p, r, q0, qlen, L, false) || !shares(p, qlen, L, blocks)) continue;
        const int32_t* const got = p.block_tables + (size_t)r * p.max_blocks_per_req;
        bool same = true;
#pragma unroll 8
        for (int i = (int)(threadIdx.x & 31); i < blocks; i += 32)
          same &= __ldg(got + i) == __ldg(want + i);
        if (!same) report_error(p.err, PA_DEVERR_PREFIX, r);
      }
    }
    __syncthreads();  // s_leader is read before the next group's
  }
}

template <bool SHARED>
__global__ void __launch_bounds__(kPlanThreads) pa_plan_kernel(PlanParams p) {
  // The lengths and tables may come from the grid before, and so may what the
  // cascade prefix pass reads, which this grid lets start next.
  if (!p.early_start) griddep_wait();
  // When the next grid has work that needs no plan (the cascade prefix
  // pass), let it start now; a grid that would only wait at its top for the
  // plan is released at the end of this one instead (starting it early
  // measured slower).
  if (p.early_trigger) griddep_launch_dependents();
  if constexpr (SHARED) {
    if (blockIdx.x > 0) {
      check_shared_tables(p);
      return;
    }
  }
  __shared__ long long scan_sm[32];
  __shared__ int bucket_cnt[kTileBuckets];
  __shared__ int bucket_pos[kTileBuckets];
  __shared__ int s_steps;    // prefill steps (item x key tile) of the batch
  __shared__ int s_workers;  // split-KV workers the slicing uses
  // Per-token scratch: {request, keys to attend}, then the compacted units'
  // first positions. In shared memory when the batch fits, else in the
  // workspace.
  extern __shared__ int2 dsm[];
  const int T = p.num_tokens;
  const bool in_smem = T <= kPlanSmemTokens;
  int2* const raw = in_smem ? dsm : p.raw;
  int* const ubase = in_smem ? reinterpret_cast<int*>(dsm + T) : nullptr;
  // a prefill work item is a pair of 128-row tiles: 2 * 128 / G chunk tokens
  const int tok_per_item = 2 * (128 / p.group);
  if (p.use_prefill)
    for (int b = threadIdx.x; b < kTileBuckets; b += blockDim.x) bucket_cnt[b] = 0;
  for (int t = threadIdx.x; t < T; t += blockDim.x) raw[t] = make_int2(-1, 0);
  if (threadIdx.x == 0) s_steps = 0;
  __syncthreads();

  // a request is valid when its span lies in [0, T] and its lengths agree
  auto check = [&](int r, int& q0, int& qlen, int& L, bool report) -> bool {
    return check_request(p, r, q0, qlen, L, report);
  };
  auto tile_nkv = [&](int L, int ctx, int j0) -> int {  // 128-key tiles the item needs
    const int last = min(L - 1, ctx + j0 + tok_per_item - 1);  // last key of the item's rows
    if (p.window > 0) return win_tiles(ctx + j0, last, p.window, p.sinks).n;
    return last / 128 + 1;
  };

  if (p.prefix_blocks > 0) {  // every table starts with request 0's prefix blocks
    // kCheckBatch independent loads per thread before any compare: one DRAM
    // round trip per batch rather than one per entry
    constexpr int kCheckBatch = 8;
    const long long n = (long long)(p.num_reqs - 1) * p.prefix_blocks;
    for (long long i0 = threadIdx.x; i0 < n; i0 += (long long)kCheckBatch * blockDim.x) {
      int got[kCheckBatch], want[kCheckBatch];
#pragma unroll
      for (int k = 0; k < kCheckBatch; ++k) {
        const long long i = i0 + (long long)k * blockDim.x;
        got[k] = want[k] = 0;
        if (i < n) {
          const int r = 1 + (int)(i / p.prefix_blocks), b = (int)(i % p.prefix_blocks);
          got[k] = __ldg(p.block_tables + (size_t)r * p.max_blocks_per_req + b);
          want[k] = __ldg(p.block_tables + b);
        }
      }
#pragma unroll
      for (int k = 0; k < kCheckBatch; ++k)
        if (got[k] != want[k])
          report_error(p.err, PA_DEVERR_PREFIX,
                       1 + (int)((i0 + (long long)k * blockDim.x) / p.prefix_blocks));
    }
  }
  // shared: of every group, its tokens that share the prefix (how many, the first
  // and behind the last) and the first request of theirs
  __shared__ int s_first[SHARED ? kMaxSharedGroups : 1], s_count[SHARED ? kMaxSharedGroups : 1];
  __shared__ int s_lo[SHARED ? kMaxSharedGroups : 1], s_hi[SHARED ? kMaxSharedGroups : 1];
  __shared__ int s_tiles[SHARED ? kMaxSharedGroups : 1];  // key tiles of its prefix; 0: not shared
  // its pairs of row tiles: full ones, and a split one or none
  __shared__ int s_full[SHARED ? kMaxSharedGroups : 1], s_split[SHARED ? kMaxSharedGroups : 1];
  __shared__ int s_start[SHARED ? kMaxSharedGroups + 1 : 1], s_len[SHARED ? kMaxSharedGroups : 1];
  __shared__ unsigned long long s_best, s_saved;
  __shared__ int s_pairs;  // pairs of row tiles of the groups that could share
  // of each candidate for the chunk length: items of a kv head, steps of the longest
  __shared__ int s_items[SHARED ? kSharedCandidates : 1], s_longest[SHARED ? kSharedCandidates : 1];
  bool sharing = false;  // whether any group does, and it pays (the same for every thread)
  // what this thread's (first) request is, kept from one pass over them to the next
  int my_q0 = 0, my_qlen = 0, my_L = 0, my_group = -1, my_blocks = 0;
  bool my_valid = false;
  if constexpr (SHARED) {
    // a thread's first group is loaded beside its first request: one round trip
    const int g0 = (int)threadIdx.x;
    const int start0 = g0 <= p.num_groups ? __ldg(p.group_start + g0) : 0;
    const int len0 = g0 < p.num_groups ? __ldg(p.prefix_lens + g0) : 0;
    if (threadIdx.x < p.num_reqs)
      my_valid = check(threadIdx.x, my_q0, my_qlen, my_L, true);
    for (int g = g0; g <= p.num_groups; g += blockDim.x) {
      s_start[g] = g == g0 ? start0 : __ldg(p.group_start + g);
      if (g == p.num_groups) break;
      s_len[g] = g == g0 ? len0 : __ldg(p.prefix_lens + g);
      s_first[g] = s_lo[g] = 0x7fffffff;
      s_count[g] = s_hi[g] = 0;
    }
    for (int t = threadIdx.x; t < T; t += blockDim.x) p.tok_parts[t] = 0;
    __syncthreads();
    for (int r = threadIdx.x; r < p.num_reqs; r += blockDim.x) {
      int q0 = my_q0, qlen = my_qlen, L = my_L, blocks;
      const bool mine = r == (int)threadIdx.x;
      if (mine ? !my_valid : !check(r, q0, qlen, L, true)) continue;
      int g = shared_group(p, s_start, s_len, r, &blocks);
      if (g >= 0 && !shares(p, qlen, L, blocks)) g = -1;
      if (mine) {
        my_group = g;
        my_blocks = blocks;
      }
      if (g < 0) continue;
      atomicMin(&s_first[g], r);
      atomicAdd(&s_count[g], qlen);
      atomicMin(&s_lo[g], q0);
      atomicMax(&s_hi[g], q0 + qlen);
    }
    if (threadIdx.x < kSharedCandidates) s_items[threadIdx.x] = s_longest[threadIdx.x] = 0;
    if (threadIdx.x == 0) {
      s_best = ~0ull;
      s_saved = 0ull;
      s_pairs = 0;
    }
    __syncthreads();
    // what sharing saves of reading, and whether that pays for the prefix pass
    // (atomics of 64 bits on shared memory are loops: one per warp)
    unsigned long long saved = 0;
    int shared_pairs = 0;
    for (int g = threadIdx.x; g < p.num_groups; g += blockDim.x)
      if (s_count[g] >= kSharedMinTokens) {
        saved += (unsigned long long)(s_count[g] - 1) * (unsigned)(s_len[g] / kBlockSize) *
                     (unsigned)p.position_bytes +
                 (s_len[g] >= kSharedLong ? p.shared_min_bytes : 0ull);
        shared_pairs += (s_hi[g] - s_lo[g] + tok_per_item - 1) / tok_per_item;
      }
    if ((int)(threadIdx.x & ~31u) < p.num_groups) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        saved += __shfl_xor_sync(kFull, saved, o);
        shared_pairs += __shfl_xor_sync(kFull, shared_pairs, o);
      }
      if ((threadIdx.x & 31) == 0) {
        atomicAdd(&s_saved, saved);
        atomicAdd(&s_pairs, shared_pairs);
      }
    }
    __syncthreads();
    const unsigned rounds =
        (unsigned)(((long long)s_pairs * p.num_kv_heads + p.num_sms - 1) / p.num_sms);
    sharing = s_saved > 0 && s_saved >= p.shared_min_bytes * rounds;
  }
  if (SHARED && sharing) {
    for (int g = threadIdx.x; g < p.num_groups; g += blockDim.x) {
      s_tiles[g] = s_count[g] >= kSharedMinTokens ? (s_len[g] + 127) / 128 : 0;
      const int n = s_tiles[g] > 0 ? s_hi[g] - s_lo[g] : 1;
      const int pairs = (n + tok_per_item - 1) / tok_per_item;
      s_full[g] = pairs - (shared_split(n - (pairs - 1) * tok_per_item, p.group) ? 1 : 0);
      s_split[g] = pairs - s_full[g];
    }
    __syncthreads();
    // The key chunks' length: of each candidate, the time of the rounds that its items
    // take on the SMs, in steps. Many groups: every fourth length, and more threads to
    // each (planning of 256 groups 30 -> 20 us, of 1024 68 -> 33).
    const int step = p.num_groups > 64 ? 4 : 1, cands = kSharedCandidates / step;
    {
      const int c = (int)threadIdx.x % cands, ct = p.chunk_tiles + c * step;
      int items = 0, longest = 0;  // steps
      // (an estimate: the divisions need not be exact)
      const float by = 1.f / (float)ct, by_split = 1.f / (float)shared_len(ct, true);
      for (int g = (int)threadIdx.x / cands; g < p.num_groups; g += (int)blockDim.x / cands) {
        const int tiles = s_tiles[g];
        if (tiles == 0) continue;
        const int full = s_full[g], split = s_split[g];
        items += full * (int)ceilf((float)tiles * by) + split * (int)ceilf((float)tiles * by_split);
        longest = max(longest, min(ct, full > 0 ? tiles : (2 * tiles + 2) / 3));
      }
      if (items > 0) {
        atomicAdd(&s_items[c], items);
        atomicMax(&s_longest[c], longest);
      }
    }
    __syncthreads();
    if ((int)threadIdx.x < cands) {
      const int ct = p.chunk_tiles + (int)threadIdx.x * step;
      const float rounds =
          ceilf((float)s_items[threadIdx.x] * (float)p.num_kv_heads / (float)p.num_sms);
      const float cost = rounds * (float)(s_longest[threadIdx.x] + kSharedItemSteps);
      unsigned long long best = (unsigned long long)__float_as_uint(cost) << 32 | (unsigned)ct;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long other = __shfl_xor_sync(kFull, best, o);
        best = other < best ? other : best;
      }
      if ((threadIdx.x & 31) == 0) atomicMin(&s_best, best);
    }
    __syncthreads();
  }
  const int chunk_tiles = sharing ? (int)(unsigned)s_best : 1;
  for (int r = threadIdx.x; r < p.num_reqs; r += blockDim.x) {
    int q0 = my_q0, qlen = my_qlen, L = my_L;
    const bool mine = SHARED && r == (int)threadIdx.x;
    if (mine ? !my_valid : !check(r, q0, qlen, L, !SHARED)) continue;
    const int ctx = L - qlen;
    if (p.use_prefill && qlen >= kPrefillMinQlen) {
      int steps = 0;
      for (int j0 = 0; j0 < qlen; j0 += tok_per_item) {
        const int nkv = tile_nkv(L, ctx, j0);
        atomicAdd(&bucket_cnt[min(nkv, kTileBuckets - 1)], p.num_kv_heads);
        steps += nkv;
      }
      if (p.overlap) atomicAdd(&s_steps, steps * p.num_kv_heads);
      continue;  // these tokens are not on the split-KV path
    }
    if constexpr (SHARED) {
      int g = my_group, blocks = my_blocks;
      if (!mine) {
        g = shared_group(p, s_start, s_len, r, &blocks);
        if (g >= 0 && !shares(p, qlen, L, blocks)) g = -1;
      }
      if (!sharing || g < 0 || s_count[g] < kSharedMinTokens) blocks = 0;
      const int at = r * p.max_blocks_per_req + blocks;
      for (int j = 0; j < qlen; ++j) {
        raw[q0 + j] = make_int2(at, ctx + j + 1 - blocks * kBlockSize);
        if (blocks > 0) {
          const int left = s_hi[g] - (q0 + j - ((q0 + j - s_lo[g]) & (tok_per_item - 1)));
          p.tok_parts[q0 + j] = shared_parts((blocks + 7) / 8, chunk_tiles, shared_split(left, p.group));
        }
      }
    } else {
      for (int j = 0; j < qlen; ++j) raw[q0 + j] = make_int2(r, ctx + j + 1);
    }
  }
  __syncthreads();
  if (p.use_prefill) {  // positions of the buckets, longest tiles first (exclusive scan, descending)
    static_assert(kTileBuckets <= kPlanThreads, "one bucket per thread");
    const int b = kTileBuckets - 1 - (int)threadIdx.x;  // blockDim is kPlanThreads here
    long long total;
    const long long ex = block_exclusive_scan(b >= 0 ? bucket_cnt[b] : 0, &total, scan_sm);
    if (b >= 0) bucket_pos[b] = (int)ex;
    if (threadIdx.x == 0) p.header->num_tiles = (int)total;
  } else if (threadIdx.x == 0) {
    p.header->num_tiles = 0;
  }
  __syncthreads();
  if (p.use_prefill) {
    for (int r = threadIdx.x; r < p.num_reqs; r += blockDim.x) {
      int q0, qlen, L;
      if (!check(r, q0, qlen, L, false) || qlen < kPrefillMinQlen) continue;
      const int ctx = L - qlen;
      for (int j0 = 0; j0 < qlen; j0 += tok_per_item) {
        const int nkv = tile_nkv(L, ctx, j0);
        const int at = atomicAdd(&bucket_pos[min(nkv, kTileBuckets - 1)], p.num_kv_heads);
        for (int kv = 0; kv < p.num_kv_heads; ++kv) p.tiles[at + kv] = PrefillTile{r, kv, j0, nkv};
      }
    }
  }
  if (SHARED && !sharing) {
    if (threadIdx.x == 0) p.header->num_prefix_items = 0;
  } else if constexpr (SHARED) {  // the prefix pass's items, group after group
    __shared__ int s_at[kMaxSharedGroups + 1];
    long long run = 0;
    for (int c0 = 0; c0 < p.num_groups; c0 += blockDim.x) {
      const int g = c0 + threadIdx.x;
      long long n = 0;
      if (g < p.num_groups && s_tiles[g] > 0)
        n = ((long long)s_full[g] * shared_chunks(s_tiles[g], chunk_tiles, false) +
             s_split[g] * shared_chunks(s_tiles[g], chunk_tiles, true)) * p.num_kv_heads;
      long long total;
      const long long ex = block_exclusive_scan(n, &total, scan_sm);
      // (an overfull list, which spans that overlap can make, is cut below)
      if (g < p.num_groups) s_at[g] = (int)min(run + ex, (long long)p.max_items + 1);
      run += total;
    }
    const int n = (int)min(run, (long long)p.max_items);
    if (threadIdx.x == 0) {
      s_at[p.num_groups] = n;
      p.header->num_prefix_items = n;
      if (run > n) report_error(p.err, PA_DEVERR_QSL, p.num_reqs);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      int lo = 0, hi = p.num_groups;  // s_at[lo] <= i < s_at[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_at[mid] <= i) lo = mid; else hi = mid;
      }
      const int tiles = s_tiles[lo], chunks = shared_chunks(tiles, chunk_tiles, false);
      // kv heads innermost, then chunks: neighbouring items read neighbouring keys
      int k = i - s_at[lo];
      SharedItem it;
      it.kv = k % p.num_kv_heads;
      k /= p.num_kv_heads;
      it.req = s_first[lo];
      it.tok_end = s_hi[lo];
      // only the group's last pair can be split, with fewer chunks than the others
      const int pair = min(k / chunks, s_full[lo] + s_split[lo] - 1), chunk = k - pair * chunks;
      it.tok0 = s_lo[lo] + pair * tok_per_item;
      const bool split = pair == s_full[lo];
      const int len = shared_len(chunk_tiles, split);
      it.i0 = chunk * len;
      it.n = min(len, tiles - it.i0);
      it.L = s_len[lo];
      it.part = split ? 2 * chunk : chunk;  // (the chunks before are whole)
      if (split && it.n > 1) it.kv |= kSharedSplit;
      p.shared_items[i] = it;
    }
    __syncthreads();  // scan_sm is used again
  }
  // compaction: tokens with keys become units with their first flattened position
  constexpr long long kLow = (1LL << 40) - 1;
  long long run_k = 0, run_w = 0;
  for (int c0 = 0; c0 < T; c0 += blockDim.x) {
    const int t = c0 + threadIdx.x;
    const int2 u = t < T ? raw[t] : make_int2(-1, 0);
    // blocks on the split-KV path: all the token sees, less a cascade prefix
    // (windowed: those that hold a key it attends to)
    const int nb = max(0, win_span(u.y, p.window, p.sinks).nb - p.prefix_blocks);
    // (token-major split-KV: one position per block, every kv head at once)
    const long long packed =
        ((long long)(nb > 0) << 40) | ((long long)nb * (p.token_major ? 1 : p.num_kv_heads));
    long long total;
    const long long ex = block_exclusive_scan(packed, &total, scan_sm);  // syncs: raw reads done
    if (nb > 0) {
      const int k = (int)(run_k + (ex >> 40));
      const int base = (int)(run_w + (ex & kLow));
      p.units[k] = UnitInfo{t, u.x, u.y, base};
      if (ubase) ubase[k] = base;
    }
    run_k += total >> 40;
    run_w += total & kLow;
  }
  const int K = (int)run_k, W = (int)run_w;
  if (threadIdx.x == 0) {
    p.units[K] = UnitInfo{T, -1, 0, W};  // base[K] = W
    if (ubase) ubase[K] = W;
    p.header->num_units = K;
    p.header->num_positions = W;
    // Overlapped mixed batch: the fewest SMs c that finish the prefill steps
    // (a margin ahead of) the split-KV work on the other S - c, if that beats
    // running the two one after the other. The split-KV time on n SMs is
    // bytes / min(n x per-SM rate, copy peak); the chunks alone on every SM
    // end at about 1.6x their even share (the longest items set the end).
    int ctas = p.num_sms, workers = p.num_workers;
    if (p.overlap && p.use_prefill && W > 0 && s_steps > 0) {
      const int S_ = p.num_sms;
      const float step_us = p.window > 0 ? kWindowStepUs : kPrefillStepUs;
      const float pre = step_us * (float)s_steps;  // SM x us
      const float bytes = (float)W * (float)p.position_bytes;
      auto dec_us = [&](int n) {
        return fmaxf(bytes / ((float)n * kDecodeSmBytesPerUs), bytes / kHbmBytesPerUs);
      };
      // smallest c with pre / c <= margin x dec_us(S - c), per branch of the max
      const float c1 = pre * (float)S_ * kDecodeSmBytesPerUs /
                       (kOverlapMargin * bytes + pre * kDecodeSmBytesPerUs);
      const float c2 = pre * kHbmBytesPerUs / (kOverlapMargin * bytes);
      const int c = max(1, (int)ceilf(fminf(fminf(c1, c2), (float)S_)));
      const float serial = 1.6f * pre / (float)S_ + dec_us(S_);
      if (p.prefill_ctas_override > 0) {  // the caller's share (at most half the SMs)
        ctas = min(p.prefill_ctas_override, S_ / 2);
        workers = min(workers, S_ - ctas);
      } else if (c <= S_ / 4 && dec_us(S_ - c) < serial) {
        ctas = c;
        workers = min(workers, S_ - c);
      }
    }
    p.header->prefill_ctas = ctas;
    p.header->decode_workers = workers;
    s_workers = workers;
  }
  // each split-KV worker's first unit (same worker count and slicing as the
  // split-KV kernel), found by binary search over the units' first positions
  __syncthreads();
  if (ubase) {
    const int NW = plan_workers(W, s_workers, p.min_pos);
    for (int w = threadIdx.x; w < NW; w += blockDim.x) {
      // (worker_begin; a division of 32 bits where it does)
      const int S = (unsigned long long)W * (unsigned)NW < 1ull << 32
                        ? (int)((unsigned)w * (unsigned)W / (unsigned)NW)
                        : worker_begin(w, W, NW);
      int lo = 0, hi = K;  // ubase[lo] <= S < ubase[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (ubase[mid] <= S) lo = mid; else hi = mid;
      }
      p.worker_unit[w] = lo;
    }
  }
  // Let the grid before this one (the KV write on the same stream) finish
  // before this grid completes: whoever waits on the plan then also sees the
  // newly written K/V.
  if (!p.early_trigger) griddep_launch_dependents();
  griddep_wait();
}

namespace {
template <bool SHARED>
cudaError_t launch_plan_t(const PlanParams& p, cudaStream_t s) {
  auto kern = pa_plan_kernel<SHARED>;
  const int smem = p.num_tokens <= kPlanSmemTokens
                       ? (int)(sizeof(int2) * p.num_tokens + sizeof(int) * (p.num_tokens + 1))
                       : 0;
  static bool attr_set[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(sizeof(int2) * kPlanSmemTokens + sizeof(int) * (kPlanSmemTokens + 1)));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  // Launched as a programmatic dependent of the previous grid, which it waits
  // for at its start; with early_start (the KV write, which makes nothing that
  // a plan needs) before completing.
  cudaLaunchConfig_t cfg = {};
  // shared calls: CTAs of their own check the groups' tables
  if (SHARED) {
    const int checks = check_parts(p.num_groups) * p.num_groups;  // at most 128, or of one part
    cfg.gridDim = dim3(1 + (checks > 128 && checks > p.num_sms - 1 ? max(128, p.num_sms - 1) : checks));
  } else {
    cfg.gridDim = dim3(1);
  }
  // A batch with no tensor-core work needs no bucket sort: a block sized to the
  // batch (fewer warps per barrier) plans it faster.
  int threads = kPlanThreads;
  if (!p.use_prefill) {
    int need = p.num_tokens > p.num_reqs ? p.num_tokens : p.num_reqs;
    // (on CUDA cores a shared call's tokens have several split-KV workers each, whose
    // first units are looked up one per thread)
    if (SHARED && !p.token_major) need *= 4;
    if (SHARED && need < kSharedCandidates) need = kSharedCandidates;
    // a cascade's prefix check reads (requests - 1) x prefix blocks entries
    if (p.prefix_blocks > 0 && (long long)(p.num_reqs - 1) * p.prefix_blocks > need)
      need = kPlanThreads;
    threads = need <= 128 ? 128 : need <= 256 ? 256 : need <= 512 ? 512 : kPlanThreads;
  }
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}
}  // namespace

cudaError_t launch_plan(const PlanParams& p, cudaStream_t s) {
  return p.num_groups > 0 ? launch_plan_t<true>(p, s) : launch_plan_t<false>(p, s);
}

}  // namespace pa
