// C ABI of libpagedattn: argument validation, per-device set-up, the device
// error word, optional launch timers and dispatch to the kernels.
//
// Validation happens before any CUDA call, so a malformed call is rejected
// without touching (or needing) a GPU.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <nvtx3/nvToolsExt.h>

#include <atomic>
#include <mutex>

#include "pa_api.h"
#include "pa_internal.h"

namespace pa {

// The device error word: [0] code (PA_DEVERR_*), [1] detail. One per device,
// in static device memory; kernels receive its address as an argument.
__device__ unsigned long long g_device_error[2];

namespace {

constexpr int kMaxDevices = 64;
constexpr int kMaxRopeHeads = 65536;  // a token's elements are counted in 32 bits

// Per-device set-up, done once. The cached device address of the error word
// stays valid for the life of the CUDA context: the library does not support
// cudaDeviceReset of a device it has been used on.
struct DeviceState {
  std::atomic<bool> ready{false};
  int num_sms = 0;
  unsigned long long* err = nullptr;
};

std::mutex g_mutex;
DeviceState g_devices[kMaxDevices];
std::atomic<long long> g_launches{0};
std::atomic<int> g_self_plan{1};  // pa_set_option(PA_OPT_DECODE_SELF_PLAN, ...)
std::atomic<int> g_decode_tc{1};  // pa_set_option(PA_OPT_DECODE_TC, ...): 0 off, 1 auto, 2 on
std::atomic<int> g_max_workers{0};  // pa_set_option(PA_OPT_DECODE_MAX_WORKERS, ...): 0 = no cap
std::atomic<int> g_mixed_overlap{1};  // pa_set_option(PA_OPT_MIXED_OVERLAP, ...)
std::atomic<int> g_token_major{1};  // pa_set_option(PA_OPT_DECODE_TOKEN_MAJOR, ...)
std::atomic<int> g_cascade_overlap{1};  // pa_set_option(PA_OPT_CASCADE_OVERLAP, ...)
std::atomic<int> g_tm_ctas{2};  // pa_set_option(PA_OPT_DECODE_TM_CTAS_PER_SM, ...)
std::atomic<int> g_write_overlap{0};  // pa_set_option(PA_OPT_WRITE_OVERLAP, ...)
std::atomic<int> g_mixed_ctas{0};  // pa_set_option(PA_OPT_MIXED_PREFILL_CTAS, ...): 0 = planned
constexpr int kNumTimers = 8;  // write, plan, decode, prefill, cascade prefix, merge, weights, evict
cudaEvent_t g_timer_start[kNumTimers] = {};
cudaEvent_t g_timer_stop[kNumTimers] = {};

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

pa_status device_state(DeviceState** out) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return PA_ERR_CUDA;
  DeviceState& d = g_devices[dev];
  if (!d.ready.load(std::memory_order_acquire)) {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!d.ready.load(std::memory_order_relaxed)) {
      int sms = 0;
      if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return PA_ERR_CUDA;
      void* err = nullptr;
      if (cudaGetSymbolAddress(&err, g_device_error) != cudaSuccess) return PA_ERR_CUDA;
      d.num_sms = sms;
      d.err = static_cast<unsigned long long*>(err);
      d.ready.store(true, std::memory_order_release);
    }
  }
  *out = &d;
  return PA_OK;
}

// An NVTX range around a call's launches (header-only NVTX: nothing happens
// unless a profiler is attached), named after the entry point.
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

struct TimerScope {
  int id;
  cudaStream_t s;
  TimerScope(int kernel, cudaStream_t stream) : id(kernel), s(stream) {
    if (g_timer_start[id]) cudaEventRecord(g_timer_start[id], s);
  }
  ~TimerScope() {
    if (g_timer_stop[id]) cudaEventRecord(g_timer_stop[id], s);
  }
};

bool supported_group(int g) { return g == 1 || g == 2 || g == 4 || g == 8; }

}  // namespace

pa_status check_attention_args(const void* q, const void* k_cache, const void* v_cache,
                               const int32_t* block_tables, const int32_t* seq_lens,
                               const int32_t* query_start_loc, float scale, const void* out,
                               int num_reqs, int num_tokens, int num_q_heads, int num_kv_heads,
                               int head_dim, int block_size, int num_blocks,
                               int max_blocks_per_req, int max_query_len, int max_seq_len,
                               int prefix_len, int kv_fp8, float k_scale, float v_scale,
                               bool* nothing_to_do) {
  *nothing_to_do = false;
  if (kv_fp8 && !(k_scale > 0.f && k_scale < INFINITY && v_scale > 0.f && v_scale < INFINITY))
    return PA_ERR_INVALID_ARG;
  if (kv_fp8 && prefix_len > 0) return PA_ERR_UNSUPPORTED;  // no FP8 cascade
  if (num_reqs < 0 || num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
      head_dim <= 0 || num_blocks < 0 || max_blocks_per_req < 0 || max_query_len < 0 ||
      max_seq_len < 0)
    return PA_ERR_INVALID_ARG;
  if (num_q_heads % num_kv_heads != 0) return PA_ERR_INVALID_ARG;
  if (block_size != kBlockSize || (head_dim != 64 && head_dim != 128) ||
      !supported_group(num_q_heads / num_kv_heads))
    return PA_ERR_UNSUPPORTED;
  if (!(scale == scale)) return PA_ERR_INVALID_ARG;  // NaN scale
  if (num_reqs == 0 || num_tokens == 0) {
    *nothing_to_do = true;
    return PA_OK;
  }
  if (!q || !k_cache || !v_cache || !block_tables || !seq_lens || !query_start_loc || !out)
    return PA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(block_tables) & 3u) ||
      (reinterpret_cast<uintptr_t>(seq_lens) & 3u) ||
      (reinterpret_cast<uintptr_t>(query_start_loc) & 3u))
    return PA_ERR_INVALID_ARG;
  // flattened work positions must fit a 32-bit int: tokens x Hkv x blocks per token
  const long long max_blocks = ((long long)max_seq_len + kBlockSize - 1) / kBlockSize;
  if ((long long)num_tokens * num_kv_heads * max_blocks >= (1LL << 31))
    return PA_ERR_UNSUPPORTED;
  // a cascade prefix is whole blocks, inside the tables, and leaves every
  // request at least one key of its own
  if (prefix_len > 0 && (prefix_len / kBlockSize > max_blocks_per_req || prefix_len >= max_seq_len))
    return PA_ERR_INVALID_ARG;
  return PA_OK;
}

}  // namespace pa

using namespace pa;

extern "C" {

int pa_version(void) { return 100; }

long long pa_launch_count(void) { return g_launches.load(); }

const char* pa_status_string(int status) {
  switch (status) {
    case PA_OK: return "PA_OK";
    case PA_ERR_INVALID_ARG: return "PA_ERR_INVALID_ARG: invalid argument";
    case PA_ERR_UNSUPPORTED: return "PA_ERR_UNSUPPORTED: unsupported block_size / head_dim / group";
    case PA_ERR_WORKSPACE: return "PA_ERR_WORKSPACE: workspace missing or too small";
    case PA_ERR_CUDA: return "PA_ERR_CUDA: CUDA runtime or launch failure";
    case PA_ERR_BOUNDS: return "PA_ERR_BOUNDS: index outside its valid range";
    case PA_ERR_TIMEOUT: return "PA_ERR_TIMEOUT: a bounded device wait gave up";
    default: return "unknown pa_status";
  }
}

pa_status pa_init(void) {
  DeviceState* d = nullptr;
  return device_state(&d);
}

}  // extern "C"

namespace {

pa_status write_kv_impl(const void* k, const void* v, const int64_t* slot_mapping, void* k_cache,
                        void* v_cache, int kv_fp8, float k_scale, float v_scale, int num_tokens,
                        int num_kv_heads, int head_dim, int block_size, int num_blocks,
                        void* stream) {
  if (num_tokens < 0 || num_kv_heads <= 0 || head_dim <= 0 || num_blocks < 0)
    return PA_ERR_INVALID_ARG;
  if (kv_fp8 && !(k_scale > 0.f && k_scale < INFINITY && v_scale > 0.f && v_scale < INFINITY))
    return PA_ERR_INVALID_ARG;
  if (block_size != kBlockSize || head_dim % 8 != 0) return PA_ERR_UNSUPPORTED;
  const NvtxRange range(kv_fp8 ? "pa_write_kv_fp8" : "pa_write_kv");
  if (num_tokens == 0) return PA_OK;
  if (!k || !v || !slot_mapping || !k_cache || !v_cache) return PA_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
    return PA_ERR_INVALID_ARG;
  DeviceState* d = nullptr;
  if (pa_status st = device_state(&d)) return st;
  WriteParams p;
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.slot_mapping = slot_mapping;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.kv_fp8 = kv_fp8;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.num_tokens = num_tokens;
  p.num_kv_heads = num_kv_heads;
  p.head_dim = head_dim;
  p.num_slots = (long long)num_blocks * kBlockSize;
  p.err = d->err;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TimerScope timer(0, s);
  const cudaError_t e = launch_write_kv(p, s);
  g_launches.fetch_add(1);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status norm_rope_write_impl(const void* q, const void* k, const void* v, long long q_stride,
                               long long k_stride, long long v_stride, const int32_t* positions,
                               const float* cos_sin, const void* q_weight, const void* k_weight,
                               float eps, int rotary_dim, int interleaved, int max_position,
                               const int64_t* slot_mapping, void* q_out, void* k_cache,
                               void* v_cache, int kv_fp8, float k_scale, float v_scale,
                               int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                               int block_size, int num_blocks, void* stream) {
  if (num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || num_blocks < 0 ||
      rotary_dim < 0 || rotary_dim > head_dim || max_position < 0 || !(eps >= 0.f && eps < INFINITY))
    return PA_ERR_INVALID_ARG;
  if (kv_fp8 && !(k_scale > 0.f && k_scale < INFINITY && v_scale > 0.f && v_scale < INFINITY))
    return PA_ERR_INVALID_ARG;
  if (block_size != kBlockSize || (head_dim != 64 && head_dim != 128) || rotary_dim % 16 != 0 ||
      num_q_heads > kMaxRopeHeads || num_kv_heads > kMaxRopeHeads)
    return PA_ERR_UNSUPPORTED;
  const NvtxRange range(kv_fp8 ? "pa_norm_rope_write_kv_fp8" : "pa_norm_rope_write_kv");
  if (num_tokens == 0) return PA_OK;
  if (!q || !k || !v || !slot_mapping || !q_out || !k_cache || !v_cache ||
      (rotary_dim > 0 && (!positions || !cos_sin)))
    return PA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) ||
      !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(q_weight) ||
      !aligned16(k_weight) || !aligned16(cos_sin) ||
      (reinterpret_cast<uintptr_t>(positions) & 3u) ||
      (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
    return PA_ERR_INVALID_ARG;
  const long long q_row = (long long)num_q_heads * head_dim;
  const long long kv_row = (long long)num_kv_heads * head_dim;
  if (q_stride < q_row || k_stride < kv_row || v_stride < kv_row || q_stride % 8 != 0 ||
      k_stride % 8 != 0 || v_stride % 8 != 0)
    return PA_ERR_INVALID_ARG;
  if (q_out == q && q_stride != q_row) return PA_ERR_INVALID_ARG;  // rows would overtake each other
  DeviceState* d = nullptr;
  if (pa_status st = device_state(&d)) return st;
  NormRopeParams p;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.positions = positions;
  p.cos_sin = cos_sin;
  p.q_weight = static_cast<const uint16_t*>(q_weight);
  p.k_weight = static_cast<const uint16_t*>(k_weight);
  p.eps = eps;
  p.rotary_dim = rotary_dim;
  p.interleaved = interleaved ? 1 : 0;
  p.max_position = rotary_dim > 0 ? max_position : 1;  // no table: position 0 stands for all
  p.slot_mapping = slot_mapping;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.kv_fp8 = kv_fp8;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.num_tokens = num_tokens;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.num_slots = (long long)num_blocks * kBlockSize;
  p.err = d->err;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TimerScope timer(0, s);
  const cudaError_t e = launch_norm_rope_write(p, head_dim, d->num_sms, s);
  g_launches.fetch_add(1);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

extern "C" {

pa_status pa_norm_rope_write_kv(const void* q, const void* k, const void* v, long long q_stride,
                                long long k_stride, long long v_stride, const int32_t* positions,
                                const float* cos_sin, const void* q_weight, const void* k_weight,
                                float eps, int rotary_dim, int interleaved, int max_position,
                                const int64_t* slot_mapping, void* q_out, void* k_cache,
                                void* v_cache, int num_tokens, int num_q_heads, int num_kv_heads,
                                int head_dim, int block_size, int num_blocks, void* stream) {
  return norm_rope_write_impl(q, k, v, q_stride, k_stride, v_stride, positions, cos_sin, q_weight,
                              k_weight, eps, rotary_dim, interleaved, max_position, slot_mapping,
                              q_out, k_cache, v_cache, 0, 1.f, 1.f, num_tokens, num_q_heads,
                              num_kv_heads, head_dim, block_size, num_blocks, stream);
}

pa_status pa_norm_rope_write_kv_fp8(const void* q, const void* k, const void* v,
                                    long long q_stride, long long k_stride, long long v_stride,
                                    const int32_t* positions, const float* cos_sin,
                                    const void* q_weight, const void* k_weight, float eps,
                                    int rotary_dim, int interleaved, int max_position,
                                    const int64_t* slot_mapping, void* q_out, void* k_cache,
                                    void* v_cache, float k_scale, float v_scale, int num_tokens,
                                    int num_q_heads, int num_kv_heads, int head_dim,
                                    int block_size, int num_blocks, void* stream) {
  return norm_rope_write_impl(q, k, v, q_stride, k_stride, v_stride, positions, cos_sin, q_weight,
                              k_weight, eps, rotary_dim, interleaved, max_position, slot_mapping,
                              q_out, k_cache, v_cache, 1, k_scale, v_scale, num_tokens,
                              num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, stream);
}

pa_status pa_write_kv(const void* k, const void* v, const int64_t* slot_mapping, void* k_cache,
                      void* v_cache, int num_tokens, int num_kv_heads, int head_dim,
                      int block_size, int num_blocks, void* stream) {
  return write_kv_impl(k, v, slot_mapping, k_cache, v_cache, 0, 1.f, 1.f, num_tokens,
                       num_kv_heads, head_dim, block_size, num_blocks, stream);
}

pa_status pa_write_kv_fp8(const void* k, const void* v, const int64_t* slot_mapping,
                          void* k_cache, void* v_cache, float k_scale, float v_scale,
                          int num_tokens, int num_kv_heads, int head_dim, int block_size,
                          int num_blocks, void* stream) {
  return write_kv_impl(k, v, slot_mapping, k_cache, v_cache, 1, k_scale, v_scale, num_tokens,
                       num_kv_heads, head_dim, block_size, num_blocks, stream);
}

size_t pa_attention_workspace_size(int num_reqs, int num_tokens, int num_q_heads,
                                   int num_kv_heads, int head_dim) {
  if (num_reqs < 0 || num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
      head_dim <= 0 || num_q_heads % num_kv_heads != 0)
    return 0;
  return ws_layout(num_reqs, num_tokens, num_q_heads, num_kv_heads, head_dim).total;
}

size_t pa_attention_cascade_workspace_size(int num_reqs, int num_tokens, int num_q_heads,
                                           int num_kv_heads, int head_dim) {
  const size_t base =
      pa_attention_workspace_size(num_reqs, num_tokens, num_q_heads, num_kv_heads, head_dim);
  if (base == 0) return 0;
  return base + prefix_partials_bytes(num_tokens, num_q_heads, num_kv_heads, head_dim);
}

}  // extern "C"

namespace {

// pa_attention and pa_attention_cascade (prefix_len > 0).
pa_status attention_impl(const void* q, const void* k_cache, const void* v_cache,
                         const int32_t* block_tables, const int32_t* seq_lens,
                         const int32_t* query_start_loc, float scale, void* out, int num_reqs,
                         int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                         int block_size, int num_blocks, int max_blocks_per_req,
                         int max_query_len, int max_seq_len, int prefix_len, int window,
                         int sinks, int kv_fp8, float k_scale, float v_scale, void* workspace,
                         size_t workspace_bytes, void* stream) {
  bool nothing = false;
  const bool windowed = window > 0;
  // a window that holds every key of the batch hides none
  if (window >= max_seq_len) window = sinks = 0;
  // the most keys a token's blocks can span (it sizes the flattened work)
  const long long span = (long long)window + sinks + 3 * kBlockSize;
  const int seen = window > 0 && span < max_seq_len ? (int)span : max_seq_len;
  if (pa_status st = check_attention_args(
          q, k_cache, v_cache, block_tables, seq_lens, query_start_loc, scale, out, num_reqs,
          num_tokens, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
          max_blocks_per_req, max_query_len, seen, prefix_len, kv_fp8, k_scale, v_scale,
          &nothing))
    return st;
  if (nothing) return PA_OK;
  if (windowed && num_blocks < 1) return PA_ERR_INVALID_ARG;  // no block to attend to
  const WsLayout lay = ws_layout(num_reqs, num_tokens, num_q_heads, num_kv_heads, head_dim);
  const size_t need =
      lay.total + (prefix_len > 0
                       ? prefix_partials_bytes(num_tokens, num_q_heads, num_kv_heads, head_dim)
                       : 0);
  if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return PA_ERR_WORKSPACE;

  DeviceState* d = nullptr;
  if (pa_status st = device_state(&d)) return st;
  const NvtxRange range(prefix_len > 0 ? "pa_attention_cascade"
                        : window > 0   ? (kv_fp8 ? "pa_attention_window_fp8" : "pa_attention_window")
                                       : (kv_fp8 ? "pa_attention_fp8" : "pa_attention"));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  unsigned char* ws = static_cast<unsigned char*>(workspace);

  const int group = num_q_heads / num_kv_heads;
  // cascade: prefix key chunks, all non-empty (they divide the key tiles evenly)
  int chunks = 0;
  if (prefix_len > 0) {
    const int nkt = (prefix_len + 127) / 128;
    const int c = prefix_chunks(num_tokens, num_kv_heads, group, nkt);
    const int per = (nkt + c - 1) / c;
    chunks = (nkt + per - 1) / per;
  }
  float* const prefix_partials =
      prefix_len > 0 ? reinterpret_cast<float*>(ws + lay.total) : nullptr;

  PlanParams pp;
  pp.qsl = query_start_loc;
  pp.seq_lens = seq_lens;
  pp.block_tables = block_tables;
  pp.prefix_blocks = prefix_len / kBlockSize;
  // a decode-only batch (every span at most one token) plans itself inside
  // the split-KV kernel: no planner launch
  const int self_plan = (g_self_plan.load() && prefix_len == 0 && max_query_len <= 1 &&
                         num_reqs <= kSelfPlanMaxReqs) ? 1 : 0;
  pp.early_start = g_write_overlap.load();
  pp.early_trigger = prefix_len > 0 ? 1 : 0;
  pp.num_reqs = num_reqs;
  pp.num_tokens = num_tokens;
  pp.num_kv_heads = num_kv_heads;
  pp.max_blocks_per_req = max_blocks_per_req;
  pp.max_query_len = max_query_len;
  pp.max_seq_len = max_seq_len;
  pp.group = group;
  // a cascade sends every span to the split-KV path
  pp.use_prefill = (prefix_len == 0 && max_query_len >= kPrefillMinQlen) ? 1 : 0;
  const int occ_cap =
      prefix_len > 0 ? PA_DEC_OCC_CAP_CASCADE : (kv_fp8 ? PA_DEC_OCC_CAP_FP8 : PA_DEC_OCC_CAP);
  // The tensor-core split-KV kernel takes the groups whose arithmetic per
  // cached byte outgrows the CUDA cores (by default G >= PA_DECODE_TC_MIN_GROUP),
  // except a cascade's suffix pass: its short suffixes leave each CTA a few
  // tiles per (token, kv head), and the CUDA-core kernel's many warps hide
  // the per-(token, kv head) epilogue better (measured 39 vs 76 us on the
  // prefix-sharing batch).
  const int tc_mode = g_decode_tc.load();
  const bool use_tc = tc_mode != 0 &&
                      decode_tc_supported(head_dim, group, kv_fp8 != 0, prefix_len / kBlockSize) &&
                      (tc_mode == 2 || (group >= PA_DECODE_TC_MIN_GROUP && prefix_len == 0));
  // A cascade on the CUDA-core suffix pass may run its prefix pass on a few
  // SMs (about two prefix items each) beside the suffix pass on the rest; the
  // merge pass then folds every (token, kv head).
  const int c_overlap = (g_cascade_overlap.load() && prefix_len > 0 && !use_tc) ? 1 : 0;
  int prefix_ctas = 0;
  if (c_overlap) {
    const int items = prefix_pairs(num_tokens, group) * num_kv_heads * chunks;
    prefix_ctas = (items + 1) / 2;
    if (prefix_ctas > d->num_sms / 4) prefix_ctas = d->num_sms / 4;
    if (prefix_ctas < 1) prefix_ctas = 1;
  }
  const int dec_sms = d->num_sms - prefix_ctas;  // SMs the split-KV grid fills
  // An E4M3 cache over eight KV heads takes the token-major tiles (one block
  // of every KV head per tile) on the tensor cores.
  // Windowed calls leave little work, where a token-major worker's start and its
  // many-partial merge can outweigh its faster tiles: by the tokens on this path
  // and the blocks they attend to at most. G = 4 (us, other tiles / token-major):
  // 8 tokens of 502 blocks 39.5 / 40.7, 8 of 1001 64.3 / 60.0, 16 of 129 25.3 /
  // 25.4, 32 of 33 19.5 / 18.3; G = 8: 8 of 1001 69.2 / 77.3, 32 of 129 45.9 /
  // 49.7, 32 of 502 124.1 / 119.8, 48 of 33 30.5 / 29.9. And below 64 blocks per SM
  // one CTA per SM is mostly the better (G = 4, one / two: 32 of 129 38.6 / 39.8,
  // 64 of 66 38.3 / 40.3, 64 of 502 175.5 / 171.1; but 64 of 33 25.9 / 21.5).
  const long long win_tokens =
      pp.use_prefill  // spans of one token, if the others have the longest's length
          ? num_reqs - ((long long)num_tokens - num_reqs) / (max_query_len - 1)
          : num_tokens;
  const long long win_keys = (long long)window + sinks;
  const long long win_blocks =
      win_tokens * (((win_keys < max_seq_len ? win_keys : max_seq_len) + kBlockSize - 1) / kBlockSize);
  const bool win_tm = group <= 4 ? 5 * win_tokens >= d->num_sms || win_blocks >= 30LL * d->num_sms
                                 : 10 * win_tokens >= 3LL * d->num_sms ||
                                       win_blocks >= 100LL * d->num_sms;
  const int tm_cps = window > 0 && win_blocks < 64LL * d->num_sms ? 1 : g_tm_ctas.load();
  const bool use_tm =
      use_tc && kv_fp8 && g_token_major.load() && (window == 0 || win_tm) &&
      decode_tm_supported(head_dim, group, num_kv_heads, decode_tm_workers(group, d->num_sms, tm_cps));
  const int launched = use_tm   ? decode_tm_workers(group, d->num_sms, tm_cps)
                       : use_tc ? decode_tc_workers(d->num_sms)
                                : decode_workers(head_dim, pp.group, kv_fp8 != 0, window > 0, dec_sms,
                                                occ_cap);
  if (launched <= 0) return PA_ERR_CUDA;
  const int cap = g_max_workers.load();
  pp.num_workers = (cap > 0 && cap < launched) ? cap : launched;
  pp.token_major = use_tm ? 1 : 0;
  pp.window = window;
  pp.sinks = sinks;
  // A window leaves short units, and a batch of a few of them is a chain of
  // blocks in a handful of warps: there the CUDA-core kernel's workers take
  // single blocks (four tokens of a 16-key window at head_dim 64: 7.3 us per
  // call against 16 us with eight blocks each). The tensor-core kernels' workers
  // keep a whole tile.
  pp.min_pos = window > 0 && !use_tc ? 1 : PA_DEC_MIN_POS;
  // A mixed batch on the tensor-core split-KV kernel (bf16) may run its
  // prefill chunks on a few SMs beside the split-KV work (the planner decides
  // how many, or none); the E4M3 path keeps its query-split pass between them.
  const int overlap = (g_mixed_overlap.load() && pp.use_prefill && use_tc && !kv_fp8) ? 1 : 0;
  pp.overlap = overlap;
  pp.prefill_ctas_override = g_mixed_ctas.load();
  pp.num_sms = d->num_sms;
  pp.position_bytes = 2 * kBlockSize * head_dim * 2;  // K and V of one 16-key block
  pp.header = reinterpret_cast<WsHeader*>(ws + lay.header_off);
  pp.units = reinterpret_cast<UnitInfo*>(ws + lay.units_off);
  pp.tiles = reinterpret_cast<PrefillTile*>(ws + lay.tiles_off);
  pp.raw = reinterpret_cast<int2*>(ws + lay.raw_off);
  pp.worker_unit = reinterpret_cast<int*>(ws + lay.workers_off);
  pp.err = d->err;
  if (!self_plan) {
    TimerScope timer(1, s);
    const cudaError_t e = launch_plan(pp, s);
    g_launches.fetch_add(1);
    if (e != cudaSuccess) return PA_ERR_CUDA;
  }

  if (pp.use_prefill || prefix_len > 0) {
    PrefillLaunch pl;
    pl.prefix_len = prefix_len;
    pl.prefix_chunks = chunks;
    pl.slot_floats = lay.slot_floats;
    pl.prefix_partials = prefix_partials;
    pl.kv_fp8 = kv_fp8;
    pl.v_scale = kv_fp8 ? v_scale : 1.f;
    pl.q = q;
    pl.k_cache = k_cache;
    pl.v_cache = v_cache;
    pl.qsl = query_start_loc;
    pl.seq_lens = seq_lens;
    pl.block_tables = block_tables;
    pl.out = static_cast<uint16_t*>(out);
    pl.header = pp.header;
    pl.tiles = pp.tiles;
    pl.num_tokens = num_tokens;
    pl.num_q_heads = num_q_heads;
    pl.num_kv_heads = num_kv_heads;
    pl.head_dim = head_dim;
    pl.num_blocks = num_blocks;
    pl.bt_stride = max_blocks_per_req;
    pl.scale_log2 = scale * 1.4426950408889634f * (kv_fp8 ? k_scale : 1.f);
    pl.overlap = prefix_len > 0 ? c_overlap : overlap;
    pl.prefix_ctas = prefix_ctas;
    pl.window = window;
    pl.sinks = sinks;
    pl.err = d->err;
    TimerScope timer(prefix_len > 0 ? 4 : 3, s);
    const cudaError_t e = launch_prefill(pl, d->num_sms, s);
    g_launches.fetch_add(1);
    if (e != cudaSuccess) return PA_ERR_CUDA;
  }

  DecodeParams dp;
  dp.q = static_cast<const uint16_t*>(q);
  dp.k_cache = k_cache;
  dp.v_cache = v_cache;
  dp.v_scale = kv_fp8 ? v_scale : 1.f;
  dp.block_tables = block_tables;
  dp.out = static_cast<uint16_t*>(out);
  dp.bt_stride = max_blocks_per_req;
  dp.num_q_heads = num_q_heads;
  dp.num_kv_heads = num_kv_heads;
  dp.num_blocks = num_blocks;
  // scores in base-2 units; an E4M3 cache's k_scale rides on q
  dp.scale_log2 = scale * 1.4426950408889634f * (kv_fp8 ? k_scale : 1.f);
  dp.header = pp.header;
  dp.units = pp.units;
  dp.worker_unit = num_tokens <= kPlanSmemTokens ? pp.worker_unit : nullptr;
  dp.partials = reinterpret_cast<float*>(ws + lay.partials_off);
  dp.slot_floats = lay.slot_floats;
  dp.key_start_blocks = prefix_len / kBlockSize;
  dp.prefix_partials = prefix_partials;
  dp.prefix_chunks = chunks;
  dp.num_tokens = num_tokens;
  dp.self_plan = self_plan;
  dp.early_start = pp.early_start;
  dp.num_reqs = num_reqs;
  dp.max_blocks_per_req = max_blocks_per_req;
  dp.max_query_len = max_query_len;
  dp.max_seq_len = max_seq_len;
  dp.qsl = query_start_loc;
  dp.seq_lens = seq_lens;
  dp.header_out = pp.header;
  dp.merge_tasks = reinterpret_cast<int4*>(ws + lay.tasks_off);
  dp.max_workers = cap > 0 ? cap : kMaxDecodeWorkers;
  dp.qsplit = ws + lay.qsplit_off;
  dp.qinv = reinterpret_cast<const float*>(ws + lay.qinv_off);
  dp.overlap = (overlap || c_overlap) ? 1 : 0;
  dp.fold_later = c_overlap;
  dp.window = window;
  dp.sinks = sinks;
  dp.min_pos = pp.min_pos;
  dp.err = d->err;
  if (use_tc && kv_fp8) {  // the E4M3 tensor-core kernel takes the queries split
    const cudaError_t e = launch_qsplit(dp, group, s);
    g_launches.fetch_add(1);
    if (e != cudaSuccess) return PA_ERR_CUDA;
  }
  int launched_workers = 0;
  {
    TimerScope timer(2, s);
    const cudaError_t e =
        use_tm   ? launch_decode_tm(dp, group, d->num_sms, tm_cps, s, &launched_workers)
        : use_tc ? launch_decode_tc(dp, group, kv_fp8 != 0, d->num_sms, s, &launched_workers)
                 : launch_decode(dp, head_dim, group, kv_fp8 != 0, dec_sms, occ_cap, s,
                                 &launched_workers);
    g_launches.fetch_add(1);
    if (e != cudaSuccess) return PA_ERR_CUDA;
  }
  // the slicing's worker count, as the split-KV kernel computes it
  const int workers = (cap > 0 && cap < launched_workers) ? cap : launched_workers;

  MergeParams mp;
  mp.header = pp.header;
  mp.tasks = dp.merge_tasks;
  mp.partials = dp.partials;
  mp.slot_floats = lay.slot_floats;
  mp.num_workers = workers;
  mp.workers_from_header = overlap;
  mp.token_major = pp.token_major;
  mp.min_pos = pp.min_pos;
  mp.num_q_heads = num_q_heads;
  mp.num_kv_heads = num_kv_heads;
  mp.num_tokens = num_tokens;
  mp.key_start_blocks = dp.key_start_blocks;
  mp.prefix_partials = prefix_partials;
  mp.prefix_chunks = chunks;
  mp.v_scale = dp.v_scale;
  mp.out = dp.out;
  mp.all_units = c_overlap;
  mp.units = pp.units;
  if (workers > 1 || c_overlap) {
    TimerScope timer(5, s);
    const cudaError_t e = launch_merge(mp, head_dim, group, s);
    g_launches.fetch_add(1);
    if (e != cudaSuccess) return PA_ERR_CUDA;
  }
  return PA_OK;
}

}  // namespace

extern "C" {

pa_status pa_attention(const void* q, const void* k_cache, const void* v_cache,
                       const int32_t* block_tables, const int32_t* seq_lens,
                       const int32_t* query_start_loc, float scale, void* out, int num_reqs,
                       int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                       int block_size, int num_blocks, int max_blocks_per_req,
                       int max_query_len, int max_seq_len, void* workspace,
                       size_t workspace_bytes, void* stream) {
  return attention_impl(q, k_cache, v_cache, block_tables, seq_lens, query_start_loc, scale, out,
                        num_reqs, num_tokens, num_q_heads, num_kv_heads, head_dim, block_size,
                        num_blocks, max_blocks_per_req, max_query_len, max_seq_len, 0, 0, 0, 0,
                        1.f, 1.f, workspace, workspace_bytes, stream);
}

pa_status pa_attention_fp8(const void* q, const void* k_cache, const void* v_cache,
                           const int32_t* block_tables, const int32_t* seq_lens,
                           const int32_t* query_start_loc, float scale, float k_scale,
                           float v_scale, void* out, int num_reqs, int num_tokens,
                           int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                           int num_blocks, int max_blocks_per_req, int max_query_len,
                           int max_seq_len, void* workspace, size_t workspace_bytes,
                           void* stream) {
  return attention_impl(q, k_cache, v_cache, block_tables, seq_lens, query_start_loc, scale, out,
                        num_reqs, num_tokens, num_q_heads, num_kv_heads, head_dim, block_size,
                        num_blocks, max_blocks_per_req, max_query_len, max_seq_len, 0, 0, 0, 1,
                        k_scale, v_scale, workspace, workspace_bytes, stream);
}

pa_status pa_attention_cascade(const void* q, const void* k_cache, const void* v_cache,
                               const int32_t* block_tables, const int32_t* seq_lens,
                               const int32_t* query_start_loc, float scale, void* out,
                               int num_reqs, int num_tokens, int num_q_heads, int num_kv_heads,
                               int head_dim, int block_size, int num_blocks,
                               int max_blocks_per_req, int max_query_len, int max_seq_len,
                               int common_prefix_len, void* workspace, size_t workspace_bytes,
                               void* stream) {
  if (common_prefix_len <= 0 || common_prefix_len % kBlockSize != 0) return PA_ERR_INVALID_ARG;
  return attention_impl(q, k_cache, v_cache, block_tables, seq_lens, query_start_loc, scale, out,
                        num_reqs, num_tokens, num_q_heads, num_kv_heads, head_dim, block_size,
                        num_blocks, max_blocks_per_req, max_query_len, max_seq_len,
                        common_prefix_len, 0, 0, 0, 1.f, 1.f, workspace, workspace_bytes, stream);
}

pa_status pa_attention_window(const void* q, const void* k_cache, const void* v_cache,
                              const int32_t* block_tables, const int32_t* seq_lens,
                              const int32_t* query_start_loc, float scale, void* out,
                              int num_reqs, int num_tokens, int num_q_heads, int num_kv_heads,
                              int head_dim, int block_size, int num_blocks,
                              int max_blocks_per_req, int max_query_len, int max_seq_len,
                              int window, int sinks, void* workspace, size_t workspace_bytes,
                              void* stream) {
  if (window < 1 || sinks < 0) return PA_ERR_INVALID_ARG;
  return attention_impl(q, k_cache, v_cache, block_tables, seq_lens, query_start_loc, scale, out,
                        num_reqs, num_tokens, num_q_heads, num_kv_heads, head_dim, block_size,
                        num_blocks, max_blocks_per_req, max_query_len, max_seq_len, 0, window,
                        sinks, 0, 1.f, 1.f, workspace, workspace_bytes, stream);
}

pa_status pa_attention_window_fp8(const void* q, const void* k_cache, const void* v_cache,
                                  const int32_t* block_tables, const int32_t* seq_lens,
                                  const int32_t* query_start_loc, float scale, float k_scale,
                                  float v_scale, void* out, int num_reqs, int num_tokens,
                                  int num_q_heads, int num_kv_heads, int head_dim,
                                  int block_size, int num_blocks, int max_blocks_per_req,
                                  int max_query_len, int max_seq_len, int window, int sinks,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  if (window < 1 || sinks < 0) return PA_ERR_INVALID_ARG;
  return attention_impl(q, k_cache, v_cache, block_tables, seq_lens, query_start_loc, scale, out,
                        num_reqs, num_tokens, num_q_heads, num_kv_heads, head_dim, block_size,
                        num_blocks, max_blocks_per_req, max_query_len, max_seq_len, 0, window,
                        sinks, 1, k_scale, v_scale, workspace, workspace_bytes, stream);
}

size_t pa_attention_weights_workspace_size(int num_reqs, int num_tokens, int num_q_heads,
                                           int num_kv_heads, int head_dim, int max_query_len,
                                           int max_seq_len) {
  if (num_reqs < 0 || num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
      head_dim <= 0 || num_q_heads % num_kv_heads != 0 || max_query_len < 0 || max_seq_len < 0 ||
      !supported_group(num_q_heads / num_kv_heads))
    return 0;
  const size_t n = weights_layout(num_reqs, num_tokens, num_q_heads, num_kv_heads, max_query_len,
                                  max_seq_len).total;
  return n ? n : 256;
}

}  // extern "C"

namespace {

pa_status weights_impl(const void* q, const void* k_cache, const int32_t* block_tables,
                       const int32_t* seq_lens, const int32_t* query_start_loc, float scale,
                       int kv_fp8, float k_scale, const float* weights, float* out,
                       long long weights_stride, int num_reqs, int num_tokens, int num_q_heads,
                       int num_kv_heads, int head_dim, int block_size, int num_blocks,
                       int max_blocks_per_req, int max_query_len, int max_seq_len,
                       void* workspace, size_t workspace_bytes, void* stream) {
  bool nothing = false;
  // pa_attention's checks; there is no V here, out is checked below, and no
  // work is flattened over the keys (so their number does not count here)
  if (pa_status st = check_attention_args(
          q, k_cache, k_cache, block_tables, seq_lens, query_start_loc, scale, q, num_reqs,
          num_tokens, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
          max_blocks_per_req, max_query_len, max_seq_len < 1 ? max_seq_len : 1, 0, kv_fp8, k_scale,
          1.f, &nothing))
    return st;
  if (weights_stride < 0) return PA_ERR_INVALID_ARG;
  if (nothing) return PA_OK;
  if (num_blocks < 1) return PA_ERR_INVALID_ARG;  // no block to read
  if (!weights || !out || (reinterpret_cast<uintptr_t>(weights) & 3u) ||
      (reinterpret_cast<uintptr_t>(out) & 3u))
    return PA_ERR_INVALID_ARG;
  if (max_query_len == 0 || max_seq_len == 0) return PA_OK;  // no request can have a new token
  if (max_seq_len > (1 << 30)) return PA_ERR_UNSUPPORTED;  // key positions are 32-bit
  const WeightsLayout lay = weights_layout(num_reqs, num_tokens, num_q_heads, num_kv_heads,
                                           max_query_len, max_seq_len);
  // grids and work lists (with some room for parts) are indexed with 32 bits
  const long long rh = (long long)num_reqs * num_kv_heads;
  if (rh * (lay.padded_len / 128 + 1) >= (1LL << 31) - (1 << 14) ||
      (long long)lay.num_slots * num_kv_heads * 16 >= (1LL << 31))
    return PA_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < lay.total || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return PA_ERR_WORKSPACE;
  DeviceState* d = nullptr;
  if (pa_status st = device_state(&d)) return st;
  const NvtxRange range(kv_fp8 ? "pa_attention_weights_fp8" : "pa_attention_weights");
  unsigned char* const ws = static_cast<unsigned char*>(workspace);
  WeightsParams p;
  p.q = static_cast<const uint16_t*>(q);
  p.k_cache = k_cache;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.qsl = query_start_loc;
  p.weights = weights;
  p.out = out;
  p.weights_stride = weights_stride;
  p.scale_log2 = scale * 1.4426950408889634f * (kv_fp8 ? k_scale : 1.f);
  p.num_reqs = num_reqs;
  p.num_tokens = num_tokens;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = num_q_heads / num_kv_heads;
  p.num_blocks = num_blocks;
  p.bt_stride = max_blocks_per_req;
  p.max_query_len = max_query_len;
  p.max_seq_len = max_seq_len;
  p.num_chunks = lay.num_chunks;
  p.padded_len = lay.padded_len;
  p.stored_rows = lay.stored_rows;
  p.num_slots = lay.num_slots;
  p.max_items[0] = lay.max_items[0];
  p.max_items[1] = lay.max_items[1];
  p.cluster = 0;
  p.stats = reinterpret_cast<float*>(ws + lay.stats_off);
  p.scores = reinterpret_cast<float*>(ws + lay.scores_off);
  p.counts = reinterpret_cast<int*>(ws + lay.counts_off);
  p.num_counters = lay.num_counters;
  p.num_sms = d->num_sms;
  p.counters = reinterpret_cast<int*>(ws + lay.counters_off);
  p.items[0] = reinterpret_cast<int4*>(ws + lay.items1_off);
  p.items[1] = reinterpret_cast<int4*>(ws + lay.items2_off);
  p.neg_lse = reinterpret_cast<float*>(ws + lay.lse_off);
  p.partial = reinterpret_cast<float2*>(ws + lay.partial_off);
  p.sums = reinterpret_cast<float*>(ws + lay.sums_off);
  p.err = d->err;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TimerScope timer(6, s);
  int launches = 0;
  const cudaError_t e = launch_weights(p, head_dim, kv_fp8 != 0, d->num_sms, s, &launches);
  g_launches.fetch_add(launches);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

extern "C" {

pa_status pa_attention_weights(const void* q, const void* k_cache, const int32_t* block_tables,
                               const int32_t* seq_lens, const int32_t* query_start_loc,
                               float scale, const float* weights, float* out,
                               long long weights_stride, int num_reqs, int num_tokens,
                               int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                               int num_blocks, int max_blocks_per_req, int max_query_len,
                               int max_seq_len, void* workspace, size_t workspace_bytes,
                               void* stream) {
  return weights_impl(q, k_cache, block_tables, seq_lens, query_start_loc, scale, 0, 1.f, weights,
                      out, weights_stride, num_reqs, num_tokens, num_q_heads, num_kv_heads,
                      head_dim, block_size, num_blocks, max_blocks_per_req, max_query_len,
                      max_seq_len, workspace, workspace_bytes, stream);
}

pa_status pa_attention_weights_fp8(const void* q, const void* k_cache,
                                   const int32_t* block_tables, const int32_t* seq_lens,
                                   const int32_t* query_start_loc, float scale, float k_scale,
                                   const float* weights, float* out, long long weights_stride,
                                   int num_reqs, int num_tokens, int num_q_heads,
                                   int num_kv_heads, int head_dim, int block_size, int num_blocks,
                                   int max_blocks_per_req, int max_query_len, int max_seq_len,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  return weights_impl(q, k_cache, block_tables, seq_lens, query_start_loc, scale, 1, k_scale,
                      weights, out, weights_stride, num_reqs, num_tokens, num_q_heads,
                      num_kv_heads, head_dim, block_size, num_blocks, max_blocks_per_req,
                      max_query_len, max_seq_len, workspace, workspace_bytes, stream);
}

pa_status pa_evict_kv(void* k_cache, void* v_cache, const int32_t* block_tables,
                      const int32_t* seq_lens, const float* weights,
                      const int32_t* new_block_tables, int32_t* new_seq_lens, int32_t* kept,
                      float* new_weights, int num_reqs, int num_kv_heads, int head_dim,
                      int elem_bytes, int block_size, int num_blocks, int max_blocks_per_req,
                      int max_new_blocks, long long weights_stride, long long new_weights_stride,
                      int max_seq_len, int keep, int recent, int sinks, void* stream) {
  if (num_reqs < 0 || num_kv_heads <= 0 || head_dim <= 0 || num_blocks < 0 ||
      max_blocks_per_req < 0 || max_new_blocks < 0 || weights_stride < 0 || max_seq_len < 0 ||
      keep < 1 || recent < 0 || sinks < 0 || (long long)sinks + recent > keep)
    return PA_ERR_INVALID_ARG;
  if (block_size != kBlockSize || (head_dim != 64 && head_dim != 128) ||
      (elem_bytes != 1 && elem_bytes != 2))
    return PA_ERR_UNSUPPORTED;
  if (max_new_blocks < (keep - 1) / kBlockSize + 1 || (new_weights && new_weights_stride < keep))
    return PA_ERR_INVALID_ARG;
  const NvtxRange range("pa_evict_kv");
  if (num_reqs == 0) return PA_OK;
  if (!k_cache || !v_cache || !block_tables || !seq_lens || !weights || !new_block_tables ||
      !new_seq_lens || !kept || new_weights == weights || new_seq_lens == seq_lens)
    return PA_ERR_INVALID_ARG;
  const void* words[] = {block_tables, seq_lens,     weights, new_block_tables,
                         new_seq_lens, kept, new_weights};
  for (const void* w : words)
    if (reinterpret_cast<uintptr_t>(w) & 3u) return PA_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_INVALID_ARG;
  // the row lists are one CTA per (request, KV head) and 64 kept tokens
  if ((long long)num_reqs * num_kv_heads * ((keep - 1) / 64 + 1) >= (1LL << 31))
    return PA_ERR_UNSUPPORTED;
  DeviceState* d = nullptr;
  if (pa_status st = device_state(&d)) return st;
  EvictParams p;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.weights = weights;
  p.new_block_tables = new_block_tables;
  p.new_seq_lens = new_seq_lens;
  p.kept = kept;
  p.new_weights = new_weights;
  p.num_reqs = num_reqs;
  p.num_kv_heads = num_kv_heads;
  p.num_blocks = num_blocks;
  p.max_blocks_per_req = max_blocks_per_req;
  p.max_new_blocks = max_new_blocks;
  p.weights_stride = weights_stride;
  p.new_weights_stride = new_weights_stride;
  p.max_seq_len = max_seq_len;
  p.keep = keep;
  p.recent = recent;
  p.sinks = sinks;
  p.cluster = 1;
  p.err = d->err;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TimerScope timer(7, s);
  const cudaError_t e = launch_evict(p, head_dim * elem_bytes, d->num_sms, s);
  g_launches.fetch_add(max_seq_len > keep ? 2 : 1);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// The struct forms.
size_t pa_args_size(int which) {
  switch (which) {
    case 0: return sizeof(pa_norm_rope_write_args);
    case 1: return sizeof(pa_window_args);
    case 2: return sizeof(pa_weights_args);
    case 3: return sizeof(pa_evict_args);
  }
  return 0;
}

pa_status pa_norm_rope_write_kv_args(const pa_norm_rope_write_args* a) {
  if (!a) return PA_ERR_INVALID_ARG;
  return norm_rope_write_impl(a->q, a->k, a->v, a->q_stride, a->k_stride, a->v_stride, a->positions,
                              a->cos_sin, a->q_weight, a->k_weight, a->eps, a->rotary_dim,
                              a->interleaved, a->max_position, a->slot_mapping, a->q_out,
                              a->k_cache, a->v_cache, a->kv_fp8 ? 1 : 0, a->kv_fp8 ? a->k_scale : 1.f,
                              a->kv_fp8 ? a->v_scale : 1.f, a->num_tokens, a->num_q_heads,
                              a->num_kv_heads, a->head_dim, a->block_size, a->num_blocks, a->stream);
}

pa_status pa_attention_window_args(const pa_window_args* a) {
  if (!a) return PA_ERR_INVALID_ARG;
  if (a->kv_fp8)
    return pa_attention_window_fp8(
        a->q, a->k_cache, a->v_cache, a->block_tables, a->seq_lens, a->query_start_loc, a->scale,
        a->k_scale, a->v_scale, a->out, a->num_reqs, a->num_tokens, a->num_q_heads, a->num_kv_heads,
        a->head_dim, a->block_size, a->num_blocks, a->max_blocks_per_req, a->max_query_len,
        a->max_seq_len, a->window, a->sinks, a->workspace, a->workspace_bytes, a->stream);
  return pa_attention_window(a->q, a->k_cache, a->v_cache, a->block_tables, a->seq_lens,
                             a->query_start_loc, a->scale, a->out, a->num_reqs, a->num_tokens,
                             a->num_q_heads, a->num_kv_heads, a->head_dim, a->block_size,
                             a->num_blocks, a->max_blocks_per_req, a->max_query_len, a->max_seq_len,
                             a->window, a->sinks, a->workspace, a->workspace_bytes, a->stream);
}

pa_status pa_attention_weights_args(const pa_weights_args* a) {
  if (!a) return PA_ERR_INVALID_ARG;
  return weights_impl(a->q, a->k_cache, a->block_tables, a->seq_lens, a->query_start_loc, a->scale,
                      a->kv_fp8 ? 1 : 0, a->kv_fp8 ? a->k_scale : 1.f, a->weights, a->out,
                      a->weights_stride, a->num_reqs, a->num_tokens, a->num_q_heads,
                      a->num_kv_heads, a->head_dim, a->block_size, a->num_blocks,
                      a->max_blocks_per_req, a->max_query_len, a->max_seq_len, a->workspace,
                      a->workspace_bytes, a->stream);
}

pa_status pa_evict_kv_args(const pa_evict_args* a) {
  if (!a) return PA_ERR_INVALID_ARG;
  return pa_evict_kv(a->k_cache, a->v_cache, a->block_tables, a->seq_lens, a->weights,
                     a->new_block_tables, a->new_seq_lens, a->kept, a->new_weights, a->num_reqs,
                     a->num_kv_heads, a->head_dim, a->elem_bytes, a->block_size, a->num_blocks,
                     a->max_blocks_per_req, a->max_new_blocks, a->weights_stride,
                     a->new_weights_stride, a->max_seq_len, a->keep, a->recent, a->sinks, a->stream);
}

pa_status pa_mapped_pointer(const void* host_ptr, void** device_ptr) {
  if (host_ptr == nullptr || device_ptr == nullptr) return PA_ERR_INVALID_ARG;
  cudaPointerAttributes a;
  if (cudaPointerGetAttributes(&a, host_ptr) != cudaSuccess) {
    cudaGetLastError();  // clear the error the query recorded
    return PA_ERR_INVALID_ARG;
  }
  if (a.type != cudaMemoryTypeHost) return PA_ERR_INVALID_ARG;
  void* d = nullptr;
  if (cudaHostGetDevicePointer(&d, const_cast<void*>(host_ptr), 0) != cudaSuccess || !d) {
    cudaGetLastError();
    return PA_ERR_CUDA;
  }
  *device_ptr = d;
  return PA_OK;
}

pa_status pa_get_device_error(int* code, long long* detail, int clear) {
  DeviceState* d = nullptr;
  if (pa_status st = device_state(&d)) return st;
  unsigned long long w[2] = {0, 0};
  if (cudaMemcpy(w, d->err, sizeof w, cudaMemcpyDeviceToHost) != cudaSuccess) return PA_ERR_CUDA;
  if (code) *code = (int)w[0];
  if (detail) *detail = (long long)w[1];
  if (clear) {
    const unsigned long long z[2] = {0, 0};
    if (cudaMemcpy(d->err, z, sizeof z, cudaMemcpyHostToDevice) != cudaSuccess) return PA_ERR_CUDA;
  }
  return PA_OK;
}

pa_status pa_set_option(int option, int value) {
  switch (option) {
    case PA_OPT_DECODE_SELF_PLAN:
      g_self_plan.store(value ? 1 : 0);
      return PA_OK;
    case PA_OPT_DECODE_TC:
      if (value < 0 || value > 2) return PA_ERR_INVALID_ARG;
      g_decode_tc.store(value);
      return PA_OK;
    case PA_OPT_CASCADE_OVERLAP:
      g_cascade_overlap.store(value ? 1 : 0);
      return PA_OK;
    case PA_OPT_DECODE_TOKEN_MAJOR:
      g_token_major.store(value ? 1 : 0);
      return PA_OK;
    case PA_OPT_DECODE_TM_CTAS_PER_SM:
      if (value != 1 && value != 2) return PA_ERR_INVALID_ARG;
      g_tm_ctas.store(value);
      return PA_OK;
    case PA_OPT_MIXED_PREFILL_CTAS:
      if (value < 0) return PA_ERR_INVALID_ARG;
      g_mixed_ctas.store(value);
      return PA_OK;
    case PA_OPT_WRITE_OVERLAP:
      if (value != 0 && value != 1) return PA_ERR_INVALID_ARG;
      g_write_overlap.store(value);
      return PA_OK;
    case PA_OPT_MIXED_OVERLAP:
      g_mixed_overlap.store(value ? 1 : 0);
      return PA_OK;
    case PA_OPT_DECODE_MAX_WORKERS:
      if (value < 0) return PA_ERR_INVALID_ARG;
      g_max_workers.store(value);
      return PA_OK;
  }
  return PA_ERR_INVALID_ARG;
}

pa_status pa_set_kernel_timer(int kernel_id, void* start_event, void* stop_event) {
  if (kernel_id < 0 || kernel_id >= kNumTimers) return PA_ERR_INVALID_ARG;
  if ((start_event == nullptr) != (stop_event == nullptr)) return PA_ERR_INVALID_ARG;
  g_timer_start[kernel_id] = static_cast<cudaEvent_t>(start_event);
  g_timer_stop[kernel_id] = static_cast<cudaEvent_t>(stop_event);
  return PA_OK;
}

}  // extern "C"
