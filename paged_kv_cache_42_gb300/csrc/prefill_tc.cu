// Prefill-chunk attention and a cascade's prefix pass: the kernel is in
// prefill_body.cuh; here are the tensor-map encoder and the dispatch.
#include <cudaTypedefs.h>

#include <mutex>

#include "prefill_body.cuh"

namespace pa {

// ---------------------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------------------
namespace {

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

bool get_encoder() {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return g_encode != nullptr;
}

bool encode_bf16(CUtensorMap* m, int rank, const void* ptr, const cuuint64_t* dims,
                 const cuuint64_t* strides_bytes, const cuuint32_t* box,
                 CUtensorMapDataType dtype = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16) {
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  const CUresult r = g_encode(m, dtype, rank, const_cast<void*>(ptr),
                              dims, strides_bytes, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

}  // namespace

bool encode_tmap_bf16_2d(void* tmap, const void* ptr, uint64_t inner, uint64_t rows,
                         uint64_t row_stride_bytes, uint32_t box_inner, uint32_t box_rows) {
  if (!get_encoder()) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)rows};
  const cuuint64_t str[1] = {(cuuint64_t)row_stride_bytes};
  const cuuint32_t box[2] = {box_inner, box_rows};
  return encode_bf16(static_cast<CUtensorMap*>(tmap), 2, ptr, dims, str, box);
}

namespace {
bool encode_tmap_any(void* tmap, int rank, const void* ptr, const uint64_t* dims,
                     const uint64_t* strides_bytes, const uint32_t* box, CUtensorMapDataType dt) {
  if (!get_encoder() || rank < 1 || rank > 5) return false;
  cuuint64_t d[5], st[4];
  cuuint32_t b[5];
  for (int i = 0; i < rank; ++i) {
    d[i] = (cuuint64_t)dims[i];
    b[i] = (cuuint32_t)box[i];
    if (i + 1 < rank) st[i] = (cuuint64_t)strides_bytes[i];
  }
  return encode_bf16(static_cast<CUtensorMap*>(tmap), rank, ptr, d, st, b, dt);
}
}  // namespace

bool encode_tmap_bf16(void* tmap, int rank, const void* ptr, const uint64_t* dims,
                      const uint64_t* strides_bytes, const uint32_t* box) {
  return encode_tmap_any(tmap, rank, ptr, dims, strides_bytes, box,
                         CU_TENSOR_MAP_DATA_TYPE_BFLOAT16);
}

bool encode_tmap_u8(void* tmap, int rank, const void* ptr, const uint64_t* dims,
                    const uint64_t* strides_bytes, const uint32_t* box) {
  return encode_tmap_any(tmap, rank, ptr, dims, strides_bytes, box, CU_TENSOR_MAP_DATA_TYPE_UINT8);
}

cudaError_t launch_prefill(const PrefillLaunch& a, int num_sms, cudaStream_t s) {
  if (!get_encoder()) return cudaErrorNotSupported;
  if (a.shared_items != nullptr) return launch_prefill_groups(a, num_sms, s);
  if (a.kv_fp8) {
    if (a.prefix_len > 0) return cudaErrorNotSupported;  // no FP8 cascade
    if (a.kv_fp8 == 2)  // windows have no row-scaled form
      return a.window > 0 ? cudaErrorNotSupported : launch_prefill_mode<kChunks, 2, false>(a, num_sms, s);
    return a.window > 0 ? launch_prefill_mode<kChunks, 1, true>(a, num_sms, s)
                        : launch_prefill_mode<kChunks, 1, false>(a, num_sms, s);
  }
  if (a.window > 0)  // never with a prefix
    return launch_prefill_mode<kChunks, 0, true>(a, num_sms, s);
  return a.prefix_len > 0 ? launch_prefill_mode<kOnePrefix, 0, false>(a, num_sms, s)
                          : launch_prefill_mode<kChunks, 0, false>(a, num_sms, s);
}

}  // namespace pa
