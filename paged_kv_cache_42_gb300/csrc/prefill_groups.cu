// The prefix pass of a shared call (groups of requests, each with its own
// prefix): the kGroups instantiations of the tensor-core kernel, over every cache
// format.
#include "prefill_body.cuh"

namespace pa {

cudaError_t launch_prefill_groups(const PrefillLaunch& a, int num_sms, cudaStream_t s) {
  switch (a.kv_fp8) {
    case 0: return launch_prefill_mode<kGroups, 0, false>(a, num_sms, s);
    case 1: return launch_prefill_mode<kGroups, 1, false>(a, num_sms, s);
    case 2: return launch_prefill_mode<kGroups, 2, false>(a, num_sms, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace pa
