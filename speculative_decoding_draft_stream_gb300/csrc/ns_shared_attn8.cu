// attend_shared over a cache of 8 bits (ns_shared_attn.cuh, PageConverter in ns_paged_mode.cuh).
#include "ns_shared_attn.cuh"

namespace ns {

cudaError_t prepare_shared_attn8() { return prepare_all<true>(); }

cudaError_t launch_shared_attn8(const PagedAttnArgs &a, const int32_t *groups, int n_groups, int dtype, int dim,
                                int sms, cudaStream_t st) {
  return launch_any<true>(a, groups, n_groups, dtype, dim, sms, st);
}

}  // namespace ns
