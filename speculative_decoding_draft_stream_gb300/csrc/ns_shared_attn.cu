// attend_shared over a cache of 16 bits (ns_shared_attn.cuh).
#include "ns_shared_attn.cuh"

namespace ns {

int64_t shared_attn_ws(int n_seqs, int n_groups, int n, int q_heads, int kv_heads, int dim, int sms) {
  return Layout(shape_of(n_seqs, n_groups, n, q_heads, kv_heads, sms), n_seqs, n_groups, dim).bytes;
}

cudaError_t prepare_shared_attn() {
  const cudaError_t e = prepare_all<false>();
  return e == cudaSuccess ? prepare_shared_attn8() : e;
}

cudaError_t launch_shared_attn(const PagedAttnArgs &a, const int32_t *groups, int n_groups, int dtype, int dim,
                               int sms, cudaStream_t st) {
  if (a.k_exp) return launch_shared_attn8(a, groups, n_groups, dtype, dim, sms, st);
  return launch_any<false>(a, groups, n_groups, dtype, dim, sms, st);
}

}  // namespace ns
