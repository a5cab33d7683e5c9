// Many rows over a paged cache of 16 bits (ns_paged_tree.cuh).
#include "ns_paged_tree.cuh"

namespace ns {

bool paged_umma_ok(const PagedAttnArgs &a) {
  const int64_t s[9] = {a.q_seq, a.q_token, a.q_head, a.k_page, a.k_head, a.k_token, a.v_page, a.v_head, a.v_token};
  for (int64_t x : s)
    if (x <= 0 || x % 8 || x >= (int64_t)1 << 39) return false;
  return reinterpret_cast<uintptr_t>(a.q) % 16 == 0;
}

cudaError_t prepare_paged_umma() { return prepare_all<false>(); }

cudaError_t launch_paged_umma(const PagedAttnArgs &a, int dtype, int dim, int sms, cudaStream_t st) {
  return launch_any<false>(a, dtype, dim, sms, st);
}

}  // namespace ns
