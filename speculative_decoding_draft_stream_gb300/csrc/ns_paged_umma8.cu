// Many rows over a paged cache of 8 bits (ns_paged_tree.cuh, PageConverter in ns_paged_mode.cuh).
#include "ns_paged_tree.cuh"

namespace ns {

bool paged_umma8_ok(const PagedAttnArgs &a) {
  const int64_t q[3] = {a.q_seq, a.q_token, a.q_head};
  for (int64_t x : q)
    if (x <= 0 || x % 8 || x >= (int64_t)1 << 39) return false;
  const int64_t c[6] = {a.k_page, a.k_head, a.k_token, a.v_page, a.v_head, a.v_token};
  for (int64_t x : c)
    if (x <= 0 || x % 16 || x >= (int64_t)1 << 40) return false;
  return reinterpret_cast<uintptr_t>(a.q) % 16 == 0;
}

cudaError_t prepare_paged_umma8() { return prepare_all<true>(); }

cudaError_t launch_paged_umma8(const PagedAttnArgs &a, int dtype, int dim, int sms, cudaStream_t st) {
  return launch_any<true>(a, dtype, dim, sms, st);
}

}  // namespace ns
