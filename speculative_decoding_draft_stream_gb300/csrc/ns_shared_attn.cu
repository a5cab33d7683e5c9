// attend_shared: whether a call shares, and the kernels over a cache of 16 bits (ns_shared_attn.cuh).
#include <algorithm>

#include "ns_shared_attn.cuh"

namespace ns {

// Whether a call shares.  Beyond 128 rows to a sequence its own tokens fill the row tiles, and all that sharing saves
// is reading; and few keys are read again from L2 sooner than a plan, the parts and their merge take.  Measured, not
// shared and shared, 32 heads on 8, 128 columns, bf16, pages of 16 (us in a graph; MB by max_len):
//   one token:  8 sequences behind 500 (19 MB) 13.3, 20.6;  behind 2101 (69) 18.3, 21.8;  behind 4000 (129) 24.0, 25.1;
//     behind 8000 (254) 35.6, 28.3;  16 behind 2101 (140) 25.5, 24.9;  24 (211) 32.2, 28.0;  32 behind 500 (81) 19.5,
//     29.1;  behind 2000 (268) 38.0, 30.5;  2 behind 16000 (126) 25.9, 31.9
//   16 sequences behind 6007:  4 new tokens 52.7, 32.3;  8: 70.7, 39.6;  16: 70.8, 54.7;  32 (128 rows): 73.7, 72.9;
//     60 (240 rows): 88, 113
// Groups of one member on average, and contexts of less than a tile by max_len, have nothing to share.  What the plan,
// the row tiles and the parts cost then (one new token, 8, 32; not shared, shared):
//   32 heads on 8, 128 columns:  1 sequence behind 16000 19.9, 28.9; 29.0, 29.0; 29.5, 29.7;  64 behind 3000 128, 159;
//     149, 164; 160, 183;  the same of 8 bits 81.5, 202.5; 193, 204; 202, 220
//   12 on 4, 64 columns:  16 behind 2101 14.6, 29.9; 22.3, 29.4; 22.7, 30.9;  1 behind 16000 10.8, 25.4; 29.6, 25.7;
//     29.9, 26.7 (row tiles of one sequence with their keys split, which attend_paged does not have)
static bool pays(const PagedAttnArgs &a, int n_groups, int dim) {
  if (n_groups >= a.n_seqs || a.max_len - a.n < kKeys) return false;
  constexpr int64_t kFew = 128LL << 20;
  const int64_t bytes = (int64_t)a.n_seqs * a.max_len * a.kv_heads * dim * (a.k_exp ? 2 : 4);
  return a.n * a.group <= 128 && (bytes > kFew || a.n * a.group > 16);
}

int64_t shared_attn_ws(int n_seqs, int n_groups, int n, int q_heads, int kv_heads, int dim, int sms) {
  const int64_t shared = Layout(shape_of(n_seqs, n_groups, n, q_heads, kv_heads, sms), n_seqs, n_groups, dim).bytes;
  return std::max(n * (q_heads / kv_heads) <= 128 ? shared : 0, paged_attn_ws(n_seqs, n, q_heads, kv_heads, dim, sms));
}

cudaError_t prepare_shared_attn() {
  const cudaError_t e = prepare_all<false>();
  return e == cudaSuccess ? prepare_shared_attn8() : e;
}

cudaError_t launch_shared_attn(const PagedAttnArgs &a, const int32_t *groups, int n_groups, int dtype, int dim,
                               int sms, const PagedFit &fit, cudaStream_t st) {
  if (!pays(a, n_groups, dim)) {
    PagedAttnArgs own = a;
    own.groups = groups, own.n_groups = n_groups;
    return a.k_exp ? launch_paged_attn8(own, dtype, dim, sms, fit, st)
                   : launch_paged_attn(own, dtype, dim, sms, fit, st);
  }
  if (a.k_exp) return launch_shared_attn8(a, groups, n_groups, dtype, dim, sms, st);
  return launch_any<false>(a, groups, n_groups, dtype, dim, sms, st);
}

}  // namespace ns
