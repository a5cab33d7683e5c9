// attend_shared: whether a call shares, and the kernels over a cache of 16 bits (ns_shared_attn.cuh).
#include <algorithm>

#include "ns_shared_attn.cuh"

namespace ns {

// Whether a call shares.  Beyond 128 rows to a sequence its own tokens fill the row tiles, and all that sharing saves
// is reading; and few keys are read again from L2 sooner than a plan, the parts and their merge take.  Measured, not
// shared and shared, bf16, pages of 16: members behind so many positions (g of m: in g groups), 80 of their own; MB of
// keys and values by max_len; us in a graph.  One new token:
//   32 heads on 8, 128 columns:  8 behind 2101 (68 MB) 18.5, 22.8;  4000 (128) 23.2, 24.5;  8000 (253) 35.4, 28.0
//     16 behind 2101 (136) 24.8, 26.1;  32 behind 2000 (260) 38.1, 32.7
//     4 of 16 behind 1000 (270) 40.9, 45.2;  4000 (1020) 117, 58;  2 behind 16000 (126) 25.3, 32.0;  64000 (501) 68, 76
//   28 on 4, 128 columns:  8 behind 8000 (126) 24.1, 26.3;  16000 (251) 36.0, 29.9;  32 behind 2000 (130) 25.8, 27.4
//     4 of 16 behind 1000 (135) 27.6, 31.2;  4000 (510) 63, 38
//   12 on 4, 64 columns:  8 behind 16000 (126) 22.2, 28.1;  4 of 16 behind 4000 (255) 42.2, 34.7
//   16 on 1, 128 columns:  4 of 16 behind 4000 (128) 26.2, 28.2;  9000 (284) 40.3, 33.2
//   8 bits, 32 on 8:  8 behind 8000 (126) 28.1, 32.3;  16000 (251) 43.1, 39.5;  32 behind 2000 (130) 31.2, 38.4
//     4 of 16 behind 1000 (135) 33.8, 56.3;  4000 (510) 81, 67
//   8 bits, 28 on 4:  4 of 16 behind 4000 (255) 48.9, 43.6;  8 of 8 49.0, 51.2;  16 on 1:  4 of 16 behind 9000 (142)
//     42.4, 35.4
// More rows, 32 on 8: 20 rows; 64; 128 (over 8 bits these take longer, so positions count, and not their bytes):
//   16 behind 1000 (68 MB) 25.3, 27.2; 25.6, 34.3; 28.1, 36.5;  8 bits 31.6, 30.4; 31.9, 38.2; 34.2, 41.9
//   4 of 4 behind 4000 (255) 51.6, 36.0; 52.0, 45.5; 56.6, 61.5;  8 bits 64.5, 41.7; 64.3, 51.4; 70.0, 76.1
//   16 behind 6007 (381) 69.8, 36.6; 69.8, 53.0; 72.7, 68.8;  8 bits 88.6, 43.1; 88.8, 62.7; 91.5, 87.8
//   the same with 240 rows 88, 113
// So the bound is between 136 and 251 MB, but for two members, short prompts of many, 128 rows just above it and small
// differences.
// Groups of one member on average, and contexts of less than a tile by max_len, have nothing to share.  What the plan,
// the row tiles and the parts cost then (one new token, 8, 32; not shared, shared):
//   32 heads on 8, 128 columns:  1 sequence behind 16000 19.9, 28.9; 29.0, 29.0; 29.5, 29.7;  64 behind 3000 128, 159;
//     149, 164; 160, 183;  the same of 8 bits 81.5, 202.5; 193, 204; 202, 220
//   12 on 4, 64 columns:  16 behind 2101 14.6, 29.9; 22.3, 29.4; 22.7, 30.9;  1 behind 16000 10.8, 25.4; 29.6, 25.7;
//     29.9, 26.7 (row tiles of one sequence with their keys split, which attend_paged does not have)
static bool pays(const PagedAttnArgs &a, int n_groups, int dim) {
  if (n_groups >= a.n_seqs || a.max_len - a.n < kKeys) return false;
  const int rows = a.n * a.group;
  constexpr int64_t kFew = 192LL << 20;
  const int64_t bytes = (int64_t)a.n_seqs * a.max_len * a.kv_heads * dim * (a.k_exp && rows <= 16 ? 2 : 4);
  return rows <= 128 && bytes > kFew;
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
