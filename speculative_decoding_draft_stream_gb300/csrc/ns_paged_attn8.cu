// Attention of a sequence's new tokens over a paged key-value cache of 8 bits
// (ns_paged_rows.cuh has the kernel and its mathematics).
#include "ns_paged_rows.cuh"

namespace ns {
namespace {

// Which kernel a call takes.  Up to 8 rows are worth their own: 32 heads on 8, 128 columns, 16 sequences of 2300 tokens,
// pages of 64, by 8 and by 16 rows (us in a graph): 4 rows 24.8, 28.3; 8 rows 26.3, 30.0; one sequence of 4097: 8.8,
// 10.0; 9.4, 10.9.  By 16 rows and on the tensor cores: 12 rows 31.8, 49.0; 16 rows 35.0, 48.9.  On the tensor cores
// and by 64 rows: 20 rows 51.9, 57.3; 64 rows 52.4, 69.2; 240 rows 73.2, 199.8.
//
// Line or clusters go by the rule for 16 bits (ns_paged_attn.cu), with tiles of twice the keys.  Line, small, large, one
// new token, bf16:
//   32 heads on 8, 128 columns, 1 sequence:  100 tokens 8.4, 6.0;  4097: 13.7, 8.6;  16000: 19.4, 18.4;
//     2 sequences:  4097: 14.7, 9.9;  12000: 22.2, 19.0
//   28 on 4, 128 columns, 1 sequence:  100: 8.4, 6.6, 7.7;  4097: 12.9, 9.0, 9.2;  16000: 24.9, 15.1, 12.3;
//     32000 (8 tiles): 24.4, 24.4, 20.7;  5 sequences:  4097: 15.5, 10.8;  12000: 25.6, 21.5;  24000: 36.6, 34.8
//   12 on 4, 64 columns, 1 sequence:  1000: 10.0, 5.3, 5.5;  8000: 14.2, 8.4, 6.7;  32000: 25.4, 20.0, 13.6
template <typename T, int D>
cudaError_t by_rows(const PagedAttnArgs &a, int sms, const PagedFit &fit, cudaStream_t st) {
  if (a.n * a.group <= 8) return few_rows<T, D, 0, true>(a, sms, fit, st);
  if (a.n * a.group <= 16) return few_rows<T, D, 1, true>(a, sms, fit, st);
  if (paged_umma8_ok(a)) return launch_paged_umma8(a, Type<T>::kBf16 ? NS_DTYPE_BF16 : NS_DTYPE_F16, D, sms, st);
  return launch<T, D, 4, true>(a, sms, st);
}
template <typename T>
cudaError_t by_dim(const PagedAttnArgs &a, int dim, int sms, const PagedFit &fit, cudaStream_t st) {
  return dim == 128 ? by_rows<T, 128>(a, sms, fit, st) : by_rows<T, 64>(a, sms, fit, st);
}

}  // namespace

cudaError_t prepare_paged_attn8(PagedFit *fit) {
  cudaError_t e = prepare_all<__nv_bfloat16, 128, true>(fit);
  if (e == cudaSuccess) e = prepare_all<__nv_bfloat16, 64, true>(fit);
  if (e == cudaSuccess) e = prepare_all<__half, 128, true>(fit);
  if (e == cudaSuccess) e = prepare_all<__half, 64, true>(fit);
  return e == cudaSuccess ? prepare_paged_umma8() : e;
}

cudaError_t launch_paged_attn8(const PagedAttnArgs &a, int dtype, int dim, int sms, const PagedFit &fit,
                               cudaStream_t st) {
  return dtype == NS_DTYPE_BF16 ? by_dim<__nv_bfloat16>(a, dim, sms, fit, st) : by_dim<__half>(a, dim, sms, fit, st);
}

}  // namespace ns
