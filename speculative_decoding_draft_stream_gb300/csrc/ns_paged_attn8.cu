// Attention of a sequence's new tokens over a paged key-value cache of 8 bits
// (ns_paged_rows.cuh has the kernel and its mathematics).
#include "ns_paged_rows.cuh"

namespace ns {
namespace {

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
