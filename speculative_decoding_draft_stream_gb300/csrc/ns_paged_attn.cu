// Attention of a sequence's new tokens over a paged key-value cache of 16 bits:
// which kernel a call takes (ns_paged_rows.cuh, ns_paged_umma.cu).
#include "ns_paged_rows.cuh"

namespace ns {
namespace {

// Up to 16 rows the keys are what costs: each is fetched once and the warps
// split them.  A call whose items fit on the GPU as clusters, all at once, with
// up to 12 (64 columns: 16) tiles to a CTA, takes clusters: of large CTAs where
// small ones would have more than one tile each and the large ones still fit (7
// clusters of 128 columns and 14 of 64, 21 and 33 of small ones).  Measured,
// line, small, large, one new token, bf16 (us in a graph):
//   32 heads on 8, 128 columns, 1 sequence:  100 tokens 8.5, 5.0, 10.1;  4097: 15.3, 8.6, 15.1;
//     8000: 17.0, 13.1;  12000: 18.4, 17.7;  16000: 20.0, 22.3
//     2 sequences:  100: 8.7, 5.5;  4097: 16.4, 9.9;  12000: 23.7, 22.9;  16000: 31.9, 30.8;  24000: 41.9, 44.1
//   28 on 4, 128 columns, 1 sequence:  100: 8.6, 5.2, 5.9;  2000: 10.0, 5.8, 5.8;  8000: 18.3, 11.6, 9.9;
//     16000: 20.0, 19.0, 14.9;  24000 (12 tiles): 21.6, 26.7, 20.3;  32000: 22.9, 35.5, 26.3
//     5 sequences:  4097: 16.6, 10.7;  12000: 30.9, 26.3;  16000: 36.4, 33.8
//   12 on 4, 64 columns, 1 sequence:  1000: 9.0, 4.4, 4.6;  8000: 17.7, 9.4, 7.5;  32000 (16 tiles): 23.8, 26.6, 19.2
//     4 sequences:  12000: 18.4, 15.0;  16000: 20.2, 18.8;  24000: 25.4, 30.3
//   32 heads on 8, 128 columns, 4 sequences (two waves):  100: 8.8, 10.0;  600: 10.5, 9.9;  2000: 15.1, 12.8;
//     4097: 18.4, 19.2
// Clusters of 8 large CTAs took 11.3 us for the 4097 tokens of one sequence.
// Above 16 rows the products cost: they belong on the tensor cores of
// ns_paged_umma.cu, which want queries that TMA can fetch (16-byte aligned,
// strides multiples of 8); other queries take 64 rows a CTA here.  Measured
// with 16 sequences of 2300 tokens, 32 heads on 8, 128 columns, pages of 64, by
// 16 rows here and there (us): 4 rows 34.6, 40.8; 16 rows 38.1, 40.7; 20 rows
// (twice 16) 49.5, 40.6; 64 rows 88.2, 40.9.  64 rows a CTA here: 16 draft
// trees of 60 nodes behind 512 to 4096 tokens (240 rows) 169, there 60.
template <typename T, int D>
cudaError_t by_rows(const PagedAttnArgs &a, int sms, const PagedFit &fit, cudaStream_t st) {
  if (a.n * a.group <= 16) return few_rows<T, D, 1, false>(a, sms, fit, st);
  if (paged_umma_ok(a)) return launch_paged_umma(a, Type<T>::kBf16 ? NS_DTYPE_BF16 : NS_DTYPE_F16, D, sms, st);
  return launch<T, D, 4, false>(a, sms, st);
}
template <typename T>
cudaError_t by_dim(const PagedAttnArgs &a, int dim, int sms, const PagedFit &fit, cudaStream_t st) {
  return dim == 128 ? by_rows<T, 128>(a, sms, fit, st) : by_rows<T, 64>(a, sms, fit, st);
}

__global__ void __launch_bounds__(256) groups_kernel(const PagedAttnArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");  // (what writes the groups may still run until then)
  look_at_groups(a.groups, a.n_groups, a.n_seqs, a.err);
}
}  // namespace

cudaError_t launch_groups(const PagedAttnArgs &a, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = st;
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(256);
  return cudaLaunchKernelEx(&cfg, groups_kernel, a);
}

int64_t paged_attn_ws(int n_seqs, int n, int q_heads, int kv_heads, int dim, int sms) {
  // two parts for each CTA: up to 4 sms CTAs of 16 rows, or sms CTAs of 256 (3 sms of 64 are no more)
  const int64_t rows = n * (q_heads / kv_heads) <= 16 ? (int64_t)kPerSm<64> * sms * 2 * 16 : (int64_t)sms * 2 * 256;
  return (((int64_t)(n_seqs + 1) * 8 + 255) & ~(int64_t)255) + rows * (dim + 2) * 4;
}

cudaError_t prepare_paged_attn(PagedFit *fit) {
  cudaError_t e = prepare_all<__nv_bfloat16, 128, false>(fit);
  if (e == cudaSuccess) e = prepare_all<__nv_bfloat16, 64, false>(fit);
  if (e == cudaSuccess) e = prepare_all<__half, 128, false>(fit);
  if (e == cudaSuccess) e = prepare_all<__half, 64, false>(fit);
  if (e == cudaSuccess) e = prepare_paged_umma();
  return e == cudaSuccess ? prepare_paged_attn8(fit) : e;
}

cudaError_t launch_paged_attn(const PagedAttnArgs &a, int dtype, int dim, int sms, const PagedFit &fit,
                              cudaStream_t st) {
  return dtype == NS_DTYPE_BF16 ? by_dim<__nv_bfloat16>(a, dim, sms, fit, st) : by_dim<__half>(a, dim, sms, fit, st);
}

}  // namespace ns
