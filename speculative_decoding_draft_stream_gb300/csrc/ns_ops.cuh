// Declarations shared by the serving operators (include/nanospec_ops.h):
// the launch wrappers that the C ABI (ns_ops_api.cu) calls.  Each operator's
// arguments are checked there; the kernels check what only the device sees.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/nanospec_ops.h"

namespace ns {

// Paged cache (ns_pages.cu).
cudaError_t launch_pages_truncate(const ns_kv_pages &c, const int32_t *seqs, const int32_t *new_len, int n,
                                  uint32_t *err, cudaStream_t st);
cudaError_t launch_pages_fork(const ns_kv_pages &c, const int32_t *src, const int32_t *dst, int n, uint32_t *err,
                              cudaStream_t st);
int64_t pages_extend_ws(const ns_kv_pages &c, int n);
// (sc: the exponents of a cache of 8 bits, or NULL)
cudaError_t launch_pages_extend(const ns_kv_pages &c, const ns_kv_scales *sc, const int32_t *seqs,
                                const int32_t *n_new, int n, void *ws, uint32_t *err, cudaStream_t st);
cudaError_t launch_pages_write(const ns_kv_pages &c, int layer, const int32_t *seqs, const int32_t *cu, int n,
                               const void *k_new, const void *v_new, int64_t k_token, int64_t k_head,
                               int64_t v_token, int64_t v_head, int tokens, uint32_t *err, cudaStream_t st);
cudaError_t launch_pages_write_scaled(const ns_kv_pages &c, const ns_kv_scales &sc, int layer, const int32_t *seqs,
                                      const int32_t *cu, int n, const void *k_new, const void *v_new, int dtype,
                                      int64_t k_token, int64_t k_head, int64_t v_token, int64_t v_head, int tokens,
                                      uint32_t *err, cudaStream_t st);
cudaError_t launch_pages_read(const ns_kv_pages &c, const ns_kv_scales *sc, int layer, const int32_t *seqs,
                              const int32_t *cu, int n, void *k, void *v, int dtype, int64_t k_token, int64_t k_head,
                              int64_t v_token, int64_t v_head, int tokens, uint32_t *err, cudaStream_t st);
cudaError_t launch_pages_compact(const ns_kv_pages &c, const ns_kv_scales *sc, const int32_t *seqs,
                                 const int32_t *base, const int32_t *keep, int keep_ld, const int32_t *n_keep, int n,
                                 uint32_t *err, cudaStream_t st);
cudaError_t launch_pages_copy(const ns_kv_pages &c, const ns_kv_scales *sc, const int32_t *src, const int32_t *dst,
                              int n, uint32_t *err, cudaStream_t st);

// Norms and rotation of heads (ns_rotate.cu).
struct RotateArgs {
  const void *q, *k;
  int32_t tokens, q_heads, kv_heads, rotary;
  int64_t q_token, q_head, k_token, k_head;
  const int32_t *positions;
  const double *inv_freq;
  const void *q_weight, *k_weight;
  float eps;  // negative: no norm
  void *q_out, *k_out;
  int64_t qo_token, qo_head, ko_token, ko_head;
};
cudaError_t launch_rotate(const RotateArgs &a, int dtype, int dim, bool neighbours, int sms, cudaStream_t st);

// Log probabilities (ns_logprobs.cu).
struct LogprobArgs {
  const void *logits;
  int32_t rows, V;
  int64_t ld;
  float inv_temperature;
  const int32_t *ids;
  int32_t n_ids, k;
  float *logprobs, *entropy, *lse;
  int32_t *top_ids;
  float *top_logprobs;
  uint32_t *err;
};
cudaError_t launch_logprobs(const LogprobArgs &a, int dtype, int sms, cudaStream_t st);

// Attention over a paged cache (ns_paged_attn.cu).
struct PagedAttnArgs {
  const void *q, *k, *v;
  int32_t n_seqs, n, q_heads, kv_heads, group;
  int64_t q_seq, q_token, q_head;
  int64_t k_page, k_head, k_token, v_page, v_head, v_token;
  int32_t n_pages, page_shift, table_ld, max_seqs, max_len;
  const int32_t *table, *lengths, *seqs;
  const int64_t *mask;
  float scale;
  void *out;
  float *lse;
  void *ws;
  uint32_t *err;
  const uint8_t *k_exp, *v_exp;  // a cache of 8 bits: each row's exponent
  int64_t ke_head, ve_head;
  int32_t kp16, kt16, vp16, vt16, kep8, vep8;  // its strides in units of 16 (exponents: 8) bytes
  const int32_t *groups;  // to be looked at, of a call of ns_attend_shared that does not share
  int32_t n_groups;
};
// What a device holds of the kernels for few rows (found when it is first used).
struct PagedFit {
  // resident at once: cache of 16 bits, of 8, of 8 with 8 rows; dtype; dim 64, 128; small, large
  int clusters[3][2][2][2];
};
cudaError_t launch_groups(const PagedAttnArgs &a, cudaStream_t st);  // looks at them, after what was launched before
int64_t paged_attn_ws(int n_seqs, int n, int q_heads, int kv_heads, int dim, int sms);
cudaError_t prepare_paged_attn(PagedFit *fit);
cudaError_t launch_paged_attn(const PagedAttnArgs &a, int dtype, int dim, int sms, const PagedFit &fit,
                              cudaStream_t st);

// The same over a cache of 8 bits (ns_paged_attn8.cu).
cudaError_t prepare_paged_attn8(PagedFit *fit);
cudaError_t launch_paged_attn8(const PagedAttnArgs &a, int dtype, int dim, int sms, const PagedFit &fit,
                               cudaStream_t st);

// The same for more than 16 rows, on tcgen05 (ns_paged_umma.cu).
bool paged_umma_ok(const PagedAttnArgs &a);
cudaError_t prepare_paged_umma();
cudaError_t launch_paged_umma(const PagedAttnArgs &a, int dtype, int dim, int sms, cudaStream_t st);
// and over a cache of 8 bits (ns_paged_umma8.cu).
bool paged_umma8_ok(const PagedAttnArgs &a);
cudaError_t prepare_paged_umma8();
cudaError_t launch_paged_umma8(const PagedAttnArgs &a, int dtype, int dim, int sms, cudaStream_t st);

// The same for groups of sequences that begin with the same pages (ns_shared_attn.cuh).
int64_t shared_attn_ws(int n_seqs, int n_groups, int n, int q_heads, int kv_heads, int dim, int sms);
cudaError_t prepare_shared_attn();
cudaError_t launch_shared_attn(const PagedAttnArgs &a, const int32_t *groups, int n_groups, int dtype, int dim,
                               int sms, const PagedFit &fit, cudaStream_t st);
// and over a cache of 8 bits (ns_shared_attn8.cu).
cudaError_t prepare_shared_attn8();
cudaError_t launch_shared_attn8(const PagedAttnArgs &a, const int32_t *groups, int n_groups, int dtype, int dim,
                                int sms, cudaStream_t st);

// Attention over whole prompts (ns_prompt_attn.cu).
struct PromptAttnArgs {
  const void *q, *k, *v;
  int32_t tokens, q_heads, kv_heads, group;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head;
  const int32_t *cu;
  int32_t n_seqs, max_len;
  float scale;
  void *out;
  float *lse;
  uint32_t *err;
};
cudaError_t prepare_prompt_attn();
cudaError_t launch_prompt_attn(const PromptAttnArgs &a, int dtype, int dim, int sms, cudaStream_t st);

}  // namespace ns
