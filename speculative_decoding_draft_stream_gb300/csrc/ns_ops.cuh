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
cudaError_t launch_pages_extend(const ns_kv_pages &c, const int32_t *seqs, const int32_t *n_new, int n, void *ws,
                                uint32_t *err, cudaStream_t st);
cudaError_t launch_pages_write(const ns_kv_pages &c, int layer, const int32_t *seqs, const int32_t *cu, int n,
                               const void *k_new, const void *v_new, int64_t k_token, int64_t k_head,
                               int64_t v_token, int64_t v_head, int tokens, uint32_t *err, cudaStream_t st);
cudaError_t launch_pages_compact(const ns_kv_pages &c, const int32_t *seqs, const int32_t *base, const int32_t *keep,
                                 int keep_ld, const int32_t *n_keep, int n, uint32_t *err, cudaStream_t st);
cudaError_t launch_pages_copy(const ns_kv_pages &c, const int32_t *src, const int32_t *dst, int n, uint32_t *err,
                              cudaStream_t st);

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
};
// What a device holds of the kernels for few rows (found when it is first used).
struct PagedFit {
  int clusters[2][2][2];  // resident at once: dtype, dim 64 or 128, small or large CTAs
};
int64_t paged_attn_ws(int n_seqs, int n, int q_heads, int kv_heads, int dim, int sms);
cudaError_t prepare_paged_attn(PagedFit *fit);
cudaError_t launch_paged_attn(const PagedAttnArgs &a, int dtype, int dim, int sms, const PagedFit &fit,
                              cudaStream_t st);

// The same for more than 16 rows, on tcgen05 (ns_paged_umma.cu).
bool paged_umma_ok(const PagedAttnArgs &a);
cudaError_t prepare_paged_umma();
cudaError_t launch_paged_umma(const PagedAttnArgs &a, int dtype, int dim, int sms, cudaStream_t st);

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
