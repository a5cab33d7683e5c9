// C ABI of the serving operators (declared in include/nanospec_ops.h):
// argument checks on the host, then the launches on the caller's stream.
#include <cmath>
#include <mutex>

#include "ns_ops.cuh"

namespace {

__device__ uint32_t g_ops_flags;  // sticky flags of a device (one copy per device)

constexpr int kMaxDevices = 64;

struct Device {
  bool ready = false;
  int sms = 0;
  ns::PagedFit fit{};
  uint32_t *flags = nullptr;
};
std::mutex g_mutex;
Device g_devices[kMaxDevices];

// The current device, its kernels prepared.  The first call on a device sets
// the kernels' limits; later ones only read.
ns_status current(const Device **out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return NS_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return NS_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_mutex);
  Device &d = g_devices[dev];
  if (!d.ready) {
    void *p = nullptr;
    if (cudaGetSymbolAddress(&p, g_ops_flags) != cudaSuccess) return NS_ERR_CUDA;
    if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return NS_ERR_CUDA;
    if (ns::prepare_paged_attn(&d.fit) != cudaSuccess || ns::prepare_prompt_attn() != cudaSuccess) return NS_ERR_CUDA;
    d.flags = static_cast<uint32_t *>(p);
    d.ready = true;
  }
  *out = &d;
  return NS_OK;
}

ns_status done(cudaError_t e) { return e == cudaSuccess ? NS_OK : NS_ERR_CUDA; }

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
// Whether each pointer may be read as 32-bit words (NULL may).
template <typename... P>
bool words(const P *...p) {
  return (... && aligned(p, 4));
}

bool attn_type(int dtype, int dim) {
  return (dtype == NS_DTYPE_BF16 || dtype == NS_DTYPE_F16) && (dim == 64 || dim == 128);
}
bool heads_ok(int q, int kv) { return q >= 1 && kv >= 1 && q <= 65535 && q % kv == 0; }
bool by8(int64_t s) { return s % 8 == 0; }
// An axis of one place is never stepped along: whatever its stride is, it becomes `row`.
int64_t step(int64_t s, int places, int row) { return places == 1 ? row : s; }
// A stride (elements) that a TMA map takes.
bool map_stride(int64_t &s, int places, int row) {
  s = step(s, places, row);
  return s > 0 && by8(s) && s < (int64_t)1 << 39;
}

bool cache_ok(const ns_kv_pages *c) {
  if (!c || !c->k || !c->v || !c->table || !c->lengths || !c->refs) return false;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->table, 4) || !aligned(c->lengths, 4) ||
      !aligned(c->refs, 4))
    return false;
  const int64_t strides[8] = {c->k_layer, c->k_page, c->k_head, c->k_token, c->v_layer, c->v_page, c->v_head, c->v_token};
  for (int64_t s : strides)
    if (s % 16) return false;
  return c->layers >= 1 && c->pages >= 1 && c->heads >= 1 && c->page_size >= 1 && c->row_bytes >= 16 &&
         c->row_bytes % 16 == 0 && c->row_bytes <= 65536 && c->max_seqs >= 1 && c->table_ld >= 1 &&
         c->table_ld <= (1 << 20) && (int64_t)c->table_ld * c->page_size <= 0x7fffffffLL &&
         (int64_t)c->page_size * c->row_bytes <= 0x7fffffffLL / 16 && (int64_t)c->heads * c->row_bytes <= 0x7fffffffLL;
}
bool page_seqs(int n) { return n >= 0 && n <= NS_MAX_PAGE_SEQS; }

}  // namespace

extern "C" {

ns_status ns_ops_get_error(uint32_t *flags, int32_t clear) {
  if (!flags) return NS_ERR_ARG;
  const Device *d = nullptr;
  if (ns_status s = current(&d)) return s;
  if (cudaDeviceSynchronize() != cudaSuccess) return NS_ERR_CUDA;
  if (cudaMemcpy(flags, d->flags, 4, cudaMemcpyDeviceToHost) != cudaSuccess) return NS_ERR_CUDA;
  if (clear && cudaMemset(d->flags, 0, 4) != cudaSuccess) return NS_ERR_CUDA;
  return NS_OK;
}

ns_status ns_attend_prompt(const void *d_q, const void *d_k, const void *d_v, int32_t dtype, int32_t tokens,
                           int32_t q_heads, int32_t kv_heads, int32_t dim, int64_t q_token, int64_t q_head,
                           int64_t k_token, int64_t k_head, int64_t v_token, int64_t v_head, const int32_t *d_cu,
                           int32_t n_seqs, int32_t max_len, float scale, void *d_out, float *d_lse,
                           ns_stream stream) {
  if (!attn_type(dtype, dim) || !heads_ok(q_heads, kv_heads) || tokens < 0 || n_seqs < 0 || n_seqs > 65535 ||
      max_len < 0 || !std::isfinite(scale) || scale <= 0.f)
    return NS_ERR_ARG;
  if (tokens == 0 || n_seqs == 0 || max_len == 0) return NS_OK;
  if (!d_q || !d_k || !d_v || !d_cu || !d_out || !aligned(d_q, 16) || !aligned(d_k, 16) || !aligned(d_v, 16) ||
      !aligned(d_out, 16) || !aligned(d_lse, 4) || !aligned(d_cu, 4) || !map_stride(q_token, tokens, dim) ||
      !map_stride(k_token, tokens, dim) || !map_stride(v_token, tokens, dim) || !map_stride(q_head, q_heads, dim) ||
      !map_stride(k_head, kv_heads, dim) || !map_stride(v_head, kv_heads, dim))
    return NS_ERR_ARG;
  const Device *d = nullptr;
  if (ns_status s = current(&d)) return s;
  ns::PromptAttnArgs a{};
  a.q = d_q, a.k = d_k, a.v = d_v;
  a.tokens = tokens, a.q_heads = q_heads, a.kv_heads = kv_heads, a.group = q_heads / kv_heads;
  a.q_token = q_token, a.q_head = q_head, a.k_token = k_token, a.k_head = k_head, a.v_token = v_token;
  a.v_head = v_head;
  a.cu = d_cu, a.n_seqs = n_seqs, a.max_len = max_len < tokens ? max_len : tokens;
  a.scale = scale, a.out = d_out, a.lse = d_lse, a.err = d->flags;
  return done(ns::launch_prompt_attn(a, dtype, dim, d->sms, static_cast<cudaStream_t>(stream)));
}

int64_t ns_attend_paged_workspace(int32_t n_seqs, int32_t n, int32_t q_heads, int32_t kv_heads, int32_t dim) {
  if (n_seqs < 0 || n_seqs > NS_MAX_ATTEND_SEQS || n < 1 || n > NS_MAX_NEW || !heads_ok(q_heads, kv_heads) ||
      (dim != 64 && dim != 128))
    return 0;
  const Device *d = nullptr;
  if (current(&d)) return 0;
  return ns::paged_attn_ws(n_seqs, n, q_heads, kv_heads, dim, d->sms);
}

ns_status ns_attend_paged(const void *d_q, int32_t dtype, int32_t n_seqs, int32_t n, int32_t q_heads,
                          int32_t kv_heads, int32_t dim, int64_t q_seq, int64_t q_token, int64_t q_head,
                          const void *d_k, const void *d_v, int32_t n_pages, int32_t page_size, int64_t k_page,
                          int64_t k_head, int64_t k_token, int64_t v_page, int64_t v_head, int64_t v_token,
                          const int32_t *d_table, int32_t table_ld, int32_t max_seqs, const int32_t *d_lengths,
                          const int32_t *d_seqs, const int64_t *d_mask, float scale, int32_t max_len, void *d_out,
                          float *d_lse, void *d_ws, int64_t ws_bytes, ns_stream stream) {
  if (!attn_type(dtype, dim) || !heads_ok(q_heads, kv_heads) || n_seqs < 0 || n_seqs > NS_MAX_ATTEND_SEQS || n < 1 ||
      n > NS_MAX_NEW || n_pages < 1 || page_size < 8 || page_size > 1024 || (page_size & (page_size - 1)) ||
      table_ld < 1 || max_seqs < 1 || (int64_t)table_ld * page_size > NS_MAX_POSITIONS || max_len < 0 ||
      !std::isfinite(scale) || scale <= 0.f)
    return NS_ERR_ARG;
  if (n_seqs == 0) return NS_OK;
  if (!d_q || !d_k || !d_v || !d_table || !d_lengths || !d_seqs || !d_out || !d_ws || !aligned(d_q, 4) ||
      !aligned(d_k, 16) || !aligned(d_v, 16) || !aligned(d_out, 16) || !aligned(d_lse, 4) || !aligned(d_table, 4) ||
      !aligned(d_lengths, 4) || !aligned(d_seqs, 4) || !aligned(d_mask, 8) || !aligned(d_ws, 16) || q_seq % 2 ||
      q_token % 2 || q_head % 2 || !by8(k_page) || !by8(k_head) || !by8(k_token) || !by8(v_page) || !by8(v_head) ||
      !by8(v_token))
    return NS_ERR_ARG;
  const Device *d = nullptr;
  if (ns_status s = current(&d)) return s;
  if (ws_bytes < ns::paged_attn_ws(n_seqs, n, q_heads, kv_heads, dim, d->sms)) return NS_ERR_ARG;
  ns::PagedAttnArgs a{};
  a.q = d_q, a.k = d_k, a.v = d_v;
  a.n_seqs = n_seqs, a.n = n, a.q_heads = q_heads, a.kv_heads = kv_heads, a.group = q_heads / kv_heads;
  a.q_seq = step(q_seq, n_seqs, dim), a.q_token = step(q_token, n, dim), a.q_head = step(q_head, q_heads, dim);
  a.k_page = step(k_page, n_pages, dim), a.k_head = step(k_head, kv_heads, dim), a.k_token = k_token;
  a.v_page = step(v_page, n_pages, dim), a.v_head = step(v_head, kv_heads, dim), a.v_token = v_token;
  a.n_pages = n_pages, a.table_ld = table_ld, a.max_seqs = max_seqs;
  while ((1 << a.page_shift) < page_size) ++a.page_shift;
  const int64_t most = (int64_t)table_ld * page_size;
  a.max_len = max_len == 0 || max_len > most ? (int32_t)most : max_len;
  a.table = d_table, a.lengths = d_lengths, a.seqs = d_seqs, a.mask = d_mask;
  a.scale = scale, a.out = d_out, a.lse = d_lse, a.ws = d_ws, a.err = d->flags;
  return done(ns::launch_paged_attn(a, dtype, dim, d->sms, d->fit, static_cast<cudaStream_t>(stream)));
}

ns_status ns_pages_truncate(const ns_kv_pages *c, const int32_t *d_seqs, const int32_t *d_new_len, int32_t n,
                            ns_stream stream) {
  if (!cache_ok(c) || !page_seqs(n) || (n > 0 && !d_seqs) || !words(d_seqs, d_new_len)) return NS_ERR_ARG;
  if (n == 0) return NS_OK;
  const Device *d = nullptr;
  if (ns_status s = current(&d)) return s;
  return done(ns::launch_pages_truncate(*c, d_seqs, d_new_len, n, d->flags, static_cast<cudaStream_t>(stream)));
}

ns_status ns_pages_fork(const ns_kv_pages *c, const int32_t *d_src, const int32_t *d_dst, int32_t n,
                        ns_stream stream) {
  if (!cache_ok(c) || !page_seqs(n) || (n > 0 && (!d_src || !d_dst)) || !words(d_src, d_dst)) return NS_ERR_ARG;
  if (n == 0) return NS_OK;
  const Device *d = nullptr;
  if (ns_status s = current(&d)) return s;
  return done(ns::launch_pages_fork(*c, d_src, d_dst, n, d->flags, static_cast<cudaStream_t>(stream)));
}

int64_t ns_pages_workspace(const ns_kv_pages *c, int32_t n) {
  return cache_ok(c) && page_seqs(n) ? ns::pages_extend_ws(*c, n) : 0;
}

ns_status ns_pages_extend(const ns_kv_pages *c, const int32_t *d_seqs, const int32_t *d_n_new, int32_t n, void *d_ws,
                          int64_t ws_bytes, ns_stream stream) {
  if (!cache_ok(c) || !page_seqs(n) || (n > 0 && (!d_seqs || !d_n_new || !d_ws || !aligned(d_ws, 16))) ||
      !words(d_seqs, d_n_new))
    return NS_ERR_ARG;
  if (n == 0) return NS_OK;
  if (ws_bytes < ns::pages_extend_ws(*c, n)) return NS_ERR_ARG;
  const Device *d = nullptr;
  if (ns_status s = current(&d)) return s;
  return done(ns::launch_pages_extend(*c, d_seqs, d_n_new, n, d_ws, d->flags, static_cast<cudaStream_t>(stream)));
}

ns_status ns_pages_write(const ns_kv_pages *c, int32_t layer, const int32_t *d_seqs, const int32_t *d_cu, int32_t n,
                         const void *d_k_new, const void *d_v_new, int64_t k_token, int64_t k_head, int64_t v_token,
                         int64_t v_head, int32_t tokens, ns_stream stream) {
  if (!cache_ok(c) || layer < 0 || layer >= c->layers || !page_seqs(n) || tokens < 0) return NS_ERR_ARG;
  if (n == 0 || tokens == 0) return NS_OK;
  if (!d_seqs || !d_cu || !d_k_new || !d_v_new || !aligned(d_k_new, 16) || !aligned(d_v_new, 16) || k_token % 16 ||
      k_head % 16 || v_token % 16 || v_head % 16 || !words(d_seqs, d_cu))
    return NS_ERR_ARG;
  const Device *d = nullptr;
  if (ns_status s = current(&d)) return s;
  return done(ns::launch_pages_write(*c, layer, d_seqs, d_cu, n, d_k_new, d_v_new, k_token, k_head, v_token, v_head,
                                     tokens, d->flags, static_cast<cudaStream_t>(stream)));
}

ns_status ns_pages_compact(const ns_kv_pages *c, const int32_t *d_seqs, const int32_t *d_base, const int32_t *d_keep,
                           int32_t keep_ld, const int32_t *d_n_keep, int32_t n, ns_stream stream) {
  if (!cache_ok(c) || !page_seqs(n) || keep_ld < 0 || (n > 0 && (!d_seqs || !d_base || !d_n_keep)) ||
      (n > 0 && keep_ld > 0 && !d_keep) || !words(d_seqs, d_base, d_keep, d_n_keep))
    return NS_ERR_ARG;
  if (n == 0) return NS_OK;
  const Device *d = nullptr;
  if (ns_status s = current(&d)) return s;
  return done(ns::launch_pages_compact(*c, d_seqs, d_base, d_keep, keep_ld, d_n_keep, n, d->flags,
                                       static_cast<cudaStream_t>(stream)));
}

ns_status ns_pages_copy(const ns_kv_pages *c, const int32_t *d_src, const int32_t *d_dst, int32_t n,
                        ns_stream stream) {
  if (!cache_ok(c) || n < 0 || (n > 0 && (!d_src || !d_dst)) || !words(d_src, d_dst)) return NS_ERR_ARG;
  if (n == 0) return NS_OK;
  const Device *d = nullptr;
  if (ns_status s = current(&d)) return s;
  return done(ns::launch_pages_copy(*c, d_src, d_dst, n, d->flags, static_cast<cudaStream_t>(stream)));
}

ns_status ns_token_logprobs(const void *d_logits, int32_t dtype, int32_t rows, int32_t V, int64_t ld,
                            float temperature, const int32_t *d_ids, int32_t n_ids, int32_t k, float *d_logprobs,
                            float *d_entropy, float *d_lse, int32_t *d_top_ids, float *d_top_logprobs,
                            ns_stream stream) {
  if (dtype < NS_DTYPE_BF16 || dtype > NS_DTYPE_F32 || rows < 0 || V < 1 || V > (1 << 30) || ld < V || n_ids < 0 ||
      k < 0 || k > NS_MAX_ALTERNATIVES || !std::isfinite(temperature) || !(temperature > 0.f) ||
      !std::isfinite(1.f / temperature * 1.4426950408889634f))  // the kernels' log2(e) / T
    return NS_ERR_ARG;
  if (rows == 0) return NS_OK;
  if (rows > (1 << 27) || !d_logits || !aligned(d_logits, dtype == NS_DTYPE_F32 ? 4 : 2) ||
      (n_ids > 0 && (!d_ids || !d_logprobs)) || (k > 0 && (!d_top_ids || !d_top_logprobs)) ||
      !words(d_ids, d_logprobs, d_entropy, d_lse, d_top_ids, d_top_logprobs))
    return NS_ERR_ARG;
  const Device *d = nullptr;
  if (ns_status s = current(&d)) return s;
  ns::LogprobArgs a{};
  a.logits = d_logits, a.rows = rows, a.V = V, a.ld = ld, a.inv_temperature = 1.f / temperature;
  a.ids = d_ids, a.n_ids = n_ids, a.k = k, a.logprobs = d_logprobs, a.entropy = d_entropy, a.lse = d_lse;
  a.top_ids = d_top_ids, a.top_logprobs = d_top_logprobs, a.err = d->flags;
  return done(ns::launch_logprobs(a, dtype, d->sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
