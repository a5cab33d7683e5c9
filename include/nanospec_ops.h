/*
 * nanospec_ops.h — C ABI of the serving operators around the draft head
 * (GB300, sm_103a): norms and rotation of heads, attention over whole prompts, attention of new tokens
 * over a paged key-value cache, the cache's bookkeeping and data movement,
 * and log probabilities of given tokens.
 *
 * The conventions of nanospec.h hold (device pointers, asynchronous on the
 * given stream, NS_ERR_ARG before anything is enqueued).  These calls need no
 * handle and allocate nothing: what they keep between their kernels goes into
 * a workspace that the caller gives, and may be used again by the next call
 * on the same stream.  Strides are in elements unless a name says bytes.
 * Pointers are aligned to what they point to (NS_ERR_ARG), or as a call says.
 *
 * Problems that only the device can see (a sequence, page or token id out of
 * range, no free page) set a sticky flag in a word of the library, one for
 * each device, read by ns_ops_get_error; what is out of range is skipped, and
 * nothing outside the given buffers is read or written.
 */
#ifndef NANOSPEC_OPS_H
#define NANOSPEC_OPS_H

#include "nanospec.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further flags of ns_ops_get_error (NS_FLAG_BAD_ID and NS_FLAG_TIMEOUT as in nanospec.h). */
#define NS_FLAG_NO_PAGES 0x10u    /* ns_pages_extend found too few free pages and changed nothing      */
#define NS_FLAG_BAD_SEQ 0x20u     /* a sequence, length or kept position was invalid and was skipped    */
#define NS_FLAG_SHARED_PAGE 0x40u /* a row of a page that another sequence holds too was not written    */

/* Element types. */
#define NS_DTYPE_BF16 0
#define NS_DTYPE_F16 1
#define NS_DTYPE_F32 2

#define NS_MAX_NEW 64          /* new tokens of a sequence in ns_attend_paged (NS_MAX_ROWS)  */
#define NS_MAX_ATTEND_SEQS 4096 /* sequences of one ns_attend_paged call                      */
#define NS_MAX_GROUPS 512      /* groups of one ns_attend_shared call                         */
#define NS_MAX_POSITIONS 0x7ffffe00 /* table_ld * page_size of ns_attend_paged: ends of tiles fit 31 bits */
#define NS_MAX_ALTERNATIVES 32 /* k of ns_token_logprobs                                      */

/* The sticky flags of the current device (synchronises it); clears them when `clear` is non-zero. */
NS_API ns_status ns_ops_get_error(uint32_t *flags, int32_t clear);

/*
 * Norms of queries and keys for each head and their rotation by position, in
 * one pass.  A row x (one token, one head) of `dim` columns becomes
 *   y = x * w / sqrt(mean(x^2) + eps)   (eps negative: no norm, y = x),
 * and then the pairs i of its first `rotary` columns, (i, i + rotary / 2) or,
 * with `neighbours`, (2i, 2i + 1), turn by t = position * inv_freq[i]:
 *   (a, b) -> (a cos t - b sin t, b cos t + a sin t).
 *   d_q   [tokens x q_heads x dim], d_k [tokens x kv_heads x dim] (NULL with
 *         kv_heads 0) of `dtype` (bf16 or f16), rows of dim consecutive
 *         elements, strides in elements, multiples of 8; 16-byte aligned
 *   d_positions int32 [tokens]; d_inv_freq fp64 [rotary / 2], finite; rotary a
 *         multiple of 16, 0 to dim
 *   d_q_weight, d_k_weight [dim] of `dtype`, 16-byte aligned, or NULL (ones);
 *         NULL without a norm
 *   d_q_out, d_k_out as d_q and d_k, with strides of their own; an output may
 *         be its input (the same address and strides), and may not overlap the
 *         inputs otherwise
 * dim is 64 or 128.  All arithmetic is fp32 and rounded once; angles are taken
 * modulo a turn in 64-bit fixed point and are good to about 2^-26 of a turn,
 * at far positions as at near ones.
 */
NS_API ns_status ns_norm_rotate(const void *d_q, const void *d_k, int32_t dtype, int32_t tokens, int32_t q_heads,
                                int32_t kv_heads, int32_t dim, int64_t q_token, int64_t q_head, int64_t k_token,
                                int64_t k_head, const int32_t *d_positions, const double *d_inv_freq, int32_t rotary,
                                int32_t neighbours, const void *d_q_weight, const void *d_k_weight, float eps,
                                void *d_q_out, void *d_k_out, int64_t qo_token, int64_t qo_head, int64_t ko_token,
                                int64_t ko_head, ns_stream stream);

/*
 * Attention over whole prompts: causal, grouped heads, sequences packed one
 * after the other.  For token i of a sequence and query head h, whose
 * key-value head is h / (q_heads / kv_heads):
 *   out_i = sum_j softmax_j(scale * q_i . k_j) v_j   over j <= i of its sequence,
 *   lse_i = log sum_j exp(scale * q_i . k_j).
 *   d_q   [tokens x q_heads x dim], d_k, d_v [tokens x kv_heads x dim], of
 *         `dtype` (bf16 or f16), rows of dim consecutive elements, token and
 *         head strides in elements, positive multiples of 8 (any for an axis
 *         of one); 16-byte aligned
 *   d_cu  int32 [n_seqs + 1]: sequence s holds tokens d_cu[s] .. d_cu[s+1] - 1
 *         (0 first, not decreasing, `tokens` last; empty sequences are fine)
 *   max_len  HOST: no sequence is longer (tokens past it are not computed and
 *         flag NS_FLAG_BAD_SEQ; with 0, or no sequences, the call does
 *         nothing).  It takes part in how the keys are split, so results of
 *         another bound may differ by their rounding
 *   d_out [tokens x q_heads x dim] of `dtype`, contiguous; d_lse fp32 [tokens x q_heads] or NULL
 * dim is 64 or 128.  Scores, softmax sums and the output's sums are fp32; the
 * probabilities are rounded to `dtype` before the product with v.  A value of
 * v that is not finite reaches only rows that see it; bf16 values with |v| times
 * a sequence's length / 64 of 2^113 and more may overflow in the sums.
 */
NS_API ns_status ns_attend_prompt(const void *d_q, const void *d_k, const void *d_v, int32_t dtype, int32_t tokens,
                                  int32_t q_heads, int32_t kv_heads, int32_t dim, int64_t q_token, int64_t q_head,
                                  int64_t k_token, int64_t k_head, int64_t v_token, int64_t v_head,
                                  const int32_t *d_cu, int32_t n_seqs, int32_t max_len, float scale, void *d_out,
                                  float *d_lse, ns_stream stream);

/*
 * Attention of the new tokens of n_seqs sequences over one layer of a paged
 * key-value cache.  Call sequence b is cache sequence s = d_seqs[b], which
 * holds len = d_lengths[s] positions, the last n of them the new tokens
 * (their keys and values are in the cache already).  Position p lives in page
 * d_table[s * table_ld + p / page_size], row p % page_size.  New token i (at
 * position len - n + i) sees every position before len - n, and new token j
 * where bit j of d_mask[b * n + i] is set; d_mask NULL means j <= i (a chain).
 * No row sees the positions of a page whose id is out of range
 * (NS_FLAG_BAD_ID).  A row that sees nothing (len 0, or an empty mask and no
 * context) gives zeros and an lse of -inf.
 *   d_q    [n_seqs x n x q_heads x dim], strides in elements (even; more than 16 rows, n * q_heads / kv_heads,
 *          take about a third of the time with positive multiples of 8, as which an axis of one counts, and 16-byte
 *          alignment)
 *   d_k, d_v  [n_pages x kv_heads x page_size x dim] of one layer, strides in
 *          elements (multiples of 8): page, head, token
 *   d_mask int64 [n_seqs x n] or NULL
 *   max_len  HOST: a bound on the lengths (0: table_ld * page_size) by which
 *          the keys are split; results depend on it by their rounding alone,
 *          and a length above it is attended all the same
 *   d_out  [n_seqs x n x q_heads x dim] contiguous, 16-byte aligned, d_lse fp32 [n_seqs x n x q_heads] or NULL
 *   d_ws   device workspace of ns_attend_paged_workspace(...) bytes, 16-byte
 *          aligned, contents immaterial
 * 1 <= n <= NS_MAX_NEW, dim 64 or 128, page_size a power of two from 8 to 1024,
 * table_ld * page_size at most NS_MAX_POSITIONS.
 * Scores, softmax sums and the output's sums are fp32; the probabilities are
 * rounded to `dtype` before the product with v, as in ns_attend_prompt.  With
 * more than 16 rows, as there, a sum of the output may pass its final size on
 * its way by 2^15 for each 64 keys: bf16 values v with |v| len / 64 of 2^113
 * and more may overflow (16 rows: |v| len of 2^128).
 */
NS_API int64_t ns_attend_paged_workspace(int32_t n_seqs, int32_t n, int32_t q_heads, int32_t kv_heads, int32_t dim);
NS_API ns_status ns_attend_paged(const void *d_q, int32_t dtype, int32_t n_seqs, int32_t n, int32_t q_heads,
                                 int32_t kv_heads, int32_t dim, int64_t q_seq, int64_t q_token, int64_t q_head,
                                 const void *d_k, const void *d_v, int32_t n_pages, int32_t page_size, int64_t k_page,
                                 int64_t k_head, int64_t k_token, int64_t v_page, int64_t v_head, int64_t v_token,
                                 const int32_t *d_table, int32_t table_ld, int32_t max_seqs, const int32_t *d_lengths,
                                 const int32_t *d_seqs, const int64_t *d_mask, float scale, int32_t max_len,
                                 void *d_out, float *d_lse, void *d_ws, int64_t ws_bytes, ns_stream stream);

/*
 * ns_attend_paged for groups of sequences that begin with the same pages, as
 * samples of one prompt do after ns_pages_fork: call sequences d_groups[g] ..
 * d_groups[g+1] - 1 (int32 [n_groups + 1], 0 first, not decreasing, n_seqs
 * last) are group g.  How much its members share is found in the table: the
 * positions in pages that stand at the beginning of every member's row and are
 * context for all of them, in whole tiles of 128.  They are read once for each
 * 256 rows of the group (new tokens and the query heads of a key-value head)
 * and the rest of each sequence as in ns_attend_paged; results differ from its
 * by their rounding alone (and values are as large as it takes them with more
 * than 16 rows).  Where sharing would not pay (more than 128 rows to
 * a sequence; up to 192 MB of keys and values by max_len, with more than 16
 * rows counted as of 16 bits; no fewer groups than sequences, or by max_len
 * less than 128 positions of context) the call is that call.  Groups that are not as said are flagged
 * (NS_FLAG_BAD_SEQ) and nothing is shared; a sequence that is invalid ends its
 * group's sharing.
 * The sequences' queries follow one another as the tokens do: q_seq is
 * n * q_token, unless n or n_seqs is 1.  d_q is 16-byte aligned, its strides
 * positive multiples of 8, as d_k's and d_v's are.  d_ws: device workspace of
 * ns_attend_shared_workspace(...) bytes, 16-byte aligned, contents immaterial.
 */
NS_API int64_t ns_attend_shared_workspace(int32_t n_seqs, int32_t n_groups, int32_t n, int32_t q_heads,
                                          int32_t kv_heads, int32_t dim);
NS_API ns_status ns_attend_shared(const void *d_q, int32_t dtype, int32_t n_seqs, int32_t n, int32_t q_heads,
                                  int32_t kv_heads, int32_t dim, int64_t q_seq, int64_t q_token, int64_t q_head,
                                  const void *d_k, const void *d_v, int32_t n_pages, int32_t page_size, int64_t k_page,
                                  int64_t k_head, int64_t k_token, int64_t v_page, int64_t v_head, int64_t v_token,
                                  const int32_t *d_table, int32_t table_ld, int32_t max_seqs, const int32_t *d_lengths,
                                  const int32_t *d_seqs, const int32_t *d_groups, int32_t n_groups,
                                  const int64_t *d_mask, float scale, int32_t max_len, void *d_out, float *d_lse,
                                  void *d_ws, int64_t ws_bytes, ns_stream stream);

/*
 * A paged key-value cache of several layers, as the ns_pages_* calls see it.
 * A page holds page_size positions of every layer and head.  Row (layer,
 * page, head, position) starts at k + layer * k_layer + page * k_page +
 * head * k_head + row * k_token BYTES and is row_bytes long; strides and row_bytes
 * are multiples of 16, v likewise.
 *   table    int32 [max_seqs x table_ld]: the pages of each sequence in
 *            order, -1 past the last
 *   lengths  int32 [max_seqs]: positions each sequence holds;
 *            ceil(length / page_size) pages of its table row are in use
 *   refs     int32 [pages]: how many sequences hold each page (0: free)
 * Sequences in one call must be distinct; a repeated or out-of-range one is
 * skipped and flags NS_FLAG_BAD_SEQ.  Calls on one cache must be ordered.
 */
typedef struct ns_kv_pages {
  void *k, *v;
  int64_t k_layer, k_page, k_head, k_token; /* bytes */
  int64_t v_layer, v_page, v_head, v_token; /* bytes */
  int32_t layers, pages, heads, page_size, row_bytes;
  int32_t max_seqs, table_ld;
  int32_t *table, *lengths, *refs;
} ns_kv_pages;

/*
 * The exponents of a cache of 8 bits, whose rows are row_bytes (64 or 128)
 * codes in e4m3: a row with exponent byte b stands for code * 2^(b - 127), and
 * for NaN in each element where b is 255.  Bytes [layers x pages x heads x
 * page_size], a page's positions one after the other; strides in bytes.
 * page_size, strides and addresses are multiples of 8.
 *
 * ns_pages_write_scaled rounds a row to the smallest power of two by which it
 * fits: e = ceil(log2(max |x| / 448)), within +-40; codes are x 2^-e to nearest
 * even (what is above 448 2^40 saturates), the byte is e + 127.  A row that
 * holds an infinity or NaN gets 255.  Bytes below 87 and from 168 to 254, which
 * no call writes, may lose precision in ns_attend_paged_scaled.
 */
typedef struct ns_kv_scales {
  uint8_t *k, *v;
  int64_t k_layer, k_page, k_head;
  int64_t v_layer, v_page, v_head;
} ns_kv_scales;

/* Most sequences of one ns_pages_* call. */
#define NS_MAX_PAGE_SEQS 8192

/*
 * Shortens sequences d_seqs[0 .. n) to d_new_len[i] positions (NULL: to 0,
 * which frees them): each page past the last one needed loses this holder.
 * A sequence that is not longer stays as it is.
 */
NS_API ns_status ns_pages_truncate(const ns_kv_pages *c, const int32_t *d_seqs, const int32_t *d_new_len, int32_t n,
                                   ns_stream stream);

/*
 * Sequence d_dst[i], which must be empty, becomes a copy of d_src[i]: it
 * holds the same pages (no data moves).  A destination may not be a source of
 * the same call.
 */
NS_API ns_status ns_pages_fork(const ns_kv_pages *c, const int32_t *d_src, const int32_t *d_dst, int32_t n,
                               ns_stream stream);

/*
 * Lengthens sequence d_seqs[i] by d_n_new[i] positions and gives it the pages
 * for them.  Where its last page is partly filled and held by another
 * sequence too when the call begins, it gets a copy of that page (of every
 * layer) in its place.  Free pages are given lowest id first, in call order,
 * a sequence's copy before its new pages.  When they do not suffice, the call
 * changes nothing and flags NS_FLAG_NO_PAGES; a sequence that would outgrow
 * its table row is skipped and flags NS_FLAG_BAD_SEQ.
 * d_ws: ns_pages_workspace bytes, 16-byte aligned.
 */
NS_API int64_t ns_pages_workspace(const ns_kv_pages *c, int32_t n);
NS_API ns_status ns_pages_extend(const ns_kv_pages *c, const int32_t *d_seqs, const int32_t *d_n_new, int32_t n,
                                 void *d_ws, int64_t ws_bytes, ns_stream stream);

/*
 * Writes new keys and values into one layer: tokens d_cu[i] .. d_cu[i+1] - 1
 * of d_k_new / d_v_new ([tokens x heads x row_bytes], strides in bytes,
 * multiples of 16) are the last positions of sequence d_seqs[i].  d_cu int32
 * [n + 1].  A row of a page that another sequence holds too is not written
 * (NS_FLAG_SHARED_PAGE).
 */
NS_API ns_status ns_pages_write(const ns_kv_pages *c, int32_t layer, const int32_t *d_seqs, const int32_t *d_cu,
                                int32_t n, const void *d_k_new, const void *d_v_new, int64_t k_token, int64_t k_head,
                                int64_t v_token, int64_t v_head, int32_t tokens, ns_stream stream);

/*
 * Keeps some of each sequence's positions from d_base[i] on and drops the
 * rest: in every layer, position base + t takes the row of position base +
 * d_keep[i * keep_ld + t] for t < d_n_keep[i]; then the sequence is shortened
 * to base + n_keep (as ns_pages_truncate does).  d_keep is strictly
 * increasing.  An entry that is not, or is past the sequence's end, is
 * skipped and flags NS_FLAG_BAD_SEQ; a row whose new page another sequence
 * holds too is not written (NS_FLAG_SHARED_PAGE).
 */
NS_API ns_status ns_pages_compact(const ns_kv_pages *c, const int32_t *d_seqs, const int32_t *d_base,
                                  const int32_t *d_keep, int32_t keep_ld, const int32_t *d_n_keep, int32_t n,
                                  ns_stream stream);

/*
 * Copies pages d_src[i] onto pages d_dst[i], i < n, in every layer.  A
 * destination may be neither another destination nor a source.  Refs, table
 * and lengths are left alone.  Ids out of range are skipped (NS_FLAG_BAD_ID).
 */
NS_API ns_status ns_pages_copy(const ns_kv_pages *c, const int32_t *d_src, const int32_t *d_dst, int32_t n,
                               ns_stream stream);

/*
 * The calls above that move rows, over a cache of 8 bits: the exponents move
 * along.  (ns_pages_truncate and ns_pages_fork move none and take any cache.)
 */
NS_API ns_status ns_pages_extend_scaled(const ns_kv_pages *c, const ns_kv_scales *s, const int32_t *d_seqs,
                                        const int32_t *d_n_new, int32_t n, void *d_ws, int64_t ws_bytes,
                                        ns_stream stream);
NS_API ns_status ns_pages_compact_scaled(const ns_kv_pages *c, const ns_kv_scales *s, const int32_t *d_seqs,
                                         const int32_t *d_base, const int32_t *d_keep, int32_t keep_ld,
                                         const int32_t *d_n_keep, int32_t n, ns_stream stream);
NS_API ns_status ns_pages_copy_scaled(const ns_kv_pages *c, const ns_kv_scales *s, const int32_t *d_src,
                                      const int32_t *d_dst, int32_t n, ns_stream stream);

/* ns_pages_write into a cache of 8 bits: rows of row_bytes elements of `dtype` (bf16 or f16), rounded as said above. */
NS_API ns_status ns_pages_write_scaled(const ns_kv_pages *c, const ns_kv_scales *s, int32_t layer,
                                       const int32_t *d_seqs, const int32_t *d_cu, int32_t n, const void *d_k_new,
                                       const void *d_v_new, int32_t dtype, int64_t k_token, int64_t k_head,
                                       int64_t v_token, int64_t v_head, int32_t tokens, ns_stream stream);

/*
 * The other way round: tokens d_cu[i] .. d_cu[i+1] - 1 of d_k and d_v become
 * the last positions of sequence d_seqs[i] in one layer, bytes as they are or,
 * with s, what the codes stand for, in `dtype` (bf16 or f16; ignored without
 * s; f16 rounds what is above its range to infinity).  A sequence may stand
 * there more than once.  Tokens of an invalid sequence or page are not written.
 */
NS_API ns_status ns_pages_read(const ns_kv_pages *c, const ns_kv_scales *s, int32_t layer, const int32_t *d_seqs,
                               const int32_t *d_cu, int32_t n, void *d_k, void *d_v, int32_t dtype, int64_t k_token,
                               int64_t k_head, int64_t v_token, int64_t v_head, int32_t tokens, ns_stream stream);

/*
 * ns_attend_paged over one layer of a cache of 8 bits: d_k and d_v are codes
 * [n_pages x kv_heads x page_size x dim] with strides in bytes, multiples of
 * 16, d_k_exp and d_v_exp their exponents [n_pages x kv_heads x page_size],
 * strides of page and head multiples of 8, as the addresses are.  `dtype` is
 * that of d_q and d_out.  The products see the codes' values exactly; bf16
 * queries become fp16 with a row's largest element at 1 to 2, so that one below
 * 2^-14 of that is off by up to 2^-25 of it, and probabilities are rounded to
 * fp16 with the value's scale in them (up to 16 rows, or queries as said at d_q
 * that TMA cannot fetch); or queries stay as they are and probabilities are
 * rounded to `dtype`.  Those rows in fp16 see what an fp16 holds: a code times
 * its power of two is rounded below 2^-14, and beyond 65504, which rows written
 * from fp16 are not, is 65504.
 */
NS_API ns_status ns_attend_paged_scaled(const void *d_q, int32_t dtype, int32_t n_seqs, int32_t n, int32_t q_heads,
                                        int32_t kv_heads, int32_t dim, int64_t q_seq, int64_t q_token, int64_t q_head,
                                        const void *d_k, const void *d_v, int32_t n_pages, int32_t page_size,
                                        int64_t k_page, int64_t k_head, int64_t k_token, int64_t v_page,
                                        int64_t v_head, int64_t v_token, const uint8_t *d_k_exp,
                                        const uint8_t *d_v_exp, int64_t ke_page, int64_t ke_head, int64_t ve_page,
                                        int64_t ve_head, const int32_t *d_table, int32_t table_ld, int32_t max_seqs,
                                        const int32_t *d_lengths, const int32_t *d_seqs, const int64_t *d_mask,
                                        float scale, int32_t max_len, void *d_out, float *d_lse, void *d_ws,
                                        int64_t ws_bytes, ns_stream stream);

/* ns_attend_shared over one layer of a cache of 8 bits, as ns_attend_paged_scaled has it (positive strides). */
NS_API ns_status ns_attend_shared_scaled(const void *d_q, int32_t dtype, int32_t n_seqs, int32_t n, int32_t q_heads,
                                         int32_t kv_heads, int32_t dim, int64_t q_seq, int64_t q_token,
                                         int64_t q_head, const void *d_k, const void *d_v, int32_t n_pages,
                                         int32_t page_size, int64_t k_page, int64_t k_head, int64_t k_token,
                                         int64_t v_page, int64_t v_head, int64_t v_token, const uint8_t *d_k_exp,
                                         const uint8_t *d_v_exp, int64_t ke_page, int64_t ke_head, int64_t ve_page,
                                         int64_t ve_head, const int32_t *d_table, int32_t table_ld, int32_t max_seqs,
                                         const int32_t *d_lengths, const int32_t *d_seqs, const int32_t *d_groups,
                                         int32_t n_groups, const int64_t *d_mask, float scale, int32_t max_len,
                                         void *d_out, float *d_lse, void *d_ws, int64_t ws_bytes, ns_stream stream);

/*
 * Log probabilities of given tokens under softmax(logits / temperature), with
 * the distribution's entropy and the k most probable tokens:
 *   d_logits  [rows x V] of dtype (fp32, bf16 or f16), row stride ld elements
 *   d_ids     int32 [rows x n_ids] (NULL with n_ids 0); an id outside [0, V)
 *             gives NaN and, unless it is -1 (an empty place), flags NS_FLAG_BAD_ID
 *   d_logprobs fp32 [rows x n_ids], d_entropy fp32 [rows] or NULL (natural
 *             logarithm), d_lse fp32 [rows] or NULL: log sum exp(logits / temperature)
 *   d_top_ids int32 [rows x k], d_top_logprobs fp32 [rows x k] (0 <= k <=
 *             NS_MAX_ALTERNATIVES): ordered by logit, ties to the smaller id, as
 *             every top-k of this library; NaN never ranks, places left over
 *             hold -1 and -inf
 *   temperature  positive, and log2(e) / temperature finite in fp32 (from
 *             about 4.3e-39 on)
 * A logit of -inf has probability 0.  A row of nothing but -inf has lse and
 * log probabilities of -inf and entropy 0; a row that holds a NaN or +inf has
 * NaN for each of these values, as the formula does.  Sums are fp32.
 */
NS_API ns_status ns_token_logprobs(const void *d_logits, int32_t dtype, int32_t rows, int32_t V, int64_t ld,
                                   float temperature, const int32_t *d_ids, int32_t n_ids, int32_t k,
                                   float *d_logprobs, float *d_entropy, float *d_lse, int32_t *d_top_ids,
                                   float *d_top_logprobs, ns_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* NANOSPEC_OPS_H */
