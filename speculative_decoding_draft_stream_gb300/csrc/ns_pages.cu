// The paged key-value cache: who holds which page, and the rows that move.
//
// A page is free when its reference count is 0, so the counts are the whole
// state of the pool: no free list has to be kept consistent, every change is
// an integer add (whose order does not matter), and pages are given lowest id
// first, so a sequence of calls always gives the same table.
//
// Bookkeeping kernels are latency-bound (a few dependent loads of a few
// words): 2.5 to 3.5 us each in a graph, launched into each other's ends.  An
// extension also looks through the counts from page 0 on, 8192 at a time, until
// it has enough: behind 90000 taken pages that is 16 us more, behind 360000 68 us.
// The data movers are bound by HBM: each row is read and written once with
// 16-byte accesses, several per lane in flight.  16 sequences that give up
// their last step, append 60 nodes and keep 5 of them in 16 layers take 20 us
// for four calls; 64 children with their 64 MB of copied last pages 34 us;
// 8 sequences of 4001 new rows of which every second stays in 12 layers 166 us
// (393 MB read and 332 MB written by the compaction: 126 us of it).
#include "ns_internal.cuh"
#include "ns_ops.cuh"

namespace ns {
namespace {

constexpr int kSeqThreads = 128;      // truncate, fork: one CTA per sequence
constexpr int kExtendThreads = 1024;  // extend: one CTA
constexpr int kListHere = 2048;       // given pages that extend lists in shared memory
constexpr int kMoveThreads = 256;
constexpr int kMoveWarps = kMoveThreads / kWarp;
constexpr int kUnroll = 8;  // 16-byte loads a lane keeps in flight in the movers

// Each kernel may be launched while the one before it ends; it waits for that
// one's writes before it reads anything, and lets the next one be launched.
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.dynamicSmemBytes = smem;
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

__host__ __device__ inline int pages_for(long long len, int page) { return (int)((len + page - 1) / page); }

// Whether entry i of ids also stands before i (the later one is skipped).
// Called by a whole CTA; the answer is the same in every thread.
__device__ __forceinline__ bool repeated(const int32_t *ids, int i) {
  const int32_t mine = ids[i];
  int hit = 0;
  for (int j = threadIdx.x; j < i; j += blockDim.x) hit |= ids[j] == mine;
  return __syncthreads_or(hit) != 0;
}

__device__ __forceinline__ bool seq_ok(const ns_kv_pages &c, int s) { return s >= 0 && s < c.max_seqs; }
__device__ __forceinline__ bool len_ok(const ns_kv_pages &c, int len) {
  return len >= 0 && (long long)len <= (long long)c.table_ld * c.page_size;
}

// Drops this holder from the pages of table row `row` in slots [from, to).
__device__ __forceinline__ void drop_pages(const ns_kv_pages &c, int32_t *row, int from, int to, uint32_t *err) {
  for (int q = from + (int)threadIdx.x; q < to; q += blockDim.x) {
    const int p = row[q];
    row[q] = -1;
    if (p < 0 || p >= c.pages) {
      set_flag(err, NS_FLAG_BAD_ID);
      continue;
    }
    if (atomicSub(c.refs + p, 1) <= 0) {  // a count that was free already: undo
      atomicAdd(c.refs + p, 1);
      set_flag(err, NS_FLAG_BAD_ID);
    }
  }
}

// Truncation, and the second half of compaction (base given: to base +
// new_len, where new_len is at most `most`, the rows that could be kept).
__global__ void __launch_bounds__(kSeqThreads) truncate_kernel(ns_kv_pages c, const int32_t *seqs,
                                                               const int32_t *new_len, const int32_t *base,
                                                               int most, uint32_t *err) {
  wait_for_previous();
  const int i = blockIdx.x;
  const int s = seqs[i];
  const bool again = repeated(seqs, i);
  if (again || !seq_ok(c, s)) {
    if (threadIdx.x == 0) set_flag(err, NS_FLAG_BAD_SEQ);
    return;
  }
  const int len = c.lengths[s];
  const long long want = (long long)(new_len ? new_len[i] : 0) + (base ? base[i] : 0);
  if (!len_ok(c, len) || want < 0 || (new_len && (new_len[i] < 0 || new_len[i] > most)) || (base && base[i] < 0)) {
    if (threadIdx.x == 0) set_flag(err, NS_FLAG_BAD_SEQ);
    return;
  }
  if (want >= len) return;
  drop_pages(c, c.table + (size_t)s * c.table_ld, pages_for(want, c.page_size), pages_for(len, c.page_size), err);
  __syncthreads();  // every thread has read the old length
  if (threadIdx.x == 0) c.lengths[s] = (int)want;
}

__global__ void __launch_bounds__(kSeqThreads) fork_kernel(ns_kv_pages c, const int32_t *src, const int32_t *dst,
                                                           int n, uint32_t *err) {
  wait_for_previous();
  const int i = blockIdx.x;
  const int a = src[i], b = dst[i];
  int clash = 0;  // the destination is another entry's destination (the first wins) or any entry's source
  for (int j = threadIdx.x; j < n; j += blockDim.x) clash |= (j < i && dst[j] == b) || src[j] == b;
  clash = __syncthreads_or(clash);
  if (clash || !seq_ok(c, a) || !seq_ok(c, b)) {
    if (threadIdx.x == 0) set_flag(err, NS_FLAG_BAD_SEQ);
    return;
  }
  const int len = c.lengths[a];
  if (!len_ok(c, len) || c.lengths[b] != 0) {
    if (threadIdx.x == 0) set_flag(err, NS_FLAG_BAD_SEQ);
    return;
  }
  const int held = pages_for(len, c.page_size);
  const int32_t *from = c.table + (size_t)a * c.table_ld;
  int32_t *to = c.table + (size_t)b * c.table_ld;
  for (int q = threadIdx.x; q < held; q += blockDim.x) {
    const int p = from[q];
    to[q] = p;
    if (p >= 0 && p < c.pages)
      atomicAdd(c.refs + p, 1);
    else
      set_flag(err, NS_FLAG_BAD_ID);
  }
  __syncthreads();  // every thread has seen the destination empty
  if (threadIdx.x == 0) c.lengths[b] = len;
}

// Workspace of an extension, int32 words: [0] copies, [1] unused, then per
// sequence its first new slot (-1: skipped), its rank among the given pages,
// their number, and the page to copy (-1: none); the copies' sources and
// destinations; the free pages found.
struct ExtendWs {
  int32_t *n_copies, *first, *start, *count, *shared, *src, *dst, *list;
  __host__ __device__ ExtendWs(void *p, int n) {
    int32_t *w = static_cast<int32_t *>(p);
    n_copies = w;
    first = w + 4;
    start = first + n;
    count = start + n;
    shared = count + n;
    src = shared + n;
    dst = src + n;
    list = dst + n;
  }
};

constexpr int extend_smem(int n) { return ((n <= kExtendThreads ? 5 * n : n) + kListHere) * 4; }
static_assert(extend_smem(NS_MAX_PAGE_SEQS) <= 47 * 1024, "shared memory without opting in");

// One CTA: what each sequence needs (a scan over the call's order), then the
// lowest free pages (a scan over the counts, which ends once there are
// enough), then the table rows, one warp per sequence.  What it takes is its
// chain of dependent loads (ids, lengths, last pages, their counts), so what
// the threads tell each other stays in shared memory where it fits (up to
// kExtendThreads sequences, kListHere pages), and in the workspace otherwise.
__global__ void __launch_bounds__(kExtendThreads) extend_kernel(ns_kv_pages c, const int32_t *seqs,
                                                                const int32_t *n_new, int n, void *ws,
                                                                uint32_t *err) {
  __shared__ int sh[kExtendThreads / kWarp];
  extern __shared__ int s_ids[];  // [n], then (extend_smem) start, first, count, shared [n] and the list
  ExtendWs w(ws, n);
  const bool here = n <= kExtendThreads;
  if (here) w.start = s_ids + n, w.first = w.start + n, w.count = w.first + n, w.shared = w.count + n;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  wait_for_previous();
  // the first pages' counts, on their way while the needs are found
  constexpr int kPer = 8;
  int r[kPer];
#pragma unroll
  for (int q = 0; q < kPer; ++q) r[q] = tid * kPer + q < c.pages ? c.refs[tid * kPer + q] : 1;
  for (int i = tid; i < n; i += kExtendThreads) s_ids[i] = seqs[i];
  __syncthreads();

  long long total = 0;  // pages wanted; may pass 32 bits only where it is refused below
  int copies = 0, grown = 0, before = 0;  // (the new length, and the copies before this sequence's, when `here`)
  for (int i0 = 0; i0 < n; i0 += kExtendThreads) {
    const int i = i0 + tid;
    int count = 0, first = -1, shared = -1;
    if (i < n) {
      const int s = s_ids[i], add = n_new[i];
      bool ok = seq_ok(c, s);
      const int len = ok ? c.lengths[s] : 0;
      int again = 0;  // (while the length is on its way)
#pragma unroll 8
      for (int j = 0; j < i; ++j) again |= s_ids[j] == s;
      ok = ok && add >= 0 && !again;
      grown = (int)min((long long)len + add, 0x7fffffffLL);
      ok = ok && len_ok(c, len) && (long long)len + add <= (long long)c.table_ld * c.page_size;
      if (ok) {
        first = pages_for(len, c.page_size);
        const int want = pages_for((long long)len + add, c.page_size);
        if (add > 0 && len % c.page_size != 0) {  // the next position is in a page that is held already
          const int p = c.table[(size_t)s * c.table_ld + first - 1];
          if (p < 0 || p >= c.pages) {
            ok = false;
            first = -1;
            set_flag(err, NS_FLAG_BAD_ID);
          } else if (c.refs[p] > 1) {
            shared = p;
            --first;
          }
        }
        if (ok) count = want - first;
      } else {
        set_flag(err, NS_FLAG_BAD_SEQ);
      }
    }
    int sum, csum;
    const int off = block_exclusive_scan(count, sh, &sum);
    const int coff = block_exclusive_scan(shared >= 0 ? 1 : 0, sh, &csum);
    before = coff;
    if (i < n) {
      // start saturates: a call that wants more pages than exist is refused
      w.start[i] = total + off > 0x3fffffffLL ? 0x3fffffff : (int)(total + off);
      w.first[i] = first;
      w.count[i] = count;
      w.shared[i] = shared;
      if (shared >= 0) w.src[copies + coff] = shared;
    }
    total += sum;
    copies += csum;
  }

  // the `total` lowest free pages, in order
  bool enough = total <= c.pages;
  if (total <= kListHere) w.list = s_ids + (here ? 5 * n : n);
  int found = 0;
  if (enough && total > 0) {
    for (int p0 = 0; p0 < c.pages && found < total; p0 += kExtendThreads * kPer) {
      const int p = p0 + tid * kPer;
      uint32_t free_bits = 0;
      if (p0 > 0) {
#pragma unroll
        for (int q = 0; q < kPer; ++q) r[q] = p + q < c.pages ? c.refs[p + q] : 1;
      }
#pragma unroll
      for (int q = 0; q < kPer; ++q) free_bits |= (r[q] == 0 ? 1u : 0u) << q;
      int sum;
      int at = found + block_exclusive_scan(__popc(free_bits), sh, &sum);
      for (; free_bits && at < total; free_bits &= free_bits - 1, ++at) w.list[at] = p + __ffs(free_bits) - 1;
      found += sum;
    }
    enough = found >= total;
  }
  if (!enough) {
    if (tid == 0) {
      set_flag(err, NS_FLAG_NO_PAGES);
      *w.n_copies = 0;
    }
    return;
  }
  if (tid == 0) *w.n_copies = copies;
  __syncthreads();  // the list, and every sequence's entry

  int done = 0;  // copies of the chunks before
  for (int i0 = 0; i0 < n; i0 += kExtendThreads) {
    const int i = i0 + tid;
    int csum = 0;
    const int coff = here ? before : block_exclusive_scan(i < n && w.shared[i] >= 0 ? 1 : 0, sh, &csum);
    if (i < n && w.first[i] >= 0) {
      const int s = s_ids[i];
      c.lengths[s] = here ? grown : c.lengths[s] + n_new[i];
      if (w.shared[i] >= 0) {
        w.dst[done + coff] = w.list[w.start[i]];
        atomicSub(c.refs + w.shared[i], 1);
      }
    }
    done += csum;
  }
  for (int i = warp; i < n; i += kExtendThreads / kWarp) {
    if (w.first[i] < 0) continue;
    int32_t *row = c.table + (size_t)s_ids[i] * c.table_ld + w.first[i];
    for (int q = lane; q < w.count[i]; q += kWarp) {
      const int p = w.list[w.start[i] + q];
      row[q] = p;
      atomicAdd(c.refs + p, 1);  // 0 -> 1
    }
  }
}

// Copies whole pages.  A warp takes one (page pair, layer, head) of k or v:
// page_size rows of row_bytes, 16 bytes a lane.  The pairs' number is on the
// device when n_ptr is given (at most n).
__global__ void __launch_bounds__(kMoveThreads) copy_pages_kernel(ns_kv_pages c, const int32_t *src,
                                                                  const int32_t *dst, const int32_t *n_ptr, int n,
                                                                  uint32_t *err) {
  wait_for_previous();
  const int lane = threadIdx.x & 31;
  const int pairs = n_ptr ? min(*n_ptr, n) : n;
  const long long items = (long long)pairs * c.layers * c.heads * 2;
  const int cols = c.row_bytes / 16, units = c.page_size * cols;
  for (long long it = (long long)blockIdx.x * kMoveWarps + (threadIdx.x >> 5); it < items;
       it += (long long)gridDim.x * kMoveWarps) {
    const int kv = (int)(it & 1);
    const long long u = it >> 1;
    const int head = (int)(u % c.heads), layer = (int)(u / c.heads % c.layers), i = (int)(u / c.heads / c.layers);
    const int a = src[i], b = dst[i];
    if (a < 0 || a >= c.pages || b < 0 || b >= c.pages) {
      if (lane == 0) set_flag(err, NS_FLAG_BAD_ID);
      continue;
    }
    const int64_t sp = kv ? c.v_page : c.k_page, st = kv ? c.v_token : c.k_token;
    char *base = static_cast<char *>(kv ? c.v : c.k) + layer * (kv ? c.v_layer : c.k_layer) +
                 head * (kv ? c.v_head : c.k_head);
    const char *from = base + a * sp;
    char *to = base + b * sp;
    for (int x0 = lane; x0 < units; x0 += kWarp * kUnroll) {
      uint4 val[kUnroll];
#pragma unroll
      for (int q = 0; q < kUnroll; ++q) {
        const int x = x0 + q * kWarp;
        if (x < units) val[q] = __ldcs(reinterpret_cast<const uint4 *>(from + x / cols * st + x % cols * 16));
      }
#pragma unroll
      for (int q = 0; q < kUnroll; ++q) {
        const int x = x0 + q * kWarp;
        if (x < units) *reinterpret_cast<uint4 *>(to + x / cols * st + x % cols * 16) = val[q];
      }
    }
  }
}

// New rows of one layer: a warp per token, its 16-byte pieces of every head
// of k and v over the lanes.  Only the first of a repeated sequence is
// written: up to kWarpLooks sequences each warp looks through the entries
// before its own; of more, the CTA looks once for all of its warps.  Measured,
// by warps and by the CTA: 8 sequences of 4001 tokens 35.6, 36.9 us; 64 of one
// token 3.6, 3.8; 256 of one 4.1, 3.9; 8192 of one 23.7, 15.5.
constexpr int kWarpLooks = 128;
__global__ void __launch_bounds__(kMoveThreads) write_kernel(ns_kv_pages c, int layer, const int32_t *seqs,
                                                             const int32_t *cu, int n, const void *k_rows,
                                                             const void *v_rows, int64_t k_token, int64_t k_head,
                                                             int64_t v_token, int64_t v_head, int tokens,
                                                             uint32_t *err) {
  __shared__ int s_seq[kMoveWarps], s_at[kMoveWarps];  // each warp's sequence, and its place in the call
  __shared__ uint32_t s_again;                         // warps whose sequence stands before that place too
  wait_for_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * kMoveWarps + warp;
  int lo = 0, t0 = 0, t1 = 0, s = -1, len = 0;
  if (t < tokens) {  // the last i with cu[i] <= t, a 32nd of what is left at a time
    for (int size = n; size > 1;) {
      const int step = (size + 31) / 32, at = lo + lane * step;
      const uint32_t before = __ballot_sync(0xffffffffu, lane * step < size && cu[at] <= t);
      const int last = before ? 31 - __clz(before) : 0;
      lo += last * step;
      size = min(step, size - last * step);
    }
    t0 = cu[lo], t1 = cu[lo + 1], s = seqs[lo];
    if (seq_ok(c, s)) len = c.lengths[s];
  }
  uint32_t again = 0;  // (found while the length is on its way)
  if (n <= kWarpLooks) {
#pragma unroll
    for (int j = lane; j < kWarpLooks; j += kWarp)
      if (j < lo && seqs[j] == s) again = 1;
    again = __reduce_or_sync(0xffffffffu, again);
  } else {
    if (lane == 0) s_seq[warp] = s, s_at[warp] = t < tokens ? lo : -1;
    if (threadIdx.x == 0) s_again = 0;
    __syncthreads();
    int most = 0, all = NS_MAX_PAGE_SEQS, who[kMoveWarps];
#pragma unroll
    for (int w = 0; w < kMoveWarps; ++w) {
      who[w] = s_seq[w];
      most = max(most, s_at[w]), all = min(all, s_at[w] >= 0 ? s_at[w] : all);
    }
    int j = threadIdx.x;
#pragma unroll 4
    for (; j < all; j += kMoveThreads) {  // before every warp's place
      const int x = seqs[j];
#pragma unroll
      for (int w = 0; w < kMoveWarps; ++w)
        if (x == who[w]) again |= 1u << w;
    }
    for (; j < most; j += kMoveThreads) {
      const int x = seqs[j];
#pragma unroll
      for (int w = 0; w < kMoveWarps; ++w)
        if (x == who[w] && j < s_at[w]) again |= 1u << w;
    }
    again = __reduce_or_sync(0xffffffffu, again);
    if (lane == 0 && again) atomicOr(&s_again, again);
    __syncthreads();
    again = s_again >> warp & 1;
  }
  if (t < t0 || t >= t1) return;  // a token of no sequence
  const long long pos = (long long)len - (t1 - t);
  if (!seq_ok(c, s) || again || !len_ok(c, len) || pos < 0) {
    if (lane == 0) set_flag(err, NS_FLAG_BAD_SEQ);
    return;
  }
  const int page = c.table[(size_t)s * c.table_ld + (int)(pos / c.page_size)], r = (int)(pos % c.page_size);
  if (page < 0 || page >= c.pages) {
    if (lane == 0) set_flag(err, NS_FLAG_BAD_ID);
    return;
  }
  if (c.refs[page] > 1) {
    if (lane == 0) set_flag(err, NS_FLAG_SHARED_PAGE);
    return;
  }
  const int cols = c.row_bytes / 16, units = c.heads * cols;
  char *kd = static_cast<char *>(c.k) + layer * c.k_layer + page * c.k_page + r * c.k_token;
  char *vd = static_cast<char *>(c.v) + layer * c.v_layer + page * c.v_page + r * c.v_token;
  const char *ks = static_cast<const char *>(k_rows) + t * k_token;
  const char *vs = static_cast<const char *>(v_rows) + t * v_token;
  for (int x0 = lane; x0 < units; x0 += kWarp * 4) {
    uint4 a[4], b[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int x = x0 + q * kWarp;
      if (x < units) {
        a[q] = __ldcs(reinterpret_cast<const uint4 *>(ks + x / cols * k_head + x % cols * 16));
        b[q] = __ldcs(reinterpret_cast<const uint4 *>(vs + x / cols * v_head + x % cols * 16));
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int x = x0 + q * kWarp;
      if (x < units) {
        *reinterpret_cast<uint4 *>(kd + x / cols * c.k_head + x % cols * 16) = a[q];
        *reinterpret_cast<uint4 *>(vd + x / cols * c.v_head + x % cols * 16) = b[q];
      }
    }
  }
}

// Kept rows move down.  A CTA takes one sequence, k or v, and kMoverWarps of
// its (layer, head, part of the row), a warp each.  It walks the
// kept rows in order, kMoveRows at a time: the threads find each row's two
// places, for the next rows while these move, and every warp moves its part
// of them, kMoveBatch 16-byte pieces a lane: all loads of a batch, then its
// stores.  Row t comes from keep[t] >= t, so a batch's destinations lie before
// every later batch's sources, and within a batch the loads come first: the
// move is in place.
//
// Bound by HBM when there are many rows; the batch is what keeps enough bytes
// in flight when there are few (layer, head) parts.
constexpr int kMoverWarps = 4;
constexpr int kMoveRows = 128;
constexpr int kMoveBatch = 16;
__global__ void __launch_bounds__(kMoverWarps * 32, 4)
    compact_kernel(ns_kv_pages c, const int32_t *seqs, const int32_t *base, const int32_t *keep, int keep_ld,
                   const int32_t *n_keep, int seg_bytes, uint32_t *err) {
  __shared__ long long s_from[2][kMoveRows], s_to[2][kMoveRows];  // -1: stays
  wait_for_previous();
  const int tid = threadIdx.x, lane = tid & 31, i = blockIdx.z, kv = blockIdx.y;
  const int s = seqs[i], m = n_keep[i], b0 = base[i];
  const bool again = repeated(seqs, i);  // only the first of a repeated sequence
  const int len = seq_ok(c, s) ? c.lengths[s] : -1;
  if (again || !seq_ok(c, s) || m < 0 || m > keep_ld || b0 < 0 || !len_ok(c, len)) {
    if (tid == 0) set_flag(err, NS_FLAG_BAD_SEQ);
    return;
  }
  const int32_t *row = c.table + (size_t)s * c.table_ld;
  const int32_t *kp = keep + (size_t)i * keep_ld;
  const int64_t sp = kv ? c.v_page : c.k_page, st = kv ? c.v_token : c.k_token;
  auto find = [&](int t0) {  // the places of rows t0 .. t0 + kMoveRows - 1
    const int t = t0 + tid, slot = (t0 / kMoveRows) & 1;
    long long src = -1, dst = -1;
    if (t < m) {
      const int from = kp[t];
      if (from < t || (t > 0 && from <= kp[t - 1]) || (long long)b0 + from >= len) {
        set_flag(err, NS_FLAG_BAD_SEQ);
      } else if (from != t) {
        const int p = b0 + from, d = b0 + t;
        const int pa = row[p / c.page_size], pb = row[d / c.page_size];
        if (pa < 0 || pa >= c.pages || pb < 0 || pb >= c.pages) {
          set_flag(err, NS_FLAG_BAD_ID);
        } else if (c.refs[pb] > 1) {
          set_flag(err, NS_FLAG_SHARED_PAGE);
        } else {
          src = pa * sp + p % c.page_size * st;
          dst = pb * sp + d % c.page_size * st;
        }
      }
    }
    s_from[slot][tid] = src;
    s_to[slot][tid] = dst;
  };
  static_assert(kMoveRows == kMoverWarps * 32, "a thread finds one row's places");
  const int segs = (c.row_bytes + seg_bytes - 1) / seg_bytes;
  const int u = blockIdx.x * kMoverWarps + (tid >> 5);
  const bool mine = u < c.layers * c.heads * segs;
  const int seg = u % segs, head = u / segs % c.heads, layer = u / segs / c.heads;
  char *data = static_cast<char *>(kv ? c.v : c.k) + (mine ? layer : 0) * (kv ? c.v_layer : c.k_layer) +
               head * (kv ? c.v_head : c.k_head) + seg * seg_bytes;
  const int cols = min(c.row_bytes - seg * seg_bytes, seg_bytes) / 16;  // lanes a row takes
  const int per = kWarp / cols, sub = lane / cols;          // rows a warp moves at once
  data += lane % cols * 16;
  if (m > 0) find(0);
  for (int t0 = 0; t0 < m; t0 += kMoveRows) {
    __syncthreads();  // the places are there, and nobody reads the other ones any more
    if (t0 + kMoveRows < m) find(t0 + kMoveRows);
    if (!mine) continue;
    const int slot = (t0 / kMoveRows) & 1, rows = min(kMoveRows, m - t0);
    for (int q0 = 0; q0 < rows; q0 += per * kMoveBatch) {
      uint4 val[kMoveBatch];
#pragma unroll
      for (int q = 0; q < kMoveBatch; ++q) {
        const int t = q0 + q * per + sub;
        if (sub < per && t < rows && s_from[slot][t] >= 0)
          val[q] = __ldcs(reinterpret_cast<const uint4 *>(data + s_from[slot][t]));
      }
      __syncwarp();  // every load of the batch before its stores
#pragma unroll
      for (int q = 0; q < kMoveBatch; ++q) {
        const int t = q0 + q * per + sub;
        if (sub < per && t < rows && s_to[slot][t] >= 0) *reinterpret_cast<uint4 *>(data + s_to[slot][t]) = val[q];
      }
      __syncwarp();
    }
  }
}

unsigned grid_for(long long items, long long most) {
  const long long g = (items + kMoveWarps - 1) / kMoveWarps;
  return (unsigned)(g < 1 ? 1 : g > most ? most : g);
}

}  // namespace

cudaError_t launch_pages_truncate(const ns_kv_pages &c, const int32_t *seqs, const int32_t *new_len, int n,
                                  uint32_t *err, cudaStream_t st) {
  return launch(truncate_kernel, dim3(n), kSeqThreads, 0, st, c, seqs, new_len, nullptr, 0x7fffffff, err);
}

cudaError_t launch_pages_fork(const ns_kv_pages &c, const int32_t *src, const int32_t *dst, int n, uint32_t *err,
                              cudaStream_t st) {
  return launch(fork_kernel, dim3(n), kSeqThreads, 0, st, c, src, dst, n, err);
}

int64_t pages_extend_ws(const ns_kv_pages &c, int n) { return 4 * (4 + 6 * (int64_t)n + c.pages); }

cudaError_t launch_pages_extend(const ns_kv_pages &c, const int32_t *seqs, const int32_t *n_new, int n, void *ws,
                                uint32_t *err, cudaStream_t st) {
  cudaError_t e = launch(extend_kernel, dim3(1), kExtendThreads, extend_smem(n), st, c, seqs, n_new, n, ws, err);
  if (e != cudaSuccess) return e;
  const ExtendWs w(ws, n);
  const unsigned grid = grid_for((long long)n * c.layers * c.heads * 2, 2432);
  return launch(copy_pages_kernel, dim3(grid), kMoveThreads, 0, st, c, w.src, w.dst, w.n_copies, n, err);
}

cudaError_t launch_pages_write(const ns_kv_pages &c, int layer, const int32_t *seqs, const int32_t *cu, int n,
                               const void *k_new, const void *v_new, int64_t k_token, int64_t k_head,
                               int64_t v_token, int64_t v_head, int tokens, uint32_t *err, cudaStream_t st) {
  return launch(write_kernel, dim3((tokens + kMoveWarps - 1) / kMoveWarps), kMoveThreads, 0, st, c, layer, seqs, cu, n,
                k_new, v_new, k_token, k_head, v_token, v_head, tokens, err);
}

cudaError_t launch_pages_compact(const ns_kv_pages &c, const int32_t *seqs, const int32_t *base, const int32_t *keep,
                                 int keep_ld, const int32_t *n_keep, int n, uint32_t *err, cudaStream_t st) {
  // A warp takes up to 512 bytes of a row, less where the CTAs are too few to keep HBM busy: 16001 rows of 12 x 4
  // x 256 bytes of k and v move in 163 us by whole rows (192 CTAs), in about 118 us by halves.
  constexpr int kEnough = 304;
  int seg_bytes = 512;
  auto ctas = [&](int seg) {
    return ((long long)c.layers * c.heads * ((c.row_bytes + seg - 1) / seg) + kMoverWarps - 1) / kMoverWarps * 2 * n;
  };
  while (seg_bytes > 128 && ctas(seg_bytes) < kEnough) seg_bytes /= 2;
  const long long units = (long long)c.layers * c.heads * ((c.row_bytes + seg_bytes - 1) / seg_bytes);
  if (units > 0x7fffffffLL - kMoverWarps) return cudaErrorInvalidValue;
  if (keep_ld > 0) {
    const dim3 grid((unsigned)((units + kMoverWarps - 1) / kMoverWarps), 2, (unsigned)n);
    cudaError_t e = launch(compact_kernel, grid, kMoverWarps * 32, 0, st, c, seqs, base, keep, keep_ld, n_keep,
                           seg_bytes, err);
    if (e != cudaSuccess) return e;
  }
  return launch(truncate_kernel, dim3(n), kSeqThreads, 0, st, c, seqs, n_keep, base, keep_ld, err);
}

cudaError_t launch_pages_copy(const ns_kv_pages &c, const int32_t *src, const int32_t *dst, int n, uint32_t *err,
                              cudaStream_t st) {
  const dim3 grid(grid_for((long long)n * c.layers * c.heads * 2, 2432));
  return launch(copy_pages_kernel, grid, kMoveThreads, 0, st, c, src, dst, nullptr, n, err);
}

}  // namespace ns
