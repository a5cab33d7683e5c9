// Attention of new tokens for groups of sequences that begin with the same
// pages (samples of one prompt, after a fork), on the 5th-generation tensor
// cores (ns_umma_attn.cuh has the kernel).
//
// Mathematics: a row's keys are cut in two, what its group shares and the rest,
// and each part i gives (m_i, l_i, o_i) with l = sum 2^(x - m), o = sum 2^(x - m) v;
//   out = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i,   M = max m_i.
// The shared part is the same keys for every member, so the new tokens of all
// members are stacked into tiles of 128 rows, and the prefix is read, and
// multiplied, once for each 256 of them instead of once for each sequence.
//
// Three kernels:
//   plan    a cluster of eight CTAs to a group compares its members' pages: how
//           many whole tiles of 128 positions, all of them context, they share;
//   attend  prefixes (items of 256 stacked rows and the prefix's tiles) and then
//           tails (items of one sequence, as in ns_paged_umma.cu) in one line of
//           tiles, of which every CTA has an equal share; every piece of an item
//           that a CTA has leaves its rows' parts in the workspace;
//   merge   adds up each row's parts, prefix and tail, in the line's order.
// Item i of the line and CTA c meet in at most one piece, and i + c grows from
// piece to piece, so it is the piece's place.  No atomics whose order matters:
// the same inputs give the same bits.
//
// What bounds it: for few rows the chain of three kernels, each waiting for the
// one before (8 sequences of one prompt of 2101 tokens, 32 heads on 8: 23 us,
// and 18 where each reads it from L2, which the rule in ns_shared_attn.cu then
// prefers); for many sequences the items' starts and the parts' way through
// L2 (64 of four prompts of 3001 to 16000 tokens, 28 heads on 4, fp16: 55 us;
// without sharing 162); for trees the products of all rows, shared or not.
#pragma once

#include "ns_paged_mode.cuh"

namespace ns {
namespace {

using attn::kNegInf;
using fa::kKeys;
using paged::quotient;

struct SharedArgs {
  const int32_t *table, *lengths, *seqs, *groups;
  const int64_t *mask;
  int32_t n_seqs, n_groups, n, q_heads, group, pack, per_tile, units, tail_blocks, tail_rows;
  int32_t page_shift, table_ld, max_seqs, n_pages;
  float c;  // scale * log2(e)
  void *out;
  float *lse;
  uint32_t *err;
  // the plan: of each group its first sequence, members, shared tiles and the first's sequence in the cache; then of
  // each sequence the cache's, its length, the tiles that it shares and its group
  int4 *plan;
  // the line: tiles before each group's items and then each sequence's, and all; prefix items before each group's
  long long *cum;
  int32_t *items_before;
  // parts of prefix items (256 rows) and of tail items (tail_rows), (m, l) and o, column by column
  float2 *part_ml, *tail_ml;
  float *part_o, *tail_o;
  paged::Exponents rows;  // (of 8 bits)
  paged::Pairs pairs;     // (Mode's P)
};

// ---------------------------------------------------------------------------
// Plan
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 256, kPlanCtas = 8;
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads) plan_kernel(const SharedArgs a) {
  __shared__ int s_most[kPlanCtas];  // what each CTA of the cluster found (in CTA 0's)
  __shared__ int s_min;
  const int g = blockIdx.x / kPlanCtas, rank = blockIdx.x % kPlanCtas, tid = threadIdx.x;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  auto cluster_sync = []() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  };
  auto valid = [&](int s, int &len) {
    len = s >= 0 && s < a.max_seqs ? a.lengths[s] : -1;
    return len >= 0 && (long long)len <= ((long long)a.table_ld << a.page_shift);
  };
  // Groups that do not cover the sequences one after the other: nothing is shared, the first has them all.
  const int from = a.groups[g], to = a.groups[g + 1];
  int bad = a.groups[0] != 0 || a.groups[a.n_groups] != a.n_seqs;
  for (int i = tid; i < a.n_groups; i += kPlanThreads) bad |= a.groups[i] < 0 || a.groups[i + 1] < a.groups[i];
  if (tid == 0) s_min = 0x7fffffff;
  bad = __syncthreads_or(bad);
  const int first = bad ? 0 : from, members = bad ? (g == 0 ? a.n_seqs : 0) : to - from;
  // positions that every member has as context, and in whole pages
  int most = bad || members < 2 ? 0 : 0x7fffffff;
  for (int i = tid; i < members; i += kPlanThreads) {
    int len;
    if (valid(a.seqs[first + i], len))
      most = min(most, max(0, len - a.n) >> a.page_shift);
    else
      most = 0;
  }
  most = __reduce_min_sync(0xffffffffu, most);
  if ((tid & 31) == 0) atomicMin(&s_min, most);
  __syncthreads();
  most = s_min;  // pages
  __syncthreads();
  if (most > 0) {  // (and less than 2^31: there are two members at least)
    const int32_t *lead = a.table + (size_t)a.seqs[first] * a.table_ld;
    int same = most;
    for (int i = 1 + rank; i < members; i += kPlanCtas) {
      const int32_t *row = a.table + (size_t)a.seqs[first + i] * a.table_ld;
#pragma unroll 4
      for (int p = tid; p < same; p += kPlanThreads)
        if (row[p] != lead[p]) same = min(same, p);
    }
    same = __reduce_min_sync(0xffffffffu, same);
    if ((tid & 31) == 0) atomicMin(&s_min, same);
  }
  cluster_sync();  // all have begun, and found their part
  uint32_t there;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(there) : "r"(smem_u32(s_most)));
  if (tid == 0) asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(there + 4 * rank), "r"(s_min) : "memory");
  cluster_sync();
  most = 0x7fffffff;
#pragma unroll
  for (int i = 0; i < kPlanCtas; ++i) {
    int x;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(there + 4 * i) : "memory");
    most = min(most, x);
  }
  if (members == 0) most = 0;
  const int shared = (int)(((long long)most << a.page_shift) / kKeys);
  if (rank == 0 && tid == 0) {
    a.plan[g] = make_int4(first, members, shared, members > 0 ? a.seqs[first] : 0);
    if (bad && g == 0) set_flag(a.err, NS_FLAG_BAD_SEQ);
  }
  for (int i = rank * kPlanThreads + tid; i < members; i += kPlanCtas * kPlanThreads) {
    const int s = a.seqs[first + i];
    int len;
    if (!valid(s, len)) {
      set_flag(a.err, NS_FLAG_BAD_SEQ);
      len = 0;
    }
    a.plan[a.n_groups + first + i] = make_int4(s, len, shared, g);
  }
  cluster_sync();  // nobody leaves before its memory has been read
}

// ---------------------------------------------------------------------------
// Attend
// ---------------------------------------------------------------------------
template <bool S>
struct Work {
  int n0, n1, hidden;
  int seq, len;       // the cache's sequence (a prefix: its group's first), the end of the keys
  int tok0, tok_end;  // the call's tokens (sequence * n + new token): first row tile's first, and where they end
  int unit;           // query heads unit * pack ..
  int j0, slot;       // first key tile; the part's place
  int ctx;            // positions that every row sees (a prefix: all)
  __device__ __forceinline__ int tiles() const { return S ? n0 + n1 : n0; }
};
constexpr int kAllSeen = 0x7fffffff;
// What an item's beginning and end take, in tiles: the line has that many more for each item, so that shares are equal
// in time.  Without: 64 sequences of 4 prompts (28 heads on 4, one new token each) 68.0 us, the CTAs with the tails
// 25 us longer at work than the others.  With 2, 3 and 4: 54.5, 54.3, 56.0 us, and 8 sequences of one prompt of 2101
// 23.8, 22.9, 24.4 (items of one row tile); 16 trees of 60 nodes behind 6007 tokens 115, 119, 120 (of two).
template <bool S>
constexpr int kItemCost = S ? 3 : 2;

// A CTA's share of the line, item by item (a whole warp): entries 0 .. n_groups - 1 are prefixes, the others tails.
// Lane l holds entry 32 chunk + l.  S: items of one row tile (attn_kernel's kSplit), otherwise of two.
template <bool S>
struct Dealer {
  static constexpr int kRowTiles = S ? 1 : 2;
  long long at, end;        // next tile, the share's end
  long long base;           // tiles before the chunk's entries
  int item_base;            // prefix items before them
  int cta, lane, l, chunk;  // l: the lane whose entry is dealt
  int nt, items;            // this lane's entry: an item's place in the line (its tiles and cost), items
  int x, y;                 // first sequence and members, or cache sequence and its length
  int from;                 // a tail's first tile, or the cache sequence of a prefix's first
  long long excl, sum;      // tiles before this lane's entry in the chunk, and of the chunk
  int item_excl, item_sum;  // prefix items

  __device__ __forceinline__ int blocks(const SharedArgs &a, int members) const {
    return (members * a.n + kRowTiles * a.per_tile - 1) / (kRowTiles * a.per_tile);
  }
  __device__ __forceinline__ void load(const SharedArgs &a, int k) {
    chunk = k;
    const int e = k * 32 + lane;
    nt = items = x = y = from = 0;
    if (e < a.n_groups + a.n_seqs) {
      const int4 r = a.plan[e];
      x = r.x, y = r.y;
      if (e < a.n_groups) {
        nt = r.z, from = r.w;
        items = nt > 0 ? a.units * blocks(a, y) : 0;
      } else {
        from = r.z;
        nt = max(1, (y + kKeys - 1) / kKeys - from);  // an empty sequence: one tile, all masked
        items = a.units * a.tail_blocks;
      }
    }
    if (nt > 0) nt += kItemCost<S>;
    const int prefix = e < a.n_groups ? items : 0;
    excl = (long long)nt * items, item_excl = prefix;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, excl, off);
      const int i = __shfl_up_sync(0xffffffffu, item_excl, off);
      if (lane >= off) excl += o, item_excl += i;
    }
    sum = __shfl_sync(0xffffffffu, excl, 31), item_sum = __shfl_sync(0xffffffffu, item_excl, 31);
    excl -= (long long)nt * items, item_excl -= prefix;
  }
  __device__ __forceinline__ void begin(const SharedArgs &a, int cta_, int ctas) {
    lane = threadIdx.x & 31, cta = cta_;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan (what the other warps do hangs on this one)
    const int entries = a.n_groups + a.n_seqs, chunks = (entries + 31) / 32;
    long long total = 0;
    int before = 0;
    for (int k = 0; k < chunks; ++k) {
      load(a, k);
      const int e = k * 32 + lane;
      if (cta == 0 && e < entries) a.cum[e] = total + excl;
      if (cta == 0 && e < a.n_groups) a.items_before[e] = before + item_excl;
      total += sum, before += item_sum;
    }
    if (cta == 0 && lane == 0) a.cum[entries] = total;
    at = quotient(total * cta, ctas), end = quotient(total * (cta + 1), ctas);
    base = 0, item_base = 0, l = 0;
    if (at >= end) return;
    for (int k = 0;; ++k) {
      if (chunks > 1) load(a, k);
      if (at < base + sum) break;
      base += sum, item_base += item_sum;
    }
  }
  __device__ __forceinline__ Work<S> next(const SharedArgs &a) {
    Work<S> w{};
    for (;;) {
      if (at >= end) return w;
      while (at >= base + sum) {
        base += sum, item_base += item_sum;
        load(a, chunk + 1);
      }
      if (piece(a, w)) return w;
    }
  }
  // The CTA's next piece of an item; false where it has nothing of the item but its cost.
  __device__ __forceinline__ bool piece(const SharedArgs &a, Work<S> &w) {
    // the entry that the next tile is in
    l = __ffs(__ballot_sync(0xffffffffu, base + excl + (long long)nt * items > at)) - 1;
    const int e = chunk * 32 + l, n = __shfl_sync(0xffffffffu, nt, l), all = __shfl_sync(0xffffffffu, items, l);
    const int p = __shfl_sync(0xffffffffu, x, l), q = __shfl_sync(0xffffffffu, y, l);
    const int first = __shfl_sync(0xffffffffu, from, l), prior = item_base + __shfl_sync(0xffffffffu, item_excl, l);
    const long long local = at - base - __shfl_sync(0xffffffffu, excl, l);
    const int item = (int)quotient(local, n), place = (int)(local - (long long)item * n);
    const int left = (int)min((long long)(n - place), end - at);  // of the line, in this item
    const int tile = max(0, place - kItemCost<S>), count = left - max(0, kItemCost<S> - place);
    at += left;
    if (count <= 0) return false;
    w.n0 = count;
    if (e < a.n_groups) {
      const int b = all / a.units;
      w.unit = item / b, w.tok0 = p * a.n + item % b * kRowTiles * a.per_tile, w.tok_end = (p + q) * a.n;
      w.seq = first, w.len = (n - kItemCost<S>) * kKeys, w.j0 = tile, w.ctx = kAllSeen, w.hidden = count;
      w.slot = prior + item + cta;
    } else {
      const int b = e - a.n_groups;
      w.unit = item / a.tail_blocks, w.tok0 = b * a.n + item % a.tail_blocks * kRowTiles * a.per_tile;
      w.tok_end = (b + 1) * a.n;
      w.seq = p, w.len = q, w.j0 = first + tile, w.ctx = q - a.n;
      w.hidden = max(0, (w.ctx > 0 ? w.ctx / kKeys : 0) - w.j0);
      w.slot = b * all + item + cta;
    }
    if (S)
      w.n1 = count / 2, w.n0 -= w.n1;
    else
      w.n1 = w.tok0 + a.per_tile < w.tok_end ? count : 0;
    return true;
  }
};

// F8: of a cache of 8 bits, whose keys and values are converted.
template <bool S, bool F8, bool P>
struct Mode {
  using Args = SharedArgs;
  using Work = ns::Work<S>;
  using Dealer = ns::Dealer<S>;
  static constexpr bool kParts = true, kSplit = S, kLiveParts = true, kWhole = false;
  static constexpr bool kCodes = F8, kHigh = F8, kPaired = P;
  static constexpr int kStageRow = 64, kRows = S ? 128 : 256;  // (of a part)

  struct Loader : paged::PageLoader<SharedArgs, Work, F8, P> {
    __device__ __forceinline__ void queries(const SharedArgs &a, const Work &w, int t, int h, uint32_t dst,
                                            const CUtensorMap *m, uint32_t bar) {
      umma::tma3(dst, m, h * 64, w.unit * a.pack, w.tok0 + t * a.per_tile, bar);
    }
  };
  template <typename T, int D>
  using Converter = paged::PageConverter<T, D, SharedArgs, Work>;
  using Wild = paged::NodeWild<Work>;

  struct Row {
    bool live;
    int64_t at;  // (its place in the output: merge's)
    int ctx;
    uint64_t word;  // new tokens that it sees
    __device__ __forceinline__ void begin(const SharedArgs &a, const Work &w, int t, int r) {
      const int in_tile = r / a.pack, tok = w.tok0 + t * a.per_tile + in_tile, node = tok - (w.tok_end - a.n);
      live = in_tile < a.per_tile && tok < w.tok_end;
      at = 0;
      ctx = w.ctx;
      word = !live || ctx == kAllSeen
                 ? 0ull
                 : (a.mask ? (uint64_t)a.mask[tok] : ~0ull >> (63 - node)) & ~0ull >> (64 - a.n);
    }
    __device__ __forceinline__ uint64_t sees(const Work &w, int j, int from) const {
      const long long d = (long long)ctx - ((w.j0 + j) * kKeys + from);  // keys of the 64 in the context
      if (d >= 64) return ~0ull;
      if (d > 0) return word << d | ((1ull << d) - 1);
      return d > -64 ? word >> -d : 0ull;
    }
  };

  template <typename T, int D>
  static __device__ __forceinline__ bool clear(const SharedArgs &, const Work &w, int j, uint8_t *tile, int lane) {
    return paged::clear_behind<D, Mode>(w, j, tile, lane);
  }

  template <int D>
  static __device__ __forceinline__ void part(const SharedArgs &a, const Work &w, int t, int r, float *&o, int &pitch,
                                              float2 *&ml) {
    const bool tail = w.ctx != kAllSeen;
    pitch = tail ? a.tail_rows : kRows;
    const int row = tail ? t * a.per_tile * a.pack + r : t * 128 + r;
    o = (tail ? a.tail_o : a.part_o) + (int64_t)w.slot * D * pitch + row;
    ml = (tail ? a.tail_ml : a.part_ml) + (int64_t)w.slot * pitch + row;
  }
};

// ---------------------------------------------------------------------------
// Merge
// ---------------------------------------------------------------------------
// A CTA has 32 rows, a lane each.  G = 8: its warps take the parts of 32
// columns in turns and add up in warp order; G = 1: each has all parts of D / 8
// columns.
constexpr int kMergeWarps = 8;
template <typename T, int D, bool S, int G>
__global__ void __launch_bounds__(kMergeWarps * 32) merge_kernel(const SharedArgs a, int ctas) {
  constexpr int N = G == 1 ? D / 8 : 32, kRowTiles = S ? 1 : 2;  // columns of a warp
  __shared__ float s_o[G][G > 1 ? N : 1][33], s_m[G][32], s_l[G][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, unit = blockIdx.y;
  const int col0 = G == 1 ? warp * N : blockIdx.z * N;
  const int row = blockIdx.x * 32 + lane, tok = row / a.pack, h = row % a.pack;
  const bool live = tok < a.n_seqs * a.n;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = live ? tok / a.n : 0, node = live ? tok % a.n : 0;
  const long long total = a.cum[a.n_groups + a.n_seqs];
  auto first_of = [&](int c) { return quotient(total * c, ctas); };
  // the row's pieces: CTAs c0 .. of an item, where (slot + c) * pitch is CTA c's part
  int pieces[2] = {0, 0}, c0[2] = {0, 0}, pitch[2] = {kRowTiles * 128, a.tail_rows};
  int64_t slot[2] = {0, 0};
  int in_part[2] = {0, 0};
  if (live) {
    const int4 mine = a.plan[a.n_groups + b];
    const int X = kRowTiles * a.per_tile, g = mine.w, nt = mine.z;
    if (nt > 0) {
      const int4 bounds = a.plan[g];
      const int v = tok - bounds.x * a.n, blocks = (bounds.y * a.n + X - 1) / X, item = unit * blocks + v / X;
      const long long from = a.cum[g] + (long long)item * (nt + kItemCost<S>) + kItemCost<S>;
      c0[0] = (int)quotient((from + 1) * ctas - 1, total);
      pieces[0] = (int)quotient((from + nt) * ctas - 1, total) - c0[0] + 1;
      slot[0] = a.items_before[g] + item;
      in_part[0] = v % X / a.per_tile * 128 + v % a.per_tile * a.pack + h;
    }
    const long long cb = a.cum[a.n_groups + b];
    const int items = a.units * a.tail_blocks, item = unit * a.tail_blocks + node / X;
    const long long n = quotient(a.cum[a.n_groups + b + 1] - cb, items), from = cb + item * n + kItemCost<S>;
    c0[1] = (int)quotient((from + 1) * ctas - 1, total);
    pieces[1] = (int)quotient((from + n - kItemCost<S>) * ctas - 1, total) - c0[1] + 1;
    slot[1] = b * items + item;
    in_part[1] = node % X * a.pack + h;
  }
  float m = kNegInf, l = 0.f, o[N];
#pragma unroll
  for (int i = 0; i < N; ++i) o[i] = 0.f;
  const int all = pieces[0] + pieces[1];
  for (int p = G == 1 ? 0 : warp; __any_sync(0xffffffffu, p < all); p += G) {
    if (p >= all) continue;
    const int k = p >= pieces[0], c = c0[k] + p - (k ? pieces[0] : 0);
    if (total < ctas && first_of(c) == first_of(c + 1)) continue;  // a CTA without tiles
    const int64_t at = (slot[k] + c) * pitch[k];
    const float2 ml = (k ? a.tail_ml : a.part_ml)[at + in_part[k]];
    const float *src = (k ? a.tail_o : a.part_o) + at * D + (int64_t)col0 * pitch[k] + in_part[k];
    float x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = src[(int64_t)i * pitch[k]];
    const float now = fmaxf(m, ml.x), safe = now == kNegInf ? 0.f : now;
    const float f0 = attn::ex2(m - safe), f1 = attn::ex2(ml.x - safe);
    m = now, l = l * f0 + ml.y * f1;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = fmaf(x[i], f1, o[i] * f0);
  }
  const int64_t at = (int64_t)tok * a.q_heads + unit * a.pack + h;
  T *out = static_cast<T *>(a.out) + at * D + col0;
  if constexpr (G == 1) {
    if (!live) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int i = 0; i < N; i += 8)
      *reinterpret_cast<uint4 *>(out + i) = make_uint4(
          attn::Type<T>::pack(o[i] * inv, o[i + 1] * inv), attn::Type<T>::pack(o[i + 2] * inv, o[i + 3] * inv),
          attn::Type<T>::pack(o[i + 4] * inv, o[i + 5] * inv), attn::Type<T>::pack(o[i + 6] * inv, o[i + 7] * inv));
    if (a.lse && warp == 0) a.lse[at] = l == 0.f ? kNegInf : (m - fa::kOffset<T> + log2f(l)) * attn::kLn2;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) s_o[warp][i][lane] = o[i];
    s_m[warp][lane] = m, s_l[warp][lane] = l;
    __syncthreads();
    // a thread has four columns of a row
    m = kNegInf, l = 0.f;
#pragma unroll
    for (int w = 0; w < G; ++w) m = fmaxf(m, s_m[w][lane]);
    const float safe = m == kNegInf ? 0.f : m;
    float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < G; ++w) {
      const float f = attn::ex2(s_m[w][lane] - safe);
      l = fmaf(s_l[w][lane], f, l);
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = fmaf(s_o[w][warp * 4 + i][lane], f, y[i]);
    }
    if (!live) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    *reinterpret_cast<uint2 *>(out + warp * 4) =
        make_uint2(attn::Type<T>::pack(y[0] * inv, y[1] * inv), attn::Type<T>::pack(y[2] * inv, y[3] * inv));
    if (a.lse && col0 == 0 && warp == 0)
      a.lse[at] = l == 0.f ? kNegInf : (m - fa::kOffset<T> + log2f(l)) * attn::kLn2;
  }
}

// ---------------------------------------------------------------------------
// Shapes, workspace and launches
// ---------------------------------------------------------------------------
struct Shape {
  bool split;  // items of one row tile
  int pack, per_tile, units, tail_blocks, tail_rows;
  int64_t parts, tails;  // places of prefix and tail parts
};
Shape shape_of(int n_seqs, int n_groups, int n, int q_heads, int kv_heads, int sms) {
  Shape s;
  const int group = q_heads / kv_heads;
  s.pack = group <= 128 ? group : 1;
  s.per_tile = 128 / s.pack, s.units = q_heads / s.pack;
  // One row tile where the groups have no more tokens than that on average: its keys keep both softmax groups busy.
  s.split = n_groups > 0 && (int64_t)n_seqs * n <= (int64_t)n_groups * s.per_tile;
  const int X = (s.split ? 1 : 2) * s.per_tile;
  s.tail_blocks = (n + X - 1) / X;
  s.tail_rows = ((n < X ? n : X) * s.pack + 7) & ~7;
  // Groups have sum ceil(tokens / X) blocks, with two members and so two tokens each at least.
  const int64_t tokens = (int64_t)n_seqs * n;
  const int64_t most = n_groups < n_seqs / 2 ? n_groups : n_seqs / 2;
  s.parts = n_seqs < 2 ? 0 : (int64_t)s.units * (tokens / X + most) + sms;
  s.tails = (int64_t)s.units * n_seqs * s.tail_blocks + sms;
  return s;
}

struct Layout {
  int64_t plan, cum, items, part_ml, tail_ml, part_o, tail_o, bytes;
  Layout(const Shape &s, int n_seqs, int n_groups, int dim) {
    int64_t at = 0;
    auto take = [&](int64_t n) {
      const int64_t was = at;
      at = (at + n + 255) & ~(int64_t)255;
      return was;
    };
    plan = take(16LL * (n_groups + n_seqs));
    cum = take(8LL * (n_groups + n_seqs + 1)), items = take(4LL * n_groups);
    part_ml = take(s.parts * (s.split ? 128 : 256) * 8), tail_ml = take(s.tails * s.tail_rows * 8);
    part_o = take(s.parts * (s.split ? 128 : 256) * dim * 4), tail_o = take(s.tails * s.tail_rows * dim * 4);
    bytes = at;
  }
};

template <typename T, int D, bool S, bool F8, bool P>
cudaError_t launch(const PagedAttnArgs &p, const Shape &s, const paged::Pairs &pairs, const int32_t *groups,
                   int n_groups, int sms, cudaStream_t st) {
  const Layout at(s, p.n_seqs, n_groups, D);
  char *ws = static_cast<char *>(p.ws);
  SharedArgs a{};
  a.table = p.table, a.lengths = p.lengths, a.seqs = p.seqs, a.groups = groups, a.mask = p.mask;
  a.n_seqs = p.n_seqs, a.n_groups = n_groups, a.n = p.n, a.q_heads = p.q_heads, a.group = p.group;
  a.pack = s.pack, a.per_tile = s.per_tile, a.units = s.units, a.tail_blocks = s.tail_blocks, a.tail_rows = s.tail_rows;
  a.page_shift = p.page_shift, a.table_ld = p.table_ld, a.max_seqs = p.max_seqs, a.n_pages = p.n_pages;
  a.c = p.scale * attn::kLog2e, a.out = p.out, a.lse = p.lse, a.err = p.err;
  a.plan = reinterpret_cast<int4 *>(ws + at.plan), a.cum = reinterpret_cast<long long *>(ws + at.cum);
  a.items_before = reinterpret_cast<int32_t *>(ws + at.items);
  a.part_ml = reinterpret_cast<float2 *>(ws + at.part_ml), a.tail_ml = reinterpret_cast<float2 *>(ws + at.tail_ml);
  a.part_o = reinterpret_cast<float *>(ws + at.part_o), a.tail_o = reinterpret_cast<float *>(ws + at.tail_o);
  a.rows = paged::exponents_of(p);
  a.pairs = pairs;
  CUtensorMap tmQ, tmK, tmV;
  const uint64_t dq[3] = {D, (uint64_t)p.q_heads, (uint64_t)p.n_seqs * p.n};
  const uint64_t sq[2] = {(uint64_t)p.q_head * 2, (uint64_t)(p.n > 1 ? p.q_token : p.q_seq) * 2};
  const uint32_t bq[3] = {64, (uint32_t)a.pack, (uint32_t)a.per_tile};
  if (!encode_16bit(&tmQ, p.q, 3, dq, sq, bq) || !paged::page_maps<D, F8, P>(p, pairs, &tmK, &tmV))
    return cudaErrorInvalidValue;
  using M = Mode<S, F8, P>;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = st;
  cfg.gridDim = dim3((unsigned)n_groups * kPlanCtas);
  cfg.blockDim = dim3(kPlanThreads);
  cudaError_t e = cudaLaunchKernelEx(&cfg, plan_kernel, a);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)sms);
  cfg.blockDim = dim3(fa::kThreadsOf<M>);
  cfg.dynamicSmemBytes = fa::Smem<D, M>::kBytes;
  e = cudaLaunchKernelEx(&cfg, fa::attn_kernel<T, D, M>, tmQ, tmK, tmV, a);
  if (e != cudaSuccess) return e;
  // an item's parts: some more than its share of the CTAs, if the prefixes are of like lengths
  const int64_t tokens = (int64_t)p.n_seqs * p.n;
  const bool many = (int64_t)sms * (S ? 1 : 2) * a.per_tile >= 4 * a.units * tokens;
  cfg.gridDim = dim3((unsigned)((tokens * a.pack + 31) / 32), (unsigned)a.units, many ? D / 32 : 1);
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.dynamicSmemBytes = 0;
  return many ? cudaLaunchKernelEx(&cfg, merge_kernel<T, D, S, 8>, a, sms)
              : cudaLaunchKernelEx(&cfg, merge_kernel<T, D, S, 1>, a, sms);
}

template <typename T, int D, bool F8, bool P>
cudaError_t by_shape(const PagedAttnArgs &p, const paged::Pairs &pairs, const int32_t *groups, int n_groups, int sms,
                     cudaStream_t st) {
  const Shape s = shape_of(p.n_seqs, n_groups, p.n, p.q_heads, p.kv_heads, sms);
  return s.split ? launch<T, D, true, F8, P>(p, s, pairs, groups, n_groups, sms, st)
                 : launch<T, D, false, F8, P>(p, s, pairs, groups, n_groups, sms, st);
}
// (as by_pages of ns_paged_tree.cuh)
template <typename T, int D, bool F8>
cudaError_t by_pages(const PagedAttnArgs &p, const int32_t *groups, int n_groups, int sms, cudaStream_t st) {
  paged::Pairs pairs{};
  if constexpr (D == 128 && !F8) {
    if (p.page_shift <= paged::kPairShift && paged::page_pairs(p, &pairs))
      return by_shape<T, D, F8, true>(p, pairs, groups, n_groups, sms, st);
  }
  return by_shape<T, D, F8, false>(p, pairs, groups, n_groups, sms, st);
}

template <typename T, int D, bool F8, bool P>
cudaError_t prepare() {
  auto set = [](auto *kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  };
  using Whole = Mode<false, F8, P>;
  using Split = Mode<true, F8, P>;
  const cudaError_t e = set(fa::attn_kernel<T, D, Whole>, fa::Smem<D, Whole>::kBytes);
  return e == cudaSuccess ? set(fa::attn_kernel<T, D, Split>, fa::Smem<D, Split>::kBytes) : e;
}
template <bool F8>
cudaError_t prepare_all() {
  cudaError_t e = prepare<__nv_bfloat16, 128, F8, false>();
  if (e == cudaSuccess) e = prepare<__nv_bfloat16, 64, F8, false>();
  if (e == cudaSuccess) e = prepare<__half, 128, F8, false>();
  if (e == cudaSuccess) e = prepare<__half, 64, F8, false>();
  if constexpr (!F8) {
    if (e == cudaSuccess) e = prepare<__nv_bfloat16, 128, F8, true>();
    if (e == cudaSuccess) e = prepare<__half, 128, F8, true>();
  }
  return e;
}
template <bool F8>
cudaError_t launch_any(const PagedAttnArgs &a, const int32_t *groups, int n_groups, int dtype, int dim, int sms,
                       cudaStream_t st) {
  if (dtype == NS_DTYPE_BF16)
    return dim == 128 ? by_pages<__nv_bfloat16, 128, F8>(a, groups, n_groups, sms, st)
                      : by_pages<__nv_bfloat16, 64, F8>(a, groups, n_groups, sms, st);
  return dim == 128 ? by_pages<__half, 128, F8>(a, groups, n_groups, sms, st)
                    : by_pages<__half, 64, F8>(a, groups, n_groups, sms, st);
}

}  // namespace
}  // namespace ns
