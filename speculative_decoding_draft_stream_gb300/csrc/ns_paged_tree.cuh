// Attention of many rows (a draft tree's nodes, or a long chain of new tokens)
// over a paged cache, on the 5th-generation tensor cores (ns_umma_attn.cuh has
// the kernel).
//
// An item is 2 * (128 / group) new tokens of one sequence, all query heads of
// one key-value head, and the sequence's keys; the CTAs have equal shares of
// all items' tiles (ns_paged_attn.cuh).  Keys and values come page by page:
// each page's part of a tile is one TMA box (of 64 columns, or of a small page's
// 128), its id fetched a tile ahead.  A page id out of range is a box outside the tensor,
// which reads as zeros; no row sees its places.  Every row sees the context whole; in the tiles from
// there on a row sees the new tokens of its mask, and what lies behind the
// sequence's end is put to zero before it is used.
//
// Bound by the products, the start of a CTA's items and the parts' way through
// L2: trees of 60 nodes behind 512 to 4096 tokens, 16 sequences, 32 heads on
// 8, bf16, pages of 16, take 56 us (0.57 PFLOP/s, 2.7 TB/s); with mma.sync
// and 64 rows to a CTA they take nearly three times as long.
//
// Over a cache of 8 bits four more warps make 16 bits of the codes that TMA has
// brought, in place of the products' wait for them: the same trees take 70.5 us
// (201 with mma.sync and 64 rows to a CTA), bound by that conversion, a tile's
// keys and values one after the other.  Without kHigh's limit 77 us.
#pragma once

#include "ns_paged_mode.cuh"

namespace ns {
namespace {

using attn::kNegInf;
using fa::kKeys;

struct TreeArgs {
  const int32_t *table, *lengths, *seqs;
  const int64_t *mask;
  int32_t n_seqs, n, q_heads, group, pack, per_tile, units, blocks;
  int32_t page_shift, table_ld, max_seqs, n_pages;
  float c;  // scale * log2(e)
  void *out;
  float *lse;
  float2 *part_ml;
  float *part_o;
  long long *cum;  // [n_seqs + 1] tiles before each sequence, for the join
  uint32_t *err;
  paged::Exponents rows;  // (of 8 bits)
  paged::Pairs pairs;     // (Mode's P)
  const int32_t *groups;  // (as PagedAttnArgs has them)
  int32_t n_groups;
};

struct Work {
  int n0, n1, hidden;
  int b, seq, len;   // the call's sequence, the cache's, its length
  int unit, node0;   // query heads unit * pack .., first new token of row tile 0
  int j0, slot;      // first key tile; the part's place (-1: the item is whole)
  int ctx;           // positions that every row sees: len - n
  __device__ __forceinline__ int tiles() const { return n0; }
};

using paged::quotient;

// A CTA's share of the line of tiles, item by item (a whole warp).  Lane l
// holds sequence 32 chunk + l of the call, so the line is walked without
// loads while it stays among 32 sequences.
struct Dealer {
  long long at, first, end, before;  // next tile, the share's bounds, tiles before sequence b
  int items, cta, lane, b, nt;
  int chunk, c_seq, c_len, c_nt;     // this lane's sequence: the cache's, its length and tiles

  __device__ __forceinline__ void load(const TreeArgs &a, int k, bool flag) {
    chunk = k;
    const int i = k * 32 + lane;
    c_nt = 0, c_len = 0, c_seq = 0;
    if (i < a.n_seqs) {
      c_seq = a.seqs[i];
      c_len = c_seq >= 0 && c_seq < a.max_seqs ? a.lengths[c_seq] : -1;
      if (c_len < 0 || (long long)c_len > ((long long)a.table_ld << a.page_shift)) {
        if (flag) set_flag(a.err, NS_FLAG_BAD_SEQ);
        c_len = 0;
      }
      c_nt = c_len > 0 ? (c_len - 1) / kKeys + 1 : 1;  // an empty sequence: one tile, all masked
    }
  }
  // tiles of the chunk's sequences up to and with this lane's
  __device__ __forceinline__ long long upto() const {
    long long sum = (long long)c_nt * items;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, sum, off);
      if (lane >= off) sum += o;
    }
    return sum;
  }
  __device__ __forceinline__ void begin(const TreeArgs &a, int cta_, int ctas) {
    lane = threadIdx.x & 31, cta = cta_, items = a.units * a.blocks;
    const int chunks = (a.n_seqs + 31) / 32;
    long long total = 0, sum = 0;
    for (int k = 0; k < chunks; ++k) {
      load(a, k, cta == 0);
      sum = upto();
      if (cta == 0 && k * 32 + lane < a.n_seqs) a.cum[k * 32 + lane] = total + sum - (long long)c_nt * items;
      total += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (cta == 0 && lane == 0) a.cum[a.n_seqs] = total;
    first = at = quotient(total * cta, ctas), end = quotient(total * (cta + 1), ctas);
    b = 0, before = 0, nt = 0;
    if (at >= end) return;
    long long passed = 0;  // the sequence with the share's first tile
    for (int k = 0; k < chunks; ++k) {
      if (chunks > 1) {
        load(a, k, false);
        sum = upto();
      }
      const uint32_t past = __ballot_sync(0xffffffffu, passed + sum > at);
      if (past) {
        const int l = __ffs(past) - 1;
        b = k * 32 + l;
        nt = __shfl_sync(0xffffffffu, c_nt, l);
        before = passed + __shfl_sync(0xffffffffu, sum, l) - (long long)nt * items;
        return;
      }
      passed += __shfl_sync(0xffffffffu, sum, 31);
    }
  }
  __device__ __forceinline__ Work next(const TreeArgs &a) {
    Work w{};
    if (at >= end) return w;
    while (at >= before + (long long)nt * items) {
      before += (long long)nt * items;
      if (++b / 32 != chunk) load(a, b / 32, false);
      nt = __shfl_sync(0xffffffffu, c_nt, b % 32);
    }
    const int len = __shfl_sync(0xffffffffu, c_len, b % 32);
    const int item = (int)quotient(at - before, nt), tile = (int)(at - before - (long long)item * nt);
    const int count = (int)min((long long)(nt - tile), end - at);
    const int ctx = len - a.n;
    w.b = b, w.seq = __shfl_sync(0xffffffffu, c_seq, b % 32), w.len = len;
    w.unit = item / a.blocks, w.node0 = item % a.blocks * 2 * a.per_tile;
    w.j0 = tile, w.ctx = ctx;
    w.n0 = count, w.n1 = w.node0 + a.per_tile < a.n ? count : 0;
    w.hidden = max(0, (ctx > 0 ? ctx / kKeys : 0) - tile);
    w.slot = tile == 0 && count == nt ? -1 : cta * 2 + (at == first ? 0 : 1);
    at += count;
    return w;
  }
};

using TreeWork = Work;
using TreeDealer = Dealer;

// F8: of a cache of 8 bits, whose keys and values are converted.
template <bool F8, bool P>
struct Mode {
  using Args = TreeArgs;
  using Work = TreeWork;
  using Dealer = TreeDealer;
  static constexpr bool kParts = true, kSplit = false, kLiveParts = false, kWhole = true;
  static constexpr bool kCodes = F8, kHigh = F8, kPaired = P;
  static constexpr int kStageRow = 64;

  struct Loader : paged::PageLoader<TreeArgs, TreeWork, F8, P> {
    __device__ __forceinline__ void queries(const TreeArgs &a, const Work &w, int t, int h, uint32_t dst,
                                            const CUtensorMap *m, uint32_t bar) {
      umma::tma4(dst, m, h * 64, w.unit * a.pack, w.node0 + t * a.per_tile, w.b, bar);
    }
  };
  template <typename T, int D>
  using Converter = paged::PageConverter<T, D, TreeArgs, TreeWork>;
  using Wild = paged::NodeWild<TreeWork>;

  struct Row {
    bool live;
    int64_t at;     // its place in the output
    int ctx;        // positions that every row sees
    uint64_t word;  // new tokens that it sees
    __device__ __forceinline__ void begin(const TreeArgs &a, const Work &w, int t, int r) {
      const int in_tile = r / a.pack, node = w.node0 + t * a.per_tile + in_tile;
      live = in_tile < a.per_tile && node < a.n;
      at = ((int64_t)w.b * a.n + node) * a.q_heads + w.unit * a.pack + r % a.pack;
      ctx = w.len - a.n;
      word = !live ? 0ull : (a.mask ? (uint64_t)a.mask[(int64_t)w.b * a.n + node] : ~0ull >> (63 - node)) &
                                ~0ull >> (64 - a.n);
    }
    __device__ __forceinline__ uint64_t sees(const Work &w, int j, int from) const {
      const int d = ctx - (w.j0 + j) * kKeys - from;  // keys of the 64 in the context
      if (d >= 64) return ~0ull;
      if (d > 0) return word << d | ((1ull << d) - 1);
      return d > -64 ? word >> -d : 0ull;
    }
  };

  template <typename T, int D>
  static __device__ __forceinline__ bool clear(const TreeArgs &, const Work &w, int j, uint8_t *tile, int lane) {
    return paged::clear_behind<D, Mode>(w, j, tile, lane);
  }

  // Where a part's row lies: 256 rows to a part, column by column.
  template <int D>
  static __device__ __forceinline__ void part(const TreeArgs &a, const Work &w, int t, int r, float *&o, int &pitch,
                                              float2 *&ml) {
    o = a.part_o + (int64_t)w.slot * D * 256 + t * 128 + r;
    pitch = 256;
    ml = a.part_ml + w.slot * 256 + t * 128 + r;
  }
};

// Joins the parts of an item that several CTAs had: a CTA has 32 of its rows,
// a lane one of them.  What it waits for are the parts' loads.  G = 1: a warp
// has an eighth of the columns and reads two parts at a time.  G = 8: the
// warps take the parts of 32 columns in turns and add up in warp order.  By
// the number of parts (launch has the rule), a whole call took, G = 1 and 8:
// 16 sequences of 512 to 4096 tokens (two or three parts) 55.7, 69.3 us; 4 of
// 2300 (five) 24.6, 27.0; 2 of 1754 (nine) 17.2, 16.1; one of 30000 (38)
// 49.1, 35.6 us.
constexpr int kJoinThreads = 256;
template <typename T, int D, int G>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const TreeArgs a, int ctas) {
  constexpr int N = G == 1 ? D / 8 : 32, kCols = 8 / G * N;  // columns of a warp, of the CTA
  constexpr int kAhead = G == 1 ? 2 : 1;
  constexpr int kPitch = kCols / 2 + 4;  // words of a row: its 16-byte pieces fall into different banks
  extern __shared__ int s_part[];        // [ctas] places of the parts
  __shared__ float s_sum[G > 1 ? G - 1 : 1][G > 1 ? N + 1 : 1][32];
  __shared__ __align__(16) uint32_t s_out[32 * kPitch];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, grp = warp % G;
  const int items = a.units * a.blocks, b = blockIdx.x / items, item = blockIdx.x % items;
  const int rl = blockIdx.y * 32 + lane, in_tile = (rl & 127) / a.pack;
  const int c_warp = warp / G * N, col0 = blockIdx.z * kCols;  // the warp's columns in the CTA's, the CTA's in the row
  const int node = (item % a.blocks * 2 + (rl >> 7)) * a.per_tile + in_tile;
  const bool live = in_tile < a.per_tile && node < a.n;
  const int64_t at = ((int64_t)b * a.n + node) * a.q_heads + item / a.blocks * a.pack + (rl & 127) % a.pack;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (b == a.n_seqs) {
    if (blockIdx.y == 0 && blockIdx.z == 0) paged::look_at_groups(a.groups, a.n_groups, a.n_seqs, a.err);
    return;
  }
  if (!__any_sync(0xffffffffu, live)) return;  // (every warp has the same rows)
  const long long total = a.cum[a.n_seqs], cb = a.cum[b];
  const long long nt = quotient(a.cum[b + 1] - cb, items);
  const long long from = cb + item * nt, to = from + nt;  // the item's tiles
  const int c0 = (int)quotient((from + 1) * ctas - 1, total), c1 = (int)quotient(to * ctas - 1, total);
  if (c0 == c1) return;  // one CTA had it all
  for (int c = c0 + tid; c <= c1; c += kJoinThreads) {
    const long long first = quotient(total * c, ctas);
    // a part is its CTA's first unless the CTA began before the item; a CTA may have no tiles at all
    s_part[c - c0] = first == quotient(total * (c + 1), ctas) ? -1 : c * 2 + (first >= from ? 0 : 1);
  }
  __syncthreads();
  const int parts = c1 - c0 + 1;
  float m = kNegInf, l = 0.f, o[N];
#pragma unroll
  for (int i = 0; i < N; ++i) o[i] = 0.f;
#pragma unroll 8
  for (int q = 0; q < parts; ++q)
    if (s_part[q] >= 0) m = fmaxf(m, a.part_ml[s_part[q] * 256 + rl].x);
  const float safe = m == kNegInf ? 0.f : m;
  for (int q0 = grp; q0 < parts; q0 += G * kAhead) {
    float x[kAhead][N];
    float2 ml[kAhead];
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      const int part = q0 + e * G < parts ? s_part[q0 + e * G] : -1;
      ml[e] = part >= 0 ? a.part_ml[part * 256 + rl] : make_float2(kNegInf, 0.f);
      const float *src = a.part_o + ((int64_t)part * D + col0 + c_warp) * 256 + rl;
#pragma unroll
      for (int i = 0; i < N; ++i) x[e][i] = part >= 0 ? src[i * 256] : 0.f;
    }
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      const float f = attn::ex2(ml[e].x - safe);
      l += ml[e].y * f;
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = fmaf(x[e][i], f, o[i]);
    }
  }
  if constexpr (G > 1) {
    if (grp > 0 && grp < parts) {
#pragma unroll
      for (int i = 0; i < N; ++i) s_sum[grp - 1][i][lane] = o[i];
      s_sum[grp - 1][N][lane] = l;
    }
    __syncthreads();
    if (grp > 0) return;
    for (int w = 1; w < min(parts, G); ++w) {
      l += s_sum[w - 1][N][lane];
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] += s_sum[w - 1][i][lane];
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < N; i += 8)
    *reinterpret_cast<uint4 *>(s_out + lane * kPitch + (c_warp + i) / 2) =
        make_uint4(attn::Type<T>::pack(o[i] * inv, o[i + 1] * inv), attn::Type<T>::pack(o[i + 2] * inv, o[i + 3] * inv),
                   attn::Type<T>::pack(o[i + 4] * inv, o[i + 5] * inv),
                   attn::Type<T>::pack(o[i + 6] * inv, o[i + 7] * inv));
  if (live && col0 + c_warp == 0 && a.lse)
    a.lse[at] = l == 0.f ? kNegInf : (m - fa::kOffset<T> + log2f(l)) * attn::kLn2;
  if (G == 1)
    __syncthreads();
  else
    __syncwarp();  // one warp is left
  const long long mine = live ? at : -1;
  constexpr int kLeft = kJoinThreads / G;
#pragma unroll
  for (int e = 0; e < 32 * kCols / 8 / kLeft; ++e) {
    const int x = e * kLeft + tid, r = x / (kCols / 8), c = x % (kCols / 8);
    const long long row = __shfl_sync(0xffffffffu, mine, r);
    if (row >= 0)
      *reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + row * D + col0 + c * 8) =
          *reinterpret_cast<const uint4 *>(s_out + r * kPitch + c * 4);
  }
}

template <typename T, int D, bool F8, bool P>
cudaError_t launch(const PagedAttnArgs &p, const paged::Pairs &pairs, int sms, cudaStream_t st) {
  TreeArgs a{};
  a.table = p.table, a.lengths = p.lengths, a.seqs = p.seqs, a.mask = p.mask;
  a.n_seqs = p.n_seqs, a.n = p.n, a.q_heads = p.q_heads, a.group = p.group;
  // All heads of a group in one tile, so that its keys are fetched once: 8 sequences of 2300 tokens, 4 new ones, group
  // 33 (64): 58.7 (104.9) us with a head to a tile, 20.4 (20.6) us so.
  a.pack = p.group <= 128 ? p.group : 1;
  a.per_tile = 128 / a.pack, a.units = p.q_heads / a.pack;
  a.blocks = (p.n + 2 * a.per_tile - 1) / (2 * a.per_tile);
  a.page_shift = p.page_shift, a.table_ld = p.table_ld, a.max_seqs = p.max_seqs, a.n_pages = p.n_pages;
  a.c = p.scale * attn::kLog2e;
  a.out = p.out, a.lse = p.lse, a.err = p.err;
  const int items = a.units * a.blocks;
  const long long most = (long long)(p.max_len > 0 ? (p.max_len - 1) / kKeys + 1 : 1) * p.n_seqs * items;
  const int ctas = (int)(most < sms ? most : sms);
  const paged::Ws ws = paged::workspace(p.ws, p.n_seqs, ctas, 256);
  a.cum = ws.cum, a.part_ml = ws.ml, a.part_o = ws.o;
  a.rows = paged::exponents_of(p);
  a.pairs = pairs;
  a.groups = p.groups, a.n_groups = p.n_groups;
  CUtensorMap tmQ, tmK, tmV;
  const uint64_t dq[4] = {D, (uint64_t)p.q_heads, (uint64_t)p.n, (uint64_t)p.n_seqs};
  const uint64_t sq[3] = {(uint64_t)p.q_head * 2, (uint64_t)p.q_token * 2, (uint64_t)p.q_seq * 2};
  const uint32_t bq[4] = {64, (uint32_t)a.pack, (uint32_t)a.per_tile, 1};
  if (!encode_16bit(&tmQ, p.q, 4, dq, sq, bq) || !paged::page_maps<D, F8, P>(p, pairs, &tmK, &tmV))
    return cudaErrorInvalidValue;
  using M = Mode<F8, P>;
  fa::attn_kernel<T, D, M><<<ctas, fa::kThreadsOf<M>, fa::Smem<D, M>::kBytes, st>>>(tmQ, tmK, tmV, a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  // an item's parts: some more than its share of the CTAs, if the sequences are of like lengths
  const bool many = ctas >= 6LL * p.n_seqs * items;
  cfg.gridDim = dim3((unsigned)((long long)p.n_seqs * items + (p.groups ? 1 : 0)), 8, many ? D / 32 : 1);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = ctas * 4;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return many ? cudaLaunchKernelEx(&cfg, tree_join_kernel<T, D, 8>, a, ctas)
              : cudaLaunchKernelEx(&cfg, tree_join_kernel<T, D, 1>, a, ctas);
}

// A page's columns in one box where pages are small: with pages of 16 the boxes, not the products, are what a tile
// takes.  16 trees of 60 nodes behind 6007 tokens, pages of 16: 102 us with a box for each 64 columns, 88 so.
template <typename T, int D, bool F8>
cudaError_t by_pages(const PagedAttnArgs &p, int sms, cudaStream_t st) {
  paged::Pairs pairs{};
  if constexpr (D == 128 && !F8) {
    if (p.page_shift <= paged::kPairShift && paged::page_pairs(p, &pairs))
      return launch<T, D, F8, true>(p, pairs, sms, st);
  }
  return launch<T, D, F8, false>(p, pairs, sms, st);
}

template <typename T, int D, bool F8, bool P>
cudaError_t prepare() {
  using M = Mode<F8, P>;
  return cudaFuncSetAttribute(fa::attn_kernel<T, D, M>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              fa::Smem<D, M>::kBytes);
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
cudaError_t launch_any(const PagedAttnArgs &a, int dtype, int dim, int sms, cudaStream_t st) {
  if (dtype == NS_DTYPE_BF16)
    return dim == 128 ? by_pages<__nv_bfloat16, 128, F8>(a, sms, st) : by_pages<__nv_bfloat16, 64, F8>(a, sms, st);
  return dim == 128 ? by_pages<__half, 128, F8>(a, sms, st) : by_pages<__half, 64, F8>(a, sms, st);
}

}  // namespace
}  // namespace ns
