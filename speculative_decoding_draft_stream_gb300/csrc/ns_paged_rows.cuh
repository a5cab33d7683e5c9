// Attention of a sequence's new tokens over a paged key-value cache.
//
// Rows: the n new tokens of a sequence and the query heads that share a
// key-value head make R = n * group query rows that read the same keys, so
// each key and value is fetched once for all of them (once for every 64 rows
// when R is larger; the repeats hit L2).
//
// Work, two ways (by_rows has the rule).  The line: the keys of every
// (sequence, key-value head, block of rows), an item, are cut into tiles of
// 64, all tiles of the call are put in one line, and each of the resident
// CTAs takes an equal, contiguous share of it.  So a batch of very different
// lengths, or one long sequence, keeps every SM busy to the end, whatever the
// lengths are (the host does not know them).  A CTA whose share begins or
// ends inside an item leaves its rows' (m, l, o) in the workspace, at most two
// of them; the join kernel, whose launch overlaps the end of this one, adds
// up the parts of such items in CTA order.  A cluster: a small call is mostly
// latency, so each item goes to one cluster, whose CTAs have equal shares of
// its tiles (of 64 or 128 keys) and join through shared memory: one launch, no
// workspace.  No atomics in either: the same inputs give the same bits.
//
// In a CTA: the next tiles are in flight (cp.async, 16 bytes, page ids
// fetched a tile ahead).  Up to 16 rows the warps split a tile's keys and
// join at the item's end; above, each of four warps has 16 rows of 64.
//
// What bounds it: HBM for one-token steps (each key is used by `group` rows,
// a few flops a byte); the mma.sync rate for 64-row blocks.  Loads and
// products of one CTA hardly overlap (a warp that issues copies waits for the
// load unit), so CTAs overlap with each other: three to an SM with two tiles
// each instead of two with three took 48 sequences of 200 to 40000 tokens (28
// heads on 4, 128 columns, fp16) from 97.6 to 91.0 us, 5.8 TB/s; with 64
// columns, four to an SM instead of two, 8 sequences of 16000 (12 heads on 4)
// from 43.8 to 33.1 us.
//
// Caches of 8 bits (F8): keys and values come as e4m3 codes with a power of two
// for each row, and become fp16 on their way into the products, which is exact.
// With ke_j and ve_j the exponents of key and value j,
//   x_j = (q . code_j) 2^ke_j scale log2(e),   y_j = x_j + ve_j,
//   o = sum 2^(y_j - m) code_j,   l = sum 2^(y_j - m) 2^-ve_j,   m = max y:
// the values' scale goes into the probability before it is rounded, so that
// fp16's range is spent on what each value adds to the result.  With ve within
// +-40 no term that counts in l is lost (2^(y - m) >= 2^-126 down to 2^-46 of
// the largest p).  bf16 queries become fp16 by a power of two of each row's
// own.  The order of a product's terms is free, so a lane's operands are runs of
// bytes: 32 columns of a key (16 of 64), and of four values 16 (8) columns each,
// paired by byte permutations; a code costs half a conversion.  A tile has twice
// the keys: as many bytes in flight.  Up to 8 rows are the columns of the
// products (Rows8), not half of 16 rows.  48 sequences of 200 to 40000 tokens
// (28 heads on 4, 128 columns, fp16, pages of 64) take 54 us, 4.9 TB/s (90 of 16
// bits): bound by HBM and by issue slots (conversions, exponents, softmax:
// half of them); with 64 keys to a tile and four CTAs to an SM 59.5 us.
#pragma once

#include <type_traits>

#include "ns_paged_attn.cuh"

namespace ns {
namespace {

using namespace paged;

// How a call is shared out (by_rows has the rule): the line, or a cluster to
// an item, of CTAs as small as the line's, two or more to an SM, or of large
// ones, one to an SM (128 columns), with twice the warps and keys.
enum Way { kLine, kSmall, kLarge };
constexpr int kCluster = 16;  // CTAs of an item: one for each row that it may have
template <int W>
constexpr int kThreads = W == kLarge ? 256 : 128;
template <int D, int W, int WM, bool F8>
constexpr int kKeys = (W == kLarge ? 128 : 64) * (F8 && WM <= 1 ? 2 : 1);  // of a tile
template <int D, bool F8>
constexpr int kRowBytes = D * (F8 ? 1 : 2);
template <int D>
constexpr int kPerSm = D == 128 ? 3 : 4;  // CTAs of the line on an SM
template <int D, int W, int WM, bool F8>
constexpr int kStages = D == 128 && W != kLarge ? 2 : F8 && WM > 1 ? 4 : 3;  // tiles in flight
constexpr int kMerge = 32 * 4 * 4;    // a lane's m, l (and padding), after its o

template <int D, int W, int WM, bool F8>
__host__ __device__ constexpr int pa_stage() {  // F8: and the exponents of keys and values
  return 2 * kKeys<D, W, WM, F8> * (kRowBytes<D, F8> + (F8 ? 1 : 0));
}
// Behind the stages: what a warp hands over to warp 0; in a cluster, (m, l)
// and o of each of its CTAs for the rows that this CTA joins.
template <int D, int WM, int W, bool F8>
__host__ __device__ constexpr int pa_smem() {
  return kStages<D, W, WM, F8> * pa_stage<D, W, WM, F8>() +
         (W != kLine ? 16 * (D + 2) * 4 : WM <= 1 ? 32 * D / (WM ? 2 : 4) * 4 + kMerge : 0);
}

// CTAs that an SM is to hold: as many as their shared memory allows (64 rows: their registers).  The line has that
// many on each SM; its equal shares would end in a second, half empty wave if it had more.
template <int D, int WM, int W>
constexpr int kResident = W == kLarge ? (D == 128 ? 1 : 2) : WM <= 1 ? kPerSm<D> : (D == 128 ? 2 : 3);
// F8: bytes of where each eight of a tile's rows lies, for each warp.
template <int D, int W, int WM>
constexpr int kPlaces = kThreads<W> / 32 * (kKeys<D, W, WM, true> / 8) * 16;
template <int D, int WM, int W, bool F8>
constexpr bool kHeld =
    // (1 KB: the system's)
    kResident<D, WM, W> * (pa_smem<D, WM, W, F8>() + 1280 + (F8 ? kPlaces<D, W, WM> : 0)) <= 228 * 1024;
template <int D, bool F8>
constexpr bool kAllHeld = kHeld<D, 1, kLine, F8> && kHeld<D, 4, kLine, F8> && kHeld<D, 1, kSmall, F8> &&
                          kHeld<D, 1, kLarge, F8>;
template <int D>
constexpr bool kHeld8 = kHeld<D, 0, kLine, true> && kHeld<D, 0, kSmall, true> && kHeld<D, 0, kLarge, true>;
static_assert(kAllHeld<128, false> && kAllHeld<64, false> && kAllHeld<128, true> && kAllHeld<64, true> && kHeld8<128> &&
                  kHeld8<64>,
              "shared memory of an SM");

// What an item's beginning and end take, in tiles: the line of 8-bit caches has that many more for each item, so that
// shares are equal in time: 48 sequences of 200 to 40000 tokens (28 heads on 4, fp16) 59.0 us without, 54.4 with 1,
// 54.1 with 2.
template <bool F8>
constexpr int kItemCost = F8 ? 1 : 0;

template <int KEYS>
__host__ __device__ inline long long pa_tiles(int len) {
  return len > 0 ? (len - 1) / KEYS + 1 : 1;
}

// Where a CTA is in the line of tiles: item (sequence b, `item` = head *
// blocks + block of rows) and its tile.
template <int KEYS>
struct Cursor {
  int b, item, tile, nt, len;
  const int32_t *table;
  __device__ __forceinline__ void enter(const PagedAttnArgs &a, uint32_t *err) {
    len = length(a, b, err);
    nt = (int)pa_tiles<KEYS>(len);
    const int s = a.seqs[b];
    table = a.table + (size_t)(s >= 0 && s < a.max_seqs ? s : 0) * a.table_ld;
  }
  __device__ __forceinline__ void next(const PagedAttnArgs &a, int items) {
    if (++tile < nt) return;
    tile = 0;
    if (++item < items) return;
    item = 0;
    if (++b < a.n_seqs) enter(a, nullptr);
  }
};

__device__ __forceinline__ uint32_t shared_at(const void *p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ uint32_t of_rank(uint32_t a, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
__device__ __forceinline__ void push(uint32_t a, float x) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(x) : "memory");
}

// Rows of a CTA's block: 16 to each of WM warps, or (WM 0, F8) 8 that every warp has, as with WM 1.  (Clusters: at
// most 16.)
template <int WM>
constexpr int kBlockRows = WM == 0 ? 8 : 16 * WM;
template <typename T, int D, int WM, int W, bool F8>
__global__ void __launch_bounds__(kThreads<W>, kResident<D, WM, W>)
    paged_attn_kernel(const PagedAttnArgs a, int blocks) {
  using C = std::conditional_t<F8, __half, T>;  // the products' type
  constexpr int kPaThreads = kThreads<W>, kPaKeys = kKeys<D, W, WM, F8>, kWarps = kPaThreads / kWarp;
  constexpr bool kFew = WM <= 1, k8 = WM == 0;
  constexpr int WK = kFew ? kWarps : kWarps / WM, NK = kPaKeys / WK, kRows = kBlockRows<WM>;
  constexpr int kRowB = kRowBytes<D, F8>, kStageB = pa_stage<D, W, WM, F8>(), kRing = kStages<D, W, WM, F8>;
  constexpr int kLanesRow = kRowB / 16;               // threads that fetch a row
  constexpr int kPass = kPaThreads / kLanesRow;       // rows a pass of the CTA fetches
  static_assert((W == kLine || kFew) && (!k8 || F8), "a cluster has 16 rows at most");
  constexpr int kCtas = kCluster;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ longlong2 s_places[F8 ? kWarps * kPaKeys / 8 : 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int wm = kFew ? 0 : warp, wk = kFew ? warp : 0;
  const int items = a.kv_heads * blocks, R = a.n * a.group;
  auto head_of = [&](int item) { return kFew ? item : item / blocks; };  // (few rows are one block)
  const uint32_t s0 = (uint32_t)__cvta_generic_to_shared(smem);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  Cursor<kPaKeys> ld;
  long long t0, t1;
  Ws ws{};
  if constexpr (W != kLine) {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // this CTA has begun
    const int at = blockIdx.x / kCtas, rank = blockIdx.x % kCtas;
    ld.b = at / items, ld.item = at % items;
    ld.enter(a, rank == 0 && ld.item == 0 ? a.err : nullptr);
    t0 = (long long)ld.nt * rank / kCtas, t1 = (long long)ld.nt * (rank + 1) / kCtas;
    ld.tile = (int)t0;
  } else {
    // where the tiles will lie, so that a CTA's shared memory does not grow with the sequences
    long long *s_cum = reinterpret_cast<long long *>(smem);
    static_assert(NS_MAX_ATTEND_SEQS * 8 <= kRing * kStageB, "room for the sequences");
    __shared__ long long s_sum[kPaThreads / kWarp];
    // tiles of the sequences before each one
    constexpr int kCost = kItemCost<F8>;
    long long total = 0;
    for (int b0 = 0; b0 < a.n_seqs; b0 += kPaThreads) {
      const int b = b0 + tid;
      const long long mine =
          b < a.n_seqs ? (pa_tiles<kPaKeys>(length(a, b, blockIdx.x == 0 ? a.err : nullptr)) + kCost) * items : 0;
      long long sum = mine;
#pragma unroll
      for (int off = 1; off < kWarp; off <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, sum, off);
        if (lane >= off) sum += o;
      }
      if (lane == kWarp - 1) s_sum[warp] = sum;
      __syncthreads();
      long long before = total;
      for (int w = 0; w < kPaThreads / kWarp; ++w) {
        if (w < warp) before += s_sum[w];
        total += s_sum[w];
      }
      if (b < a.n_seqs) s_cum[b] = before + sum - mine;
      __syncthreads();
    }
    ws = workspace(a.ws, a.n_seqs, gridDim.x, kRows);
    if (blockIdx.x == 0) {
      for (int b = tid; b < a.n_seqs; b += kPaThreads) ws.cum[b] = s_cum[b];
      if (tid == 0) ws.cum[a.n_seqs] = total;
    }
    t0 = quotient(total * blockIdx.x, gridDim.x), t1 = quotient(total * (blockIdx.x + 1), gridDim.x);
    if (t0 >= t1) return;

    auto enter_at = [&](long long t) {  // the cursor to place t of the line; the tiles before it
      int lo = 0, hi = a.n_seqs;        // the last sequence that begins at or before t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_cum[mid] <= t)
          lo = mid;
        else
          hi = mid;
      }
      ld.b = lo;
      ld.enter(a, nullptr);
      const long long local = t - s_cum[lo];
      ld.item = (int)quotient(local, ld.nt + kCost);
      ld.tile = max(0, (int)(local - (long long)ld.item * (ld.nt + kCost)) - kCost);
      return s_cum[lo] - (long long)kCost * lo * items + (long long)ld.item * ld.nt + ld.tile;
    };
    if (kCost) {  // from places of the line to tiles
      t1 = t1 == total ? total - (long long)kCost * a.n_seqs * items : enter_at(t1);
      t0 = enter_at(t0);
      if (t0 >= t1) return;
    } else {
      enter_at(t0);
    }
    __syncthreads();  // everyone is done with s_cum before the first tile comes
  }
  Cursor<kPaKeys> cu = ld;

  // page ids of the load cursor's tile, one for each eight rows, in as many lanes (-1: past the sequence's end, -2: out
  // of range)
  auto fetch_ids = [&]() {
    int id = -1;
    if (lane < kPaKeys / 8) {
      const int p = ld.tile * kPaKeys + lane * 8;
      if (p < ld.len) {
        id = ld.table[p >> a.page_shift];
        if (id < 0 || id >= a.n_pages) {
          set_flag(a.err, NS_FLAG_BAD_ID);
          id = -2;
        }
      }
    }
    return id;
  };
  // A lane has the offsets of its eight rows' first; a thread's rows are all the same one of their eight.
  const int fr = tid / kLanesRow, fc = tid % kLanesRow, pmask = (1 << a.page_shift) - 1;
  static_assert(kPass % 8 == 0, "rows of a thread");
  using E = std::conditional_t<F8, uint8_t, T>;  // an element of the cache
  const E *kbase = static_cast<const E *>(a.k) + (fr & 7) * a.k_token + fc * (16 / sizeof(E));
  const E *vbase = static_cast<const E *>(a.v) + (fr & 7) * a.v_token + fc * (16 / sizeof(E));
  const uint32_t to = F8 ? piece8<D>(fr, fc) : piece<D>(fr, fc);
  auto fetch = [&](int id, int stage) {
    if constexpr (F8) {
      // A lane finds an eight's places (products of 32 bits), which the warp then reads from shared memory.
      const uint32_t sk = s0 + stage * kStageB + to, sv = sk + kPaKeys * kRowB;
      const int p0 = ld.tile * kPaKeys, left = ld.len - p0, head = head_of(ld.item);
      const uint32_t there = __ballot_sync(0xffffffffu, id >= 0);
      longlong2 *mine = s_places + warp * (kPaKeys / 8);
      if (lane < kPaKeys / 8) {
        const int page = max(0, id), row = (p0 + lane * 8) & pmask;
        mine[lane] = make_longlong2(16 * ((int64_t)page * a.kp16 + (int64_t)row * a.kt16),
                                    16 * ((int64_t)page * a.vp16 + (int64_t)row * a.vt16));
        if (warp < 2)  // its exponents: warp 0 the keys', warp 1 the values'
          cp8(s0 + stage * kStageB + 2 * kPaKeys * kRowB + warp * kPaKeys + lane * 8,
              warp ? a.v_exp + head * a.ve_head + 8 * ((int64_t)page * a.vep8) + row
                   : a.k_exp + head * a.ke_head + 8 * ((int64_t)page * a.kep8) + row,
              id >= 0);
      }
      __syncwarp();
      const char *kh = reinterpret_cast<const char *>(kbase) + head * a.k_head;
      const char *vh = reinterpret_cast<const char *>(vbase) + head * a.v_head;
      auto rows_of = [&](auto whole) {
#pragma unroll
        for (int pass = 0; pass < kPaKeys / kPass; ++pass) {
          const int r = pass * kPass + fr, eight = r >> 3;
          const longlong2 at = mine[eight];
          const bool ok = whole.value || (r < left && (there >> eight & 1));
          cp16(sk + pass * kPass * kRowB, kh + at.x, ok);
          cp16(sv + pass * kPass * kRowB, vh + at.y, ok);
        }
      };
      constexpr uint32_t kAll = kPaKeys == 256 ? 0xffffffffu : (1u << (kPaKeys / 8 % 32)) - 1;
      if (left >= kPaKeys && (there & kAll) == kAll)
        rows_of(std::true_type{});
      else
        rows_of(std::false_type{});
      __syncwarp();  // (the places are written again for the next tile)
      return;
    }
    const uint32_t sk = s0 + stage * kStageB + to, sv = sk + kPaKeys * kRowB;
    const int left = ld.len - ld.tile * kPaKeys, head = head_of(ld.item);
    const int64_t page = id >= 0 ? id : 0, row = (ld.tile * kPaKeys + lane * 8) & pmask;
    const int64_t ko = page * a.k_page + head * a.k_head + row * a.k_token;
    const int64_t vo = page * a.v_page + head * a.v_head + row * a.v_token;
    const uint32_t there = __ballot_sync(0xffffffffu, id >= 0);
#pragma unroll
    for (int pass = 0; pass < kPaKeys / kPass; ++pass) {
      const int r = pass * kPass + fr;
      const bool ok = r < left && (there >> (r >> 3) & 1);
      const int64_t k = __shfl_sync(0xffffffffu, ko, r >> 3), v = __shfl_sync(0xffffffffu, vo, r >> 3);
      cp16(sk + pass * kPass * kRowB, kbase + k, ok);
      cp16(sv + pass * kPass * kRowB, vbase + v, ok);
    }
  };

  const float c = a.scale * kLog2e;
  long long left_ld = t1 - t0;
  int ids = fetch_ids();
  int st_ld = 0;
  constexpr int kAhead = kRing - 1;
  uint32_t missing[kAhead] = {};  // of each tile in flight: its eights of rows without a page
  auto issue = [&]() {
#pragma unroll
    for (int i = 0; i + 1 < kAhead; ++i) missing[i] = missing[i + 1];
    missing[kAhead - 1] = 0;
    if (left_ld > 0) {
      fetch(ids, st_ld);
      missing[kAhead - 1] = __ballot_sync(0xffffffffu, ids == -2);
      st_ld = st_ld + 1 == kRing ? 0 : st_ld + 1;
      --left_ld;
      if (left_ld > 0) {
        ld.next(a, items);
        ids = fetch_ids();
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) issue();

  std::conditional_t<k8, Rows8<C, D>, Rows<C, D>> rows;
  if (W != kLine) rows.clear();  // (a CTA of a short sequence may have no tile)
  uint32_t q[D / 16][k8 ? 2 : 4];
  float cq[2] = {c, c};  // of each row's scores (F8: with the power of two that its query was divided by)
  uint64_t word[2] = {0, 0};
  int st = 0;
  long long seg0 = t0;  // where the current item's share of this CTA begins
  for (long long g = t0; g < t1; ++g) {
    const int head = head_of(cu.item), rb = kFew ? 0 : cu.item % blocks;
    if (g == t0 || cu.tile == 0) {  // a new item: its queries and masks
      seg0 = g;
      rows.clear();
      const T *qs = static_cast<const T *>(a.q) + (int64_t)cu.b * a.q_seq;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = rb * kRows + wm * 16 + rows.row(h), node = r / a.group;
        word[h] = 0;
        if (r < R) {
          word[h] = a.mask ? (uint64_t)a.mask[(int64_t)cu.b * a.n + node] : ~0ull >> (63 - node);
        }
      }
      constexpr int kParts = k8 ? 2 : 4;  // words of a product's operand
#pragma unroll
      for (int h = 0; h < (k8 ? 1 : 2); ++h) {
        const int r = rb * kRows + wm * 16 + (lane >> 2) + 8 * h;
        const int node = r / a.group, qh = head * a.group + r % a.group;
        const T *src = qs + (int64_t)node * a.q_token + (int64_t)qh * a.q_head + (lane & 3) * (F8 ? D / 4 : 2);
        constexpr int kStep = F8 ? 4 : 16, kHalf = F8 ? 2 : 8;  // columns of a product, of its halves
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          q[kk][h] = r < R ? *reinterpret_cast<const uint32_t *>(src + kk * kStep) : 0u;
          q[kk][kParts / 2 + h] = r < R ? *reinterpret_cast<const uint32_t *>(src + kk * kStep + kHalf) : 0u;
        }
        if constexpr (F8 && !std::is_same_v<T, __half>) {  // bf16 -> fp16, the largest to 1 .. 2
          uint32_t most = 0;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            most = __vimax3_u16x2(most, q[kk][h] & 0x7fff7fffu, q[kk][kParts / 2 + h] & 0x7fff7fffu);
          most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, 1));
          most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, 2));
          const int e = min(max((int)(max(most & 0xffffu, most >> 16) >> 7) - 127, -126), 126);
          const float f = __uint_as_float((uint32_t)(127 - e) << 23);
          const float back = c * __uint_as_float((uint32_t)(127 + e) << 23);
          if constexpr (k8) {  // (row g's lanes have it, rows 2 t and 2 t + 1 want it)
            cq[0] = __shfl_sync(0xffffffffu, back, (lane & 3) * 8);
            cq[1] = __shfl_sync(0xffffffffu, back, (lane & 3) * 8 + 4);
          } else {
            cq[h] = back;
          }
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t &lo = q[kk][h], &hi = q[kk][kParts / 2 + h];
            const float2 x = Type<T>::unpack(lo), y = Type<T>::unpack(hi);
            lo = Type<C>::pack(x.x * f, x.y * f), hi = Type<C>::pack(y.x * f, y.y * f);
          }
        }
      }
    }
    cp_wait<kAhead - 1>();
    __syncthreads();  // the tile is there for everyone, and everyone is done with the stage to be filled next
    const uint32_t gone = missing[0];
    issue();
    const uint32_t sk = s0 + st * kStageB, sv = sk + kPaKeys * kRowB, se = sv + kPaKeys * kRowB;
    st = st + 1 == kRing ? 0 : st + 1;
    const int ctx = cu.len - a.n, p0 = cu.tile * kPaKeys, k0 = wk * NK;
    if (p0 + kPaKeys <= ctx && !gone) {
      auto none = [](int, int) { return false; };
      if constexpr (F8)
        rows.template tile8<NK, false>(q, sk, sv, se, se + kPaKeys, k0, cq, none, false);
      else
        rows.template tile<NK, false>(q, sk, sv, k0, c, none, false);
    } else {
      const int n = a.n, j0 = p0 + k0 - ctx;  // the first key's node
      bool wild = false;
      auto hidden = [&](int h, int key) {
        const int j = j0 + key;
        return (j >= 0 && (j >= n || !((word[h] >> j) & 1))) || (gone >> ((k0 + key) >> 3) & 1);
      };
      if constexpr (F8) {
        if (n > 1 || a.mask)
          wild = __any_sync(0xffffffffu, wild_codes(sv + (uint32_t)(k0 * kRowB), NK * kRowB / 16, lane, kWarp));
        rows.template tile8<NK, true>(q, sk, sv, se, se + kPaKeys, k0, cq, hidden, wild);
      } else {
        if (n > 1 || a.mask)
          wild = __any_sync(0xffffffffu, wild_pieces<T>(sv + (uint32_t)(k0 * D * 2), NK * D / 8, lane, kWarp));
        rows.template tile<NK, true>(q, sk, sv, k0, c, hidden, wild);
      }
    }
    const bool ends = cu.tile + 1 == cu.nt;
    if (ends || g + 1 == t1) {
      rows.sum_l();
      if (W != kLine) break;
      if (kFew) {  // the warps' keys join, in warp order, in warp 0
        float4 *bo = reinterpret_cast<float4 *>(smem + kRing * kStageB);
        constexpr int kParts = decltype(rows)::kParts;
        float4 *bm = bo + kParts * 32;
        for (int w = 1; w < 4; ++w) {
          if (warp == w) {
#pragma unroll
            for (int i = 0; i < kParts; ++i)
              bo[i * 32 + lane] = make_float4(rows.o[i][0], rows.o[i][1], rows.o[i][2], rows.o[i][3]);
            bm[lane] = make_float4(rows.m[0], rows.m[1], rows.l[0], rows.l[1]);
          }
          __syncthreads();
          if (warp == 0) {
            const float4 x = bm[lane];
            const float om[2] = {x.x, x.y}, ol[2] = {x.z, x.w};
            float fa[2], fb[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float to = fmaxf(rows.m[h], om[h]), safe = to == kNegInf ? 0.f : to;
              fa[h] = ex2(rows.m[h] - safe);
              fb[h] = ex2(om[h] - safe);
              rows.m[h] = to;
              rows.l[h] = rows.l[h] * fa[h] + ol[h] * fb[h];
            }
#pragma unroll
            for (int i = 0; i < kParts; ++i) {
              const float4 y = bo[i * 32 + lane];
              rows.o[i][0] = rows.o[i][0] * fa[0] + y.x * fb[0];
              rows.o[i][1] = rows.o[i][1] * fa[rows.of(1)] + y.y * fb[rows.of(1)];
              rows.o[i][2] = rows.o[i][2] * fa[rows.of(2)] + y.z * fb[rows.of(2)];
              rows.o[i][3] = rows.o[i][3] * fa[1] + y.w * fb[1];
            }
          }
          __syncthreads();
        }
      }
      if (!kFew || warp == 0) {
        const bool whole = ends && g + 1 - seg0 == cu.nt;
        const int slot = seg0 == t0 ? 0 : 1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int rl = wm * 16 + rows.row(h), r = rb * kRows + rl;
          if (r < R) {
            if (whole) {
              const int64_t at = ((int64_t)cu.b * a.n + r / a.group) * a.q_heads + head * a.group + r % a.group;
              const float inv = rows.l[h] == 0.f ? 0.f : 1.f / rows.l[h];
              T *dst = static_cast<T *>(a.out) + at * D;
              rows.template columns<F8>(h, [&](int d, float x, float y) {
                *reinterpret_cast<uint32_t *>(dst + d) = Type<T>::pack(x * inv, y * inv);
              });
              if (a.lse && rows.first()) a.lse[at] = row_lse<C>(rows.m[h], rows.l[h]);
            } else {
              const size_t at = ((size_t)blockIdx.x * 2 + slot) * kRows + rl;
              float *dst = ws.o + at * D;
              rows.template columns<F8>(
                  h, [&](int d, float x, float y) { *reinterpret_cast<float2 *>(dst + d) = make_float2(x, y); });
              if (rows.first()) ws.ml[at] = make_float2(rows.m[h], rows.l[h]);
            }
          }
        }
      }
    }
    if (g + 1 < t1) cu.next(a, items);
  }
  if constexpr (W != kLine) {
    // The warps' parts join here, and the CTAs' in CTA r for row r, both in their order.
    constexpr int kPitch = D + 8;  // of a row of a warp's part: the eight rows of a store in different banks
    static_assert(kWarps * 16 * (kPitch + 2) * 4 <= kRing * kStageB, "the parts replace the tiles");
    const int rank = blockIdx.x % kCtas, head = ld.item, b = ld.b;
    float *w_o = reinterpret_cast<float *>(smem);
    float2 *w_ml = reinterpret_cast<float2 *>(w_o + kWarps * 16 * kPitch);
    float *c_o = reinterpret_cast<float *>(smem + kRing * kStageB);  // [kCtas][D]
    float2 *c_ml = reinterpret_cast<float2 *>(c_o + kCtas * D);
    __syncthreads();  // (every tile has been waited for and used)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = rows.row(h);
      if (r < R) {
        float *dst = w_o + (warp * 16 + r) * kPitch;
        rows.template columns<F8>(
            h, [&](int d, float x, float y) { *reinterpret_cast<float2 *>(dst + d) = make_float2(x, y); });
        if (rows.first()) w_ml[warp * 16 + r] = make_float2(rows.m[h], rows.l[h]);
      }
    }
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // every CTA of the cluster has begun
    __syncthreads();
    const int col = tid % D;
    for (int r = tid / D; r < R; r += kPaThreads / D) {
      float2 p[kWarps];
      float m = kNegInf, l = 0.f, o = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        p[w] = w_ml[w * 16 + r];
        m = fmaxf(m, p[w].x);
      }
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(p[w].x - (m == kNegInf ? 0.f : m));
        l = fmaf(p[w].y, f, l);
        o = fmaf(w_o[(w * 16 + r) * kPitch + col], f, o);
      }
      push(of_rank(shared_at(c_o + rank * D + col), r), o);
      if (col < 2) push(of_rank(shared_at(c_ml + rank) + 4 * col, r), col ? l : m);
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank < R && tid < D) {
      float2 p[kCtas];
      float m = kNegInf, l = 0.f, o = 0.f;
#pragma unroll
      for (int i = 0; i < kCtas; ++i) {
        p[i] = c_ml[i];
        m = fmaxf(m, p[i].x);
      }
#pragma unroll
      for (int i = 0; i < kCtas; ++i) {
        const float f = ex2(p[i].x - (m == kNegInf ? 0.f : m));
        l = fmaf(p[i].y, f, l);
        o = fmaf(c_o[i * D + col], f, o);
      }
      const int64_t at = ((int64_t)b * a.n + rank / a.group) * a.q_heads + head * a.group + rank % a.group;
      static_cast<T *>(a.out)[at * D + col] = static_cast<T>(l == 0.f ? 0.f : o / l);
      if (a.lse && col == 0) a.lse[at] = row_lse<C>(m, l);
    }
  }
}

// The rows of an item for the join: row r of head h and block rb is new token
// (16 WM rb + r) / group.
template <int WM, bool F8>
struct Rows16 {
  int blocks;
  static constexpr int kRows = kBlockRows<WM>, kCost = kItemCost<F8>;
  static constexpr int kGroups = WM <= 1 ? 4 : 1;  // few rows may have hundreds of parts, many rows have two or three
  template <typename T>
  __device__ __forceinline__ float offset() const {
    return F8 ? Type<__half>::kOffset : Type<T>::kOffset;
  }
  __device__ __forceinline__ bool place(const PagedAttnArgs &a, int item, int rl, int &node, int &qh) const {
    const int r = item % blocks * kRows + rl;
    node = r / a.group, qh = item / blocks * a.group + r % a.group;
    return r < a.n * a.group;
  }
};

template <typename T, int D, int WM, bool F8>
cudaError_t launch(const PagedAttnArgs &a, int sms, cudaStream_t st) {
  constexpr int kRows = kBlockRows<WM>;
  const int blocks = (a.n * a.group + kRows - 1) / kRows;
  constexpr int kCtas = kResident<D, WM, kLine>;  // (on an SM)
  const long long most = pa_tiles<kKeys<D, kLine, WM, F8>>(a.max_len) * a.n_seqs * a.kv_heads * blocks;
  const int ctas = (int)(most < (long long)kCtas * sms ? most : kCtas * sms);
  paged_attn_kernel<T, D, WM, kLine, F8><<<ctas, kThreads<kLine>, pa_smem<D, WM, kLine, F8>(), st>>>(a, blocks);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int rows = a.n * a.group < kRows ? a.n * a.group : kRows;
  return launch_join<T, D>(a, Rows16<WM, F8>{blocks}, rows, a.kv_heads * blocks, ctas, st);
}

struct ClusterLaunch {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[1];
  ClusterLaunch(int items, int threads, int smem, cudaStream_t st) {
    cfg.gridDim = dim3((unsigned)items * kCluster);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kCluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
  }
};
// Clusters that the device holds at once.
template <typename T, int D, int WM, int W, bool F8, typename Fit>
auto &resident(Fit &fit) {
  return fit.clusters[F8 ? 2 - WM : 0][Type<T>::kBf16 ? NS_DTYPE_BF16 : NS_DTYPE_F16][D == 128][W == kLarge];
}

// Whether each item can have its own cluster with up to kMostTiles tiles to a
// CTA (in two waves of small CTAs: with one or two tiles).
template <int D>
constexpr int kMostTiles = D == 128 ? 12 : 16;
template <typename T, int D, int WM, int W, bool F8>
bool clusters_fit(const PagedAttnArgs &a, const PagedFit &fit) {
  constexpr int kTile = kKeys<D, W, WM, F8>;
  const bool two_waves = W == kSmall && a.max_len > kCluster * kTile / 2 && a.max_len <= 2 * kCluster * kTile;
  return (long long)a.n_seqs * a.kv_heads <= (two_waves ? 2 : 1) * resident<T, D, WM, W, F8>(fit) &&
         a.max_len <= kMostTiles<D> * kCluster * kTile;
}
template <typename T, int D, int WM, int W, bool F8>
cudaError_t launch_clusters(const PagedAttnArgs &a, cudaStream_t st) {
  ClusterLaunch l(a.n_seqs * a.kv_heads, kThreads<W>, pa_smem<D, WM, W, F8>(), st);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, paged_attn_kernel<T, D, WM, W, F8>, a, 1);
  return e != cudaSuccess || !a.groups ? e : launch_groups(a, st);
}

template <typename T, int D, int WM, int W, bool F8>
cudaError_t prepare(PagedFit *fit) {
  auto *kernel = paged_attn_kernel<T, D, WM, W, F8>;
  cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, pa_smem<D, WM, W, F8>());
  if (W == kLine) return e;
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  ClusterLaunch l(64, kThreads<W>, pa_smem<D, WM, W, F8>(), nullptr);
  return cudaOccupancyMaxActiveClusters(&resident<T, D, WM, W, F8>(*fit), kernel, &l.cfg);
}
template <typename T, int D, bool F8>
cudaError_t prepare_all(PagedFit *fit) {
  cudaError_t e = prepare<T, D, 1, kLine, F8>(fit);
  if (e == cudaSuccess) e = prepare<T, D, 4, kLine, F8>(fit);
  if (e == cudaSuccess) e = prepare<T, D, 1, kSmall, F8>(fit);
  if (e == cudaSuccess) e = prepare<T, D, 1, kLarge, F8>(fit);
  if constexpr (F8) {
    if (e == cudaSuccess) e = prepare<T, D, 0, kLine, F8>(fit);
    if (e == cudaSuccess) e = prepare<T, D, 0, kSmall, F8>(fit);
    if (e == cudaSuccess) e = prepare<T, D, 0, kLarge, F8>(fit);
  }
  return e;
}

// At most 16 rows (by_rows in ns_paged_attn.cu has the rule).
template <typename T, int D, int WM, bool F8>
cudaError_t few_rows(const PagedAttnArgs &a, int sms, const PagedFit &fit, cudaStream_t st) {
  if (a.max_len > kCluster * kKeys<D, kSmall, WM, F8> && clusters_fit<T, D, WM, kLarge, F8>(a, fit))
    return launch_clusters<T, D, WM, kLarge, F8>(a, st);
  if (clusters_fit<T, D, WM, kSmall, F8>(a, fit)) return launch_clusters<T, D, WM, kSmall, F8>(a, st);
  return launch<T, D, WM, F8>(a, sms, st);
}

}  // namespace
}  // namespace ns
