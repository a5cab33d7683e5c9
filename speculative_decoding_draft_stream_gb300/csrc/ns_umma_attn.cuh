// Attention on the 5th-generation tensor cores: the kernel that whole prompts
// (ns_prompt_attn.cu) and many rows over a paged cache (ns_paged_umma.cu) share.
//
// Mathematics: for each query row, over its keys in tiles of 128,
//   x_j = scale log2(e) q . k_j,  m = running bound of max x,
//   l = sum 2^(x_j - m),  o = sum 2^(x_j - m) v_j;   out = o / l.
// m is the first tile's maximum, and is raised (l and o multiplied by
// 2^(old - new)) only when the sum of 64 probabilities passes 2^15: any m
// that is not far below the maximum gives the same quotient, so after the
// first tile no maximum is taken (the sum is needed anyway) and the
// accumulator in tensor memory is hardly ever rewritten.  Scores, sums and o
// are fp32; a probability is rounded once, to the values' type, as an operand
// of the second product (l sums it unrounded).  With u that type's unit
// roundoff it costs at most u sum p |v|, beside the output's own u |o|; in two
// operands, a rounded one and the rest, the second product would cost twice as
// much.  fp16 probabilities are kept
// 2^6 times larger: within fp16's range under the bound on the sum, and 2^-30
// of the largest is not lost.
//
// Rows: the query heads that share a key-value head are packed with their
// tokens into tiles of 128 rows (128 / group tokens each), so a tile of keys
// is fetched once for all of them; a work item is two such row tiles and some
// key tiles.
//
// A CTA (one per SM, it keeps taking items) has five roles:
//   warp 0     TMA loads: the item's queries, then key and value tiles into a
//              ring of four;
//   warp 1     tcgen05.mma: S_i = Q_i K^T into tensor memory, O_i += P_i V
//              with P_i read from tensor memory, for the row tiles i = 0, 1 in
//              turn: while one tile's softmax runs, the other's products do;
//   warp 2     looks through the value tiles that are hidden from some rows
//              (see below);
//   warp 3     deals the items;
//   warps 4-7 and 8-11  softmax of row tile 0 and 1: a thread has a row, reads
//              its 128 scores, writes its probabilities over them (16 bits
//              each), and at the item's end scales O and stores it.
// Tensor memory: S_0, S_1, O_0, O_1, 128 fp32 columns each: all of it.
//
// Hidden values: a probability of 0 times a value that is infinite or NaN
// would be NaN, and the last tiles of an item hold values that some rows may
// not see.  Warp 2 looks for such values there; where it finds one it puts 0
// in its place and notes its column and kind, from which the rows that do see
// it set their result.
//
// A mode M says which items there are, where their rows, keys and values lie,
// what each row sees, and where its result goes:
//   Args (with pack, per_tile, c, err), Work (with n0, n1: key tiles of the
//   two row tiles, and hidden: the first that some row does not see whole),
//   Dealer, Loader, Row, Wild.
// kSplit: an item is one row tile, and row tile 1 the same rows again with
// every other tile of keys; row tile 0's threads add the two up.
//
// Every wait is bounded (NS_FLAG_TIMEOUT).
//
// What bounds it: a tile of keys costs 2048 tensor-core cycles for the two row
// tiles, and the softmax of 128 scores a thread nearly as many issue slots, so
// both have to run all the time.  16381 tokens of 32 heads on 8, 128 columns,
// bf16 take 1.40 ms, 1.57 PFLOP/s (0.83 of the measured cuBLAS burst); with the
// exponentials left out the same kernel took 1.20 ms.  What other forms took
// there: two threads to a row (640 threads) 1.76 ms, output warps of their own
// 1.43 ms, a softmax of half tiles in 128 registers 1.50 ms, two threads that
// issue products 1.42 to 1.76 ms, a ring of three tiles 1.49 ms, of five 1.44;
// a maximum of the first 64 keys alone, one loop for both halves 1.44 ms.
#pragma once

#include "ns_attn_tile.cuh"
#include "ns_internal.cuh"
#include "ns_ops.cuh"
#include "ns_umma_ptx.cuh"

namespace ns {
namespace fa {

using attn::Type;
using attn::ex2;
using attn::kNegInf;

constexpr int kThreads = 384;
constexpr int kRing = 4;             // key or value tiles in flight: keys in the even places
static_assert(kRing % 2 == 0, "keys and values take turns");
constexpr int kKeys = 128;           // keys of a tile
constexpr int kHalf = 128 * 128;     // bytes of 128 rows of 64 elements
constexpr float kLimit = 32768.f;    // a sum of 64 probabilities above this says that m is too low
constexpr int kChecks = 4;           // value tiles looked through ahead of the product
constexpr int kMissingTiles = 4;     // key tiles whose missing keys are kept (see there)
constexpr int kWorkReaders = 11;     // loads, products, hidden values, and the eight softmax warps
constexpr int kWorkBytes = 48;

template <typename T>
constexpr float kOffset = 0.f;
template <>
constexpr float kOffset<__half> = 6.f;

template <int D, typename M>
struct Smem {
  static constexpr int kTile = D / 64 * kHalf;  // a row tile of queries, or a key or value tile
  static constexpr int kQ = 0, kKV = 2 * kTile, kOut = kKV + kRing * kTile, kMisc = kOut + 8 * 32 * M::kStageRow;
  // barriers, 8 bytes each
  static constexpr int kKvFull = kMisc, kKvEmpty = kKvFull + 8 * kRing, kQFull = kKvEmpty + 8 * kRing,
                       kQEmpty = kQFull + 8, kSFull = kQEmpty + 8, kPFull = kSFull + 16, kPvHalf = kPFull + 32,
                       kOFull = kPvHalf + 16, kOEmpty = kOFull + 16, kCheck = kOEmpty + 16,
                       kMerge = kCheck + 8 * kChecks, kWFull = kMerge + 16, kWEmpty = kWFull + 16, kSlot = kWEmpty + 16, kWork = kSlot + 16,
                       kWildAny = kWork + 2 * kWorkBytes, kMissing = kWildAny + 16,
                       kWild = kMissing + 4 * kMissingTiles,
                       kEnd = kWild + 2 * (int)sizeof(typename M::Wild);
  static constexpr int kBytes = kEnd + 1024;  // the base is rounded up to 1024 bytes
  static_assert(kBytes <= 232448, "shared memory of a CTA");
};

// Key tiles of an item: both row tiles see them in turn, or (M::kSplit) they
// are one row tile twice, with every other key tile each.
template <typename M>
__device__ __forceinline__ int key_tiles(const typename M::Work &w) {
  return M::kSplit ? w.n0 + w.n1 : max(w.n0, w.n1);
}

template <typename Work>
__device__ __forceinline__ bool get_work(uint32_t base, int full, const uint8_t *g, int work_off, int i, Work &w,
                                         uint32_t *err) {
  static_assert(sizeof(Work) <= kWorkBytes, "a work slot");
  if (!umma::inline_wait(base + full + 8 * (i & 1), (i >> 1) & 1, err)) return false;
  w = *reinterpret_cast<const Work *>(g + work_off + kWorkBytes * (i & 1));
  return w.n0 > 0;
}

// The keys that eight bits say are there no page for, eight keys a bit.
__device__ __forceinline__ uint64_t eights(uint32_t bits) {
  const uint64_t x = (bits & 0xffu) * 0x0101010101010101ull & 0x8040201008040201ull;  // byte e: whether bit e is set
  return (uint64_t)__vcmpne4((uint32_t)(x >> 32), 0u) << 32 | __vcmpne4((uint32_t)x, 0u);
}

// Where the value of column d, key r of a value tile lies in it.
__device__ __forceinline__ int value_at(int r, int d) {
  return (d >> 6) * kHalf + r * 128 + ((((d & 63) >> 3) ^ (r & 7)) << 4) + (d & 7) * 2;
}

// -inf where bit e of `sees` is not set, scores from, from + 1, ... of a register array
#define NS_FA_MASK(s, from, sees)                                             \
  _Pragma("unroll") for (int e_ = 0; e_ < 64; ++e_) {                         \
    if (!(((sees) >> e_) & 1)) s[(from) + e_] = 0xff800000u;                  \
  }

template <typename T, int D, typename M>
__global__ void __launch_bounds__(kThreads, 1)
    attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ typename M::Args a) {
  using L = Smem<D, M>;
  using Work = typename M::Work;
  using Wild = typename M::Wild;
  constexpr bool kBf16 = sizeof(T) == 2 && kOffset<T> == 0.f;
  constexpr uint32_t kIdS = umma::idesc(kBf16, kKeys, false), kIdO = umma::idesc(kBf16, D, true);
  extern __shared__ uint8_t smem_raw[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t *g = smem_raw + (base - raw);
  uint32_t *err = a.err;

  if (tid == 0) {
    for (int s = 0; s < kRing; ++s) {
      mbar_init(base + L::kKvFull + 8 * s, 1);
      mbar_init(base + L::kKvEmpty + 8 * s, 1 + (s & 1));  // the products; values: and the check
    }
    mbar_init(base + L::kQFull, 1);
    mbar_init(base + L::kQEmpty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(base + L::kSFull + 8 * i, 1);
      mbar_init(base + L::kPFull + 16 * i, 128);      // the probabilities of the first 64 keys
      mbar_init(base + L::kPFull + 16 * i + 8, 128);  // and of the others
      mbar_init(base + L::kPvHalf + 8 * i, 1);        // the product with the first 64 keys is over
      mbar_init(base + L::kOFull + 8 * i, 1);
      mbar_init(base + L::kOEmpty + 8 * i, 128);
      mbar_init(base + L::kWFull + 8 * i, 1);
      mbar_init(base + L::kWEmpty + 8 * i, kWorkReaders);
    }
    mbar_init(base + L::kMerge, 128);
    for (int i = 0; i < kChecks; ++i) mbar_init(base + L::kCheck + 8 * i, 1);
    mbar_fence_init();
    umma::prefetch_map(&tmQ);
    umma::prefetch_map(&tmK);
    umma::prefetch_map(&tmV);
  }
  if (warp == 1) umma::alloc(base + L::kSlot, 512);
  umma::fence_before();
  __syncthreads();
  umma::fence_after();
  const uint32_t tmem = *reinterpret_cast<uint32_t *>(g + L::kSlot);
  if (M::kParts) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join waits for this grid

  // registers: 128 threads x 88 + 256 x 208 = 384 x 168, the launch's own
  if (warp < 4)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  if (warp == 0) {  // loads
    Work w;
    typename M::Loader loader;
    int it = 0;  // ring position: K0 V0 K1 V1 ... over all items
    // Key tile x (over all items) leaves its missing keys in word x % kMissingTiles.  They are read before the
    // softmax hands over tile x's probabilities, scores of tile x + 1 are issued after that, and key tile x + 3 is
    // loaded after those are over: a word is not written again before it was read.
    static_assert(!M::kParts || kMissingTiles > kRing / 2, "the words outlive their tiles");
    uint32_t *missing = reinterpret_cast<uint32_t *>(g + L::kMissing);
    bool ok = true;
    auto wait = [&](uint32_t bar, int phase) {
      return __all_sync(0xffffffffu, umma::inline_wait(base + bar, phase & 1, err));
    };
    int i = 0;
    for (; ok; ++i) {
      const bool more = get_work(base, L::kWFull, g, L::kWork, i, w, err);
      if (!__all_sync(0xffffffffu, more)) break;
      loader.begin(a, w, lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(base + L::kWEmpty + 8 * (i & 1));
      if (i > 0 && !(ok = wait(L::kQEmpty, i - 1))) break;
      const int tiles = w.n1 > 0 ? 2 : 1, n = key_tiles<M>(w);
      if (lane == 0) {
        mbar_expect_tx(base + L::kQFull, tiles * a.pack * a.per_tile * D * 2);
        for (int t = 0; t < tiles; ++t)
          for (int h = 0; h < D / 64; ++h)
            loader.queries(a, w, M::kSplit ? 0 : t, h, base + L::kQ + t * L::kTile + h * kHalf, &tmQ, base + L::kQFull);
      }
      for (int j = 0; j < n && ok; ++j) {
        for (int kv = 0; kv < 2; ++kv, ++it) {
          const int s = it % kRing;
          if (it >= kRing && !(ok = wait(L::kKvEmpty + 8 * s, it / kRing - 1))) break;
          loader.template keys<D>(a, w, j, kv, base + L::kKV + s * L::kTile, kv ? &tmV : &tmK,
                                  base + L::kKvFull + 8 * s, lane, missing + it / 2 % kMissingTiles);
        }
      }
    }
    // nothing may still be landing in shared memory when the CTA leaves
    if (i > 0) wait(L::kQFull, i - 1);
    for (int q = it > kRing ? it - kRing : 0; q < it; ++q) wait(L::kKvFull + 8 * (q % kRing), q / kRing);
  } else if (warp == 1) {
    if (umma::elect()) {  // products
      // A product that waits for its operands leaves the tensor cores idle: only one or two are queued behind
      // the running one.  So each group looks whether the next one's barrier is over before its own last products.
      Work w;
      int sl = 0, ph = 0, checked = 0;  // ring slot and phase of the next tile
      int pos = 0;                      // ring position (M::kSplit)
      int np[2] = {0, 0}, no[2] = {0, 0};  // probabilities awaited, items begun, of each row tile
      bool ok = true, begun = false;
      auto next = [&]() {
        if (++sl == kRing) sl = 0, ph ^= 1;
      };
      auto peek = [&](uint32_t bar, int phase) { return umma::test_wait(base + bar, phase & 1); };
      auto wait = [&](uint32_t bar, int phase, bool seen = false) {
        if (!seen && ok) ok = umma::inline_wait(base + bar, phase & 1, err);
        umma::fence_after();
      };
      // S_t = Q_t K^T; the look at the next barrier comes before the last two products
      auto scores = [&](int t, int slot, uint32_t bar, int phase) {
        const uint64_t A = umma::desc_k(base + L::kQ + t * L::kTile), B = umma::desc_k(base + L::kKV + slot * L::kTile);
        bool seen = false;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          if (kk == D / 16 - 2) seen = peek(bar, phase);
          const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;  // in the descriptors' 16-byte units
          umma::mma_ss(tmem + t * 128, A + off, B + off, kIdS, kk != 0);
        }
        umma::commit(base + L::kSFull + 8 * t);
        return seen;
      };
      // O_t += P_t V, 64 keys
      auto values = [&](int t, int slot, int h, bool more, uint32_t bar, int phase) {
        const uint64_t V = umma::desc_mn(base + L::kKV + slot * L::kTile, kHalf);
        bool seen = false;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if (kk == 2) seen = peek(bar, phase);
          umma::mma_ts(tmem + 256 + t * 128, tmem + t * 128 + (h * 4 + kk) * 8, V + (h * 4 + kk) * (2048 >> 4), kIdO,
                       more || h > 0 || kk > 0);
        }
        return seen;
      };
      for (int i = 0; get_work(base, L::kWFull, g, L::kWork, i, w, err); ++i) {
        mbar_arrive(base + L::kWEmpty + 8 * (i & 1));
        const int n0 = w.n0, n1 = w.n1, n = max(n0, n1), hidden = w.hidden;
        wait(L::kQFull, i);
        if constexpr (M::kSplit) {
          // Key tile j goes to the scores and the accumulator of j & 1.
          const int first = pos, tiles = n0 + n1;
          auto slot = [&](int x) { return (first + x) % kRing; };
          auto filled = [&](int x) { wait(L::kKvFull + 8 * slot(x), (first + x) / kRing); };
          for (int j = 0; j < min(tiles, 2); ++j) {
            filled(2 * j);
            if (!ok) break;
            scores(j, slot(2 * j), L::kQFull, 0);
            umma::commit(base + L::kKvEmpty + 8 * slot(2 * j));
            if (j + 1 == tiles || (j == 1 && tiles == 2)) umma::commit(base + L::kQEmpty);
          }
          begun = true;
          for (int j = 0; j < tiles && ok; ++j) {
            const int t = j & 1;
            filled(2 * j + 1);
            if (j >= hidden) {
              wait(L::kCheck + 8 * (checked % kChecks), checked / kChecks);
              ++checked;
            }
            if (j < 2 && no[t] > 0) wait(L::kOEmpty + 8 * t, no[t] - 1);
            wait(L::kPFull + 16 * t, np[t]);
            if (!ok) break;
            const bool seen = values(t, slot(2 * j + 1), 0, j > 1, L::kPFull + 16 * t + 8, np[t]);
            umma::commit(base + L::kPvHalf + 8 * t);
            wait(L::kPFull + 16 * t + 8, np[t], seen);
            if (!ok) break;
            values(t, slot(2 * j + 1), 1, j > 1, L::kQFull, 0);
            ++np[t];
            if (j + 2 >= tiles) {
              umma::commit(base + L::kOFull + 8 * t);
              ++no[t];
            }
            umma::commit(base + L::kKvEmpty + 8 * slot(2 * j + 1));
            if (j + 2 < tiles) {
              filled(2 * j + 4);
              if (!ok) break;
              scores(t, slot(2 * j + 4), L::kQFull, 0);
              umma::commit(base + L::kKvEmpty + 8 * slot(2 * j + 4));
              if (j + 3 == tiles) umma::commit(base + L::kQEmpty);
            }
          }
          pos += 2 * tiles;
          sl = pos % kRing, ph = pos / kRing & 1;
          if (!ok) break;
          continue;
        }
        wait(L::kKvFull + 8 * sl, ph);
        if (!ok) break;
        scores(0, sl, L::kQFull, 0);
        if (n1 > 0) scores(1, sl, L::kQFull, 0);
        umma::commit(base + L::kKvEmpty + 8 * sl);
        if (n == 1) umma::commit(base + L::kQEmpty);
        next();
        begun = true;
        bool seen_p = false;  // the first half of row tile 0's probabilities
        for (int j = 0; j < n && ok; ++j) {
          const int sv = sl, pv = ph;
          next();
          const int sk = sl, pk = ph;
          const bool more = j + 1 < n;
          if (more) next();
          wait(L::kKvFull + 8 * sv, pv);
          if (j >= hidden) {
            wait(L::kCheck + 8 * (checked % kChecks), checked / kChecks);
            ++checked;
          }
          bool seen_k = false, seen = seen_p, have_k = false;
          seen_p = false;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int nt = t ? n1 : n0;
            if (ok && j < nt) {
              if (j == 0 && no[t] > 0) wait(L::kOEmpty + 8 * t, no[t] - 1);
              wait(L::kPFull + 16 * t, np[t], seen);
              if (!ok) break;
              seen = values(t, sv, 0, j > 0, L::kPFull + 16 * t + 8, np[t]);
              umma::commit(base + L::kPvHalf + 8 * t);
              wait(L::kPFull + 16 * t + 8, np[t], seen);
              if (!ok) break;
              seen = values(t, sv, 1, j > 0, L::kKvFull + 8 * sk, pk);
              if (!have_k) seen_k = seen;
              seen = false;
              ++np[t];
              if (j + 1 == nt) {
                umma::commit(base + L::kOFull + 8 * t);
                ++no[t];
              }
            }
            if (ok && j + 1 < nt) {
              if (!have_k) wait(L::kKvFull + 8 * sk, pk, seen_k);
              have_k = true;
              if (!ok) break;
              seen = scores(t, sk, L::kPFull + 16 * (1 - t), np[1 - t]);
              if (t == 1) seen_p = seen && j + 1 < n0;
            }
          }
          if (!ok) break;
          umma::commit(base + L::kKvEmpty + 8 * sv);
          if (more) {
            umma::commit(base + L::kKvEmpty + 8 * sk);
            if (j + 2 == n) umma::commit(base + L::kQEmpty);
          }
        }
        if (!ok) break;
      }
      // the last commit has arrived before the CTA leaves
      if (ok && begun) {
        const int last = sl ? sl - 1 : kRing - 1;
        wait(L::kKvEmpty + 8 * last, sl ? ph : ph ^ 1);
      }
    }
  } else if (warp == 2) {  // hidden values
    Work w;
    int it = 0, checked = 0;
    bool ok = true;
    for (int i = 0; ok; ++i) {
      const bool more = get_work(base, L::kWFull, g, L::kWork, i, w, err);
      if (!__all_sync(0xffffffffu, more)) break;
      Wild *wild = reinterpret_cast<Wild *>(g + L::kWild) + (i & 1);
      volatile int *any = reinterpret_cast<volatile int *>(g + L::kWildAny) + (i & 1);
      const int n = key_tiles<M>(w);
      bool reset = false;
      for (int j = 0; j < n && ok; ++j) {
        // Every value tile passes here, so that the barrier's phase is this tile's: a slot is not filled again before
        // it did.
        const int pos = it + 2 * j + 1, s = pos % kRing;
        ok = __all_sync(0xffffffffu, umma::inline_wait(base + L::kKvFull + 8 * s, (pos / kRing) & 1, err));
        if (!ok) break;
        if (j < w.hidden) {
          if (lane == 0) mbar_arrive(base + L::kKvEmpty + 8 * s);
          continue;
        }
        uint8_t *tile = g + L::kKV + s * L::kTile;
        bool touched = M::template clear<T, D>(a, w, j, tile, lane);
        if (__any_sync(0xffffffffu, attn::wild_pieces<T>(base + L::kKV + s * L::kTile, L::kTile / 16, lane, kWarp))) {
          if (!reset) {
            for (int d = lane; d < D; d += kWarp) wild->none(d);
            reset = true;
          }
          for (int d = lane; d < D; d += kWarp) {
            for (int r = 0; r < kKeys; ++r) {
              T *v = reinterpret_cast<T *>(tile + value_at(r, d));
              const float x = static_cast<float>(*v);
              if (!(fabsf(x) < __int_as_float(0x7f800000)) && wild->note(w, j, r, d, x)) *v = static_cast<T>(0.f);
            }
          }
          if (lane == 0) *any = 1;
          touched = true;
        }
        if (__any_sync(0xffffffffu, touched))
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the zeros, for the tensor core
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(base + L::kCheck + 8 * (checked % kChecks));
          mbar_arrive(base + L::kKvEmpty + 8 * s);
        }
        ++checked;
      }
      it += 2 * n;
      __syncwarp();
      if (lane == 0) mbar_arrive(base + L::kWEmpty + 8 * (i & 1));
    }
  } else if (warp == 3) {  // the items
    typename M::Dealer dealer;
    dealer.begin(a, blockIdx.x, gridDim.x);
    for (int i = 0;; ++i) {
      const Work w = dealer.next(a);
      if (i >= 2 &&
          !__all_sync(0xffffffffu, umma::inline_wait(base + L::kWEmpty + 8 * (i & 1), ((i >> 1) - 1) & 1, err)))
        break;
      if (lane == 0) {
        *reinterpret_cast<Work *>(g + L::kWork + kWorkBytes * (i & 1)) = w;
        *(reinterpret_cast<volatile int *>(g + L::kWildAny) + (i & 1)) = 0;
        mbar_arrive(base + L::kWFull + 8 * (i & 1));
      }
      __syncwarp();
      if (w.n0 == 0) break;
    }
  } else {  // softmax of row tile t
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int t = (warp - 4) >> 2, wq = warp & 3;
    const int r = wq * 32 + lane;
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tmem + t * 128 + lanes, tO = tmem + 256 + t * 128 + lanes;
    const uint64_t c2 = umma::pack2(a.c, a.c);
    Work w;
    int ns = 0, items = 0;  // scores awaited, items of this row tile begun
    int merged = 0;         // items whose two accumulators were added up (M::kSplit)
    int passed = 0;         // key tiles of the items before (M::kParts)
    bool ok = true;
    for (int i = 0; ok; ++i) {
      const bool more = get_work(base, L::kWFull, g, L::kWork, i, w, err);
      if (!__all_sync(0xffffffffu, more)) break;
      const int nt = t ? w.n1 : w.n0;
      typename M::Row row;
      row.begin(a, w, M::kSplit ? 0 : t, r);
      const bool live = row.live;
      float m = kNegInf, l = 0.f;
      for (int j = 0; j < nt; ++j, ++ns) {
        ok = __all_sync(0xffffffffu, umma::inline_wait(base + L::kSFull + 8 * t, ns & 1, err));
        if (!ok) break;
        umma::fence_after();
        const int key_tile = M::kSplit ? 2 * j + t : j;
        uint32_t s[128], p[32];
        float sum;
        // (only a cache's pages may be missing)
        const uint32_t missing =
            M::kParts ? *(reinterpret_cast<volatile uint32_t *>(g + L::kMissing) + (passed + j) % kMissingTiles) : 0u;
        const bool masked = key_tile >= w.hidden || (M::kParts && missing != 0);
        auto mask = [&](int from) {  // keys that the row does not see, among 64
          uint64_t sees = row.sees(w, key_tile, from);
          if (M::kParts && missing) sees &= ~eights(missing >> (from / 8));
          NS_FA_MASK(s, from, sees)
        };
        auto most = [&](int from) {
          float mx[2] = {kNegInf, kNegInf};
#pragma unroll
          for (int e = from; e < from + 64; e += 4) {
            mx[0] = fmaxf(fmaxf(mx[0], __uint_as_float(s[e])), __uint_as_float(s[e + 1]));
            mx[1] = fmaxf(fmaxf(mx[1], __uint_as_float(s[e + 2])), __uint_as_float(s[e + 3]));
          }
          return fmaxf(mx[0], mx[1]) * a.c;
        };
        // the probabilities of 64 keys with the m that there is, and their sum
        auto probabilities = [&](int from) {
          const float shift = kOffset<T> - (m == kNegInf ? 0.f : m);
          const uint64_t shift2 = umma::pack2(shift, shift);
          uint64_t sum2[2] = {0, 0};
#pragma unroll
          for (int e = 0; e < 64; e += 2) {
            float x, y;
            umma::unpack2(umma::fma2(umma::pack2(__uint_as_float(s[from + e]), __uint_as_float(s[from + e + 1])), c2,
                                     shift2),
                          x, y);
            x = ex2(x), y = ex2(y);
            p[e / 2] = Type<T>::pack(x, y);
            sum2[(e >> 1) & 1] = umma::add2(sum2[(e >> 1) & 1], umma::pack2(x, y));
          }
          float x, y;
          umma::unpack2(umma::add2(sum2[0], sum2[1]), x, y);
          sum = x + y;
        };
        // where the sum says that m is too low for some row: its new m, and everything before in terms of it
        auto raise = [&](bool row, float top) {
          const float was = m;
          if (row) m = fmaxf(m, top);
          const float f = row ? ex2(was - (m == kNegInf ? 0.f : m)) : 1.f;
          l *= f;
#pragma unroll 1
          for (int q = 0; q < D / 16; ++q) {
            uint32_t o[16];
            umma::ld16(tO + q * 16, o);
            umma::wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            umma::st16(tO + q * 16, o);
          }
        };
        umma::ld32(tS, s);
        umma::ld32(tS + 32, s + 32);
        umma::wait_ld();
        umma::ld32(tS + 64, s + 64);
        umma::ld32(tS + 96, s + 96);
        if (masked) mask(0);
        bool whole = false;  // the second half has come
        if (j == 0) {
          umma::wait_ld();
          if (masked) mask(64);
          whole = true;
          m = fmaxf(most(0), most(64));
        }
        probabilities(0);
        if (j > 0) {
          const bool low = live && (sum > kLimit || m == kNegInf);
          if (__any_sync(0xffffffffu, low)) {
            umma::wait_ld();
            if (masked) mask(64);
            whole = true;
            // the accumulator is still: S of this tile came after the last product into it
            raise(low, fmaxf(most(0), most(64)));
            probabilities(0);
          }
        }
        umma::st32(tS, p);
        umma::wait_st();
        umma::fence_before();
        mbar_arrive(base + L::kPFull + 16 * t);
        l += sum;
        if (!whole) {
          umma::wait_ld();
          if (masked) mask(64);
        }
        probabilities(64);
        if (j > 0) {
          const bool low = live && sum > kLimit;
          if (__any_sync(0xffffffffu, low)) {
            // the product with the first half must be over before the accumulator is touched
            ok = __all_sync(0xffffffffu, umma::inline_wait(base + L::kPvHalf + 8 * t, ns & 1, err));
            umma::fence_after();
            raise(low, most(64));
            probabilities(64);
          }
        }
        umma::st32(tS + 32, p);
        l += sum;
        umma::wait_st();
        umma::fence_before();
        mbar_arrive(base + L::kPFull + 16 * t + 8);
        if (!ok) break;
      }
      if (!ok) break;
      passed += key_tiles<M>(w);
      if (nt > 0) {
        ok = __all_sync(0xffffffffu, umma::inline_wait(base + L::kOFull + 8 * t, items & 1, err));
        if (!ok) break;
        ++items;
        umma::fence_after();
        float f0 = 1.f, f1 = 0.f;
        if constexpr (M::kSplit) {
          float2 *hand = reinterpret_cast<float2 *>(g + L::kOut + (4 + wq) * 32 * M::kStageRow) + lane;
          if (t == 1) {  // row tile 0's thread of the same row has the rest of it
            *hand = make_float2(m, l);
            mbar_arrive(base + L::kMerge);
          } else if (w.n1 > 0) {
            ok = __all_sync(0xffffffffu, umma::inline_wait(base + L::kMerge, merged & 1, err)) &&
                 __all_sync(0xffffffffu, umma::inline_wait(base + L::kOFull + 8, merged & 1, err));
            if (!ok) break;
            ++merged;
            umma::fence_after();
            const float2 o = *hand;
            const float top = fmaxf(m, o.x), safe = top == kNegInf ? 0.f : top;
            f0 = ex2(m - safe), f1 = ex2(o.x - safe);
            l = l * f0 + o.y * f1;
            m = top;
          }
        }
        const bool wild = *(reinterpret_cast<volatile int *>(g + L::kWildAny) + (i & 1)) != 0;
        const Wild *wd = reinterpret_cast<const Wild *>(g + L::kWild) + (i & 1);
        // some columns at a time through shared memory, so that a store covers whole lines of a few rows
        constexpr int kRow = M::kStageRow, kChunks = kRow / 16, kWords = kRow / 4;
        uint8_t *stage = g + L::kOut + (warp - 4) * 32 * kRow;
        auto place = [&](int r, int c) { return stage + r * kRow + ((c ^ ((r / (8 / kChunks)) % kChunks)) << 4); };
        auto flush = [&](long long to, int off) {  // the staged 32 rows to their addresses `to` (0: none) + off
          __syncwarp();
#pragma unroll
          for (int e = 0; e < kChunks; ++e) {
            const int r = e * (32 / kChunks) + lane / kChunks;
            const long long at = __shfl_sync(0xffffffffu, to, r);
            const uint4 x = *reinterpret_cast<const uint4 *>(place(r, lane % kChunks));
            if (at) *reinterpret_cast<uint4 *>(at + off + lane % kChunks * 16) = x;
          }
          __syncwarp();
        };
        auto fixed = [&](uint32_t o, int d) {  // a row that sees a value that is not finite
          const int kind = wd->seen(row, d);
          return kind == 0 ? o : kind == 1 ? 0x7fffffffu : __float_as_uint(__uint_as_float(o) + (kind == 2 ? -kNegInf : kNegInf));
        };
        auto drained = [&]() {  // the accumulator may be written again
          umma::fence_before();
          mbar_arrive(base + L::kOEmpty + 8 * t);
          if (M::kSplit && w.n1 > 0) mbar_arrive(base + L::kOEmpty + 8);
        };
        if (M::kSplit && t == 1) {
        } else if (!M::kParts || w.slot < 0) {
          const float inv = l == 0.f ? 0.f : 1.f / l;
          const long long to = live ? reinterpret_cast<long long>(static_cast<T *>(a.out) + row.at * D) : 0;
#pragma unroll 1
          for (int q = 0; q < D / (2 * kWords); ++q) {
            uint32_t o[2 * kWords];
#pragma unroll
            for (int e = 0; e < 2 * kWords; e += 32) umma::ld32(tO + q * 2 * kWords + e, o + e);
            if constexpr (M::kSplit) {
              if (w.n1 > 0) {
                uint32_t o1[2 * kWords];
#pragma unroll
                for (int e = 0; e < 2 * kWords; e += 32) umma::ld32(tO + 128 + q * 2 * kWords + e, o1 + e);
                umma::wait_ld();
#pragma unroll
                for (int e = 0; e < 2 * kWords; ++e)
                  o[e] = __float_as_uint(__uint_as_float(o[e]) * f0 + __uint_as_float(o1[e]) * f1);
              }
            }
            umma::wait_ld();
            if (q + 1 == D / (2 * kWords)) drained();
            if (wild) {
#pragma unroll
              for (int e = 0; e < 2 * kWords; ++e) o[e] = fixed(o[e], q * 2 * kWords + e);
            }
#pragma unroll
            for (int e = 0; e < 2 * kWords; e += 8)
              *reinterpret_cast<uint4 *>(place(lane, e >> 3)) =
                  make_uint4(Type<T>::pack(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv),
                             Type<T>::pack(__uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv),
                             Type<T>::pack(__uint_as_float(o[e + 4]) * inv, __uint_as_float(o[e + 5]) * inv),
                             Type<T>::pack(__uint_as_float(o[e + 6]) * inv, __uint_as_float(o[e + 7]) * inv));
            flush(to, q * kRow);
          }
          if (live && a.lse) a.lse[row.at] = l == 0.f ? kNegInf : (m - kOffset<T> + log2f(l)) * attn::kLn2;
        } else {  // a part: fp32 sums for the join, column by column (32 rows of a column are one line)
          float *to = a.part_o + (int64_t)w.slot * D * 256 + t * 128 + r;
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            umma::ld32(tO + q * 32, o);
            umma::wait_ld();
            if (q + 1 == D / 32) drained();
            if (wild) {
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = fixed(o[e], q * 32 + e);
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) to[(q * 32 + e) * 256] = __uint_as_float(o[e]);
          }
          a.part_ml[w.slot * 256 + t * 128 + r] = make_float2(m, l);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(base + L::kWEmpty + 8 * (i & 1));
    }
  }
  umma::fence_before();
  __syncthreads();
  umma::fence_after();
  if (warp == 1) umma::dealloc(tmem, 512);
}

}  // namespace fa
}  // namespace ns
