// Causal attention over whole packed prompts, on the 5th-generation tensor
// cores.
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
// of the second product (l sums it unrounded).  fp16 probabilities are kept
// 2^6 times larger: within fp16's range under the bound on the sum, and 2^-30
// of the largest is not lost.
//
// Rows: the query heads that share a key-value head are packed with their
// tokens into tiles of 128 rows (128 / group tokens each), so a tile of keys
// is fetched once for all of them; a work item is two such row tiles.
//
// A CTA (one per SM, it keeps taking items, longest first) has five roles:
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
// not see: later tokens, and tokens of the next sequence.  Warp 2 looks for
// such values there; where it finds one it puts 0 in its place and notes, per
// column, the first position of each kind, from which the rows that do see it
// set their result.
//
// Every wait is bounded (NS_FLAG_TIMEOUT).
#include "ns_attn_tile.cuh"
#include "ns_internal.cuh"
#include "ns_ops.cuh"
#include "ns_umma_ptx.cuh"

namespace ns {
namespace {

using attn::Type;
using attn::ex2;
using attn::kNegInf;

constexpr int kFaThreads = 384;
constexpr int kFaRing = 4;       // key or value tiles in flight
constexpr int kFaKeys = 128;     // keys of a tile
constexpr int kFaHalf = 128 * 128;  // bytes of 128 rows of 64 elements
constexpr float kFaLimit = 32768.f;  // a sum of 64 probabilities above this says that m is too low
constexpr int kFaChecks = 4;     // value tiles looked through ahead of the product

template <typename T>
constexpr float kFaOffset = 0.f;
template <>
constexpr float kFaOffset<__half> = 6.f;

struct Work {
  int seq0, len;     // the sequence's first token and its length
  int tok0;          // first token of row tile 0
  int unit;          // query heads unit * pack .. + pack - 1
  int n0, n1;        // key tiles of the row tiles (0: no such row tile); n0 = 0: no more work
};
struct Wild {  // first positions of values that are not finite, from the first looked-through tile on
  uint16_t nan[128], pos[128], neg[128];
};
constexpr uint16_t kNever = 0xffff;

template <int D>
struct FaSmem {
  static constexpr int kTile = D / 64 * kFaHalf;  // a row tile of queries, or a key or value tile
  static constexpr int kQ = 0, kKV = 2 * kTile, kOut = kKV + kFaRing * kTile, kMisc = kOut + 8 * 4096;
  // barriers, 8 bytes each
  static constexpr int kKvFull = kMisc, kKvEmpty = kKvFull + 8 * kFaRing, kQFull = kKvEmpty + 8 * kFaRing,
                       kQEmpty = kQFull + 8, kSFull = kQEmpty + 8, kPFull = kSFull + 16, kPvHalf = kPFull + 32, kOFull = kPvHalf + 16,
                       kOEmpty = kOFull + 16, kCheck = kOEmpty + 16, kWFull = kCheck + 8 * kFaChecks,
                       kWEmpty = kWFull + 16, kSlot = kWEmpty + 16, kWork = kSlot + 16, kWildAny = kWork + 2 * 32,
                       kWild = kWildAny + 16, kEnd = kWild + 2 * (int)sizeof(Wild);
  static constexpr int kBytes = kEnd + 1024;  // the base is rounded up to 1024 bytes
};
static_assert(FaSmem<128>::kBytes <= 232448, "shared memory of a CTA");
constexpr int kWorkReaders = 11;  // producer, MMA, checker, and the eight softmax warps

struct FaArgs {
  const int32_t *cu;
  int32_t tokens, n_seqs, max_len, q_heads, group, pack, per_tile, units;
  float c;  // scale * log2(e)
  void *out;
  float *lse;
  uint32_t *err;
};

// The position of an item's first value tile that is hidden from some rows.
__device__ __forceinline__ int first_hidden_tile(const Work &w) { return (w.tok0 + 1) / kFaKeys; }

__device__ __forceinline__ bool get_work(uint32_t base, int full, const uint8_t *g, int work_off, int i, Work &w,
                                         uint32_t *err) {
  if (!umma::inline_wait(base + full + 8 * (i & 1), (i >> 1) & 1, err)) return false;
  w = *reinterpret_cast<const Work *>(g + work_off + 32 * (i & 1));
  return w.n0 > 0;
}

// A sequence's first token and its length (0 where its bounds are invalid).
__device__ __forceinline__ int sequence(const FaArgs &a, int s, int &len) {
  const int t0 = a.cu[s], t1 = a.cu[s + 1];
  len = t0 < 0 || t1 < t0 || t1 > a.tokens ? 0 : min(t1 - t0, a.max_len);
  return t0;
}

// The items of CTA `cta` in order (a whole warp).  All items, longest first,
// are in one line: block x of tokens (from the last), sequence, unit; the CTAs
// take turns forth and back, so each gets a like share of every length.  A
// lane keeps the longest of its 32nd of the sequences, so at each x only
// groups that reach it are looked at.
struct Dealer {
  int cta, ctas, lane, block, size;
  int most;                // blocks of the lane's group's longest sequence
  int x, s;                // where the line is: block, and the lane's sequence
  uint32_t groups, live;   // groups left at x; sequences of the 32 at s that reach x
  int t0, len;             // of the lane's sequence
  int before, here;        // items before these 32 sequences, and of them
  int turn, mine;          // the CTA's next item

  __device__ __forceinline__ void begin(const FaArgs &a, int cta_, int ctas_) {
    cta = cta_, ctas = ctas_, lane = threadIdx.x & 31, block = 2 * a.per_tile;
    size = (a.n_seqs + 1023) / 1024 * 32;
    most = 0;
    for (int q = lane * size; q < min(a.n_seqs, (lane + 1) * size); ++q) {
      int n;
      sequence(a, q, n);
      if (cta == 0 && a.cu[q + 1] - a.cu[q] != n) set_flag(a.err, NS_FLAG_BAD_SEQ);
      most = max(most, (n + block - 1) / block);
    }
    x = __reduce_max_sync(0xffffffffu, most);
    groups = 0, s = 0, before = 0, here = 0, turn = 0, mine = cta;
  }
  // the next 32 sequences that reach x, or some of the next lower x; false at the end
  __device__ __forceinline__ bool advance(const FaArgs &a) {
    before += here;
    const int g0 = groups ? (__ffs(groups) - 1) * size : 0;
    if (groups && s - lane + 32 < g0 + size) {
      s += 32;
    } else {
      groups &= groups - 1;
      while (groups == 0) {
        if (--x < 0) return false;
        groups = __ballot_sync(0xffffffffu, most > x);
      }
      s = (__ffs(groups) - 1) * size + lane;
    }
    t0 = len = 0;
    if (s < a.n_seqs) t0 = sequence(a, s, len);
    live = __ballot_sync(0xffffffffu, len > x * block);
    here = __popc(live) * a.units;
    return true;
  }
  __device__ __forceinline__ Work next(const FaArgs &a) {
    Work w{};
    while (mine >= before + here)
      if (!advance(a)) return w;
    const int from = __fns(live, 0, (mine - before) / a.units + 1);
    w.seq0 = __shfl_sync(0xffffffffu, t0, from);
    w.len = __shfl_sync(0xffffffffu, len, from);
    w.tok0 = x * block;
    w.unit = (mine - before) % a.units;
    w.n0 = (min(w.len, w.tok0 + a.per_tile) + kFaKeys - 1) / kFaKeys;
    w.n1 = w.tok0 + a.per_tile < w.len ? (min(w.len, w.tok0 + block) + kFaKeys - 1) / kFaKeys : 0;
    ++turn;
    mine = turn * ctas + ((turn & 1) ? ctas - 1 - cta : cta);
    return w;
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(kFaThreads, 1)
    prompt_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ FaArgs a) {
  using L = FaSmem<D>;
  constexpr bool kBf16 = sizeof(T) == 2 && kFaOffset<T> == 0.f;
  constexpr uint32_t kIdS = umma::idesc(kBf16, kFaKeys, false), kIdO = umma::idesc(kBf16, D, true);
  extern __shared__ uint8_t smem_raw[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t *g = smem_raw + (base - raw);
  uint32_t *err = a.err;

  if (tid == 0) {
    for (int s = 0; s < kFaRing; ++s) {
      mbar_init(base + L::kKvFull + 8 * s, 1);
      mbar_init(base + L::kKvEmpty + 8 * s, 1);
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
    for (int i = 0; i < kFaChecks; ++i) mbar_init(base + L::kCheck + 8 * i, 1);
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

  // registers: 128 threads x 88 + 256 x 208 = 384 x 168, the launch's own
  if (warp < 4)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  if (warp == 0) {
    if (lane == 0) {  // loads
      Work w;
      int it = 0;  // ring position: K0 V0 K1 V1 ... over all items
      bool ok = true;
      int i = 0;
      for (; ok && get_work(base, L::kWFull, g, L::kWork, i, w, err); ++i) {
        mbar_arrive(base + L::kWEmpty + 8 * (i & 1));
        if (i > 0 && !(ok = umma::inline_wait(base + L::kQEmpty, (i - 1) & 1, err))) break;
        const int tiles = w.n1 > 0 ? 2 : 1, n = max(w.n0, w.n1);
        const int rows = a.pack * a.per_tile;
        mbar_expect_tx(base + L::kQFull, tiles * rows * D * 2);
        for (int t = 0; t < tiles; ++t)
          for (int h = 0; h < D / 64; ++h)
            umma::tma3(base + L::kQ + t * L::kTile + h * kFaHalf, &tmQ, h * 64, w.unit * a.pack,
                       w.seq0 + w.tok0 + t * a.per_tile, base + L::kQFull);
        const int kvh = w.unit * a.pack / a.group;
        for (int j = 0; j < n && ok; ++j) {
          for (int kv = 0; kv < 2; ++kv, ++it) {
            const int s = it % kFaRing;
            if (it >= kFaRing && !(ok = umma::inline_wait(base + L::kKvEmpty + 8 * s, (it / kFaRing - 1) & 1, err))) break;
            mbar_expect_tx(base + L::kKvFull + 8 * s, L::kTile);
            for (int h = 0; h < D / 64; ++h)
              umma::tma3(base + L::kKV + s * L::kTile + h * kFaHalf, kv ? &tmV : &tmK, h * 64, kvh,
                         w.seq0 + j * kFaKeys, base + L::kKvFull + 8 * s);
          }
        }
      }
      // nothing may still be landing in shared memory when the CTA leaves
      if (i > 0) umma::inline_wait(base + L::kQFull, (i - 1) & 1, err);
      for (int q = it > kFaRing ? it - kFaRing : 0; q < it; ++q)
        umma::inline_wait(base + L::kKvFull + 8 * (q % kFaRing), (q / kFaRing) & 1, err);
    }
  } else if (warp == 1) {
    if (umma::elect()) {  // products
      // A product that waits for its operands leaves the tensor cores idle: only one or two are queued behind
      // the running one.  So each group looks whether the next one's barrier is over before its own last products.
      Work w;
      int sl = 0, ph = 0, checked = 0;  // ring slot and phase of the next tile
      int np[2] = {0, 0}, no[2] = {0, 0};  // probabilities awaited, items begun, of each row tile
      bool ok = true, begun = false;
      auto next = [&]() {
        if (++sl == kFaRing) sl = 0, ph ^= 1;
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
          const uint32_t off = ((kk >> 2) * kFaHalf + (kk & 3) * 32) >> 4;  // in the descriptors' 16-byte units
          umma::mma_ss(tmem + t * 128, A + off, B + off, kIdS, kk != 0);
        }
        umma::commit(base + L::kSFull + 8 * t);
        return seen;
      };
      // O_t += P_t V, 64 keys
      auto values = [&](int t, int slot, int h, bool more, uint32_t bar, int phase) {
        const uint64_t V = umma::desc_mn(base + L::kKV + slot * L::kTile, kFaHalf);
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
        const int n0 = w.n0, n1 = w.n1, n = max(n0, n1), hidden = first_hidden_tile(w);
        wait(L::kQFull, i);
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
            wait(L::kCheck + 8 * (checked % kFaChecks), checked / kFaChecks);
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
        const int last = sl ? sl - 1 : kFaRing - 1;
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
      const int n = max(w.n0, w.n1), hidden = first_hidden_tile(w);
      bool reset = false;
      for (int j = hidden; j < n && ok; ++j) {
        const int pos = it + 2 * j + 1, s = pos % kFaRing;
        ok = __all_sync(0xffffffffu, umma::inline_wait(base + L::kKvFull + 8 * s, (pos / kFaRing) & 1, err));
        if (!ok) break;
        const uint32_t V = base + L::kKV + s * L::kTile;
        if (__any_sync(0xffffffffu, attn::wild_pieces<T>(V, L::kTile / 16, lane, kWarp))) {
          if (!reset) {
            for (int d = lane; d < D; d += kWarp) wild->nan[d] = wild->pos[d] = wild->neg[d] = kNever;
            reset = true;
          }
          for (int d = lane; d < D; d += kWarp) {
            for (int r = 0; r < kFaKeys; ++r) {
              T *v = reinterpret_cast<T *>(g + L::kKV + s * L::kTile + (d >> 6) * kFaHalf + r * 128 +
                                           ((((d & 63) >> 3) ^ (r & 7)) << 4) + (d & 7) * 2);
              const float x = static_cast<float>(*v);
              if (!(fabsf(x) < __int_as_float(0x7f800000))) {
                const uint16_t at = (uint16_t)((j - hidden) * kFaKeys + r);
                if (x != x)
                  wild->nan[d] = min(wild->nan[d], at);
                else if (x > 0.f)
                  wild->pos[d] = min(wild->pos[d], at);
                else
                  wild->neg[d] = min(wild->neg[d], at);
                *v = static_cast<T>(0.f);
              }
            }
          }
          if (lane == 0) *any = 1;
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the zeros, for the tensor core
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(base + L::kCheck + 8 * (checked % kFaChecks));
        ++checked;
      }
      it += 2 * n;
      __syncwarp();
      if (lane == 0) mbar_arrive(base + L::kWEmpty + 8 * (i & 1));
    }
  } else if (warp == 3) {  // the items
    Dealer dealer;
    dealer.begin(a, blockIdx.x, gridDim.x);
    for (int i = 0;; ++i) {
      const Work w = dealer.next(a);
      if (i >= 2 &&
          !__all_sync(0xffffffffu, umma::inline_wait(base + L::kWEmpty + 8 * (i & 1), ((i >> 1) - 1) & 1, err)))
        break;
      if (lane == 0) {
        *reinterpret_cast<Work *>(g + L::kWork + 32 * (i & 1)) = w;
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
    const int tok_r = r / a.pack, head_r = r % a.pack;  // the row's token in the tile and head in the unit
    const bool row_used = tok_r < a.per_tile;
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tmem + t * 128 + lanes, tO = tmem + 256 + t * 128 + lanes;
    const uint64_t c2 = umma::pack2(a.c, a.c);
    Work w;
    int ns = 0, items = 0;  // scores awaited, items of this row tile begun
    bool ok = true;
    for (int i = 0; ok; ++i) {
      const bool more = get_work(base, L::kWFull, g, L::kWork, i, w, err);
      if (!__all_sync(0xffffffffu, more)) break;
      const int nt = t ? w.n1 : w.n0;
      const int tok = w.tok0 + t * a.per_tile + tok_r;  // position in the sequence
      const bool live = row_used && tok < w.len;
      float m = kNegInf, l = 0.f;
      const int clear = (w.tok0 + t * a.per_tile + 1) / kFaKeys;  // tiles that every row sees whole
      for (int j = 0; j < nt; ++j, ++ns) {
        ok = __all_sync(0xffffffffu, umma::inline_wait(base + L::kSFull + 8 * t, ns & 1, err));
        if (!ok) break;
        umma::fence_after();
        uint32_t s[128], p[32];
        float sum;
        auto mask = [&](int from) {  // keys after the row's token, among 64
          const int see = tok + 1 - j * kFaKeys;
#pragma unroll
          for (int e = from; e < from + 64; ++e)
            if (e >= see) s[e] = 0xff800000u;
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
          const float shift = kFaOffset<T> - (m == kNegInf ? 0.f : m);
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
        if (j >= clear) mask(0);
        bool whole = false;  // the second half has come
        if (j == 0) {
          umma::wait_ld();
          if (j >= clear) mask(64);
          whole = true;
          m = fmaxf(most(0), most(64));
        }
        probabilities(0);
        if (j > 0) {
          const bool low = live && (sum > kFaLimit || m == kNegInf);
          if (__any_sync(0xffffffffu, low)) {
            umma::wait_ld();
            if (j >= clear) mask(64);
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
          if (j >= clear) mask(64);
        }
        probabilities(64);
        if (j > 0) {
          const bool low = live && sum > kFaLimit;
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
      if (nt > 0) {
        ok = __all_sync(0xffffffffu, umma::inline_wait(base + L::kOFull + 8 * t, items & 1, err));
        if (!ok) break;
        ++items;
        umma::fence_after();
        const int64_t at = (int64_t)(w.seq0 + tok) * a.q_heads + w.unit * a.pack + head_r;
        const float inv = 1.f / l;
        const bool wild = *(reinterpret_cast<volatile int *>(g + L::kWildAny) + (i & 1)) != 0;
        const Wild *wd = reinterpret_cast<const Wild *>(g + L::kWild) + (i & 1);
        const int upto = tok - first_hidden_tile(w) * kFaKeys;  // last position the row sees
        // 64 columns at a time through shared memory, so that a store covers whole lines of a few rows
        uint8_t *stage = g + L::kOut + (warp - 4) * 4096;
        const long long row_at = live ? at : -1;
#pragma unroll 1
        for (int q = 0; q < D / 64; ++q) {
          uint32_t o[64];
          umma::ld32(tO + q * 64, o);
          umma::ld32(tO + q * 64 + 32, o + 32);
          umma::wait_ld();
          if (q == D / 64 - 1) {
            umma::fence_before();
            mbar_arrive(base + L::kOEmpty + 8 * t);
          }
          if (wild) {
#pragma unroll
            for (int e = 0; e < 64; ++e) {
              const int d = q * 64 + e;
              const bool n = (int)wd->nan[d] <= upto, p = (int)wd->pos[d] <= upto, b = (int)wd->neg[d] <= upto;
              if (n || (p && b))
                o[e] = 0x7fffffffu;
              else if (p || b)
                o[e] = __float_as_uint(__uint_as_float(o[e]) + (p ? -kNegInf : kNegInf));
            }
          }
#pragma unroll
          for (int e = 0; e < 64; e += 8)
            *reinterpret_cast<uint4 *>(stage + lane * 128 + (((e >> 3) ^ (lane & 7)) << 4)) =
                make_uint4(Type<T>::pack(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv),
                           Type<T>::pack(__uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv),
                           Type<T>::pack(__uint_as_float(o[e + 4]) * inv, __uint_as_float(o[e + 5]) * inv),
                           Type<T>::pack(__uint_as_float(o[e + 6]) * inv, __uint_as_float(o[e + 7]) * inv));
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int row = e * 4 + (lane >> 3);
            const long long to = __shfl_sync(0xffffffffu, row_at, row);
            const uint4 x = *reinterpret_cast<const uint4 *>(stage + row * 128 + (((lane & 7) ^ (row & 7)) << 4));
            if (to >= 0) *reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + to * D + q * 64 + (lane & 7) * 8) = x;
          }
          __syncwarp();
        }
        if (live && a.lse) a.lse[at] = (m - kFaOffset<T> + log2f(l)) * attn::kLn2;
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

template <typename T, int D>
cudaError_t launch(const PromptAttnArgs &p, int sms, cudaStream_t st) {
  FaArgs a{};
  a.cu = p.cu, a.tokens = p.tokens, a.n_seqs = p.n_seqs, a.max_len = p.max_len;
  a.q_heads = p.q_heads, a.group = p.group;
  // heads packed into a row tile: all of a group's, up to 32 (then at most a fifth of the rows is left over)
  a.pack = p.group <= 32 ? p.group : 1;
  a.per_tile = 128 / a.pack, a.units = p.q_heads / a.pack;
  a.c = p.scale * attn::kLog2e;
  a.out = p.out, a.lse = p.lse, a.err = p.err;
  CUtensorMap tmQ, tmK, tmV;
  const uint64_t dq[3] = {D, (uint64_t)p.q_heads, (uint64_t)p.tokens}, dk[3] = {D, (uint64_t)p.kv_heads, (uint64_t)p.tokens};
  const uint64_t sq[2] = {(uint64_t)p.q_head * 2, (uint64_t)p.q_token * 2};
  const uint64_t sk[2] = {(uint64_t)p.k_head * 2, (uint64_t)p.k_token * 2};
  const uint64_t sv[2] = {(uint64_t)p.v_head * 2, (uint64_t)p.v_token * 2};
  const uint32_t bq[3] = {64, (uint32_t)a.pack, (uint32_t)a.per_tile}, bk[3] = {64, 1, kFaKeys};
  if (!encode_16bit(&tmQ, p.q, 3, dq, sq, bq) || !encode_16bit(&tmK, p.k, 3, dk, sk, bk) ||
      !encode_16bit(&tmV, p.v, 3, dk, sv, bk))
    return cudaErrorInvalidValue;
  const long long items =
      (long long)((p.max_len + 2 * a.per_tile - 1) / (2 * a.per_tile)) * p.n_seqs * a.units;
  prompt_attn_kernel<T, D><<<(unsigned)(items < sms ? items : sms), kFaThreads, FaSmem<D>::kBytes, st>>>(tmQ, tmK, tmV,
                                                                                                        a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t prepare_prompt_attn() {
  cudaError_t e = cudaSuccess;
  auto set = [&](const void *f, int bytes) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  };
  set((const void *)prompt_attn_kernel<__nv_bfloat16, 128>, FaSmem<128>::kBytes);
  set((const void *)prompt_attn_kernel<__nv_bfloat16, 64>, FaSmem<64>::kBytes);
  set((const void *)prompt_attn_kernel<__half, 128>, FaSmem<128>::kBytes);
  set((const void *)prompt_attn_kernel<__half, 64>, FaSmem<64>::kBytes);
  return e;
}

cudaError_t launch_prompt_attn(const PromptAttnArgs &a, int dtype, int dim, int sms, cudaStream_t st) {
  if (dtype == NS_DTYPE_BF16)
    return dim == 128 ? launch<__nv_bfloat16, 128>(a, sms, st) : launch<__nv_bfloat16, 64>(a, sms, st);
  return dim == 128 ? launch<__half, 128>(a, sms, st) : launch<__half, 64>(a, sms, st);
}

}  // namespace ns
