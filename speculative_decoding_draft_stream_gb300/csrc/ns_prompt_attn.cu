// Causal attention over whole packed prompts, on the 5th-generation tensor
// cores (ns_umma_attn.cuh has the kernel).
//
// An item is two tiles of 128 rows of one sequence and the keys up to its last
// token: 2 * (128 / group) consecutive tokens of all query heads of one
// key-value head, or 256 tokens of one head; in calls of few items, one tile
// of one head with its keys split in two (launch has the rules).  Items are
// dealt longest first, so that the CTAs end together.  A row sees the keys up
// to its own token; what lies behind it in the item's last tiles are later
// tokens and the next sequence's.
//
// Bound by the products (see there) for long sequences: 16381 tokens, 32 heads
// on 8, 1.40 ms.  For batches of shorter ones each item's start and end, where
// only one of softmax and products runs, are a third: 16 sequences of 130 to
// 2047 tokens, 28 heads on 4, 147 us, 1.02 PFLOP/s.  A few short ones are
// latency: four of up to 200 tokens, 12 heads on 4 of 64 columns, 8.0 us; one
// of 1967 tokens, 8 heads, 21 us (16 key tiles one after the other: 30 us).
#include <algorithm>

#include "ns_umma_attn.cuh"

namespace ns {
namespace {

using fa::kKeys;

struct FaArgs {
  const int32_t *cu;
  int32_t tokens, n_seqs, max_len, q_heads, group, pack, per_tile, units;
  float c;  // scale * log2(e)
  void *out;
  float *lse;
  float2 *part_ml;  // unused: items are whole
  float *part_o;
  uint32_t *err;
};

struct Work {
  int n0, n1, hidden;
  int seq0, len;     // the sequence's first token and its length
  int tok0;          // first token of row tile 0
  int unit;          // query heads unit * pack .. + pack - 1
  int slot;          // unused: items are whole
};

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
template <bool S>
struct Dealer {
  int cta, ctas, lane, block, size;
  int most;                // blocks of the lane's group's longest sequence
  int x, s;                // where the line is: block, and the lane's sequence
  uint32_t groups, live;   // groups left at x; sequences of the 32 at s that reach x
  int t0, len;             // of the lane's sequence
  int before, here;        // items before these 32 sequences, and of them
  int turn, mine;          // the CTA's next item

  __device__ __forceinline__ void begin(const FaArgs &a, int cta_, int ctas_) {
    cta = cta_, ctas = ctas_, lane = threadIdx.x & 31, block = (S ? 1 : 2) * a.per_tile;
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
    w.hidden = (w.tok0 + 1) / kKeys;  // tile 0's first token sees the tiles before whole
    w.n0 = (min(w.len, w.tok0 + a.per_tile) + kKeys - 1) / kKeys;
    if (S)
      w.n1 = w.n0 / 2, w.n0 -= w.n1;
    else
      w.n1 = w.tok0 + a.per_tile < w.len ? (min(w.len, w.tok0 + block) + kKeys - 1) / kKeys : 0;
    ++turn;
    mine = turn * ctas + ((turn & 1) ? ctas - 1 - cta : cta);
    return w;
  }
};

template <bool S>
struct Mode {
  using Args = FaArgs;
  using Work = ns::Work;
  using Dealer = ns::Dealer<S>;
  static constexpr bool kParts = false, kSplit = S, kWhole = true, kCodes = false, kHigh = false, kPaired = false;
  static constexpr int kStageRow = 128;

  struct Loader {
    __device__ __forceinline__ void begin(const FaArgs &, const Work &, int) {}
    __device__ __forceinline__ void queries(const FaArgs &a, const Work &w, int t, int h, uint32_t dst,
                                            const CUtensorMap *m, uint32_t bar) {
      umma::tma3(dst, m, h * 64, w.unit * a.pack, w.seq0 + w.tok0 + t * a.per_tile, bar);
    }
    template <int D>
    __device__ __forceinline__ void keys(const FaArgs &a, const Work &w, int j, int, uint32_t dst,
                                         const CUtensorMap *m, uint32_t bar, int lane, uint32_t *) {
      if (lane == 0) {
        mbar_expect_tx(bar, kKeys * D * 2);
        for (int h = 0; h < D / 64; ++h)
          umma::tma3(dst + h * fa::kHalf, m, h * 64, w.unit * a.pack / a.group, w.seq0 + j * kKeys, bar);
      }
      __syncwarp();
    }
  };

  struct Row {
    int tok;       // position in the sequence
    bool live;
    int64_t at;    // its place in the output
    int first;     // position of the first looked-through tile
    __device__ __forceinline__ void begin(const FaArgs &a, const Work &w, int t, int r) {
      const int in_tile = r / a.pack;
      tok = w.tok0 + t * a.per_tile + in_tile;
      live = in_tile < a.per_tile && tok < w.len;
      at = (int64_t)(w.seq0 + tok) * a.q_heads + w.unit * a.pack + r % a.pack;
      first = w.hidden * kKeys;
    }
    __device__ __forceinline__ uint64_t sees(const Work &, int j, int from) const {
      const int n = tok + 1 - j * kKeys - from;
      return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1;
    }
  };

  struct Wild {  // first positions of values that are not finite, from the first looked-through tile on
    uint16_t nan[128], pos[128], neg[128];
    static constexpr uint16_t kNever = 0xffff;
    __device__ __forceinline__ void none(int d) { nan[d] = pos[d] = neg[d] = kNever; }
    __device__ __forceinline__ bool note(const Work &w, int j, int r, int d, float x) {
      const uint16_t at = (uint16_t)((j - w.hidden) * kKeys + r);
      uint16_t &f = x != x ? nan[d] : x > 0.f ? pos[d] : neg[d];
      f = f < at ? f : at;
      return true;
    }
    // 0: none, 1: NaN (or infinities of both signs), 2: inf, 3: -inf
    __device__ __forceinline__ int seen(const Row &row, int d) const {
      const int upto = row.tok - row.first;
      const bool n = (int)nan[d] <= upto, p = (int)pos[d] <= upto, b = (int)neg[d] <= upto;
      return n || (p && b) ? 1 : p ? 2 : b ? 3 : 0;
    }
  };

  template <typename T, int D>
  static __device__ __forceinline__ bool clear(const FaArgs &, const Work &, int, uint8_t *, int) {
    return false;
  }
};

template <typename T, int D>
cudaError_t launch(const PromptAttnArgs &p, int sms, cudaStream_t st) {
  FaArgs a{};
  a.cu = p.cu, a.tokens = p.tokens, a.n_seqs = p.n_seqs, a.max_len = p.max_len;
  a.q_heads = p.q_heads, a.group = p.group;
  // Few row tiles (no more than SMs, a head to a tile; 7/4 of them with long keys): an item is one of them, and where
  // there is more than one key tile its keys are split over both halves of the CTA.  One prompt, us without and with:
  // 567 tokens, 28 heads on 4 15.2, 12.3; 1967, 8 on 8 30.1, 21.3; 4000, 8 on 8 (1.7 tiles an SM) 52.8, 39.0; 1000, 32
  // on 8 (1.7) 19.2, 19.9; 1300, 32 on 8 (2.3) 22.5, 27.3; one of 50, 32 on 8 8.6, 7.6 (one key tile); but ten of 1 to
  // 3, 16 on 1 (1.05) 9.5, 14.0.
  const long long blocks = (p.max_len + 127) / 128;
  const long long tiles = std::min((long long)p.tokens / 128 + p.n_seqs, blocks * p.n_seqs) * p.q_heads;
  const bool few = tiles <= sms || (4 * tiles <= 7LL * sms && p.max_len >= 1024);
  const bool split = few && p.max_len > kKeys;
  // Otherwise the heads of a group in one tile of 128 / group tokens, or a tile of 128 tokens for each head.  The first
  // leaves fewer of the products behind the diagonal: 16 sequences of 130 to 2047 tokens, 28 heads on 4: 146.5 us, 168.2
  // with a head to a tile; 32 on 2 181.8, 213.0.  But its few tokens have many rows of queries, keys of the same tiles
  // for every CTA, and no more items: one sequence of 2000 tokens with 8 heads on 1 takes 30.1, 29.6 us; 16 on 1 41.6,
  // 30.7; 32 on 1 77.8, 36.3; 64 on 1 148.5, 64.4.
  a.pack = !few && (p.group <= 8 || (p.group <= 32 && p.n_seqs >= 8)) ? p.group : 1;
  a.per_tile = 128 / a.pack, a.units = p.q_heads / a.pack;
  a.c = p.scale * attn::kLog2e;
  a.out = p.out, a.lse = p.lse, a.err = p.err;
  CUtensorMap tmQ, tmK, tmV;
  const uint64_t dq[3] = {D, (uint64_t)p.q_heads, (uint64_t)p.tokens}, dk[3] = {D, (uint64_t)p.kv_heads, (uint64_t)p.tokens};
  const uint64_t sq[2] = {(uint64_t)p.q_head * 2, (uint64_t)p.q_token * 2};
  const uint64_t sk[2] = {(uint64_t)p.k_head * 2, (uint64_t)p.k_token * 2};
  const uint64_t sv[2] = {(uint64_t)p.v_head * 2, (uint64_t)p.v_token * 2};
  const uint32_t bq[3] = {64, (uint32_t)a.pack, (uint32_t)a.per_tile}, bk[3] = {64, 1, kKeys};
  if (!encode_16bit(&tmQ, p.q, 3, dq, sq, bq) || !encode_16bit(&tmK, p.k, 3, dk, sk, bk) ||
      !encode_16bit(&tmV, p.v, 3, dk, sv, bk))
    return cudaErrorInvalidValue;
  const int block = (split ? 1 : 2) * a.per_tile;
  const long long items = (long long)((p.max_len + block - 1) / block) * p.n_seqs * a.units;
  const unsigned ctas = (unsigned)(items < sms ? items : sms);
  if (split)
    fa::attn_kernel<T, D, Mode<true>><<<ctas, fa::kThreads, fa::Smem<D, Mode<true>>::kBytes, st>>>(tmQ, tmK, tmV, a);
  else
    fa::attn_kernel<T, D, Mode<false>><<<ctas, fa::kThreads, fa::Smem<D, Mode<false>>::kBytes, st>>>(tmQ, tmK, tmV, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t prepare_prompt_attn() {
  cudaError_t e = cudaSuccess;
  auto set = [&](const void *f, int bytes) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  };
  set((const void *)fa::attn_kernel<__nv_bfloat16, 128, Mode<false>>, fa::Smem<128, Mode<false>>::kBytes);
  set((const void *)fa::attn_kernel<__nv_bfloat16, 64, Mode<false>>, fa::Smem<64, Mode<false>>::kBytes);
  set((const void *)fa::attn_kernel<__half, 128, Mode<false>>, fa::Smem<128, Mode<false>>::kBytes);
  set((const void *)fa::attn_kernel<__half, 64, Mode<false>>, fa::Smem<64, Mode<false>>::kBytes);
  set((const void *)fa::attn_kernel<__nv_bfloat16, 128, Mode<true>>, fa::Smem<128, Mode<true>>::kBytes);
  set((const void *)fa::attn_kernel<__nv_bfloat16, 64, Mode<true>>, fa::Smem<64, Mode<true>>::kBytes);
  set((const void *)fa::attn_kernel<__half, 128, Mode<true>>, fa::Smem<128, Mode<true>>::kBytes);
  set((const void *)fa::attn_kernel<__half, 64, Mode<true>>, fa::Smem<64, Mode<true>>::kBytes);
  return e;
}

cudaError_t launch_prompt_attn(const PromptAttnArgs &a, int dtype, int dim, int sms, cudaStream_t st) {
  if (dtype == NS_DTYPE_BF16)
    return dim == 128 ? launch<__nv_bfloat16, 128>(a, sms, st) : launch<__nv_bfloat16, 64>(a, sms, st);
  return dim == 128 ? launch<__half, 128>(a, sms, st) : launch<__half, 64>(a, sms, st);
}

}  // namespace ns
