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
template <int W>
constexpr int kKeys = W == kLarge ? 128 : 64;  // of a tile
template <int D>
constexpr int kPerSm = D == 128 ? 3 : 4;  // CTAs of the line on an SM
template <int D, int W>
constexpr int kStages = D == 128 && W != kLarge ? 2 : 3;  // tiles in flight
constexpr int kMerge = 32 * 4 * 4;    // a lane's m, l (and padding), after its o

template <int D, int W>
__host__ __device__ constexpr int pa_stage() {
  return 2 * kKeys<W> * D * 2;
}
// Behind the stages: what a warp hands over to warp 0; in a cluster, (m, l)
// and o of each of its CTAs for the rows that this CTA joins.
template <int D, int WM, int W>
__host__ __device__ constexpr int pa_smem() {
  return kStages<D, W> * pa_stage<D, W>() + (W != kLine ? 16 * (D + 2) * 4 : WM == 1 ? 32 * D / 2 * 4 + kMerge : 0);
}

// CTAs that an SM is to hold: as many as their shared memory allows (64 rows: their registers).  The line has that
// many on each SM; its equal shares would end in a second, half empty wave if it had more.
template <int D, int WM, int W>
constexpr int kResident = W == kLarge ? (D == 128 ? 1 : 2) : WM == 1 ? kPerSm<D> : (D == 128 ? 2 : 3);
template <int D, int WM, int W>
constexpr bool kHeld = kResident<D, WM, W> * (pa_smem<D, WM, W>() + 1280) <= 228 * 1024;  // (1 KB is the system's)
static_assert(kHeld<128, 1, kLine> && kHeld<64, 1, kLine> && kHeld<128, 4, kLine> && kHeld<64, 4, kLine> &&
                  kHeld<128, 1, kSmall> && kHeld<64, 1, kSmall> && kHeld<128, 1, kLarge> && kHeld<64, 1, kLarge>,
              "shared memory of an SM");

template <int W>
__host__ __device__ inline long long pa_tiles(int len) {
  return len > 0 ? (len - 1) / kKeys<W> + 1 : 1;
}

// Where a CTA is in the line of tiles: item (sequence b, `item` = head *
// blocks + block of rows) and its tile.
template <int W>
struct Cursor {
  int b, item, tile, nt, len;
  const int32_t *table;
  __device__ __forceinline__ void enter(const PagedAttnArgs &a, uint32_t *err) {
    len = length(a, b, err);
    nt = (int)pa_tiles<W>(len);
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

// (Clusters: at most 16 rows.)
template <typename T, int D, int WM, int W>
__global__ void __launch_bounds__(kThreads<W>, kResident<D, WM, W>)
    paged_attn_kernel(const PagedAttnArgs a, int blocks) {
  constexpr int kPaThreads = kThreads<W>, kPaKeys = kKeys<W>, kWarps = kPaThreads / kWarp;
  constexpr int WK = kWarps / WM, NK = kPaKeys / WK, kRows = 16 * WM;
  constexpr int kLanesRow = D / 8;                    // threads that fetch a row
  constexpr int kPass = kPaThreads / kLanesRow;       // rows a pass of the CTA fetches
  static_assert(W == kLine || WM == 1, "a cluster has 16 rows");
  constexpr int C = kCluster;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int wm = WM == 1 ? 0 : warp, wk = WM == 1 ? warp : 0;
  const int items = a.kv_heads * blocks, R = a.n * a.group;
  const uint32_t s0 = (uint32_t)__cvta_generic_to_shared(smem);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  Cursor<W> ld;
  long long t0, t1;
  Ws ws{};
  if constexpr (W != kLine) {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // this CTA has begun
    const int at = blockIdx.x / C, rank = blockIdx.x % C;
    ld.b = at / items, ld.item = at % items;
    ld.enter(a, rank == 0 && ld.item == 0 ? a.err : nullptr);
    t0 = (long long)ld.nt * rank / C, t1 = (long long)ld.nt * (rank + 1) / C;
    ld.tile = (int)t0;
  } else {
    // where the tiles will lie, so that a CTA's shared memory does not grow with the sequences
    long long *s_cum = reinterpret_cast<long long *>(smem);
    static_assert(NS_MAX_ATTEND_SEQS * 8 <= kStages<D, W> * pa_stage<D, W>(), "room for the sequences");
    __shared__ long long s_sum[kPaThreads / kWarp];
    // tiles of the sequences before each one
    long long total = 0;
    for (int b0 = 0; b0 < a.n_seqs; b0 += kPaThreads) {
      const int b = b0 + tid;
      const long long mine = b < a.n_seqs ? pa_tiles<W>(length(a, b, blockIdx.x == 0 ? a.err : nullptr)) * items : 0;
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

    {
      int lo = 0, hi = a.n_seqs;  // the last sequence that begins at or before t0
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_cum[mid] <= t0)
          lo = mid;
        else
          hi = mid;
      }
      ld.b = lo;
      ld.enter(a, nullptr);
      const long long local = t0 - s_cum[lo];
      ld.item = (int)quotient(local, ld.nt);
      ld.tile = (int)(local - (long long)ld.item * ld.nt);
    }
    __syncthreads();  // everyone is done with s_cum before the first tile comes
  }
  Cursor<W> cu = ld;

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
  const T *kbase = static_cast<const T *>(a.k) + (fr & 7) * a.k_token + fc * 8;
  const T *vbase = static_cast<const T *>(a.v) + (fr & 7) * a.v_token + fc * 8;
  const uint32_t to = piece<D>(fr, fc);
  auto fetch = [&](int id, int stage) {
    const uint32_t sk = s0 + stage * pa_stage<D, W>() + to, sv = sk + kPaKeys * D * 2;
    const int left = ld.len - ld.tile * kPaKeys, head = ld.item / blocks;
    const int64_t page = id >= 0 ? id : 0, row = (ld.tile * kPaKeys + lane * 8) & pmask;
    const int64_t ko = page * a.k_page + head * a.k_head + row * a.k_token;
    const int64_t vo = page * a.v_page + head * a.v_head + row * a.v_token;
    const uint32_t there = __ballot_sync(0xffffffffu, id >= 0);
#pragma unroll
    for (int pass = 0; pass < kPaKeys / kPass; ++pass) {
      const int r = pass * kPass + fr;
      const bool ok = r < left && (there >> (r >> 3) & 1);
      const int64_t k = __shfl_sync(0xffffffffu, ko, r >> 3), v = __shfl_sync(0xffffffffu, vo, r >> 3);
      cp16(sk + pass * kPass * D * 2, kbase + k, ok);
      cp16(sv + pass * kPass * D * 2, vbase + v, ok);
    }
  };

  const float c = a.scale * kLog2e;
  long long left_ld = t1 - t0;
  int ids = fetch_ids();
  int st_ld = 0;
  constexpr int kAhead = kStages<D, W> - 1;
  uint32_t missing[kAhead] = {};  // of each tile in flight: its eights of rows without a page
  auto issue = [&]() {
#pragma unroll
    for (int i = 0; i + 1 < kAhead; ++i) missing[i] = missing[i + 1];
    missing[kAhead - 1] = 0;
    if (left_ld > 0) {
      fetch(ids, st_ld);
      missing[kAhead - 1] = __ballot_sync(0xffffffffu, ids == -2);
      st_ld = st_ld + 1 == kStages<D, W> ? 0 : st_ld + 1;
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

  Rows<T, D> rows;
  if (W != kLine) rows.clear();  // (a CTA of a short sequence may have no tile)
  uint32_t q[D / 16][4];
  uint64_t word[2] = {0, 0};
  int st = 0;
  long long seg0 = t0;  // where the current item's share of this CTA begins
  for (long long g = t0; g < t1; ++g) {
    const int head = cu.item / blocks, rb = cu.item % blocks;
    if (g == t0 || cu.tile == 0) {  // a new item: its queries and masks
      seg0 = g;
      rows.clear();
      const T *qs = static_cast<const T *>(a.q) + (int64_t)cu.b * a.q_seq;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = rb * kRows + wm * 16 + (lane >> 2) + 8 * h;
        const int node = r / a.group, qh = head * a.group + r % a.group;
        word[h] = 0;
        if (r < R) {
          word[h] = a.mask ? (uint64_t)a.mask[(int64_t)cu.b * a.n + node] : ~0ull >> (63 - node);
        }
        const T *src = qs + (int64_t)node * a.q_token + (int64_t)qh * a.q_head + (lane & 3) * 2;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          q[kk][h] = r < R ? *reinterpret_cast<const uint32_t *>(src + kk * 16) : 0u;
          q[kk][2 + h] = r < R ? *reinterpret_cast<const uint32_t *>(src + kk * 16 + 8) : 0u;
        }
      }
    }
    cp_wait<kAhead - 1>();
    __syncthreads();  // the tile is there for everyone, and everyone is done with the stage to be filled next
    const uint32_t gone = missing[0];
    issue();
    const uint32_t sk = s0 + st * pa_stage<D, W>(), sv = sk + kPaKeys * D * 2;
    st = st + 1 == kStages<D, W> ? 0 : st + 1;
    const int ctx = cu.len - a.n, p0 = cu.tile * kPaKeys, k0 = wk * NK;
    if (p0 + kPaKeys <= ctx && !gone) {
      rows.template tile<NK, false>(q, sk, sv, k0, c, [](int, int) { return false; }, false);
    } else {
      const int n = a.n, j0 = p0 + k0 - ctx;  // the first key's node
      bool wild = false;
      if (n > 1 || a.mask)
        wild = __any_sync(0xffffffffu, wild_pieces<T>(sv + (uint32_t)(k0 * D * 2), NK * D / 8, lane, kWarp));
      rows.template tile<NK, true>(
          q, sk, sv, k0, c,
          [&](int h, int key) {
            const int j = j0 + key;
            return (j >= 0 && (j >= n || !((word[h] >> j) & 1))) || (gone >> ((k0 + key) >> 3) & 1);
          },
          wild);
    }
    const bool ends = cu.tile + 1 == cu.nt;
    if (ends || g + 1 == t1) {
      rows.sum_l();
      if (W != kLine) break;
      if (WM == 1) {  // the warps' keys join, in warp order, in warp 0
        float4 *bo = reinterpret_cast<float4 *>(smem + kStages<D, W> * pa_stage<D, W>());
        float4 *bm = bo + (D / 8) * 32;
        for (int w = 1; w < 4; ++w) {
          if (warp == w) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
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
            for (int i = 0; i < D / 8; ++i) {
              const float4 y = bo[i * 32 + lane];
              rows.o[i][0] = rows.o[i][0] * fa[0] + y.x * fb[0];
              rows.o[i][1] = rows.o[i][1] * fa[0] + y.y * fb[0];
              rows.o[i][2] = rows.o[i][2] * fa[1] + y.z * fb[1];
              rows.o[i][3] = rows.o[i][3] * fa[1] + y.w * fb[1];
            }
          }
          __syncthreads();
        }
      }
      if (WM > 1 || warp == 0) {
        const bool whole = ends && g + 1 - seg0 == cu.nt;
        const int slot = seg0 == t0 ? 0 : 1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int rl = wm * 16 + (lane >> 2) + 8 * h, r = rb * kRows + rl;
          if (r < R) {
            if (whole) {
              const int64_t at = ((int64_t)cu.b * a.n + r / a.group) * a.q_heads + head * a.group + r % a.group;
              const float inv = rows.l[h] == 0.f ? 0.f : 1.f / rows.l[h];
              uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<T *>(a.out) + at * D) + (lane & 3);
#pragma unroll
              for (int i = 0; i < D / 8; ++i)
                dst[i * 4] = Type<T>::pack(rows.o[i][2 * h] * inv, rows.o[i][2 * h + 1] * inv);
              if (a.lse && (lane & 3) == 0) a.lse[at] = row_lse<T>(rows.m[h], rows.l[h]);
            } else {
              const size_t at = ((size_t)blockIdx.x * 2 + slot) * kRows + rl;
              float2 *dst = reinterpret_cast<float2 *>(ws.o + at * D) + (lane & 3);
#pragma unroll
              for (int i = 0; i < D / 8; ++i) dst[i * 4] = make_float2(rows.o[i][2 * h], rows.o[i][2 * h + 1]);
              if ((lane & 3) == 0) ws.ml[at] = make_float2(rows.m[h], rows.l[h]);
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
    static_assert(kWarps * 16 * (kPitch + 2) * 4 <= kStages<D, W> * pa_stage<D, W>(), "the parts replace the tiles");
    const int rank = blockIdx.x % C, head = ld.item, b = ld.b;
    float *w_o = reinterpret_cast<float *>(smem);
    float2 *w_ml = reinterpret_cast<float2 *>(w_o + kWarps * 16 * kPitch);
    float *c_o = reinterpret_cast<float *>(smem + kStages<D, W> * pa_stage<D, W>());  // [C][D]
    float2 *c_ml = reinterpret_cast<float2 *>(c_o + C * D);
    __syncthreads();  // (every tile has been waited for and used)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = (lane >> 2) + 8 * h;
      if (r < R) {
        float2 *dst = reinterpret_cast<float2 *>(w_o + (warp * 16 + r) * kPitch) + (lane & 3);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) dst[i * 4] = make_float2(rows.o[i][2 * h], rows.o[i][2 * h + 1]);
        if ((lane & 3) == 0) w_ml[warp * 16 + r] = make_float2(rows.m[h], rows.l[h]);
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
      float2 p[C];
      float m = kNegInf, l = 0.f, o = 0.f;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        p[i] = c_ml[i];
        m = fmaxf(m, p[i].x);
      }
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const float f = ex2(p[i].x - (m == kNegInf ? 0.f : m));
        l = fmaf(p[i].y, f, l);
        o = fmaf(c_o[i * D + col], f, o);
      }
      const int64_t at = ((int64_t)b * a.n + rank / a.group) * a.q_heads + head * a.group + rank % a.group;
      static_cast<T *>(a.out)[at * D + col] = static_cast<T>(l == 0.f ? 0.f : o / l);
      if (a.lse && col == 0) a.lse[at] = row_lse<T>(m, l);
    }
  }
}

// The rows of an item for the join: row r of head h and block rb is new token
// (16 WM rb + r) / group.
template <int WM>
struct Rows16 {
  int blocks;
  static constexpr int kRows = 16 * WM;
  static constexpr int kGroups = WM == 1 ? 4 : 1;  // few rows may have hundreds of parts, many rows have two or three
  template <typename T>
  __device__ __forceinline__ float offset() const {
    return Type<T>::kOffset;
  }
  __device__ __forceinline__ bool place(const PagedAttnArgs &a, int item, int rl, int &node, int &qh) const {
    const int r = item % blocks * kRows + rl;
    node = r / a.group, qh = item / blocks * a.group + r % a.group;
    return r < a.n * a.group;
  }
};

template <typename T, int D, int WM>
cudaError_t launch(const PagedAttnArgs &a, int sms, cudaStream_t st) {
  constexpr int kRows = 16 * WM;
  const int blocks = (a.n * a.group + kRows - 1) / kRows;
  constexpr int kCtas = kResident<D, WM, kLine>;
  const long long most = pa_tiles<kLine>(a.max_len) * a.n_seqs * a.kv_heads * blocks;
  const int ctas = (int)(most < (long long)kCtas * sms ? most : kCtas * sms);
  paged_attn_kernel<T, D, WM, kLine><<<ctas, kThreads<kLine>, pa_smem<D, WM, kLine>(), st>>>(a, blocks);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int rows = a.n * a.group < kRows ? a.n * a.group : kRows;
  return launch_join<T, D>(a, Rows16<WM>{blocks}, rows, a.kv_heads * blocks, ctas, st);
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
template <typename T, int D, int W, typename Fit>
auto &resident(Fit &fit) {
  return fit.clusters[Type<T>::kBf16 ? NS_DTYPE_BF16 : NS_DTYPE_F16][D == 128][W == kLarge];
}

// Whether each item can have its own cluster with up to kMostTiles tiles to a
// CTA (in two waves of small CTAs: with one or two tiles).
template <int D>
constexpr int kMostTiles = D == 128 ? 12 : 16;
template <typename T, int D, int W>
bool clusters_fit(const PagedAttnArgs &a, const PagedFit &fit) {
  const bool two_waves = W == kSmall && a.max_len > kCluster * kKeys<W> / 2 && a.max_len <= 2 * kCluster * kKeys<W>;
  return (long long)a.n_seqs * a.kv_heads <= (two_waves ? 2 : 1) * resident<T, D, W>(fit) &&
         a.max_len <= kMostTiles<D> * kCluster * kKeys<W>;
}
template <typename T, int D, int W>
cudaError_t launch_clusters(const PagedAttnArgs &a, cudaStream_t st) {
  ClusterLaunch l(a.n_seqs * a.kv_heads, kThreads<W>, pa_smem<D, 1, W>(), st);
  return cudaLaunchKernelEx(&l.cfg, paged_attn_kernel<T, D, 1, W>, a, 1);
}

template <typename T, int D, int WM, int W>
cudaError_t prepare(PagedFit *fit) {
  cudaError_t e = cudaFuncSetAttribute(paged_attn_kernel<T, D, WM, W>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       pa_smem<D, WM, W>());
  if (W == kLine) return e;
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(paged_attn_kernel<T, D, WM, W>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  ClusterLaunch l(64, kThreads<W>, pa_smem<D, 1, W>(), nullptr);
  return cudaOccupancyMaxActiveClusters(&resident<T, D, W>(*fit), paged_attn_kernel<T, D, WM, W>, &l.cfg);
}

// Up to 16 rows the keys are what costs: each is fetched once and the warps
// split them.  A call whose items fit on the GPU as clusters, all at once, with
// up to 12 (64 columns: 16) tiles to a CTA, takes clusters: of large CTAs where
// small ones would have more than one tile each and the large ones still fit (7
// clusters of 128 columns and 14 of 64, 21 and 33 of small ones).  Measured,
// line, small, large, one new token, bf16 (us in a graph):
//   32 heads on 8, 128 columns, 1 sequence:  100 tokens 8.5, 5.0, 10.1;  4097: 15.3, 8.6, 15.1;
//     8000: 17.0, 13.1;  12000: 18.4, 17.7;  16000: 20.0, 22.3
//     2 sequences:  100: 8.7, 5.5;  4097: 16.4, 9.9;  12000: 23.7, 22.9;  16000: 31.9, 30.8;  24000: 41.9, 44.1
//   28 on 4, 128 columns, 1 sequence:  100: 8.6, 5.2, 5.9;  2000: 10.0, 5.8, 5.8;  8000: 18.3, 11.6, 9.9;
//     16000: 20.0, 19.0, 14.9;  24000 (12 tiles): 21.6, 26.7, 20.3;  32000: 22.9, 35.5, 26.3
//     5 sequences:  4097: 16.6, 10.7;  12000: 30.9, 26.3;  16000: 36.4, 33.8
//   12 on 4, 64 columns, 1 sequence:  1000: 9.0, 4.4, 4.6;  8000: 17.7, 9.4, 7.5;  32000 (16 tiles): 23.8, 26.6, 19.2
//     4 sequences:  12000: 18.4, 15.0;  16000: 20.2, 18.8;  24000: 25.4, 30.3
//   32 heads on 8, 128 columns, 4 sequences (two waves):  100: 8.8, 10.0;  600: 10.5, 9.9;  2000: 15.1, 12.8;
//     4097: 18.4, 19.2
// Clusters of 8 large CTAs took 11.3 us for the 4097 tokens of one sequence.
// Above 16 rows the products cost: they belong on the tensor cores of
// ns_paged_umma.cu, which want queries that TMA can fetch (16-byte aligned,
// strides multiples of 8); other queries take 64 rows a CTA here.  Measured
// with 16 sequences of 2300 tokens, 32 heads on 8, 128 columns, pages of 64, by
// 16 rows here and there (us): 4 rows 34.6, 40.8; 16 rows 38.1, 40.7; 20 rows
// (twice 16) 49.5, 40.6; 64 rows 88.2, 40.9.  64 rows a CTA here: 16 draft
// trees of 60 nodes behind 512 to 4096 tokens (240 rows) 169, there 60.
template <typename T, int D>
cudaError_t by_rows(const PagedAttnArgs &a, int sms, const PagedFit &fit, cudaStream_t st) {
  if (a.n * a.group <= 16) {
    if (a.max_len > kCluster * kKeys<kSmall> && clusters_fit<T, D, kLarge>(a, fit))
      return launch_clusters<T, D, kLarge>(a, st);
    if (clusters_fit<T, D, kSmall>(a, fit)) return launch_clusters<T, D, kSmall>(a, st);
    return launch<T, D, 1>(a, sms, st);
  }
  if (paged_umma_ok(a)) return launch_paged_umma(a, Type<T>::kBf16 ? NS_DTYPE_BF16 : NS_DTYPE_F16, D, sms, st);
  return launch<T, D, 4>(a, sms, st);
}
template <typename T>
cudaError_t by_dim(const PagedAttnArgs &a, int dim, int sms, const PagedFit &fit, cudaStream_t st) {
  return dim == 128 ? by_rows<T, 128>(a, sms, fit, st) : by_rows<T, 64>(a, sms, fit, st);
}
template <typename T, int D>
cudaError_t prepare_all(PagedFit *fit) {
  cudaError_t e = prepare<T, D, 1, kLine>(fit);
  if (e == cudaSuccess) e = prepare<T, D, 4, kLine>(fit);
  if (e == cudaSuccess) e = prepare<T, D, 1, kSmall>(fit);
  if (e == cudaSuccess) e = prepare<T, D, 1, kLarge>(fit);
  return e;
}

}  // namespace

int64_t paged_attn_ws(int n_seqs, int n, int q_heads, int kv_heads, int dim, int sms) {
  // two parts for each CTA: up to 4 sms CTAs of 16 rows, or sms CTAs of 256 (3 sms of 64 are no more)
  const int64_t rows = n * (q_heads / kv_heads) <= 16 ? (int64_t)kPerSm<64> * sms * 2 * 16 : (int64_t)sms * 2 * 256;
  return (((int64_t)(n_seqs + 1) * 8 + 255) & ~(int64_t)255) + rows * (dim + 2) * 4;
}

cudaError_t prepare_paged_attn(PagedFit *fit) {
  cudaError_t e = prepare_all<__nv_bfloat16, 128>(fit);
  if (e == cudaSuccess) e = prepare_all<__nv_bfloat16, 64>(fit);
  if (e == cudaSuccess) e = prepare_all<__half, 128>(fit);
  if (e == cudaSuccess) e = prepare_all<__half, 64>(fit);
  return e == cudaSuccess ? prepare_paged_umma() : e;
}

cudaError_t launch_paged_attn(const PagedAttnArgs &a, int dtype, int dim, int sms, const PagedFit &fit,
                              cudaStream_t st) {
  return dtype == NS_DTYPE_BF16 ? by_dim<__nv_bfloat16>(a, dim, sms, fit, st) : by_dim<__half>(a, dim, sms, fit, st);
}

}  // namespace ns
