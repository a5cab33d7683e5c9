// Attention of a sequence's new tokens over a paged key-value cache.
//
// Rows: the n new tokens of a sequence and the query heads that share a
// key-value head make R = n * group query rows that read the same keys, so
// each key and value is fetched once for all of them (once for every 64 rows
// when R is larger; the repeats hit L2).
//
// Work: the keys of every (sequence, key-value head, block of rows) are cut
// into tiles of 64, all tiles of the call are put in one line, and each of
// the resident CTAs takes an equal, contiguous share of it.  So a batch of
// very different lengths, or one long sequence, keeps every SM busy to the
// end, whatever the lengths are (the host does not know them).  A CTA whose
// share begins or ends inside an item leaves its rows' (m, l, o) in the
// workspace, at most two of them; the join kernel, whose launch overlaps the
// end of this one, adds up the parts of such items in CTA order.  No atomics:
// the same inputs give the same bits.
//
// In a CTA: keys and values of three tiles are in flight (cp.async, 16 bytes,
// page ids fetched a tile ahead).  Up to 16 rows the four warps split a
// tile's keys and join at the item's end; above, each warp has 16 rows of 64.
//
// What bounds it: HBM for one-token steps (each key is used by `group` rows,
// a few flops a byte); the mma.sync rate for 64-row blocks.
#include "ns_paged_attn.cuh"

namespace ns {
namespace {

using namespace paged;

constexpr int kPaThreads = 128;
constexpr int kPaKeys = 64;   // keys of a tile
constexpr int kPaStages = 3;
constexpr int kPaMerge = 32 * 4 * 4;  // a lane's m, l (and padding), after its o

template <int D>
__host__ __device__ constexpr int pa_stage() {
  return 2 * kPaKeys * D * 2;
}
template <int D, int WM>
__host__ __device__ constexpr int pa_smem() {
  return kPaStages * pa_stage<D>() + (WM == 1 ? 32 * D / 2 * 4 + kPaMerge : 0);
}

__host__ __device__ inline long long pa_tiles(int len) { return len > 0 ? (len + kPaKeys - 1) / kPaKeys : 1; }

// Where a CTA is in the line of tiles: item (sequence b, `item` = head *
// blocks + block of rows) and its tile.
struct Cursor {
  int b, item, tile, nt, len;
  const int32_t *table;
  __device__ __forceinline__ void enter(const PagedAttnArgs &a) {
    len = length(a, b, nullptr);
    nt = (int)pa_tiles(len);
    const int s = a.seqs[b];
    table = a.table + (size_t)(s >= 0 && s < a.max_seqs ? s : 0) * a.table_ld;
  }
  __device__ __forceinline__ void next(const PagedAttnArgs &a, int items) {
    if (++tile < nt) return;
    tile = 0;
    if (++item < items) return;
    item = 0;
    if (++b < a.n_seqs) enter(a);
  }
};

template <typename T, int D, int WM>
__global__ void __launch_bounds__(kPaThreads) paged_attn_kernel(const PagedAttnArgs a, int blocks) {
  constexpr int WK = 4 / WM, NK = kPaKeys / WK, kRows = 16 * WM;
  constexpr int kLanesRow = D / 8;                    // threads that fetch a row
  constexpr int kPass = kPaThreads / kLanesRow;       // rows a pass of the CTA fetches
  extern __shared__ __align__(128) uint8_t smem[];
  long long *s_cum = reinterpret_cast<long long *>(smem + pa_smem<D, WM>());
  __shared__ long long s_sum[kPaThreads / kWarp];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int wm = WM == 1 ? 0 : warp, wk = WM == 1 ? warp : 0;
  const int items = a.kv_heads * blocks, R = a.n * a.group;
  const uint32_t s0 = (uint32_t)__cvta_generic_to_shared(smem);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // tiles of the sequences before each one
  long long total = 0;
  for (int b0 = 0; b0 < a.n_seqs; b0 += kPaThreads) {
    const int b = b0 + tid;
    const long long mine = b < a.n_seqs ? pa_tiles(length(a, b, blockIdx.x == 0 ? a.err : nullptr)) * items : 0;
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
  const Ws ws = workspace(a.ws, a.n_seqs, gridDim.x, kRows);
  if (blockIdx.x == 0) {
    for (int b = tid; b < a.n_seqs; b += kPaThreads) ws.cum[b] = s_cum[b];
    if (tid == 0) ws.cum[a.n_seqs] = total;
  }
  const long long t0 = quotient(total * blockIdx.x, gridDim.x), t1 = quotient(total * (blockIdx.x + 1), gridDim.x);
  if (t0 >= t1) return;

  Cursor ld;
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
    ld.enter(a);
    const long long local = t0 - s_cum[lo];
    ld.item = (int)quotient(local, ld.nt);
    ld.tile = (int)(local - (long long)ld.item * ld.nt);
  }
  Cursor cu = ld;

  // page ids of the load cursor's tile, one for each eight rows, in lanes 0 to 7
  auto fetch_ids = [&]() {
    int id = -1;
    if (lane < 8) {
      const int p = ld.tile * kPaKeys + lane * 8;
      if (p < ld.len) {
        id = ld.table[p >> a.page_shift];
        if (id < 0 || id >= a.n_pages) {
          set_flag(a.err, NS_FLAG_BAD_ID);
          id = -1;
        }
      }
    }
    return id;
  };
  const T *kbase = static_cast<const T *>(a.k), *vbase = static_cast<const T *>(a.v);
  const int fr = tid / kLanesRow, fc = tid % kLanesRow, pmask = (1 << a.page_shift) - 1;
  auto fetch = [&](int ids, int stage) {
    const uint32_t sk = s0 + stage * pa_stage<D>(), sv = sk + kPaKeys * D * 2;
    const int head = ld.item / blocks;
#pragma unroll
    for (int pass = 0; pass < kPaKeys / kPass; ++pass) {
      const int r = pass * kPass + fr;
      const int id = __shfl_sync(0xffffffffu, ids, r >> 3);
      const int p = ld.tile * kPaKeys + r;
      const bool ok = id >= 0 && p < ld.len;
      const int64_t page = ok ? id : 0, row = ok ? p & pmask : 0;
      cp16(sk + piece<D>(r, fc), kbase + page * a.k_page + head * a.k_head + row * a.k_token + fc * 8, ok);
      cp16(sv + piece<D>(r, fc), vbase + page * a.v_page + head * a.v_head + row * a.v_token + fc * 8, ok);
    }
  };

  const float c = a.scale * kLog2e;
  long long left_ld = t1 - t0;
  int ids = fetch_ids();
  int st_ld = 0;
  auto issue = [&]() {
    if (left_ld > 0) {
      fetch(ids, st_ld);
      st_ld = st_ld + 1 == kPaStages ? 0 : st_ld + 1;
      --left_ld;
      if (left_ld > 0) {
        ld.next(a, items);
        ids = fetch_ids();
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < kPaStages - 1; ++i) issue();

  Rows<T, D> rows;
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
    cp_wait<kPaStages - 2>();
    __syncthreads();  // the tile is there for everyone, and everyone is done with the stage to be filled next
    issue();
    const uint32_t sk = s0 + st * pa_stage<D>(), sv = sk + kPaKeys * D * 2;
    st = st + 1 == kPaStages ? 0 : st + 1;
    const int ctx = cu.len - a.n, p0 = cu.tile * kPaKeys, k0 = wk * NK;
    if (p0 + kPaKeys <= ctx) {
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
            return j >= 0 && (j >= n || !((word[h] >> j) & 1));
          },
          wild);
    }
    const bool ends = cu.tile + 1 == cu.nt;
    if (ends || g + 1 == t1) {
      rows.sum_l();
      if (WM == 1) {  // the warps' keys join, in warp order, in warp 0
        float4 *bo = reinterpret_cast<float4 *>(smem + kPaStages * pa_stage<D>());
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
  const int smem = pa_smem<D, WM>() + a.n_seqs * 8;
  const long long most = pa_tiles(a.max_len) * a.n_seqs * a.kv_heads * blocks;
  const int per_sm = smem <= 113 * 1024 ? 2 : 1;
  const int ctas = (int)(most < (long long)per_sm * sms ? most : per_sm * sms);
  paged_attn_kernel<T, D, WM><<<ctas, kPaThreads, smem, st>>>(a, blocks);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int rows = a.n * a.group < kRows ? a.n * a.group : kRows;
  return launch_join<T, D>(a, Rows16<WM>{blocks}, rows, a.kv_heads * blocks, ctas, st);
}

template <typename T, int D, int WM>
cudaError_t prepare() {
  return cudaFuncSetAttribute(paged_attn_kernel<T, D, WM>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              pa_smem<D, WM>() + NS_MAX_ATTEND_SEQS * 8);
}

// Up to 16 rows the keys are what costs: each is fetched once and the warps
// split them.  Above, the products are: they belong on the tensor cores of
// ns_paged_umma.cu, which want queries that TMA can fetch (16-byte aligned,
// strides multiples of 8); other queries take 64 rows a CTA here.
template <typename T>
cudaError_t by_rows(const PagedAttnArgs &a, int dim, int sms, cudaStream_t st) {
  if (a.n * a.group <= 16) return dim == 128 ? launch<T, 128, 1>(a, sms, st) : launch<T, 64, 1>(a, sms, st);
  if (paged_umma_ok(a)) return launch_paged_umma(a, Type<T>::kBf16 ? NS_DTYPE_BF16 : NS_DTYPE_F16, dim, sms, st);
  return dim == 128 ? launch<T, 128, 4>(a, sms, st) : launch<T, 64, 4>(a, sms, st);
}

}  // namespace

int64_t paged_attn_ws(int n_seqs, int n, int q_heads, int kv_heads, int dim, int sms) {
  // two parts for each CTA: 2 sms CTAs of 16 rows, or sms CTAs of 256 (2 sms of 64 are fewer)
  const int64_t rows = n * (q_heads / kv_heads) <= 16 ? (int64_t)2 * sms * 2 * 16 : (int64_t)sms * 2 * 256;
  return (((int64_t)(n_seqs + 1) * 8 + 255) & ~(int64_t)255) + rows * (dim + 2) * 4;
}

cudaError_t prepare_paged_attn() {
  cudaError_t e = cudaSuccess;
  auto also = [&](cudaError_t x) { e = e == cudaSuccess ? x : e; };
  also(prepare<__nv_bfloat16, 128, 1>()), also(prepare<__nv_bfloat16, 128, 4>());
  also(prepare<__nv_bfloat16, 64, 1>()), also(prepare<__nv_bfloat16, 64, 4>());
  also(prepare<__half, 128, 1>()), also(prepare<__half, 128, 4>());
  also(prepare<__half, 64, 1>()), also(prepare<__half, 64, 4>());
  also(prepare_paged_umma());
  return e;
}

cudaError_t launch_paged_attn(const PagedAttnArgs &a, int dtype, int dim, int sms, cudaStream_t st) {
  return dtype == NS_DTYPE_BF16 ? by_rows<__nv_bfloat16>(a, dim, sms, st) : by_rows<__half>(a, dim, sms, st);
}

}  // namespace ns
