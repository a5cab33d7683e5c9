// What the tensor-core kernels over a paged cache share (ns_paged_umma.cu,
// ns_shared_attn.cu): keys and values page by page, and values behind a
// sequence's end or of new tokens that some rows do not see.
#pragma once

#include "ns_paged_attn.cuh"
#include "ns_umma_attn.cuh"

#include <cuda_fp16.h>

namespace ns {
namespace paged {

// A whole warp fetches key and value tiles, a lane a page.  Work has the cache's sequence (seq, len), the tiles (j0,
// tiles()) and the heads (unit); Args the table and the pages.
// F8: codes, a box of all columns to a page.  P: of 16 bits and 128 columns, a box of all columns to a page (fa::Tile),
// where heads or columns come in strides that leave a dimension for it (page_pairs).
template <typename Args, typename Work, bool F8, bool P>
struct PageLoader {
  int ids, next;  // lane l: the id of the l-th page of this tile, and of the next
  // pages of tile j that hold keys of the sequence
  __device__ __forceinline__ int pages(const Args &a, const Work &w, int j) const {
    const int rows = min(fa::kKeys, w.len - (w.j0 + j) * fa::kKeys), page = 1 << a.page_shift;
    return rows <= 0 ? 0 : page >= fa::kKeys ? 1 : (rows + page - 1) >> a.page_shift;
  }
  __device__ __forceinline__ int fetch(const Args &a, const Work &w, int j, int lane) const {
    if (j >= w.tiles() || lane >= pages(a, w, j)) return 0;
    const int p = ((w.j0 + j) * fa::kKeys >> a.page_shift) + lane;
    const int id = a.table[(size_t)w.seq * a.table_ld + p];
    if (id >= 0 && id < a.n_pages) return id;
    set_flag(a.err, NS_FLAG_BAD_ID);
    return a.n_pages;  // outside the tensor: zeros
  }
  __device__ __forceinline__ void begin(const Args &a, const Work &w, int lane) { next = fetch(a, w, 0, lane); }
  template <int D>
  __device__ __forceinline__ void keys(const Args &a, const Work &w, int j, int kv, uint32_t dst,
                                       const CUtensorMap *m, uint32_t bar, int lane, uint32_t *missing) {
    const int n = pages(a, w, j), page = 1 << a.page_shift, rows = min(page, fa::kKeys);
    if (kv == 0) {
      ids = next;
      next = fetch(a, w, j + 1, lane);
      // pages out of range, then the tile's eights of keys that lie in them
      uint32_t out = __ballot_sync(0xffffffffu, lane < n && ids == a.n_pages);
      if (out) out = __ballot_sync(0xffffffffu, lane < fa::kKeys / 8 && (out >> (lane * 8 / rows) & 1));
      if (lane == 0) *missing = out;
    }
    if (lane == 0) mbar_expect_tx(bar, n * rows * D * (F8 ? 1 : 2));
    __syncwarp();
    if (lane < n) {
      const int row = page > fa::kKeys ? (w.j0 + j) * fa::kKeys & (page - 1) : 0;
      if (F8)
        umma::tma4(dst + lane * rows * D, m, 0, row, w.unit * a.pack / a.group, ids, bar);
      else if (P)
        umma::tma5(dst + lane * rows * 256, m, 0, 0, (kv ? a.pairs.vz : a.pairs.kz) * (w.unit * a.pack / a.group),
                   (kv ? a.pairs.vw : a.pairs.kw) * (w.unit * a.pack / a.group) + row / 8, ids, bar);
      for (int h = 0; h < (F8 || P ? 0 : D / 64); ++h)
        umma::tma4(dst + h * fa::kHalf + lane * rows * 128, m, h * 64, row, w.unit * a.pack / a.group, ids, bar);
    }
    __syncwarp();
  }
};

// Where a layer's exponents lie: page strides in units of 8 bytes, heads in bytes.
struct Exponents {
  const uint8_t *ke, *ve;
  int64_t ke_head, ve_head;
  int32_t kep8, vep8;
};
inline Exponents exponents_of(const PagedAttnArgs &p) {
  return Exponents{p.k_exp, p.v_exp, p.ke_head, p.ve_head, p.kep8, p.vep8};
}
// A page of 128 columns of 16 bits in one box: dimensions are 64 columns, 8 rows, the two 64s, eights of rows, pages,
// and a head is a step of the third (heads next to each other) or of the fourth (heads a page's rows apart).
constexpr int kPairShift = 5;  // pages of up to 32
struct Pairs {
  int32_t kz, kw, vz, vw;  // a head's step in either
};
inline bool pair_steps(int64_t head, int64_t token, int page, int heads, int32_t &z, int32_t &w) {
  z = head == 128 ? 2 : 0, w = head == 128 ? 0 : page / 8;
  return head == 128 || head == token * page || heads == 1;
}
inline bool page_pairs(const PagedAttnArgs &p, Pairs *s) {
  const int page = 1 << p.page_shift;
  return pair_steps(p.k_head, p.k_token, page, p.kv_heads, s->kz, s->kw) &&
         pair_steps(p.v_head, p.v_token, page, p.kv_heads, s->vz, s->vw);
}

// Maps of a layer's keys and values, 16 bits or codes.
template <int D, bool F8, bool P>
bool page_maps(const PagedAttnArgs &p, const Pairs &s, CUtensorMap *k, CUtensorMap *v) {
  if (P) {
    const uint64_t page = 1ull << p.page_shift;
    const uint32_t box[5] = {64, 8, 2, (uint32_t)(page < fa::kKeys ? page : fa::kKeys) / 8, 1};
    auto map = [&](CUtensorMap *m, const void *at, int64_t token, int64_t in_page, int z) {
      const uint64_t heads = p.kv_heads, eights = page / 8;
      const uint64_t dims[5] = {64, 8, z ? 2 * heads : 2, z ? eights : eights * heads, (uint64_t)p.n_pages};
      const uint64_t strides[4] = {(uint64_t)token * 2, 128, (uint64_t)token * 16, (uint64_t)in_page * 2};
      return encode_16bit(m, at, 5, dims, strides, box);
    };
    return map(k, p.k, p.k_token, p.k_page, s.kz) && map(v, p.v, p.v_token, p.v_page, s.vz);
  }
  const uint64_t page = 1ull << p.page_shift, e = F8 ? 1 : 2;
  const uint64_t dims[4] = {D, page, (uint64_t)p.kv_heads, (uint64_t)p.n_pages};
  const uint64_t sk[3] = {p.k_token * e, p.k_head * e, p.k_page * e};
  const uint64_t sv[3] = {p.v_token * e, p.v_head * e, p.v_page * e};
  const uint32_t box[4] = {F8 ? D : 64, (uint32_t)(page < fa::kKeys ? page : fa::kKeys), 1, 1};
  if (F8) return encode_8bit(k, p.k, 4, dims, sk, box, D == 128) && encode_8bit(v, p.v, 4, dims, sv, box, D == 128);
  return encode_16bit(k, p.k, 4, dims, sk, box) && encode_16bit(v, p.v, 4, dims, sv, box);
}

// A warp of four that turn key and value tiles of 8 bits, which TMA has brought,
// into tiles of 16 bits in the layout of its 128-byte swizzle: piece c (16 bytes)
// of row r's half h (64 columns) at h * kHalf + r * 128 + (c ^ (r & 7)) * 16.
//
// With 128 columns a row's codes lie where its last 128 bytes will be (there is
// no room beside the ring): a warp reads its rows and then writes over them.  A
// code times its row's power of two is exact in bf16 (fp32 in between), and in
// fp16: by one multiplication of two where the power is within 2^-14 and 2^7,
// otherwise through fp32 and rounded where it is outside fp16's range.
//
// What other forms took (16 trees of 60 nodes behind 512 to 4096 tokens, 32 heads
// on 8, pages of 16; a whole call): these warps fetching the codes themselves, by
// cp.async 79 us, and 87 with the code for it in four places, which the softmax's
// instruction cache did not stand; loads a tile ahead in registers 184, with
// spills.
template <typename T, int D, typename Args, typename Work>
struct PageConverter {
  static constexpr int kPieces = D / 16;  // of a row of codes
  static constexpr int kRows = 32 / kPieces, kPass = 4 * kRows, kPasses = fa::kKeys / kPass;
  static constexpr int kAtOnce = 2;  // passes converted at once
  int next;          // lanes 0 .. 15: the page of eight rows of the next tile, as it was read (-1: none)
  uint32_t exps[2];  // the tile's exponents of keys and values: lane l has the l-th of the warp's rows

  static __device__ __forceinline__ int fetch(const Args &a, const Work &w, int j, int n, int lane) {
    const int p = (w.j0 + j) * fa::kKeys + lane * 8;
    if (j >= n || lane >= fa::kKeys / 8 || p >= w.len) return -1;
    return a.table[(size_t)w.seq * a.table_ld + (p >> a.page_shift)];
  }
  // This lane's row of a pass and piece of it: eight lanes store two pieces each of two rows, so that neighbours'
  // pieces fall into different banks.
  static __device__ __forceinline__ int row_of(int lane) {
    return D == 128 ? (lane >> 2 & 1) | lane >> 4 << 1 : lane >> 2;
  }
  static __device__ __forceinline__ int piece_of(int lane) {
    return D == 128 ? (lane & 3) | (lane >> 3 & 1) << 2 : lane & 3;
  }
  static __device__ __forceinline__ uint32_t code_at(int r, int piece) {
    return D == 128 ? r * 128 + ((piece ^ (r & 7)) << 4) : r * 64 + (piece << 4);
  }

  // The exponents of tile j, whose pages are in `next`; then the pages after it.
  __device__ __forceinline__ void exponents(const Args &a, const Work &w, int j, int n, int cw, int lane) {
    const int row = lane / kRows * kPass + cw * kRows + lane % kRows, head = w.unit * a.pack / a.group;
    const int page = __shfl_sync(0xffffffffu, next, row >> 3);
    const int pos = ((w.j0 + j) * fa::kKeys + row) & ((1 << a.page_shift) - 1);
    exps[0] = exps[1] = 127;
    if (page >= 0 && page < a.n_pages) {  // (coherent loads: this kernel may have begun before the bytes were written)
      exps[0] = a.rows.ke[head * a.rows.ke_head + 8 * ((int64_t)page * a.rows.kep8) + pos];
      exps[1] = a.rows.ve[head * a.rows.ve_head + 8 * ((int64_t)page * a.rows.vep8) + pos];
    }
    next = fetch(a, w, j + 1, n, lane);
  }
  __device__ __forceinline__ void begin(const Args &a, const Work &w, int cw, int lane, int n) {
    next = fetch(a, w, 0, n, lane);
    exponents(a, w, 0, n, cw, lane);
  }

  // 16 codes as as many T.
  static __device__ __forceinline__ void convert(const uint32_t *c, uint32_t byte, bool plain, uint32_t *to) {
    const float f = attn::scale_of(byte);
    if (attn::Type<T>::kBf16 || !plain) {
      const uint64_t f2 = umma::pack2(f, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 v = attn::Type<__half>::unpack(i & 1 ? attn::from_e4m3_hi(c[i / 2]) : attn::from_e4m3(c[i / 2]));
        float lo, hi;
        umma::unpack2(umma::mul2(umma::pack2(v.x, v.y), f2), lo, hi);
        if (!attn::Type<T>::kBf16) {  // (a NaN stays one)
          lo = lo > 65504.f ? 65504.f : lo < -65504.f ? -65504.f : lo;
          hi = hi > 65504.f ? 65504.f : hi < -65504.f ? -65504.f : hi;
        }
        to[i] = attn::Type<T>::pack(lo, hi);
      }
    } else {
      const __half2 h = __float2half2_rn(f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t v = i & 1 ? attn::from_e4m3_hi(c[i / 2]) : attn::from_e4m3(c[i / 2]);
        const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&v), h);
        to[i] = *reinterpret_cast<const uint32_t *>(&y);
      }
    }
  }

  // The tile at dst from the codes at src, with the exponents `now`.
  __device__ __forceinline__ void tile(uint32_t dst, uint32_t src, uint32_t now, int cw, int lane) const {
    const int piece = piece_of(lane), row = cw * kRows + row_of(lane);
    const bool plain = attn::Type<T>::kBf16 || __all_sync(0xffffffffu, now - 113u <= 21u);
#pragma unroll 1
    for (int p0 = 0; p0 < kPasses; p0 += kAtOnce) {
      uint32_t x[kAtOnce][4];
#pragma unroll
      for (int p = 0; p < kAtOnce; ++p) attn::lds16(src + code_at((p0 + p) * kPass + row, piece), x[p]);
      __syncwarp();  // every lane has read the rows that are written over now
#pragma unroll
      for (int p = 0; p < kAtOnce; ++p) {
        const int r = (p0 + p) * kPass + row;
        uint32_t y[8];
        convert(x[p], __shfl_sync(0xffffffffu, now, (p0 + p) * kRows + row_of(lane)), plain, y);
        const uint32_t line = dst + (piece >> 2) * fa::kHalf + r * 128;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t to = line + (((2 * piece + h) & 7) ^ (r & 7)) * 16;
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(y[4 * h]), "r"(y[4 * h + 1]),
                       "r"(y[4 * h + 2]), "r"(y[4 * h + 3])
                       : "memory");
        }
      }
    }
  }
};

template <typename Work>
struct NodeWild {  // new tokens whose value is not finite, per column
  unsigned long long nan[128], pos[128], neg[128];
  __device__ __forceinline__ void none(int d) { nan[d] = pos[d] = neg[d] = 0; }
  // (a value of the context stays: every row sees it)
  __device__ __forceinline__ bool note(const Work &w, int j, int r, int d, float x) {
    const int node = (w.j0 + j) * fa::kKeys + r - w.ctx;
    if (node < 0) return false;
    (x != x ? nan[d] : x > 0.f ? pos[d] : neg[d]) |= 1ull << node;
    return true;
  }
  template <typename R>
  __device__ __forceinline__ int seen(const R &row, int d) const {
    const bool n = nan[d] & row.word, p = pos[d] & row.word, b = neg[d] & row.word;
    return n || (p && b) ? 1 : p ? 2 : b ? 3 : 0;
  }
};

// Rows of a value tile behind the sequence's end: what the ring held before, or what their page holds.
template <int D, typename M, typename Work>
__device__ __forceinline__ bool clear_behind(const Work &w, int j, uint8_t *tile, int lane) {
  const int r0 = max(0, w.len - (w.j0 + j) * fa::kKeys);
  for (int h = 0; h < D / 64; ++h)
    for (int x = r0 * 8 + lane; x < fa::kKeys * 8; x += kWarp)
      *reinterpret_cast<uint4 *>(tile + fa::Tile<D, M>::piece(x >> 3, h, x & 7)) = make_uint4(0, 0, 0, 0);
  __syncwarp();
  return r0 < fa::kKeys;
}

}  // namespace paged
}  // namespace ns
