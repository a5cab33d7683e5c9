// What the tensor-core kernels over a paged cache share (ns_paged_umma.cu,
// ns_shared_attn.cu): keys and values page by page, and values behind a
// sequence's end or of new tokens that some rows do not see.
#pragma once

#include "ns_paged_attn.cuh"
#include "ns_umma_attn.cuh"

namespace ns {
namespace paged {

// A whole warp fetches key and value tiles, a lane a page.  Work has the cache's sequence (seq, len), the tiles (j0,
// tiles()) and the heads (unit); Args the table and the pages.
template <typename Args, typename Work>
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
    if (lane == 0) mbar_expect_tx(bar, n * rows * D * 2);
    __syncwarp();
    if (lane < n) {
      const int row = page > fa::kKeys ? (w.j0 + j) * fa::kKeys & (page - 1) : 0;
      for (int h = 0; h < D / 64; ++h)
        umma::tma4(dst + h * fa::kHalf + lane * rows * 128, m, h * 64, row, w.unit * a.pack / a.group, ids, bar);
    }
    __syncwarp();
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
template <int D, typename Work>
__device__ __forceinline__ bool clear_behind(const Work &w, int j, uint8_t *tile, int lane) {
  const int r0 = max(0, w.len - (w.j0 + j) * fa::kKeys);
  for (int h = 0; h < D / 64; ++h)
    for (int x = r0 * 8 + lane; x < fa::kKeys * 8; x += kWarp)
      reinterpret_cast<uint4 *>(tile + h * fa::kHalf)[x] = make_uint4(0, 0, 0, 0);
  __syncwarp();
  return r0 < fa::kKeys;
}

}  // namespace paged
}  // namespace ns
