// What the kernels of attention over a paged cache share: the line of tiles,
// the workspace of the parts, and the join.
//
// The keys of every (sequence, heads, block of rows) of a call, an item, are
// cut into tiles; all tiles of the call are in one line, sequence by
// sequence, and CTA c of G has tiles total c / G .. total (c + 1) / G of it.
// A CTA whose share begins or ends inside an item leaves its rows' (m, l, o)
// in the workspace, at most two of them; the join adds up the parts of such
// items in CTA order.  No atomics: the same inputs give the same bits.
#pragma once

#include "ns_attn_tile.cuh"
#include "ns_internal.cuh"
#include "ns_ops.cuh"

namespace ns {
namespace paged {

using namespace attn;

// Workspace: cum int64 [n_seqs + 1], then (m, l) and o of two parts per CTA.
struct Ws {
  long long *cum;
  float2 *ml;  // [ctas x 2 x rows]
  float *o;    // [ctas x 2 x rows x D]
};
__host__ __device__ inline Ws workspace(void *p, int n_seqs, int ctas, int rows) {
  Ws w;
  w.cum = static_cast<long long *>(p);
  const size_t c = ((size_t)(n_seqs + 1) * 8 + 255) & ~(size_t)255;
  w.ml = reinterpret_cast<float2 *>(static_cast<char *>(p) + c);
  w.o = reinterpret_cast<float *>(w.ml + (size_t)ctas * 2 * rows);
  return w;
}

// a / b of nonnegative a: 32 bits where both fit (a division of 64 bits is a
// hundred instructions, and a chain of them is a good part of a short call).
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return (a | b) >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

__device__ __forceinline__ int length(const PagedAttnArgs &a, int b, uint32_t *err) {
  const int s = a.seqs[b];
  if (s < 0 || s >= a.max_seqs) {
    if (err) set_flag(err, NS_FLAG_BAD_SEQ);
    return 0;
  }
  const int len = a.lengths[s];
  if (len < 0 || (long long)len > ((long long)a.table_ld << a.page_shift)) {
    if (err) set_flag(err, NS_FLAG_BAD_SEQ);
    return 0;
  }
  return len;
}

// Joins the parts of an item that several CTAs had.  A CTA has some rows of an
// item; kGroups warps have a row's parts in turns and join in group order.
// R says how an item's rows lie: kRows of them, kGroups, and where each goes.
constexpr int kJoinWarps = 8;
template <typename T, int D, typename R>
__global__ void __launch_bounds__(kJoinWarps * 32)
    join_kernel(const PagedAttnArgs a, const R rows, void *ws_, int items, int ctas) {
  constexpr int kRows = R::kRows, N = D / 32, G = R::kGroups, kPer = kJoinWarps / G;
  extern __shared__ int s_part[];  // [ctas] rows before each part
  __shared__ float s_o[G][kPer][D];
  __shared__ float s_l[G][kPer];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, grp = warp % G, rw = warp / G;
  const int b = blockIdx.x / items, item = blockIdx.x % items, rl = blockIdx.y * kPer + rw;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Ws ws = workspace(ws_, a.n_seqs, ctas, kRows);
  const long long total = ws.cum[a.n_seqs], cb = ws.cum[b];
  const long long nt = quotient(ws.cum[b + 1] - cb, items);
  const long long from = cb + item * nt, to = from + nt;  // the item's tiles
  const int c0 = (int)quotient((from + 1) * ctas - 1, total), c1 = (int)quotient(to * ctas - 1, total);
  if (c0 == c1) return;  // one CTA had it all
  for (int c = c0 + tid; c <= c1; c += kJoinWarps * 32) {
    const long long first = quotient(total * c, ctas);
    // a part is its CTA's first unless the CTA began before the item; a CTA may have no tiles at all
    s_part[c - c0] = first == quotient(total * (c + 1), ctas) ? -1 : (c * 2 + (first >= from ? 0 : 1)) * kRows;
  }
  __syncthreads();
  int node, qh;
  const bool live = rl < kRows && rows.place(a, item, rl, node, qh);
  const int parts = c1 - c0 + 1;
  float m = kNegInf, l = 0.f, o[N];
#pragma unroll
  for (int i = 0; i < N; ++i) o[i] = 0.f;
  if (live) {
    for (int q = lane; q < parts; q += kWarp)
      if (s_part[q] >= 0) m = fmaxf(m, ws.ml[s_part[q] + rl].x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    const float safe = m == kNegInf ? 0.f : m;
#pragma unroll 8
    for (int q = grp; q < parts; q += G) {
      if (s_part[q] < 0) continue;
      const size_t at = (size_t)s_part[q] + rl;
      const float2 ml = ws.ml[at];
      const float f = ex2(ml.x - safe);
      l += ml.y * f;
      const float *src = ws.o + at * D + lane * N;
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = fmaf(src[i], f, o[i]);
    }
  }
  if (G > 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) s_o[grp][rw][lane * N + i] = o[i];
    if (lane == 0) s_l[grp][rw] = l;
    __syncthreads();
    if (grp != 0) return;
#pragma unroll
    for (int g = 1; g < G; ++g) {
      l += s_l[g][rw];
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] += s_o[g][rw][lane * N + i];
    }
  }
  if (!live) return;
  const int64_t at = ((int64_t)b * a.n + node) * a.q_heads + qh;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<T *>(a.out) + at * D + lane * N);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) dst[i] = Type<T>::pack(o[2 * i] * inv, o[2 * i + 1] * inv);
  if (a.lse && lane == 0) a.lse[at] = l == 0.f ? kNegInf : (m - rows.template offset<T>() + log2f(l)) * kLn2;
}

// Launches the join so that it starts while the kernel before it ends.
template <typename T, int D, typename R>
cudaError_t launch_join(const PagedAttnArgs &a, const R &rows, int used_rows, int items, int ctas, cudaStream_t st) {
  constexpr int kPer = kJoinWarps / R::kGroups;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((long long)a.n_seqs * items), (unsigned)((used_rows + kPer - 1) / kPer));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.dynamicSmemBytes = ctas * 4;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<T, D, R>, a, rows, a.ws, items, ctas);
}

}  // namespace paged
}  // namespace ns
