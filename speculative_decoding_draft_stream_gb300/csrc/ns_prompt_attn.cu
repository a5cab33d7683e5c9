// Causal attention over whole packed prompts.
//
// A CTA has 64 consecutive tokens of one sequence and one query head; its
// four warps have 16 rows each and walk the keys up to their own diagonal in
// tiles of 64, two ahead in flight (cp.async).  The longest blocks come first.
#include "ns_internal.cuh"
#include "ns_ops.cuh"
#include "ns_attn_tile.cuh"

namespace ns {
namespace {

using namespace attn;

constexpr int kPrThreads = 128;
constexpr int kPrRows = 64, kPrKeys = 64, kPrStages = 3;

template <int D>
__host__ __device__ constexpr int pr_stage() {
  return 2 * kPrKeys * D * 2;
}

template <typename T, int D>
__global__ void __launch_bounds__(kPrThreads) prompt_attn_kernel(const PromptAttnArgs a) {
  constexpr int kLanesRow = D / 8, kPass = kPrThreads / kLanesRow;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int seq = blockIdx.z, head = blockIdx.y, kvh = head / a.group;
  const int t0 = a.cu[seq], t1 = a.cu[seq + 1];
  if (t0 < 0 || t1 < t0 || t1 > a.tokens) {
    if (tid == 0) set_flag(a.err, NS_FLAG_BAD_SEQ);
    return;
  }
  if (t1 - t0 > a.max_len && blockIdx.x == 0 && tid == 0) set_flag(a.err, NS_FLAG_BAD_SEQ);
  const int len = min(t1 - t0, a.max_len);
  const int r0 = ((int)gridDim.x - 1 - (int)blockIdx.x) * kPrRows;
  if (r0 >= len) return;
  const uint32_t s0 = (uint32_t)__cvta_generic_to_shared(smem);
  const T *kb = static_cast<const T *>(a.k) + (int64_t)t0 * a.k_token + (int64_t)kvh * a.k_head;
  const T *vb = static_cast<const T *>(a.v) + (int64_t)t0 * a.v_token + (int64_t)kvh * a.v_head;
  const T *qb = static_cast<const T *>(a.q) + (int64_t)t0 * a.q_token + (int64_t)head * a.q_head;
  const int last = min(len, r0 + kPrRows);  // keys this block sees
  const int tiles = (last + kPrKeys - 1) / kPrKeys;
  const int fr = tid / kLanesRow, fc = tid % kLanesRow;
  auto issue = [&](int t) {
    if (t < tiles) {
      const uint32_t sk = s0 + (t % kPrStages) * pr_stage<D>(), sv = sk + kPrKeys * D * 2;
#pragma unroll
      for (int pass = 0; pass < kPrKeys / kPass; ++pass) {
        const int r = pass * kPass + fr, p = t * kPrKeys + r;
        const bool ok = p < last;
        const int64_t row = ok ? p : 0;
        cp16(sk + piece<D>(r, fc), kb + row * a.k_token + fc * 8, ok);
        cp16(sv + piece<D>(r, fc), vb + row * a.v_token + fc * 8, ok);
      }
    }
    cp_commit();
  };
  issue(0);
  issue(1);
  uint32_t q[D / 16][4];
  const int row[2] = {r0 + warp * 16 + (lane >> 2), r0 + warp * 16 + (lane >> 2) + 8};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const bool ok = row[h] < len;
    const T *src = qb + (int64_t)(ok ? row[h] : 0) * a.q_token + (lane & 3) * 2;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      q[kk][h] = ok ? *reinterpret_cast<const uint32_t *>(src + kk * 16) : 0u;
      q[kk][2 + h] = ok ? *reinterpret_cast<const uint32_t *>(src + kk * 16 + 8) : 0u;
    }
  }
  Rows<T, D> rows;
  rows.clear();
  const float c = a.scale * kLog2e;
  for (int t = 0; t < tiles; ++t) {
    cp_wait<kPrStages - 2>();
    __syncthreads();
    issue(t + kPrStages - 1);
    const uint32_t sk = s0 + (t % kPrStages) * pr_stage<D>(), sv = sk + kPrKeys * D * 2;
    const int p0 = t * kPrKeys;
    if (p0 + kPrKeys - 1 <= r0 + warp * 16) {
      rows.template tile<kPrKeys, false>(q, sk, sv, 0, c, [](int, int) { return false; }, false);
    } else {
      const bool wild = __any_sync(0xffffffffu, wild_pieces<T>(sv, kPrKeys * D / 8, lane, kWarp));
      rows.template tile<kPrKeys, true>(q, sk, sv, 0, c, [&](int h, int key) { return p0 + key > row[h]; }, wild);
    }
  }
  rows.sum_l();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (row[h] >= len) continue;
    const int64_t at = (int64_t)(t0 + row[h]) * a.q_heads + head;
    const float inv = rows.l[h] == 0.f ? 0.f : 1.f / rows.l[h];
    uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<T *>(a.out) + at * D) + (lane & 3);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) dst[i * 4] = Type<T>::pack(rows.o[i][2 * h] * inv, rows.o[i][2 * h + 1] * inv);
    if (a.lse && (lane & 3) == 0) a.lse[at] = row_lse<T>(rows.m[h], rows.l[h]);
  }
}

template <typename T, int D>
cudaError_t launch(const PromptAttnArgs &a, cudaStream_t st) {
  const dim3 grid((unsigned)((a.max_len + kPrRows - 1) / kPrRows), (unsigned)a.q_heads, (unsigned)a.n_seqs);
  prompt_attn_kernel<T, D><<<grid, kPrThreads, kPrStages * pr_stage<D>(), st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t prepare_prompt_attn() {
  cudaError_t e = cudaSuccess;
  auto set = [&](const void *f, int bytes) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  };
  set((const void *)prompt_attn_kernel<__nv_bfloat16, 128>, kPrStages * pr_stage<128>());
  set((const void *)prompt_attn_kernel<__nv_bfloat16, 64>, kPrStages * pr_stage<64>());
  set((const void *)prompt_attn_kernel<__half, 128>, kPrStages * pr_stage<128>());
  set((const void *)prompt_attn_kernel<__half, 64>, kPrStages * pr_stage<64>());
  return e;
}

cudaError_t launch_prompt_attn(const PromptAttnArgs &a, int dtype, int dim, int sms, cudaStream_t st) {
  (void)sms;
  if (dtype == NS_DTYPE_BF16) return dim == 128 ? launch<__nv_bfloat16, 128>(a, st) : launch<__nv_bfloat16, 64>(a, st);
  return dim == 128 ? launch<__half, 128>(a, st) : launch<__half, 64>(a, st);
}

}  // namespace ns
