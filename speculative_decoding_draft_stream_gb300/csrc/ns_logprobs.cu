// Log probabilities of given tokens, entropy and top alternatives, in one
// pass over the logits.
//
// With z = x / T and m = max x, d = (x - m) / T:
//   lse = m / T + log S,           S = sum exp(d)
//   log p(x) = d - log S
//   entropy = log S - U / S,       U = sum exp(d) d
// Every thread keeps (m, S, U) of what it has read, in powers of two; when its
// maximum grows by delta, S and U move with it: S' = S 2^-delta,
// U' = 2^-delta (U - delta S).  Two such triples join the same way.
//
// The top k need no second read of the row.  A thread's maximum is m, so the
// k-th largest of the CTA's thread maxima bounds the k-th largest value from
// below, and only the k or so threads whose maximum reaches it can hold one
// of the top k: their few values alone are read again (from L2) and ranked.
//
// A row is one CTA, or a cluster of up to eight that split it and join their
// triples and lists through distributed shared memory: one launch, no
// workspace, and a fixed order of every sum.
//
// What bounds it: HBM for many rows (each logit crosses it once); for a few
// rows, latency (one wave of loads, the joins).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ns_internal.cuh"
#include "ns_ops.cuh"
#include "ns_umma_ptx.cuh"

namespace ns {
namespace {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / kWarp;
constexpr int kLpVecs = 4;        // 16-byte loads a thread keeps in flight
constexpr int kLpMaxCluster = 8;  // portable cluster size
constexpr int kLpMinSlice = 4096; // least logits of a CTA of a split row
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// max(x, lo), NaN where x is NaN
__device__ __forceinline__ float floor_nan(float x, float lo) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(lo));
  return y;
}

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4 &u, float *x) {
    x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y), x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ float one(float v) { return v; }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4 &u, float *x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ float one(__nv_bfloat16 v) { return __bfloat162float(v); }
};
template <>
struct Vec<__half> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4 &u, float *x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ float one(__half v) { return __half2float(v); }
};

constexpr float kFloorD = -200.f;  // 2^-200 is 0 in fp32: a smaller exponent adds nothing to S or U

// (m, S, U) of some logits, in powers of two.
struct Part {
  float m, s, u;
  // moves the sums to the maximum `to` >= m; c = log2(e) / T
  __device__ __forceinline__ void raise(float to, float c) {
    if (to == m) return;
    const float d = fmaxf((m - to) * c, kFloorD), f = ex2(d);
    u = f * fmaf(d, s, u);
    s *= f;
    m = to;
  }
  __device__ __forceinline__ void join(Part o, float c) {
    const float to = fmaxf(m, o.m);
    raise(to, c);
    o.raise(to, c);
    s += o.s;
    u += o.u;
  }
  template <int N>
  __device__ __forceinline__ void add(const float *x, float c) {
    float top = x[0];
#pragma unroll
    for (int i = 1; i < N; ++i) top = fmaxf(top, x[i]);
    if (top > m) raise(top, c);
    const float at = m == kNegInf ? 0.f : -m;  // nothing but -inf so far: exponents of -inf, not NaN
    if (N == 1) {
      const float d = floor_nan((x[0] + at) * c, kFloorD), e = ex2(d);
      s += e;
      u = fmaf(e, d, u);
    } else {  // two at a time
      const uint64_t at2 = umma::pack2(at, at), c2 = umma::pack2(c, c);
      uint64_t s2 = 0, u2 = 0;
#pragma unroll
      for (int i = 0; i + 1 < N; i += 2) {
        float a, b;
        umma::unpack2(umma::mul2(umma::add2(umma::pack2(x[i], x[i + 1]), at2), c2), a, b);
        a = floor_nan(a, kFloorD), b = floor_nan(b, kFloorD);
        const uint64_t e2 = umma::pack2(ex2(a), ex2(b));
        s2 = umma::add2(s2, e2);
        u2 = umma::fma2(e2, umma::pack2(a, b), u2);
      }
      float a, b;
      umma::unpack2(s2, a, b);
      s += a + b;
      umma::unpack2(u2, a, b);
      u += a + b;
    }
  }
};

__device__ __forceinline__ uint32_t peer_addr(const void *p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(r)
               : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t ld_peer(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sync_cluster() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A warp's sorted list of its k best (key, id): lane r holds the r-th.
struct WarpList {
  uint32_t key, id;
  __device__ __forceinline__ void clear() { key = 0u, id = (uint32_t)kEmptyId; }
  // ck, ci the same in every lane; ck != 0
  __device__ __forceinline__ void insert(uint32_t ck, uint32_t ci, int lane) {
    const bool ahead = key > ck || (key == ck && id < ci);
    const int pos = __popc(__ballot_sync(0xffffffffu, ahead));  // ahead holds for a prefix of the lanes
    const uint32_t pk = __shfl_up_sync(0xffffffffu, key, 1), pi = __shfl_up_sync(0xffffffffu, id, 1);
    if (lane > pos) key = pk, id = pi;
    if (lane == pos) key = ck, id = ci;
  }
};

// One row by the `split` CTAs of a cluster (split = 1: no cluster).  The
// row's 16-byte pieces are counted from the aligned address at or before its
// first logit; the pieces at its ends may be partly outside and are read
// value by value.
template <typename T, bool kSplit>
__global__ void __launch_bounds__(kLpThreads) logprob_kernel(const LogprobArgs a, int split) {
  using V = Vec<T>;
  constexpr int N = V::N;
  __shared__ Part s_part[kLpWarps];
  __shared__ Part s_all;
  __shared__ __align__(16) uint32_t s_keys[kLpThreads];
  __shared__ uint32_t s_mask[kLpWarps], s_min[kLpWarps];
  __shared__ uint32_t s_lk[kLpWarps * NS_MAX_ALTERNATIVES], s_li[kLpWarps * NS_MAX_ALTERNATIVES];
  __shared__ uint32_t s_rk[NS_MAX_ALTERNATIVES], s_ri[NS_MAX_ALTERNATIVES];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = kSplit ? (int)(blockIdx.x % split) : 0;
  const int r = kSplit ? (int)(blockIdx.x / split) : (int)blockIdx.x;
  const float c = kLog2e * a.inv_temperature;
  const T *row = static_cast<const T *>(a.logits) + (int64_t)r * a.ld;
  const int mis = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
  const uint4 *vec = reinterpret_cast<const uint4 *>(row - mis);
  const int pieces = (a.V + mis + N - 1) / N;  // of the row, ends included
  const int per = kSplit ? (pieces + split - 1) / split : pieces;
  const int v0 = rank * per, v1 = min(pieces, v0 + per);
  const int first_whole = mis ? 1 : 0, last_whole = (a.V + mis) / N;
  const int w0 = max(v0, first_whole), w1 = min(v1, last_whole);  // whole pieces of this CTA

  Part p{kNegInf, 0.f, 0.f};
  {
    const uint4 *v = vec + w0 + tid;
    int left = w1 - w0 - tid;
    for (; left > (kLpVecs - 1) * kLpThreads; left -= kLpVecs * kLpThreads, v += kLpVecs * kLpThreads) {
      uint4 u[kLpVecs];
#pragma unroll
      for (int q = 0; q < kLpVecs; ++q) u[q] = __ldg(v + q * kLpThreads);
      float x[kLpVecs * N];
#pragma unroll
      for (int q = 0; q < kLpVecs; ++q) V::unpack(u[q], x + q * N);
      p.add<kLpVecs * N>(x, c);
    }
    for (; left > 0; left -= kLpThreads, v += kLpThreads) {
      float x[N];
      V::unpack(__ldg(v), x);
      p.add<N>(x, c);
    }
  }
  // the pieces at the row's ends: threads 0 and 1 of the CTAs that have them
  const int end_piece = tid == 0 ? 0 : pieces - 1;
  const bool has_end = (tid == 0 && mis && v0 == 0) ||
                       (tid == 1 && v1 == pieces && v0 < pieces && last_whole < pieces && !(mis && pieces == 1));
  if (has_end) {
    for (int e = 0; e < N; ++e) {
      const int i = end_piece * N + e - mis;
      if (i >= 0 && i < a.V) {
        const float x = V::one(row[i]);
        p.add<1>(&x, c);
      }
    }
  }

  const uint32_t my_key = order_key(p.m);
  if (a.k > 0) s_keys[tid] = my_key;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    Part o;
    o.m = __shfl_xor_sync(0xffffffffu, p.m, off);
    o.s = __shfl_xor_sync(0xffffffffu, p.s, off);
    o.u = __shfl_xor_sync(0xffffffffu, p.u, off);
    p.join(o, c);
  }
  if (lane == 0) s_part[warp] = p;
  __syncthreads();
  if (warp == 0) {
    p = s_part[lane % kLpWarps];
#pragma unroll
    for (int off = kLpWarps / 2; off > 0; off >>= 1) {
      Part o;
      o.m = __shfl_xor_sync(0xffffffffu, p.m, off);
      o.s = __shfl_xor_sync(0xffffffffu, p.s, off);
      o.u = __shfl_xor_sync(0xffffffffu, p.u, off);
      p.join(o, c);
    }
    if (lane == 0) s_all = p;
  }

  if (a.k > 0) {
    // threads that may hold one of the CTA's k best: fewer than k maxima are larger
    int larger = 0;
    const uint4 *k4 = reinterpret_cast<const uint4 *>(s_keys);
#pragma unroll 8
    for (int q = 0; q < kLpThreads / 4; ++q) {
      const uint4 u = k4[q];
      larger += (u.x > my_key) + (u.y > my_key) + (u.z > my_key) + (u.w > my_key);
    }
    const bool mine = larger < a.k;
    const uint32_t ball = __ballot_sync(0xffffffffu, mine);
    const uint32_t low = __reduce_min_sync(0xffffffffu, mine ? my_key : 0xffffffffu);
    if (lane == 0) s_mask[warp] = ball, s_min[warp] = low;
    __syncthreads();
    uint32_t least = s_min[0];
#pragma unroll
    for (int q = 1; q < kLpWarps; ++q) least = min(least, s_min[q]);
    WarpList L;
    L.clear();
    // inserts every lane's value (x of logit i; ok: there is one) that may be among the k best
    auto offer = [&](float x, int i, bool ok) {
      const uint32_t key = ok ? order_key(x) : 0u;
      const uint32_t kk = __shfl_sync(0xffffffffu, L.key, a.k - 1), ki = __shfl_sync(0xffffffffu, L.id, a.k - 1);
      uint32_t in = __ballot_sync(0xffffffffu, key != 0u && key >= least && (key > kk || (key == kk && (uint32_t)i < ki)));
      for (; in; in &= in - 1) {
        const int from = __ffs(in) - 1;
        L.insert(__shfl_sync(0xffffffffu, key, from), (uint32_t)__shfl_sync(0xffffffffu, i, from), lane);
      }
    };
    int nth = 0;
    for (int w = 0; w < kLpWarps; ++w) {
      for (uint32_t left = s_mask[w]; left; left &= left - 1, ++nth) {
        if (nth % kLpWarps != warp) continue;
        const int owner = w * kWarp + __ffs(left) - 1;
        for (int v = w0 + owner; v < w1; v += kWarp * kLpThreads) {  // 32 of the owner's pieces at a time
          const int piece = v + lane * kLpThreads;
          const bool ok = piece < w1;
          float x[N];
          V::unpack(ok ? __ldg(vec + piece) : make_uint4(0, 0, 0, 0), x);
#pragma unroll
          for (int e = 0; e < N; ++e) offer(x[e], piece * N + e - mis, ok);
        }
        const int ep = owner == 0 ? 0 : pieces - 1;
        const bool end = (owner == 0 && mis && v0 == 0) ||
                         (owner == 1 && v1 == pieces && v0 < pieces && last_whole < pieces && !(mis && pieces == 1));
        if (end) {
          const int i = ep * N + lane - mis;
          const bool ok = lane < N && i >= 0 && i < a.V;
          offer(ok ? V::one(row[i]) : 0.f, i, ok);
        }
      }
    }
    if (lane < a.k) {
      s_lk[warp * a.k + lane] = L.key;
      s_li[warp * a.k + lane] = L.id;
    }
    __syncthreads();
    if (warp == 0) {
      uint32_t lk, li;
      warp_merge_lists(s_lk, s_li, kLpWarps, a.k, s_rk, s_ri, lk, li);
    }
  }
  __syncthreads();

  if (kSplit) {
    sync_cluster();  // every CTA's triple and list are in its shared memory
    if (rank == 0 && warp == 0) {
      Part q{kNegInf, 0.f, 0.f};
      for (int o = 0; o < split; ++o) {  // in rank order
        const uint32_t at = peer_addr(&s_all, o);
        q.join(Part{__uint_as_float(ld_peer(at)), __uint_as_float(ld_peer(at + 4)), __uint_as_float(ld_peer(at + 8))},
               c);
      }
      if (a.k > 0) {
        for (int e = lane; e < split * a.k; e += kWarp) {
          s_lk[e] = ld_peer(peer_addr(&s_rk[e % a.k], e / a.k));
          s_li[e] = ld_peer(peer_addr(&s_ri[e % a.k], e / a.k));
        }
      }
      __syncwarp();
      uint32_t lk = 0u, li = 0u;
      if (a.k > 0) warp_merge_lists(s_lk, s_li, split, a.k, s_keys, s_keys + NS_MAX_ALTERNATIVES, lk, li);
      if (lane == 0) s_all = q;  // only rank 0 reads it from here on: q is what each of its lanes holds
    }
    sync_cluster();  // no CTA leaves while rank 0 reads it
    if (rank != 0) return;
    __syncthreads();
  }
  const uint32_t *rk = kSplit ? s_keys : s_rk, *ri = kSplit ? s_keys + NS_MAX_ALTERNATIVES : s_ri;
  p = s_all;
  const float log_s = logf(p.s);
  const bool none = p.m == kNegInf && p.s == 0.f;  // nothing but -inf
  auto logprob = [&](float x) { 
    // -inf among others: (-inf - m) / T, unless the row's sums are NaN
    return none || (x == kNegInf && p.s == p.s) ? kNegInf : (x - p.m) * a.inv_temperature - log_s;
  };
  if (tid == 0) {
    if (a.lse) a.lse[r] = none ? kNegInf : p.m * a.inv_temperature + log_s;
    if (a.entropy) a.entropy[r] = none ? 0.f : log_s - kLn2 * (p.u / p.s);
  }
  if (tid < a.k) {
    const uint32_t key = rk[tid];
    a.top_ids[(int64_t)r * a.k + tid] = key ? (int32_t)ri[tid] : -1;
    a.top_logprobs[(int64_t)r * a.k + tid] = key ? logprob(key_value(key)) : kNegInf;
  }
  for (int j = tid; j < a.n_ids; j += kLpThreads) {
    const int id = a.ids[(int64_t)r * a.n_ids + j];
    float out = __int_as_float(0x7fffffff);
    if (id >= 0 && id < a.V)
      out = logprob(V::one(row[id]));
    else if (id != -1)
      set_flag(a.err, NS_FLAG_BAD_ID);
    a.logprobs[(int64_t)r * a.n_ids + j] = out;
  }
}

template <typename T>
cudaError_t launch(const LogprobArgs &a, int split, cudaStream_t st) {
  if (split == 1) {
    logprob_kernel<T, false><<<a.rows, kLpThreads, 0, st>>>(a, 1);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)a.rows * split);
  cfg.blockDim = dim3(kLpThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = split;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, logprob_kernel<T, true>, a, split);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs &a, int dtype, int sms, cudaStream_t st) {
  // a row is split until there are four CTAs for each SM, as long as each CTA keeps kLpMinSlice logits
  int split = 1;
  while (split < kLpMaxCluster && (long long)a.rows * split < 4LL * sms && a.V / (2 * split) >= kLpMinSlice) split *= 2;
  if (dtype == NS_DTYPE_F32) return launch<float>(a, split, st);
  if (dtype == NS_DTYPE_BF16) return launch<__nv_bfloat16>(a, split, st);
  return launch<__half>(a, split, st);
}

}  // namespace ns
