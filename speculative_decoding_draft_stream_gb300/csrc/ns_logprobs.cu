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
// The top k need no second read of the row.  A thread's maximum is m; the k-th
// largest of the maxima of 32 or 64 groups of threads bounds the k-th largest
// value from below, and only threads whose maximum reaches it can hold one of the
// top k: their few values alone are read again (from L2).  Those that reach
// the bound go to a buffer in any order, and each one's place is the number
// of better ones.  Where they do not fit (rows of many equal values), every
// warp keeps a sorted list of its best instead, and the lists are merged.
//
// A row is one CTA, or a cluster of up to eight that split it and join their
// triples and lists through distributed shared memory: one launch, no
// workspace, and a fixed order of every sum.
//
// What bounds it: HBM for many rows (each logit crosses it once): 2048 rows of
// 152064 in bf16 with 5 alternatives take 122 us, 5.1 TB/s (100 us without
// alternatives); the exponentials and sums that hide behind the loads are the
// rest.  For a few rows, latency: a thread's batches of kLpVecs loads follow one
// another, and what is left over comes a load at a time (one row of 128256 in
// fp32 on 8 CTAs: three batches and up to four single loads), then the second
// look and the joins.  With one given token and 10 alternatives one such row
// takes 10.2 us (6.2 without alternatives), 60 rows of 151936 13.0 us (7.5).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ns_internal.cuh"
#include "ns_ops.cuh"
#include "ns_umma_ptx.cuh"

namespace ns {
namespace {

constexpr int kLpVecs = 4;        // 16-byte loads a thread keeps in flight
constexpr int kLpMaxCluster = 8;  // portable cluster size
constexpr int kLpMinSlice = 4096; // least logits of a CTA of a split row
// Above 16 alternatives (kMany), 64 groups instead of 32: 32 groups' least
// maximum lets a third of the threads through.  Rows of 128256, by 32 and by 64 groups
// (us): 126 in fp32, k 14 17.0, 18.2; 17 18.9, 18.7; 24 23.1, 20.8; 32 75.5, 23.6;
// 298 in bf16, k 14 21.0, 21.4; 17 22.9, 21.6; 31 40.9, 27.7.
constexpr int kManyFrom = 17;
constexpr int kLpBuffer = kLpMaxCluster * NS_MAX_ALTERNATIVES;  // candidates of a CTA, or the lists of a cluster
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
  template <int N>
  __device__ __forceinline__ void add(const float *x, float c) {
    float top = x[0];
    if (N >= 8) {
      float t[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
      for (int i = 4; i + 3 < N; i += 4)
#pragma unroll
        for (int q = 0; q < 4; ++q) t[q] = fmaxf(t[q], x[i + q]);
      top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
    } else {
#pragma unroll
      for (int i = 1; i < N; ++i) top = fmaxf(top, x[i]);
    }
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
__device__ __forceinline__ void st_peer(uint32_t a, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ void st_peer(uint32_t a, const Part &p) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(p.m) : "memory");
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a + 4), "f"(p.s) : "memory");
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a + 8), "f"(p.u) : "memory");
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

// A candidate as one number: the larger is the better (key, then lower id);
// 0 is none.
__device__ __forceinline__ unsigned long long candidate(uint32_t key, uint32_t id) {
  return (unsigned long long)key << 32 | (0xffffffffu - id);
}

// The k best of n <= kLpBuffer candidates, best first, each at the place that
// the number of better ones says (a CTA; s has room for n + 1; places left
// over get 0).
template <int kLpThreads>
__device__ __forceinline__ void place_best(const unsigned long long *s, int n, int k, unsigned long long *out) {
  static_assert(kLpThreads >= kLpBuffer, "a thread places one candidate");
  const int tid = threadIdx.x;
  if (tid < n || tid < k) {
    const unsigned long long mine = tid < n ? s[tid] : 0;
    int better = 0, filled = 0;
    const ulonglong2 *s2 = reinterpret_cast<const ulonglong2 *>(s);
#pragma unroll 4
    for (int q = 0; q < (n + 1) / 2; ++q) {
      const ulonglong2 o = s2[q];
      better += o.x > mine;
      filled += o.x != 0;
      if (2 * q + 1 < n) {
        better += o.y > mine;
        filled += o.y != 0;
      }
    }
    if (mine && better < k) out[better] = mine;
    if (tid < k && tid >= filled) out[tid] = 0;
  }
}

// One row by the `split` CTAs of a cluster (split = 1: no cluster).  The
// row's 16-byte pieces are counted from the aligned address at or before its
// first logit; the pieces at its ends may be partly outside and are read
// value by value.
template <typename T, bool kSplit, bool kMany, int kLpThreads>
__global__ void __launch_bounds__(kLpThreads, 1024 / kLpThreads + 1024 / kLpThreads / 4)
    logprob_kernel(const LogprobArgs a, int split) {
  constexpr int kLpWarps = kLpThreads / kWarp;
  using V = Vec<T>;
  constexpr int N = V::N;
  constexpr int kGroups = kMany ? 64 : 32, kGroup = kLpThreads / kGroups;  // groups of threads
  __shared__ uint32_t s_group[kGroups];
  __shared__ float s_top[kLpWarps];
  __shared__ float2 s_sums[kLpWarps];
  __shared__ uint32_t s_mask[kLpWarps];
  __shared__ int s_count;
  __shared__ __align__(16) unsigned long long s_cand[kLpBuffer + 2], s_best[NS_MAX_ALTERNATIVES];
  __shared__ uint32_t s_lk[kLpWarps * NS_MAX_ALTERNATIVES], s_li[kLpWarps * NS_MAX_ALTERNATIVES];
  __shared__ uint32_t s_ok[NS_MAX_ALTERNATIVES], s_oi[NS_MAX_ALTERNATIVES];
  // rank 0's: every CTA's triple and list
  __shared__ Part s_peer[kLpMaxCluster];
  __shared__ __align__(16) unsigned long long s_lists[kSplit ? kLpBuffer + 2 : 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = kSplit ? (int)(blockIdx.x % split) : 0;
  const int r = kSplit ? (int)(blockIdx.x / split) : (int)blockIdx.x;
  const float c = kLog2e * a.inv_temperature;
  if (kSplit) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // this CTA has begun
  const T *row = static_cast<const T *>(a.logits) + (int64_t)r * a.ld;
  const int mis = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
  const uint4 *vec = reinterpret_cast<const uint4 *>(row - mis);
  const int pieces = (a.V + mis + N - 1) / N;  // of the row, ends included
  const int per = kSplit ? (pieces + split - 1) / split : pieces;
  const int v0 = rank * per, v1 = min(pieces, v0 + per);
  const int first_whole = mis ? 1 : 0, last_whole = (a.V + mis) / N;
  const int w0 = max(v0, first_whole), w1 = min(v1, last_whole);  // whole pieces of this CTA

  // the given tokens' logits, on their way while the row is read
  int my_id = -1;
  float my_x = 0.f;
  if (rank == 0 && tid < a.n_ids) {
    my_id = a.ids[(int64_t)r * a.n_ids + tid];
    if (my_id >= 0 && my_id < a.V) my_x = V::one(row[my_id]);
  }

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
  {
    uint32_t most = my_key;
#pragma unroll
    for (int off = kGroup / 2; off > 0; off >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, off));
    if (a.k > 0 && lane % kGroup == 0) s_group[tid / kGroup] = most;
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) s_top[warp] = most ? key_value(most) : kNegInf;
    if (tid == 0) s_count = 0;
  }
  __syncthreads();
  {  // the CTA's maximum, and every thread's sums in terms of it
    float top = s_top[0];
#pragma unroll
    for (int q = 1; q < kLpWarps; ++q) top = fmaxf(top, s_top[q]);
    p.raise(top, c);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      p.s += __shfl_xor_sync(0xffffffffu, p.s, off);
      p.u += __shfl_xor_sync(0xffffffffu, p.u, off);
    }
    if (lane == 0) s_sums[warp] = make_float2(p.s, p.u);
  }
  if (a.k > 0) {
    // threads that may hold one of the CTA's k best: those whose maximum reaches the k-th largest group's
    const uint32_t ga = s_group[lane], gb = kMany ? s_group[lane + kWarp * kMany] : 0u;
    int la = 0, lb = 0;  // larger groups than each
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      const uint32_t o = s_group[q];
      la += o > ga;
      if (kMany) lb += o > gb;
    }
    uint32_t least = la < a.k ? ga : 0xffffffffu;
    if (kMany && lb < a.k) least = min(least, gb);
    least = __reduce_min_sync(0xffffffffu, least);
    const uint32_t ball = __ballot_sync(0xffffffffu, my_key >= least && my_key != 0u);
    if (lane == 0) s_mask[warp] = ball;
    __syncthreads();
    // every lane's value x of logit i (ok: there is one), for each piece that an owner of the mask has read;
    // half a warp takes an owner, 16 of its pieces at a time
    auto rescan = [&](auto offer) {
      const int half = lane >> 4, hl = lane & 15;
      int nth = 0;
      for (int w = 0; w < kLpWarps; ++w) {
        uint32_t left = s_mask[w];
        while (left) {
          // the next two owners' turn is this warp's, or both are passed over
          const int o0 = __ffs(left) - 1;
          left &= left - 1;
          const int o1 = left ? __ffs(left) - 1 : -1;
          left &= left - 1;
          if (nth++ % kLpWarps != warp) continue;
          const int owner = w * kWarp + (half ? o1 : o0);
          const bool live = !half || o1 >= 0;
          for (int v = w0 + w * kWarp + o0; v < w1; v += 16 * kLpThreads) {  // (o0 < o1: o0 has at least as many)
            const int piece = v - (w * kWarp + o0) + owner + hl * kLpThreads;
            const bool ok = live && piece < w1;
            float x[N];
            V::unpack(ok ? __ldg(vec + piece) : make_uint4(0, 0, 0, 0), x);
#pragma unroll
            for (int e = 0; e < N; ++e) offer(x[e], piece * N + e - mis, ok);
          }
          const bool head = w == 0 && mis && v0 == 0;  // the row's end pieces: threads 0 and 1 of their CTAs
          const bool tail = w == 0 && v1 == pieces && v0 < pieces && last_whole < pieces && !(mis && pieces == 1);
          if ((head && o0 == 0) || (tail && (o0 == 1 || o1 == 1))) {
            const bool mine = live && ((owner == 0 && head) || (owner == 1 && tail));
            const int i = (owner == 0 ? 0 : pieces - 1) * N + hl - mis;
            const bool ok = mine && hl < N && i >= 0 && i < a.V;
            offer(ok ? V::one(row[i]) : 0.f, i, ok);
          }
        }
      }
    };
    rescan([&](float x, int i, bool ok) {
      const uint32_t key = ok ? order_key(x) : 0u;
      if (key != 0u && key >= least) {
        const int at = atomicAdd(&s_count, 1);
        if (at < kLpBuffer) s_cand[at] = candidate(key, (uint32_t)i);
      }
    });
    __syncthreads();
    if (s_count <= kLpBuffer) {
      place_best<kLpThreads>(s_cand, s_count, a.k, s_best);
    } else {
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
    rescan(offer);
      if (lane < a.k) {
        s_lk[warp * a.k + lane] = L.key;
        s_li[warp * a.k + lane] = L.id;
      }
      __syncthreads();
      if (warp == 0) {
        uint32_t lk, li;
        warp_merge_lists(s_lk, s_li, kLpWarps, a.k, s_ok, s_oi, lk, li);
        if (lane < a.k) s_best[lane] = s_ok[lane] ? candidate(s_ok[lane], s_oi[lane]) : 0;
      }
    }
  }
  __syncthreads();

  p.s = p.u = 0.f;
#pragma unroll
  for (int q = 0; q < kLpWarps; ++q) p.s += s_sums[q].x, p.u += s_sums[q].y;
  const unsigned long long *best = s_best;
  if (kSplit) {
    // to rank 0's shared memory, once it has begun; the others leave, and rank 0 goes on when all have arrived
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (tid < a.k) st_peer(peer_addr(&s_lists[rank * a.k + tid], 0), s_best[tid]);
    if (tid == 0) st_peer(peer_addr(&s_peer[rank], 0), p);
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    if (rank != 0) return;
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    float top = s_peer[0].m;
    for (int o = 1; o < split; ++o) top = fmaxf(top, s_peer[o].m);
    p = Part{top, 0.f, 0.f};
    for (int o = 0; o < split; ++o) {  // in rank order
      Part q = s_peer[o];
      q.raise(top, c);
      p.s += q.s, p.u += q.u;
    }
    if (a.k > 0) place_best<kLpThreads>(s_lists, split * a.k, a.k, s_best);
    __syncthreads();
  }
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
    const uint32_t key = (uint32_t)(best[tid] >> 32);
    a.top_ids[(int64_t)r * a.k + tid] = key ? (int32_t)(0xffffffffu - (uint32_t)best[tid]) : -1;
    a.top_logprobs[(int64_t)r * a.k + tid] = key ? logprob(key_value(key)) : kNegInf;
  }
  for (int j = tid; j < a.n_ids; j += kLpThreads) {
    const int id = j == tid ? my_id : a.ids[(int64_t)r * a.n_ids + j];
    float out = __int_as_float(0x7fffffff);
    if (id >= 0 && id < a.V)
      out = logprob(j == tid ? my_x : V::one(row[id]));
    else if (id != -1)
      set_flag(a.err, NS_FLAG_BAD_ID);
    a.logprobs[(int64_t)r * a.n_ids + j] = out;
  }
}

// A row is split while the call has fewer than two CTAs for each SM and every
// CTA keeps kLpMinSlice logits.  In fp32 with 10 alternatives, one row of 128256
// takes 10.2 us on 8 CTAs, 10.6 on 4, 14.0 on 2, 15.2 on one; 60 rows of 151936
// take 13.0 us on 4 each, 15.2 on 8, 16.2 on 2, 20.8 on one.
// Threads of a CTA: 512 or 1024 took 27 to 55 us for those 60 rows: the joins
// wait for more warps.
constexpr int kLpThreads = 256;

template <typename T, bool kMany>
cudaError_t launch(const LogprobArgs &a, int sms, cudaStream_t st) {
  int split = 1;
  while (split < kLpMaxCluster && (long long)a.rows * split * 2 <= 2LL * sms && a.V / (2 * split) >= kLpMinSlice)
    split *= 2;
  if (split == 1) {
    logprob_kernel<T, false, kMany, kLpThreads><<<a.rows, kLpThreads, 0, st>>>(a, 1);
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
  return cudaLaunchKernelEx(&cfg, logprob_kernel<T, true, kMany, kLpThreads>, a, split);
}
template <typename T>
cudaError_t by_k(const LogprobArgs &a, int sms, cudaStream_t st) {
  return a.k >= kManyFrom ? launch<T, true>(a, sms, st) : launch<T, false>(a, sms, st);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs &a, int dtype, int sms, cudaStream_t st) {
  if (dtype == NS_DTYPE_F32) return by_k<float>(a, sms, st);
  if (dtype == NS_DTYPE_BF16) return by_k<__nv_bfloat16>(a, sms, st);
  return by_k<__half>(a, sms, st);
}

}  // namespace ns
