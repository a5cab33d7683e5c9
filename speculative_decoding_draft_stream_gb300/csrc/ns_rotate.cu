// Norms of queries and keys for each head, and their rotation by position, in
// one pass.
//
// Mathematics: a row x of D columns (one token, one head) becomes
//   y = x w / sqrt(mean(x^2) + eps)                  (without a norm: x)
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = position * f_i,
// for the pairs i of its first R columns, halves (i, i + R/2) or neighbours
// (2i, 2i + 1).  Everything is fp32 and rounded once, to the row's type.
//
// Angles: in 32 bits, position * f_i of a far token is off by whole radians'
// fractions (2^-24 of 10^6).  Only t modulo a turn counts, so f_i / 2 pi is
// kept as a 64-bit fixed-point fraction of a turn, from the 53 bits of f_i and
// 64 bits of 1 / 2 pi; its product with the position wraps by itself, and the
// upper 32 bits are the angle.  Cut there, it is off by up to 2^-32 turns, and
// as an fp32 number by up to 2^-26 turns more (24 bits of half a turn), wherever
// the position is; beside that, position * 2^-53 of f_i's own rounding.  It
// takes a few integer instructions; the same product in fp64 would wait for two
// fp64 units an SM.
//
// Layout: D / 16 lanes have a row, 16 columns each, so that every lane has
// both columns of its eight pairs and nothing is exchanged but the sum of
// squares; a lane keeps its eight cosines and sines for a chunk of the token's
// heads.  Long calls take chunks of several heads (a row's arithmetic is about
// 110 instructions a lane, a chunk's angles 350), short ones a head to each.
//
// Bound by HBM where there are many tokens, by the launch where there are few:
// 62.0 us for 335 MB (80 % of a copy's rate), 5.7 us for 15.7 MB, 2.7 us for
// one token.  Two rows' loads in flight a lane and 3 CTAs an SM: with four rows
// and 2 CTAs 64.7, 6.4 and 2.9 us, with two rows and 4 CTAs (spills) 67.9, 5.9
// and 3.3.  Chunks of at most 4 heads took 67.0 us, of 16 71.5.
#include "ns_attn_tile.cuh"
#include "ns_internal.cuh"
#include "ns_ops.cuh"

namespace ns {
namespace {

using attn::Type;

constexpr int kRotThreads = 256;
constexpr int kInFlight = 2;  // rows whose loads a lane has under way

// f / (2 pi) modulo 1 in units of 2^-64 turns.
__device__ __forceinline__ int64_t turns(double f) {
  constexpr uint64_t kInvTwoPi = 0xa2f9836e4e44152aull;  // 2^66 / (2 pi)
  const uint64_t bits = (uint64_t)__double_as_longlong(f);
  const int e = (int)(bits >> 52 & 0x7ff) - 1023;
  const uint64_t m = (bits << 11) | 1ull << 63;  // |f| = m 2^(e - 63); (subnormal f: less than 2^-1000 turns)
  const uint64_t hi = __umul64hi(m, kInvTwoPi);  // |f| / (2 pi) = hi 2^(e - 65)
  const int up = e - 1;
  const uint64_t t = up >= 64 || up <= -64 ? 0ull : up >= 0 ? hi << up : hi >> -up;
  return (int64_t)(bits >> 63 ? 0ull - t : t);
}

template <typename T, int D, bool kNeighbours>
__global__ void __launch_bounds__(kRotThreads, 3)
    rotate_kernel(const RotateArgs a, int chunk, int q_chunks, int chunks) {
  constexpr int L = D / 16, kRows = kRotThreads / L;
  __shared__ int64_t s_turns[D / 2];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int j = threadIdx.x % L;
  for (int i = threadIdx.x; i < a.rotary / 2; i += kRotThreads) s_turns[i] = turns(a.inv_freq[i]);
  const long long u = (long long)blockIdx.x * kRows + threadIdx.x / L;
  const bool live = u < (long long)a.tokens * chunks;
  const int token = live ? (int)(u / chunks) : 0, c = live ? (int)(u % chunks) : 0;
  const bool is_k = c >= q_chunks;
  const int h0 = (is_k ? c - q_chunks : c) * chunk;
  const int heads = live ? min(chunk, (is_k ? a.kv_heads : a.q_heads) - h0) : 0;
  const int64_t in_head = is_k ? a.k_head : a.q_head, out_head = is_k ? a.ko_head : a.qo_head;
  const bool turned = 16 * (j + 1) <= a.rotary;
  // this lane's two pieces of eight columns
  const int p0 = kNeighbours || !turned ? 2 * j : j, p1 = kNeighbours || !turned ? 2 * j + 1 : j + a.rotary / 16;
  const T *src = static_cast<const T *>(is_k ? a.k : a.q) + token * (is_k ? a.k_token : a.q_token) + h0 * in_head;
  T *dst = static_cast<T *>(is_k ? a.k_out : a.q_out) + token * (is_k ? a.ko_token : a.qo_token) + h0 * out_head;
  const int pos = live ? a.positions[token] : 0;
  const T *wp = static_cast<const T *>(is_k ? a.k_weight : a.q_weight);
  uint4 w[2] = {};
  if (wp) w[0] = reinterpret_cast<const uint4 *>(wp)[p0], w[1] = reinterpret_cast<const uint4 *>(wp)[p1];

  float cs[8], sn[8];
  bool angles = false;
  __syncthreads();
  for (int r0 = 0; __any_sync(0xffffffffu, r0 < heads); r0 += kInFlight) {
    uint4 x[kInFlight][2];
#pragma unroll
    for (int r = 0; r < kInFlight; ++r)
      if (r0 + r < heads) {
        const uint4 *row = reinterpret_cast<const uint4 *>(src + (r0 + r) * in_head);
        x[r][0] = row[p0], x[r][1] = row[p1];
      }
    if (!angles) {  // (while the first rows are on their way)
      angles = true;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        cs[i] = 1.f, sn[i] = 0.f;
        if (turned) {
          const int64_t t = (int64_t)((uint64_t)s_turns[8 * j + i] * (uint64_t)(int64_t)pos);
          sincospif((float)(int)(t >> 32) * 0x1p-31f, &sn[i], &cs[i]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < kInFlight; ++r) {
      if (!__any_sync(0xffffffffu, r0 + r < heads)) break;
      float v[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = reinterpret_cast<const uint32_t *>(&x[r][0])[i];
        const uint32_t hi = reinterpret_cast<const uint32_t *>(&x[r][1])[i];
        const float2 y = Type<T>::unpack(r0 + r < heads ? lo : 0u), z = Type<T>::unpack(r0 + r < heads ? hi : 0u);
        v[2 * i] = y.x, v[2 * i + 1] = y.y, v[8 + 2 * i] = z.x, v[8 + 2 * i + 1] = z.y;
      }
      if (a.eps >= 0.f) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) sum = fmaf(v[i], v[i], sum);
#pragma unroll
        for (int off = L / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        const float f = rsqrtf(fmaf(sum, 1.f / D, a.eps));
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] *= f;
        if (wp) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 y = Type<T>::unpack(reinterpret_cast<const uint32_t *>(w)[i]);
            v[2 * i] *= y.x, v[2 * i + 1] *= y.y;
          }
        }
      }
      if (turned) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float &p = kNeighbours ? v[2 * i] : v[i], &q = kNeighbours ? v[2 * i + 1] : v[8 + i];
          const float x0 = p, x1 = q;
          p = fmaf(x0, cs[i], -x1 * sn[i]);
          q = fmaf(x1, cs[i], x0 * sn[i]);
        }
      }
      if (r0 + r < heads) {
        uint4 *row = reinterpret_cast<uint4 *>(dst + (r0 + r) * out_head);
        row[p0] = make_uint4(Type<T>::pack(v[0], v[1]), Type<T>::pack(v[2], v[3]), Type<T>::pack(v[4], v[5]),
                             Type<T>::pack(v[6], v[7]));
        row[p1] = make_uint4(Type<T>::pack(v[8], v[9]), Type<T>::pack(v[10], v[11]), Type<T>::pack(v[12], v[13]),
                             Type<T>::pack(v[14], v[15]));
      }
    }
  }
}

template <typename T, int D, bool kNeighbours>
cudaError_t launch(const RotateArgs &a, int sms, cudaStream_t st) {
  // The largest chunk, up to 8 heads, that leaves each SM 64 rows at work: one of 256 rows
  // took 7.4 us for 15.7 MB where this takes 5.7, and made no difference at 335 MB.
  const long long rows = (long long)a.tokens * (a.q_heads + a.kv_heads);
  int chunk = 1;
  while (chunk < 8 && rows / (2 * chunk) >= 64LL * sms) chunk *= 2;
  const int q_chunks = (a.q_heads + chunk - 1) / chunk, chunks = q_chunks + (a.kv_heads + chunk - 1) / chunk;
  constexpr int kRows = kRotThreads / (D / 16);
  const long long ctas = ((long long)a.tokens * chunks + kRows - 1) / kRows;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kRotThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rotate_kernel<T, D, kNeighbours>, a, chunk, q_chunks, chunks);
}
template <typename T>
cudaError_t by_shape(const RotateArgs &a, int dim, bool neighbours, int sms, cudaStream_t st) {
  if (dim == 128) return neighbours ? launch<T, 128, true>(a, sms, st) : launch<T, 128, false>(a, sms, st);
  return neighbours ? launch<T, 64, true>(a, sms, st) : launch<T, 64, false>(a, sms, st);
}

}  // namespace

cudaError_t launch_rotate(const RotateArgs &a, int dtype, int dim, bool neighbours, int sms, cudaStream_t st) {
  return dtype == NS_DTYPE_BF16 ? by_shape<__nv_bfloat16>(a, dim, neighbours, sms, st)
                                : by_shape<__half>(a, dim, neighbours, sms, st);
}

}  // namespace ns
