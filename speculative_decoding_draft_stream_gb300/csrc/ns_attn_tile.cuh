// One warp's part of an attention tile on mma.sync: scores of 16 query rows
// with some keys, the running softmax, and the product with the values.
//
// A row's state is (m, l, o): m the largest scaled score so far (in powers of
// two), l = sum 2^(x - m), o = sum 2^(x - m) v.  A tile with a larger maximum
// m' first multiplies l and o by 2^(m - m').  Scores, m, l and o are fp32.
// Probabilities are rounded to the values' type for the product, whose operands
// have 16 bits (at most u sum p |v| with u its unit roundoff, beside the output's
// own u |o|); l sums them unrounded.  For fp16 they are all kept 2^8 times larger, so that
// probabilities down to 2^-32 of the largest are not lost to fp16's range.
//
// Keys and values lie in shared memory as rows of D elements whose 16-byte
// pieces are permuted: piece c of row r is at c ^ (r & 7), so the eight rows
// that an ldmatrix reads at one piece fall into different banks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace ns {
namespace attn {

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

template <typename T>
struct Type;
template <>
struct Type<__nv_bfloat16> {
  static constexpr bool kBf16 = true;
  static constexpr uint32_t kInf = 0x7f80u;  // the pattern of infinity
  static constexpr float kOffset = 0.f;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ void mma(float *d, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};
template <>
struct Type<__half> {
  static constexpr bool kBf16 = false;
  static constexpr uint32_t kInf = 0x7c00u;
  static constexpr float kOffset = 8.f;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
  }
  static __device__ __forceinline__ void mma(float *d, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t *r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t *r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
// 16 bytes to shared memory, zeros where ok is false (src is not read then)
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Byte offset of 16-byte piece c of row r in a tile of rows of D elements.
template <int D>
__device__ __forceinline__ uint32_t piece(int r, int c) {
  return (uint32_t)(r * (D * 2) + ((c ^ (r & 7)) << 4));
}

// State of 16 rows of a warp.  Lane (g = lane / 4, t = lane % 4) holds rows g
// and g + 8, columns 8 i + 2 t and + 1 of each group i of eight.
template <typename T, int D>
struct Rows {
  float o[D / 8][4];
  float m[2], l[2];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    m[0] = m[1] = kNegInf;
    l[0] = l[1] = 0.f;
  }

  // Takes in NK keys whose rows start at row k0 of the tiles at sK and sV.
  // x = score * c with c = scale * log2(e).  hidden(row of the pair, key of
  // the NK) says which places are masked, consulted when kMasked; `wild`
  // (kMasked only): the values may hold infinities or NaN, which must not
  // reach rows that do not see them.
  template <int NK, bool kMasked, typename Hidden>
  __device__ __forceinline__ void tile(const uint32_t (*q)[4], uint32_t sK, uint32_t sV, int k0, float c,
                                       const Hidden &hidden, bool wild) {
    const int lane = threadIdx.x & 31;
    float s[NK / 8][4];
#pragma unroll
    for (int i = 0; i < NK / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
    // matrices of an x4 load: keys 0-7 and 8-15, the two 8-element halves of 16
    const int kr = (lane & 7) + ((lane >> 4) << 3), kc = (lane >> 3) & 1;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
      for (int nb = 0; nb < NK / 16; ++nb) {
        uint32_t b[4];
        ldsm4(sK + piece<D>(k0 + nb * 16 + kr, kk * 2 + kc), b);
        Type<T>::mma(s[2 * nb], q[kk], b[0], b[1]);
        Type<T>::mma(s[2 * nb + 1], q[kk], b[2], b[3]);
      }
    }
    if (kMasked) {
#pragma unroll
      for (int i = 0; i < NK / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (hidden(j >> 1, i * 8 + (lane & 3) * 2 + (j & 1))) s[i][j] = kNegInf;
    }
    float shift[2], p2[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float top = kNegInf;
#pragma unroll
      for (int i = 0; i < NK / 8; ++i) top = fmaxf(top, fmaxf(s[i][2 * h], s[i][2 * h + 1]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float now = fmaxf(m[h], top * c);
      const float safe = now == kNegInf ? 0.f : now;  // nothing seen yet: exponents of -inf, not NaN
      p2[h] = ex2(m[h] - safe);
      m[h] = now;
      shift[h] = Type<T>::kOffset - safe;
    }
    float add[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NK / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = ex2(fmaf(s[i][j], c, shift[j >> 1]));
        add[j >> 1] += s[i][j];
      }
#pragma unroll
    for (int h = 0; h < 2; ++h) l[h] = l[h] * p2[h] + add[h];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      o[i][0] *= p2[0];
      o[i][1] *= p2[0];
      o[i][2] *= p2[1];
      o[i][3] *= p2[1];
    }
    if (kMasked && wild) {
      // one key at a time, and only into rows that see it
#pragma unroll 1
      for (int key = 0; key < NK; ++key) {
        float pa = 0.f, pb = 0.f;
#pragma unroll
        for (int i = 0; i < NK / 8; ++i)
          if (i == key >> 3) {
            pa = (key & 1) ? s[i][1] : s[i][0];
            pb = (key & 1) ? s[i][3] : s[i][2];
          }
        const int from = (lane & ~3) | ((key & 7) >> 1);
        pa = __shfl_sync(0xffffffffu, pa, from);
        pb = __shfl_sync(0xffffffffu, pb, from);
        const bool ha = hidden(0, key), hb = hidden(1, key);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          uint32_t w;
          asm volatile("ld.shared.b32 %0, [%1];"
                       : "=r"(w)
                       : "r"(sV + piece<D>(k0 + key, i) + (uint32_t)((lane & 3) * 4))
                       : "memory");
          const float2 v = Type<T>::unpack(w);
          if (!ha) o[i][0] = fmaf(pa, v.x, o[i][0]), o[i][1] = fmaf(pa, v.y, o[i][1]);
          if (!hb) o[i][2] = fmaf(pb, v.x, o[i][2]), o[i][3] = fmaf(pb, v.y, o[i][3]);
        }
      }
      return;
    }
    // matrices of an x4 load: keys 0-7 and 8-15 of two groups of eight columns
    const int vr = lane & 15, vc = lane >> 4;
#pragma unroll
    for (int kb = 0; kb < NK / 16; ++kb) {
      const uint32_t a[4] = {Type<T>::pack(s[2 * kb][0], s[2 * kb][1]), Type<T>::pack(s[2 * kb][2], s[2 * kb][3]),
                             Type<T>::pack(s[2 * kb + 1][0], s[2 * kb + 1][1]),
                             Type<T>::pack(s[2 * kb + 1][2], s[2 * kb + 1][3])};
#pragma unroll
      for (int db = 0; db < D / 16; ++db) {
        uint32_t b[4];
        ldsm4t(sV + piece<D>(k0 + kb * 16 + vr, db * 2 + vc), b);
        Type<T>::mma(o[2 * db], a, b[0], b[1]);
        Type<T>::mma(o[2 * db + 1], a, b[2], b[3]);
      }
    }
  }

  // The lanes of a row add up their shares of l (once, after the last tile).
  __device__ __forceinline__ void sum_l() {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
  }
};

// The log-sum-exp (natural) of a row from its (m, l), -inf for an empty row.
template <typename T>
__device__ __forceinline__ float row_lse(float m, float l) {
  return l == 0.f ? kNegInf : (m - Type<T>::kOffset + log2f(l)) * kLn2;
}

// Whether any of the n 16-byte pieces at shared address a holds an infinity
// or NaN (this thread's share of them): their exponents are all ones, so
// without the sign no finite value has a larger pattern.
template <typename T>
__device__ __forceinline__ bool wild_pieces(uint32_t a, int n, int tid, int threads) {
  uint32_t most[2] = {0, 0};  // of 16-bit halves
#pragma unroll 8
  for (int i = tid; i < n; i += threads) {
    uint32_t x[4];
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                 : "r"(a + 16u * (uint32_t)i)
                 : "memory");
    most[0] = __vimax3_u16x2(most[0], x[0] & 0x7fff7fffu, x[1] & 0x7fff7fffu);
    most[1] = __vimax3_u16x2(most[1], x[2] & 0x7fff7fffu, x[3] & 0x7fff7fffu);
  }
  const uint32_t m = __vmaxu2(most[0], most[1]);
  return (m & 0xffffu) >= Type<T>::kInf || (m >> 16) >= Type<T>::kInf;
}

}  // namespace attn
}  // namespace ns
