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
  // (the compiler may move it)
  static __device__ __forceinline__ void mma_free(float *d, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

// e4m3, two at a time (the first in the lower half), and the scale that a row's exponent byte stands for.
__device__ __forceinline__ uint16_t to_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t from_e4m3(uint32_t pair) {  // (upper half ignored)
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)pair));
  return r;
}
__device__ __forceinline__ uint32_t from_e4m3_hi(uint32_t pairs) {  // the upper two of four
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(pairs));
  return r;
}
__device__ __forceinline__ float scale_of(uint32_t byte) {
  return __uint_as_float(byte << 23 | (byte == 255u ? 0x400000u : 0u));  // 2^(byte - 127); 255: NaN
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// An 8 x 8 matrix of 16-bit elements, two of a row to a lane, transposed.
__device__ __forceinline__ uint32_t across(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
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
__device__ __forceinline__ void cp8(uint32_t dst, const void *src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(ok ? 8 : 0) : "memory");
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

// The same of rows of D bytes.  Rows of 64 share a line of 128 by twos, and the
// lines' pieces are permuted by twice the line, so that four rows two apart
// have their first 16 bytes, and their 8-byte pieces, in different banks.
template <int D>
__device__ __forceinline__ uint32_t piece8(int r, int c) {
  if (D == 128) return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4));
  return (uint32_t)((r >> 1) * 128 + ((((r & 1) * 4 + c) ^ (r & 6)) << 4));
}
__device__ __forceinline__ void lds16(uint32_t a, uint32_t *r) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void lds8(uint32_t a, uint32_t *r) {
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(a) : "memory");
}
__device__ __forceinline__ uint32_t lds1(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(a) : "memory");
  return r;
}

// State of 16 rows of a warp.  Lane (g = lane / 4, t = lane % 4) holds rows g
// and g + 8, columns 8 i + 2 t and + 1 of each group i of eight.
template <typename T, int D>
struct Rows {
  float o[D / 8][4];
  float m[2], l[2];

  static constexpr int kParts = D / 8;  // groups of o
  // The row (of its two) that o[.][j] belongs to, and where row h lies in the 16.
  static __device__ __forceinline__ int of(int j) { return j >> 1; }
  static __device__ __forceinline__ int row(int h) { return ((threadIdx.x & 31) >> 2) + 8 * h; }
  static __device__ __forceinline__ bool first() { return (threadIdx.x & 3) == 0; }  // of a row's lanes

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

  // The same with keys and values of 8 bits (T is fp16): rows of D codes at sK
  // and sV, their exponents' bytes at sKe and sVe.  cq: each row's factor c.
  // Lane (g, t) reads columns D / 4 t .. of key g of each eight, so product kk's
  // columns are D / 4 t + 4 kk .. + 3 (as q's must be), and columns D / 8 g .. of
  // values 2 t, 2 t + 1, 2 t + 8 and 2 t + 9 of each 16: its share of o has
  // columns D / 8 (2 t) + i and D / 8 (2 t + 1) + i in group i.
  template <int NK, bool kMasked, typename Hidden>
  __device__ __forceinline__ void tile8(const uint32_t (*q)[4], uint32_t sK, uint32_t sV, uint32_t sKe, uint32_t sVe,
                                        int k0, const float *cq, const Hidden &hidden, bool wild) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    static_assert(NK % 32 == 0, "a lane an exponent");
    float s[NK / 8][4];
    constexpr int kAtOnce = 4;  // eights of keys whose products take turns
#pragma unroll
    for (int i0 = 0; i0 < NK / 8; i0 += kAtOnce) {
      uint32_t w[kAtOnce][D / 16];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int row = k0 + (i0 + i) * 8 + g;
        if (D == 128) {
          lds16(sK + piece8<D>(row, 2 * t), w[i]);
          lds16(sK + piece8<D>(row, 2 * t + 1), w[i] + D / 32);
        } else {
          lds16(sK + piece8<D>(row, t), w[i]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i0 + i][j] = 0.f;
      }
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
          Type<T>::mma_free(s[i0 + i], q[kk], from_e4m3(w[i][kk]), from_e4m3_hi(w[i][kk]));
    }
    // A lane turns one key's two exponents of each 32 into factors, and the others ask it.
    float top[2] = {kNegInf, kNegInf};
    float unit[NK / 8][2];  // 2^-ve
    uint32_t bad[NK / 32];  // keys whose value is NaN
#pragma unroll
    for (int b0 = 0; b0 < NK; b0 += 32) {
      const int at = k0 + b0 + lane;
      const uint32_t bk = lds1(sKe + at), byte = lds1(sVe + at), bv = byte == 255u ? 127u : byte;
      bad[b0 / 32] = __ballot_sync(0xffffffffu, byte == 255u);
      const float f = __uint_as_float(bk << 23);  // (255: infinity, and NaN with what is added)
      // the value's byte as a number, less 127; NaN where the key's is 255
      const float add = bk == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float(0x4b000000u | bv) - 8388735.f;
      const float u = __uint_as_float((254u - bv) << 23);
#pragma unroll
      for (int i = b0 / 8; i < b0 / 8 + 4; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int from = i * 8 - b0 + 2 * t + e;
          const float ff = __shfl_sync(0xffffffffu, f, from), aa = __shfl_sync(0xffffffffu, add, from);
          unit[i][e] = __shfl_sync(0xffffffffu, u, from);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float &x = s[i][2 * h + e];
            x = fmaf(x * ff, cq[h], aa);
            if (kMasked && hidden(h, i * 8 + 2 * t + e)) x = kNegInf;
            top[h] = fmaxf(top[h], x);
          }
        }
    }
    float shift[2], p2[2];
    bool grows = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
      top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
      const float now = fmaxf(m[h], top[h]), safe = now == kNegInf ? 0.f : now;
      grows |= now > m[h];
      p2[h] = ex2(m[h] - safe);
      m[h] = now;
      shift[h] = Type<T>::kOffset - safe;
    }
    float add[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NK / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = ex2(s[i][j] + shift[j >> 1]);
        add[j >> 1] = fmaf(s[i][j], unit[i][j & 1], add[j >> 1]);
      }
    uint32_t any_bad = 0;
#pragma unroll
    for (int b = 0; b < NK / 32; ++b) any_bad |= bad[b];
    if (any_bad) {  // (after l: a value is no part of it)
#pragma unroll
      for (int i = 0; i < NK / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int key = i * 8 + 2 * t + (j & 1);
          if ((bad[key / 32] >> (key % 32) & 1) && !(kMasked && hidden(j >> 1, key)))
            s[i][j] = __uint_as_float(0x7fffffffu);
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) l[h] = l[h] * p2[h] + add[h];
    if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        o[i][0] *= p2[0];
        o[i][1] *= p2[0];
        o[i][2] *= p2[1];
        o[i][3] *= p2[1];
      }
    }
    if (kMasked && wild) {  // one key at a time, and only into rows that see it
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
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int d = D / 8 * (2 * t + e) + i;
            const float v = Type<T>::unpack(from_e4m3(lds1(sV + piece8<D>(k0 + key, d >> 4) + (d & 15)))).x;
            if (!ha) o[i][e] = fmaf(pa, v, o[i][e]);
            if (!hb) o[i][2 + e] = fmaf(pb, v, o[i][2 + e]);
          }
      }
      return;
    }
#pragma unroll
    for (int kb = 0; kb < NK / 16; ++kb) {
      uint32_t v[4][D / 32];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = k0 + kb * 16 + 2 * t + (r & 1) + (r >> 1) * 8;
        if (D == 128)
          lds16(sV + piece8<D>(row, g), v[r]);
        else
          lds8(sV + piece8<D>(row, g >> 1) + (g & 1) * 8, v[r]);
      }
      const uint32_t a[4] = {Type<T>::pack(s[2 * kb][0], s[2 * kb][1]), Type<T>::pack(s[2 * kb][2], s[2 * kb][3]),
                             Type<T>::pack(s[2 * kb + 1][0], s[2 * kb + 1][1]),
                             Type<T>::pack(s[2 * kb + 1][2], s[2 * kb + 1][3])};
#pragma unroll
      for (int x = 0; x < D / 32; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {  // columns 4 x + 2 y and the next, of keys 2 t, 2 t + 1; 2 t + 8, 2 t + 9
          const uint32_t sel = y ? 0x7362u : 0x5140u;
          const uint32_t lo = __byte_perm(v[0][x], v[1][x], sel), hi = __byte_perm(v[2][x], v[3][x], sel);
          Type<T>::mma_free(o[4 * x + 2 * y], a, from_e4m3(lo), from_e4m3(hi));
          Type<T>::mma_free(o[4 * x + 2 * y + 1], a, from_e4m3_hi(lo), from_e4m3_hi(hi));
        }
    }
  }

  // This lane's columns of row h (of its two), two neighbours at a time: to(column, o, o).
  template <bool F8, typename To>
  __device__ __forceinline__ void columns(int h, const To &to) const {
    const int t = threadIdx.x & 3;
    if constexpr (F8) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < D / 8; i += 2) to(D / 8 * (2 * t + e) + i, o[i][2 * h + e], o[i + 1][2 * h + e]);
    } else {
#pragma unroll
      for (int i = 0; i < D / 8; ++i) to(8 * i + 2 * t, o[i][2 * h], o[i][2 * h + 1]);
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

// State of 8 rows of a warp over a cache of 8 bits, the products the other way
// round: scores are K Q^T and the sums V^T P^T, so keys and columns take the
// 16 places of mma's first operand and the rows its 8 columns.  Half the
// products, scores and sums of 16 rows, of which a decoded token's heads rarely
// fill more than 8.  Lane (g, t) holds rows 2 t and 2 t + 1: columns
// D / 8 g + 2 i and + 1 in group i.  P goes from where it is computed (keys g,
// rows 2 t) to where it is an operand (rows g, keys 2 t) by movmatrix.
template <typename T, int D>
struct Rows8 {
  static constexpr int kParts = D / 16;
  float o[D / 16][4];
  float m[2], l[2];

  static __device__ __forceinline__ int of(int j) { return j & 1; }
  static __device__ __forceinline__ int row(int h) { return 2 * (threadIdx.x & 3) + h; }
  static __device__ __forceinline__ bool first() { return (threadIdx.x & 31) < 4; }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    m[0] = m[1] = kNegInf;
    l[0] = l[1] = 0.f;
  }

  // As Rows::tile8; q: row g's columns D / 4 t + 4 kk .. + 3 in product kk.
  template <int NK, bool kMasked, typename Hidden>
  __device__ __forceinline__ void tile8(const uint32_t (*q)[2], uint32_t sK, uint32_t sV, uint32_t sKe, uint32_t sVe,
                                        int k0, const float *cq, const Hidden &hidden, bool wild) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    constexpr int B = NK / 16;  // blocks of keys
    float s[B][4];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      uint32_t w[2][D / 16];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = k0 + i * 16 + r * 8 + g;
        if (D == 128) {
          lds16(sK + piece8<D>(row, 2 * t), w[r]);
          lds16(sK + piece8<D>(row, 2 * t + 1), w[r] + D / 32);
        } else {
          lds16(sK + piece8<D>(row, t), w[r]);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t a[4] = {from_e4m3(w[0][kk]), from_e4m3(w[1][kk]), from_e4m3_hi(w[0][kk]),
                               from_e4m3_hi(w[1][kk])};
        Type<T>::mma_free(s[i], a, q[kk][0], q[kk][1]);
      }
    }
    float top[2] = {kNegInf, kNegInf}, unit[B][2];
    uint32_t bad = 0;  // keys of this lane whose value is NaN
#pragma unroll
    for (int i = 0; i < B; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int key = i * 16 + e * 8 + g;
        const uint32_t bk = lds1(sKe + k0 + key), byte = lds1(sVe + k0 + key), bv = byte == 255u ? 127u : byte;
        bad |= (byte == 255u ? 1u : 0u) << (2 * i + e);
        const float f = __uint_as_float(bk << 23);  // (255: infinity, and NaN with what is added)
        const float add = bk == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float(0x4b000000u | bv) - 8388735.f;
        unit[i][e] = __uint_as_float((254u - bv) << 23);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float &x = s[i][2 * e + h];
          x = fmaf(x * f, cq[h], add);
          if (kMasked && hidden(h, key)) x = kNegInf;
          top[h] = fmaxf(top[h], x);
        }
      }
    float shift[2], p2[2];
    bool grows = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], off));
      const float now = fmaxf(m[h], top[h]), safe = now == kNegInf ? 0.f : now;
      grows |= now > m[h];
      p2[h] = ex2(m[h] - safe);
      m[h] = now;
      shift[h] = Type<T>::kOffset - safe;
    }
    float add[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < B; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = ex2(s[i][j] + shift[j & 1]);
        add[j & 1] = fmaf(s[i][j], unit[i][j >> 1], add[j & 1]);
      }
    if (bad) {  // (after l: a value is no part of it)
#pragma unroll
      for (int i = 0; i < B; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if ((bad >> (2 * i + (j >> 1)) & 1) && !(kMasked && hidden(j & 1, i * 16 + (j >> 1) * 8 + g)))
            s[i][j] = __uint_as_float(0x7fffffffu);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) l[h] = l[h] * p2[h] + add[h];
    if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] *= p2[j & 1];
    }
    if (kMasked && wild) {  // one key at a time, and only into rows that see it
#pragma unroll 1
      for (int key = 0; key < NK; ++key) {
        float p[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < B; ++i)
          if (i == key >> 4) {
            p[0] = (key & 8) ? s[i][2] : s[i][0];
            p[1] = (key & 8) ? s[i][3] : s[i][1];
          }
#pragma unroll
        for (int h = 0; h < 2; ++h) p[h] = __shfl_sync(0xffffffffu, p[h], (key & 7) * 4 + t);
        const bool gone[2] = {hidden(0, key), hidden(1, key)};
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int d = D / 8 * g + 2 * i + e;
            const float v = Type<T>::unpack(from_e4m3(lds1(sV + piece8<D>(k0 + key, d >> 4) + (d & 15)))).x;
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (!gone[h]) o[i][2 * e + h] = fmaf(p[h], v, o[i][2 * e + h]);
          }
      }
      return;
    }
#pragma unroll
    for (int kb = 0; kb < B; ++kb) {
      uint32_t v[4][D / 32];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = k0 + kb * 16 + 2 * t + (r & 1) + (r >> 1) * 8;
        if (D == 128)
          lds16(sV + piece8<D>(row, g), v[r]);
        else
          lds8(sV + piece8<D>(row, g >> 1) + (g & 1) * 8, v[r]);
      }
      const uint32_t b0 = across(Type<T>::pack(s[kb][0], s[kb][1])), b1 = across(Type<T>::pack(s[kb][2], s[kb][3]));
#pragma unroll
      for (int x = 0; x < D / 32; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {  // columns 4 x + 2 y and the next, of keys 2 t, 2 t + 1; 2 t + 8, 2 t + 9
          const uint32_t sel = y ? 0x7362u : 0x5140u;
          const uint32_t lo = __byte_perm(v[0][x], v[1][x], sel), hi = __byte_perm(v[2][x], v[3][x], sel);
          const uint32_t a[4] = {from_e4m3(lo), from_e4m3_hi(lo), from_e4m3(hi), from_e4m3_hi(hi)};
          Type<T>::mma_free(o[2 * x + y], a, b0, b1);
        }
    }
  }

  template <bool F8, typename To>
  __device__ __forceinline__ void columns(int h, const To &to) const {
    const int g = (threadIdx.x & 31) >> 2;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) to(D / 8 * g + 2 * i, o[i][h], o[i][2 + h]);
  }

  __device__ __forceinline__ void sum_l() {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], off);
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

// The same of n 16-byte pieces of e4m3 codes: NaN is all ones but the sign.
__device__ __forceinline__ bool wild_codes(uint32_t a, int n, int tid, int threads) {
  uint32_t any = 0;
#pragma unroll 8
  for (int i = tid; i < n; i += threads) {
    uint32_t x[4];
    lds16(a + 16u * (uint32_t)i, x);
#pragma unroll
    for (int j = 0; j < 4; ++j) any |= __vcmpeq4(x[j] & 0x7f7f7f7fu, 0x7f7f7f7fu);
  }
  return any != 0;
}

}  // namespace attn
}  // namespace ns
