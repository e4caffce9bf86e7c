// nvfp4.cuh -- blocks of 16 elements in NVFP4 (E2M1 codes under an E4M3 scale
// and an fp32 global scale): a thread encodes a whole block, and decodes pieces of
// 16 bytes, a block being two of a 16-bit type or four of fp32.
#pragma once

#include "rows.cuh"

namespace moe {

constexpr int kBlock16 = 16;                 // elements of a block
constexpr float kE2m1Max = 6.f, kE4m3Most = 448.f;
constexpr float kGlobalDiv = kE2m1Max * kE4m3Most;   // a group's maximum over its global scale
// The least global scale.  It keeps a block's step, 2^-9 of it at least, and
// the residuals of the quotients (2^-49 of an element of a step's size) among
// the numbers that fp32 holds exactly.
constexpr float kGlobalMin = 0x1p-80f;

// Pieces of a block, and the type of a piece's packed codes.
template <typename T>
constexpr int kPieces16 = kBlock16 / kPer16<T>;
template <int N> struct PackedCodes { using type = uint32_t; };
template <> struct PackedCodes<4> { using type = uint16_t; };

// Eight floats to E2M1, ties to even, saturating at 6; the first in the low
// nibble.
__device__ __forceinline__ uint32_t to_e2m1x8(const f32x2 *f) {
  uint32_t r;
  const float2 a = unpair(f[0]), b = unpair(f[1]), c = unpair(f[2]), d = unpair(f[3]);
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
  return r;
}

// The values of N codes under the step t, code * t.
template <int N>
__device__ __forceinline__ void code_values(uint32_t codes, float t, f32x2 *f) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const float2 p = f16x2_to_float2(e2m1x2_to_f16x2((codes >> (8 * i)) & 0xFFu));
    f[i] = mul2(pair(p.x, p.y), pair(t, t));
  }
}

// A block as it is stored.  How it is moved: by 32-byte sectors (kSectors), 16-byte
// pieces (kWhole) or elements (kElems).
enum { kSectors = 32 };
template <typename T>
using RawBlock = Raw<T, kBlock16>;
template <typename T, int A>
__device__ __forceinline__ RawBlock<T> block_load(const typename T::bits *row, int b) {
  RawBlock<T> r;
  const typename T::bits *p = row + (size_t)b * kBlock16;
  if constexpr (A == kSectors) {
#pragma unroll
    for (int i = 0; i < RawBlock<T>::kWords; i += 8)
      asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(r.w[i]), "=r"(r.w[i + 1]), "=r"(r.w[i + 2]), "=r"(r.w[i + 3]),
                     "=r"(r.w[i + 4]), "=r"(r.w[i + 5]), "=r"(r.w[i + 6]), "=r"(r.w[i + 7])
                   : "l"(reinterpret_cast<const uint32_t *>(p) + i));
  } else if constexpr (A == kWhole) {
    r = raw_load_aligned<T, kBlock16>(p);
  } else {
#pragma unroll
    for (int i = 0; i < RawBlock<T>::kWords; ++i) {
      if constexpr (sizeof(typename T::bits) == 4)
        r.w[i] = p[i];
      else
        r.w[i] = (uint32_t)p[2 * i] | (uint32_t)p[2 * i + 1] << 16;
    }
  }
  return r;
}
template <typename T, int A>
__device__ __forceinline__ void block_store(typename T::bits *row, int b, const RawBlock<T> &r) {
  typename T::bits *p = row + (size_t)b * kBlock16;
  if constexpr (A == kSectors) {
#pragma unroll
    for (int i = 0; i < RawBlock<T>::kWords; i += 8)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                       reinterpret_cast<uint32_t *>(p) + i),
                   "r"(r.w[i]), "r"(r.w[i + 1]), "r"(r.w[i + 2]), "r"(r.w[i + 3]), "r"(r.w[i + 4]),
                   "r"(r.w[i + 5]), "r"(r.w[i + 6]), "r"(r.w[i + 7])
                   : "memory");
  } else if constexpr (A == kWhole) {
#pragma unroll
    for (int i = 0; i < RawBlock<T>::kWords; i += 4)
      *reinterpret_cast<uint4 *>(reinterpret_cast<uint32_t *>(p) + i) =
          make_uint4(r.w[i], r.w[i + 1], r.w[i + 2], r.w[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < RawBlock<T>::kWords; ++i) {
      if constexpr (sizeof(typename T::bits) == 4) {
        p[i] = r.w[i];
      } else {
        p[2 * i] = (uint16_t)r.w[i];
        p[2 * i + 1] = (uint16_t)(r.w[i] >> 16);
      }
    }
  }
}

// The largest magnitude of a block; NaN if it has one.
template <typename T>
__device__ __forceinline__ float block_max(const RawBlock<T> &r) {
  float m = 0.f;
  if constexpr (sizeof(typename T::bits) == 2) {
    uint32_t w = r.w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < 8; ++i) w = T::max2(w, r.w[i] & 0x7FFF7FFFu);
    const float2 p = T::up2(w);
    m = max_nan(p.x, p.y);
  } else {
#pragma unroll
    for (int i = 0; i < 16; i += 2)
      m = max_abs_nan(m, __uint_as_float(r.w[i]), __uint_as_float(r.w[i + 1]));
  }
  return m;
}
// What a block's maximum adds to its group's: blocks with a NaN or an infinity
// have no part in it.
__device__ __forceinline__ float finite_max(float m) {
  return m < __int_as_float(0x7F800000) ? m : 0.f;
}
// The global scale of a group whose largest magnitude is m.
__device__ __forceinline__ float global_of(float m) { return fmaxf(m / kGlobalDiv, kGlobalMin); }

// The negative of a quotient a / b from y, nearly 1 / b: q = a y, corrected by its
// residual a - q b (one fma, exact) times y (Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990).  It is the float next to
// a / b unless that is within about 2^-22 units of the middle of two floats.  With y the
// float next to 1 / b no such pair lies beside a border of E2M1 or E4M3 (a search over
// every 24-bit b); with y a unit off there are a few, of b = 12582909 and 16777209 to
// 16777215 (16777212: a = 20971516, border 1.25).  The reciprocal of the chip that this
// is for is near enough there: a test takes every b, each border and the floats around
// border * b, and finds the division's codes.  (One that is rounded correctly,
// __frcp_rn, takes 32 x 1536 x 2048 bf16 from 75.6 to 79.7 us.)  The negative, as zeros keep
// their sign in it: for a = -0, q = -a y = +0, the residual q b + a = +0 and
// +0 * -y + q = +0; the quotient itself would be +0 + q = +0.
__device__ __forceinline__ f32x2 minus_quotient2(f32x2 a, f32x2 b, f32x2 minus_y) {
  const f32x2 q = mul2(a, minus_y);
  return fma2(fma2(q, b, a), minus_y, q);
}
__device__ __forceinline__ float reciprocal(float v) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// A group's scale and what its blocks' scales divide by.
struct GlobalScale {
  float g, six, inv;
  __device__ __forceinline__ explicit GlobalScale(float v)
      : g(v), six(kE2m1Max * v), inv(1.f / (kE2m1Max * v)) {}
};

// A block's scale byte from its maximum m:
//   s = e4m3(min(m / (6 g), 448)), NaN for a block with a NaN or an infinity.
// Quotients over 2^60 (a given scale far below the values) go without the
// residual, which could leave fp32's range: their scale is 448 either way.
__device__ __forceinline__ uint32_t block_scale(float m, const GlobalScale &g) {
  const float q = m * g.inv;
  float r = q < 0x1p60f ? fmaf(fmaf(-q, g.six, m), g.inv, q) : q;
  if (!(m < __int_as_float(0x7F800000))) r = __int_as_float(0x7FFFFFFF);
  return to_e4m3x2(r, 0.f) & 0xFFu;
}

// Magnitudes above 8 t down to it, where every code is 6.
template <typename T>
__device__ __forceinline__ RawBlock<T> clamped(RawBlock<T> r, float t) {
  if constexpr (sizeof(typename T::bits) == 2) {
    const uint32_t most = T::down2(8.f * t, 8.f * t);
#pragma unroll
    for (int i = 0; i < RawBlock<T>::kWords; ++i)
      r.w[i] = T::min2(r.w[i] & 0x7FFF7FFFu, most) | (r.w[i] & 0x80008000u);
  } else {
#pragma unroll
    for (int i = 0; i < RawBlock<T>::kWords; ++i)
      r.w[i] = __float_as_uint(
          copysignf(fminf(fabsf(__uint_as_float(r.w[i])), 8.f * t), __uint_as_float(r.w[i])));
  }
  return r;
}

// The codes of a block with the step t (its scale s times the global one) and the
// maximum m: e2m1(x / t), and 0 throughout where s is 0 or NaN.
template <typename T>
__device__ __forceinline__ uint2 block_codes(RawBlock<T> r, float s, float t, float m) {
  const float y = reciprocal(t);
  const f32x2 my = pair(-y, -y), tt = pair(t, t);
  // an infinite quotient has no residual (those of fp16 reach 2^88 at most)
  if constexpr (!std::is_same_v<T, F16>)
    if (!(m * y < 0x1p126f)) r = clamped<T>(r, t);
  f32x2 f[8];
  raw_up<T, kBlock16>(r, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = minus_quotient2(f[i], tt, my);
  constexpr uint32_t kSigns = 0x88888888u;   // of the negative quotients, turned
  const uint32_t live = s > 0.f ? ~0u : 0u;
  return make_uint2((to_e2m1x8(f) ^ kSigns) & live, (to_e2m1x8(f + 4) ^ kSigns) & live);
}

}  // namespace moe
