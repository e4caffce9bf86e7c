// nvfp4.cuh -- blocks of 16 elements in NVFP4 (E2M1 codes under an E4M3 scale
// and an fp32 global scale): encoding and decoding.
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

// Eight codes to floats (exact).
__device__ __forceinline__ void from_e2m1x8(uint32_t v, f32x2 *f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = f16x2_to_float2(e2m1x2_to_f16x2((v >> (8 * i)) & 0xFFu));
    f[i] = pair(p.x, p.y);
  }
}

// The largest magnitude of a block, NaN if it has one.
__device__ __forceinline__ float block_max(const f32x2 (&f)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 p = unpair(f[i]);
    m = max_abs_nan(m, p.x, p.y);
  }
  return m;
}
// What a block's maximum adds to its group's: blocks with a NaN or an infinity
// have no part in it.
__device__ __forceinline__ float finite_max(float m) { return m < __int_as_float(0x7F800000) ? m : 0.f; }

// The global scale of a group whose largest magnitude is m.
__device__ __forceinline__ float global_of(float m) { return fmaxf(m / kGlobalDiv, kGlobalMin); }

// A block's scale byte from its maximum m and the global scale g:
//   s = e4m3(min(m / (6 g), 448)), NaN for a block with a NaN or an infinity.
__device__ __forceinline__ uint32_t block_scale(float m, float g) {
  float r = m / (kE2m1Max * g);
  if (!(m < __int_as_float(0x7F800000))) r = __int_as_float(0x7FFFFFFF);
  return to_e4m3x2(r, 0.f) & 0xFFu;
}

// A block's codes, e2m1(x / t) with t the block's step s * g in fp32, and 0
// throughout where s is 0 or NaN.  The quotient is x times y = 1 / t rounded,
// corrected by its residual x - q t (one fma) times y: the nearest float to
// x / t, so that ties of the rounding to a code are where the division puts
// them (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990).  One division a block instead of one an
// element.  A quotient over 2^60 (a given global scale far below the values)
// goes without the residual, which could leave fp32's range.
__device__ __forceinline__ uint2 block_codes(f32x2 (&f)[8], float s, float t, float m) {
  if (!(s > 0.f)) return make_uint2(0u, 0u);
  const float y = 1.f / t;
  const f32x2 yy = pair(y, y), mt = pair(-t, -t);
  if (m * y < 0x1p60f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const f32x2 q = mul2(f[i], yy);
      f[i] = fma2(fma2(q, mt, f[i]), yy, q);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = mul2(f[i], yy);
  }
  return make_uint2(to_e2m1x8(f), to_e2m1x8(f + 4));
}

// The values of a block's codes, code * t.
__device__ __forceinline__ void block_values(uint2 codes, float t, f32x2 (&f)[8]) {
  from_e2m1x8(codes.x, f);
  from_e2m1x8(codes.y, f + 4);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = mul2(f[i], pair(t, t));
}

// Block b of a row of H elements (H a multiple of 16) as stored: 16-byte
// pieces (kWhole) or elements (kElems).
template <typename T>
constexpr int kPieces16 = kBlock16 / kPer16<T>;
template <typename T>
struct RawBlock {
  Raw<T, kPer16<T>> p[kPieces16<T>];
};
template <typename T, int A>
__device__ __forceinline__ RawBlock<T> block_load(const typename T::bits *row, int b, int H) {
  RawBlock<T> r;
#pragma unroll
  for (int i = 0; i < kPieces16<T>; ++i)
    r.p[i] = raw_load<T, kPer16<T>, A>(row, b * kPieces16<T> + i, H);
  return r;
}
template <typename T>
__device__ __forceinline__ void block_up(const RawBlock<T> &r, f32x2 (&f)[8]) {
  constexpr int N = kPer16<T>;
#pragma unroll
  for (int i = 0; i < kPieces16<T>; ++i) {
    f32x2 v[N / 2];
    raw_up<T, N>(r.p[i], v);
#pragma unroll
    for (int e = 0; e < N / 2; ++e) f[i * N / 2 + e] = v[e];
  }
}
template <typename T, int A>
__device__ __forceinline__ void block_store(typename T::bits *row, int b, int H,
                                            const f32x2 (&f)[8]) {
  constexpr int N = kPer16<T>;
#pragma unroll
  for (int i = 0; i < kPieces16<T>; ++i) {
    f32x2 v[N / 2];
#pragma unroll
    for (int e = 0; e < N / 2; ++e) v[e] = f[i * N / 2 + e];
    raw_store<T, N, A>(row, b * kPieces16<T> + i, H, raw_down<T>(v));
  }
}

}  // namespace moe
