// rows.cuh -- rows of 16- or 32-bit floats in chunks of eight, for the
// row-wise kernels (token dispatch and combination, RMS norm): raw loads and
// stores, and the exact or once-rounded conversions to and from fp32.
#pragma once

#include "common.cuh"

namespace moe {

// The storage types of token and expert rows.
struct BF16 {
  using bits = uint16_t;
  static __device__ __forceinline__ float up(uint16_t b) { return bf16_to_float(b); }
  static __device__ __forceinline__ uint16_t down(float f) { return float_to_bf16_rn(f); }
  // two floats, the first in the low half
  static __device__ __forceinline__ uint32_t down2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ float2 up2(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
  }
};
struct F16 {
  using bits = uint16_t;
  static __device__ __forceinline__ float up(uint16_t b) {
    float f;
    asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(b));
    return f;
  }
  static __device__ __forceinline__ uint16_t down(float f) {
    uint16_t r;
    asm("cvt.rn.f16.f32 %0, %1;" : "=h"(r) : "f"(f));
    return r;
  }
  static __device__ __forceinline__ uint32_t down2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ float2 up2(uint32_t v) { return f16x2_to_float2(v); }
};
struct F32 {
  using bits = uint32_t;
  static __device__ __forceinline__ float up(uint32_t b) { return __uint_as_float(b); }
  static __device__ __forceinline__ uint32_t down(float f) { return __float_as_uint(f); }
};

constexpr int kChunk = 8;   // elements a thread takes at a time

// Eight elements as they are stored: one 16-byte register quad, or two.
template <typename T>
struct Raw {
  static constexpr int kQuads = (int)sizeof(typename T::bits) * kChunk / 16;
  uint4 q[kQuads];
};

template <typename T>
__device__ __forceinline__ Raw<T> raw_zero() {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < Raw<T>::kQuads; ++i) r.q[i] = make_uint4(0, 0, 0, 0);
  return r;
}

// Chunk c of a row of H elements.  VEC: the row is 16-byte aligned and H is a
// multiple of 8.  Otherwise element by element, zeros behind the end.  Plain
// (coherent) loads: some callers let an output share an input's buffer.
template <typename T, bool VEC>
__device__ __forceinline__ Raw<T> raw_load(const typename T::bits *row, int c, int H) {
  Raw<T> r;
  if (VEC) {
    const uint4 *p = reinterpret_cast<const uint4 *>(row + (size_t)c * kChunk);
#pragma unroll
    for (int i = 0; i < Raw<T>::kQuads; ++i) r.q[i] = p[i];
  } else {
    const typename T::bits *p = row + (size_t)c * kChunk;
    const int left = H - c * kChunk;
    uint32_t w[Raw<T>::kQuads * 4];
    if (sizeof(typename T::bits) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = 2 * i < left ? (uint32_t)p[2 * i] : 0u;
        const uint32_t hi = 2 * i + 1 < left ? (uint32_t)p[2 * i + 1] : 0u;
        w[i] = lo | (hi << 16);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kChunk; ++i) w[i % (Raw<T>::kQuads * 4)] = i < left ? (uint32_t)p[i] : 0u;
    }
#pragma unroll
    for (int i = 0; i < Raw<T>::kQuads; ++i)
      r.q[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
  return r;
}

template <typename T, bool VEC>
__device__ __forceinline__ void raw_store(typename T::bits *row, int c, int H, const Raw<T> &r) {
  if (VEC) {
    uint4 *p = reinterpret_cast<uint4 *>(row + (size_t)c * kChunk);
#pragma unroll
    for (int i = 0; i < Raw<T>::kQuads; ++i) p[i] = r.q[i];
  } else {
    typename T::bits *p = row + (size_t)c * kChunk;
    const int left = H - c * kChunk;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      if (i >= left) continue;
      constexpr int per = 4 / (int)sizeof(typename T::bits);   // elements per 32-bit word
      const uint4 q = r.q[i / (4 * per)];
      const int k = (i / per) & 3;
      const uint32_t w = k == 0 ? q.x : k == 1 ? q.y : k == 2 ? q.z : q.w;
      p[i] = (typename T::bits)(per == 2 && (i & 1) ? w >> 16 : w);
    }
  }
}

// Exact.
template <typename T>
__device__ __forceinline__ void raw_up(const Raw<T> &r, float (&f)[kChunk]) {
  if constexpr (sizeof(typename T::bits) == 2) {
    const uint32_t w[4] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = T::up2(w[i]);
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f[4 * i] = __uint_as_float(r.q[i].x);
      f[4 * i + 1] = __uint_as_float(r.q[i].y);
      f[4 * i + 2] = __uint_as_float(r.q[i].z);
      f[4 * i + 3] = __uint_as_float(r.q[i].w);
    }
  }
}

// Rounded to nearest, ties to even.
template <typename T>
__device__ __forceinline__ Raw<T> raw_down(const float (&f)[kChunk]) {
  Raw<T> r;
  if constexpr (sizeof(typename T::bits) == 2) {
    r.q[0] = make_uint4(T::down2(f[0], f[1]), T::down2(f[2], f[3]), T::down2(f[4], f[5]),
                        T::down2(f[6], f[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      r.q[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]),
                          __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3]));
  }
  return r;
}

// ---- host ------------------------------------------------------------------

inline int dtype_bytes(int dtype) {
  switch (dtype) {
    case MOE_DTYPE_BF16:
    case MOE_DTYPE_F16: return 2;
    case MOE_DTYPE_F32: return 4;
    case MOE_DTYPE_E4M3: return 1;
    default: return 0;
  }
}

// Whether rows of `hidden` elements at p, `stride` elements apart, can be
// read and written in 16-byte pieces (NULL: not used).
inline bool rows_vector(const void *p, int64_t stride, int bytes) {
  return !p || (((uintptr_t)p & 15) == 0 && (stride * bytes) % 16 == 0);
}
// Whether p is aligned to its elements.
inline bool elem_aligned(const void *p, int bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }

}  // namespace moe
