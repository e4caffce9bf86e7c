// rows.cuh -- rows of 16- or 32-bit floats in pieces of a few elements, for
// the row-wise kernels (token dispatch and combination, RMS norm): raw loads
// and stores, and the exact or once-rounded conversions to and from fp32.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace moe {

// Two floats in one 64-bit register pair, the first in the low half: the
// packed fp32 instructions of sm_100 do both lanes in one issue, each rounded
// like the plain one.
using f32x2 = uint64_t;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpair(f32x2 v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Maxima that keep a NaN: of two, and of three magnitudes.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_abs_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Two floats to E4M3, saturating, ties to even; the first in the low byte.
__device__ __forceinline__ uint16_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The storage types of token and expert rows.  add: the sum of the elements of
// one 32-bit word, rounded once.
struct BF16 {
  using bits = uint16_t;
  static __device__ __forceinline__ uint32_t add(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  // two floats, the first in the low half
  static __device__ __forceinline__ uint32_t down2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ float2 up2(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
  }
  // the larger ones, NaN if there is one
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
};
struct F16 {
  using bits = uint16_t;
  static __device__ __forceinline__ uint32_t add(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ uint32_t down2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ float2 up2(uint32_t v) { return f16x2_to_float2(v); }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
};
struct F32 {
  using bits = uint32_t;
  static __device__ __forceinline__ uint32_t add(uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }
};

// Elements of T in the 16 bytes that a thread moves at a time.
template <typename T>
constexpr int kPer16 = 16 / (int)sizeof(typename T::bits);

// N consecutive elements as they are stored, in 32-bit words.
template <typename T, int N>
struct Raw {
  static constexpr int kWords = N * (int)sizeof(typename T::bits) / 4;
  uint32_t w[kWords];
};

template <typename T, int N>
__device__ __forceinline__ Raw<T, N> raw_zero() {
  Raw<T, N> r;
#pragma unroll
  for (int i = 0; i < Raw<T, N>::kWords; ++i) r.w[i] = 0;
  return r;
}

// The N elements at p, aligned to their bytes (at most 16).
template <typename T, int N>
__device__ __forceinline__ Raw<T, N> raw_load_aligned(const void *p) {
  constexpr int W = Raw<T, N>::kWords;
  Raw<T, N> r;
  if constexpr (W == 2) {
    const uint2 v = *static_cast<const uint2 *>(p);
    r.w[0] = v.x;
    r.w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const uint4 v = static_cast<const uint4 *>(p)[i];
      r.w[4 * i] = v.x;
      r.w[4 * i + 1] = v.y;
      r.w[4 * i + 2] = v.z;
      r.w[4 * i + 3] = v.w;
    }
  }
  return r;
}

// ---- pieces by alignment ------------------------------------------------------
//
// How the pieces of a call's rows are held and moved:
//   kWhole   16-byte aligned rows of whole pieces;
//   kHalves  8-byte aligned rows of whole 8-byte halves, two of them a piece;
//   kElems   such widths at any other alignment, element by element;
//   kDealt   other widths, element by element and dealt out in turn: element i
//            of a lane's piece is the (32 i + lane)th of the 32 N that a warp
//            holds, so that a warp's loads and stores are runs of neighbours (a
//            lane with N neighbours of its own makes four times the memory
//            wavefronts: the bf16 combine gradient at M = 2000, hidden = 1111,
//            top_k = 6 took 42.6 us, dealt out it takes 29.3).
// Which elements a thread holds depends on the width alone, not on the
// alignment, so neither do a sum's bits.
enum { kWhole = 16, kHalves = 8, kDealt = 2, kElems = 1 };

// Element i of piece c: its place in the row.
template <int N, int A>
__device__ __forceinline__ int place(int c, int i) {
  return A == kDealt ? (c & ~31) * N + (c & 31) + 32 * i : c * N + i;
}
// Whether piece c has an element of the row.
template <int N, int A>
__device__ __forceinline__ bool in_row(int c, int H) {
  return place<N, A>(c, 0) < H;
}

template <int ES> struct Elem;
template <> struct Elem<1> { using type = uint8_t; };
template <> struct Elem<2> { using type = uint16_t; };
template <> struct Elem<4> { using type = uint32_t; };

// Element i (of ES bytes) of a piece.
template <int ES>
__device__ __forceinline__ typename Elem<ES>::type elem_of(const uint4 &q, int i) {
  const int b = i * ES;
  const uint32_t w = b / 4 == 0 ? q.x : b / 4 == 1 ? q.y : b / 4 == 2 ? q.z : q.w;
  return (typename Elem<ES>::type)(w >> (8 * (b & 3)));
}

// Piece c of a row of H elements of ES bytes, zeros behind its end.
template <int ES, int A>
__device__ __forceinline__ uint4 load16(const void *row, int c, int H) {
  constexpr int N = 16 / ES;
  const char *p = static_cast<const char *>(row) + (size_t)c * 16;
  if constexpr (A == kWhole) {
    return *reinterpret_cast<const uint4 *>(p);
  } else if constexpr (A == kHalves) {
    const uint2 lo = *reinterpret_cast<const uint2 *>(p);
    const uint2 hi = c * N + N / 2 < H ? reinterpret_cast<const uint2 *>(p)[1] : make_uint2(0, 0);
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
  } else {
    const int first = place<N, A>(c, 0), left = H - first;
    const typename Elem<ES>::type *e = static_cast<const typename Elem<ES>::type *>(row) + first;
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (place<N, A>(0, i) < left)
        w[i * ES / 4] |= (uint32_t)e[place<N, A>(0, i)] << (8 * (i * ES & 3));
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}
template <int ES, int A>
__device__ __forceinline__ void store16(void *row, int c, int H, const uint4 &q) {
  constexpr int N = 16 / ES;
  char *p = static_cast<char *>(row) + (size_t)c * 16;
  if constexpr (A == kWhole) {
    *reinterpret_cast<uint4 *>(p) = q;
  } else if constexpr (A == kHalves) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(q.x, q.y);
    if (c * N + N / 2 < H) reinterpret_cast<uint2 *>(p)[1] = make_uint2(q.z, q.w);
  } else {
    const int first = place<N, A>(c, 0), left = H - first;
    typename Elem<ES>::type *e = static_cast<typename Elem<ES>::type *>(row) + first;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (place<N, A>(0, i) < left) e[place<N, A>(0, i)] = elem_of<ES>(q, i);
  }
}

// Piece c (N elements, 16 bytes, or 8 in the 16-bit type of a mixed pair) of a
// row of H elements, in_row; zeros behind the end.  Plain (coherent) loads: some
// callers let an output share an input's buffer, and under programmatic launch
// the grid in front may still write these rows when this one becomes resident
// (no ld.global.nc, which asks for data that is read-only for a grid's life).
template <typename T, int N, int A>
__device__ __forceinline__ Raw<T, N> raw_load(const typename T::bits *row, int c, int H) {
  constexpr int ES = sizeof(typename T::bits);
  if constexpr (N * ES == 16) {
    const uint4 q = load16<ES, A>(row, c, H);
    return Raw<T, N>{{q.x, q.y, q.z, q.w}};
  } else if constexpr (A == kWhole) {
    return raw_load_aligned<T, N>(row + (size_t)c * N);
  } else {
    Raw<T, N> r = raw_zero<T, N>();
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (const int e = place<N, A>(c, i); e < H)
        r.w[i * ES / 4] |= (uint32_t)row[e] << (8 * (i * ES & 3));
    return r;
  }
}
template <typename T, int N, int A>
__device__ __forceinline__ void raw_store(typename T::bits *row, int c, int H, const Raw<T, N> &r) {
  constexpr int ES = sizeof(typename T::bits);
  if constexpr (N * ES == 16) {
    store16<ES, A>(row, c, H, make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]));
  } else if constexpr (A == kWhole) {
    *reinterpret_cast<uint2 *>(row + (size_t)c * N) = make_uint2(r.w[0], r.w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (const int e = place<N, A>(c, i); e < H)
        row[e] = (typename T::bits)(r.w[i * ES / 4] >> (8 * (i * ES & 3)));
  }
}

// Exact.
template <typename T, int N>
__device__ __forceinline__ void raw_up(const Raw<T, N> &r, float (&f)[N]) {
  if constexpr (sizeof(typename T::bits) == 2) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float2 v = T::up2(r.w[i]);
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = __uint_as_float(r.w[i]);
  }
}

template <typename T, int N>
__device__ __forceinline__ void raw_up(const Raw<T, N> &r, f32x2 (&f)[N / 2]) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    if constexpr (sizeof(typename T::bits) == 2) {
      const float2 v = T::up2(r.w[i]);
      f[i] = pair(v.x, v.y);
    } else {
      f[i] = pair(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]));
    }
  }
}

template <typename T, int N>
__device__ __forceinline__ Raw<T, N> raw_add(const Raw<T, N> &a, const Raw<T, N> &b) {
  Raw<T, N> r;
#pragma unroll
  for (int i = 0; i < Raw<T, N>::kWords; ++i) r.w[i] = T::add(a.w[i], b.w[i]);
  return r;
}

// Rounded to nearest, ties to even.
template <typename T, int P>
__device__ __forceinline__ Raw<T, 2 * P> raw_down(const f32x2 (&f)[P]) {
  Raw<T, 2 * P> r;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const float2 v = unpair(f[i]);
    if constexpr (sizeof(typename T::bits) == 2) {
      r.w[i] = T::down2(v.x, v.y);
    } else {
      r.w[2 * i] = __float_as_uint(v.x);
      r.w[2 * i + 1] = __float_as_uint(v.y);
    }
  }
  return r;
}
template <typename T, int N>
__device__ __forceinline__ Raw<T, N> raw_down(const float (&f)[N]) {
  Raw<T, N> r;
  if constexpr (sizeof(typename T::bits) == 2) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) r.w[i] = T::down2(f[2 * i], f[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) r.w[i] = __float_as_uint(f[i]);
  }
  return r;
}

// ---- copies ahead (cp.async) ------------------------------------------------
//
// A thread copies pieces of rows that it will need into shared-memory slots of
// its own, one group of copies at a time, and waits for the oldest group: no
// barrier, no register holds what is in flight, and the wait ends with the
// copies themselves.

constexpr int kMaxDepth = 4;            // groups in flight
constexpr size_t kStaticBytes = 2048;   // more than a kernel's other shared memory, with which
                                        // the ring shares its limit

__device__ __forceinline__ void copy16_async(uint32_t shared, const void *global) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(shared), "l"(global) : "memory");
}
// BYTES (4 or 8) of them, zeros for the rest and for what is not `there`.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t shared, const void *global, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(shared), "l"(global),
               "n"(BYTES), "r"(there ? BYTES : 0)
               : "memory");
}
// Whether pieces of elements of ES bytes can be copied ahead: a copy moves four
// bytes at least.
template <int ES, int A>
constexpr bool kCopied = A == kWhole || A == kHalves || ES == 4;
// Copies piece c of a row of H elements of ES bytes, in_row, to a 16-byte slot.
template <int ES, int A>
__device__ __forceinline__ void copy_piece_async(uint32_t shared, const void *row, int c, int H) {
  static_assert(kCopied<ES, A>);
  constexpr int N = 16 / ES;
  const char *p = static_cast<const char *>(row) + (size_t)c * 16;
  if constexpr (A == kWhole) {
    copy16_async(shared, p);
  } else if constexpr (A == kHalves) {
    const bool there = c * N + N / 2 < H;
    copy_async<8>(shared, p, true);
    copy_async<8>(shared + 8, there ? p + 8 : p, there);
  } else {
    const char *r = static_cast<const char *>(row);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = place<N, A>(c, i);
      copy_async<ES>(shared + i * ES, r + (size_t)(e < H ? e : 0) * ES, e < H);
    }
  }
}
// The 16 bytes at a shared-memory address.
template <typename T>
__device__ __forceinline__ Raw<T, kPer16<T>> raw_load_shared(uint32_t shared) {
  Raw<T, kPer16<T>> r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3])
               : "r"(shared)
               : "memory");
  return r;
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// Until at most depth - 1 of this thread's committed groups are in flight.
__device__ __forceinline__ void copies_wait(int depth) {
  if (depth >= 4) asm volatile("cp.async.wait_group 3;" ::: "memory");
  else if (depth == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (depth == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else asm volatile("cp.async.wait_group 0;" ::: "memory");
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

// The alignment, in bytes up to 16, of rows at p that are `stride` elements of
// `bytes` apart and `hidden` long (NULL: not used).
inline int rows_alignment(const void *p, int64_t stride, int hidden, int bytes) {
  if (!p) return 16;
  const uint64_t v = (uint64_t)(uintptr_t)p | (uint64_t)(stride * bytes) |
                     (uint64_t)hidden * bytes | 16;
  return (int)(v & (~v + 1));
}
// f(integral_constant of how the pieces are moved) for an alignment in bytes of
// rows of `hidden` elements of `bytes`; MIXED: pairs of types, whose pieces have
// no halves.
template <bool MIXED = false, typename F>
int by_align(int align, int hidden, int bytes, F &&f) {
  if (align == 16) return f(std::integral_constant<int, kWhole>{});
  if constexpr (!MIXED)
    if (align == 8) return f(std::integral_constant<int, kHalves>{});
  if (hidden * bytes % (MIXED ? 16 : 8)) return f(std::integral_constant<int, kDealt>{});
  return f(std::integral_constant<int, kElems>{});
}

// Whether by_align's choice can be copied ahead (kCopied).
inline bool can_copy(int align, int bytes) { return align >= kHalves || bytes == 4; }

// Whether p is aligned to its elements.
inline bool elem_aligned(const void *p, int bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }

}  // namespace moe
