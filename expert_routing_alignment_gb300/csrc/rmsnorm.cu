// rmsnorm.cu -- residual addition with root-mean-square norm in front of the
// router (moe_add_rmsnorm), its 8-bit output, and its gradient
// (moe_add_rmsnorm_backward).
#include <math.h>

#include "common.cuh"
#include "rows.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr float kE4m3Max = 448.f;
constexpr float kScaleMin = 1.17549435e-38f;   // 2^-126, the smallest normal

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

// Sum over the threads of a row group (blockDim.x threads, whole warps):
// butterfly in the warp, then the warps' sums four by four.  One barrier, of
// the group alone; calls that follow one another take turns between two
// `red`s, whose unused places are zero.
constexpr int kRedFloats = 64;   // a multiple of four per group, 48 at most (12 of two warps)
__device__ __forceinline__ float group_sum(float v, float *red) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return v;
  float *mine = red + threadIdx.y * ((nw + 3) & ~3);
  if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(1 + threadIdx.y), "r"(blockDim.x) : "memory");
  v = 0.f;
  for (int i = 0; i < nw; i += 4) {
    const float4 q = *reinterpret_cast<const float4 *>(mine + i);
    v += (q.x + q.y) + (q.z + q.w);
  }
  return v;
}
// Before the first group_sum; the whole CTA.
__device__ __forceinline__ void clear_red(float (&red)[2][kRedFloats]) {
  const int i = threadIdx.y * blockDim.x + threadIdx.x;
  if (i < 2 * kRedFloats) red[i / kRedFloats][i % kRedFloats] = 0.f;
  for (int k = i + blockDim.x * blockDim.y; k < 2 * kRedFloats; k += blockDim.x * blockDim.y)
    red[k / kRedFloats][k % kRedFloats] = 0.f;
  __syncthreads();
}

// ---------------------------------------------------------------------------
// how rows are split and fed
// ---------------------------------------------------------------------------
//
// A row of H elements is split over TPR threads (whole warps) of CH 16-byte
// pieces each, thread i taking the pieces i, i + TPR, ...: a function of H
// and the type alone, so that a row's bits do not depend on the batch.  A CTA
// holds several such groups, each walking over rows of its own.  A thread
// copies its own pieces of the rows ahead into its own shared-memory slots
// (cp.async, `depth` rows deep), so no barrier stands between a copy and its
// use and the loads of later rows are in flight while a row waits for its sum.
struct Split {
  int ch, tpr;   // pieces a thread, threads a row
};
// `two`: the most pieces of a row that is split in two a thread.  Forward 896:
// 448 threads at hidden = 7168 (M = 4096, E4M3) 38.9 us, four pieces for each of
// 224 threads 47.1.  Gradient 512, up to 768 threads: at 896, with 72 registers
// a thread instead of 80, hidden = 4096 (M = 10007) went from 55.6 to 71.4 us.
// Widths that are dealt out by elements take 896 there too (hidden = 4097,
// M = 8000: 193 us with four pieces a thread, 126 with two).
Split split_row(int H, int per16, int two) {
  const int pieces = (H + per16 - 1) / per16;
  const int ch = pieces <= 256 ? 1 : pieces <= two ? 2 : pieces <= 2048 ? 4 : 8;
  return Split{ch, ((pieces + ch - 1) / ch + 31) / 32 * 32};
}
constexpr int kTwoForward = 896, kTwoGradient = 512;

// Rows in flight for a group so that an SM has about `flight` bytes in flight
// with `groups` groups; no more than a group has rows (`turns`).
int plan_depth(size_t stage, int groups, int64_t turns, int flight) {
  const int64_t depth = flight / (int64_t)(stage * groups);
  const int64_t most = turns < kMaxDepth ? turns : kMaxDepth;
  return depth < 1 ? 1 : depth > most ? (int)most : (int)depth;
}

// The rows of IN input arrays (the last may be NULL: not used), as the walk
// above feeds them, or, by elements of two bytes, which no copy moves, read
// straight from global memory.  (Straight against ahead: bf16 in halves, M = 8000,
// hidden = 4100, 56.6 us and 48.6, gradient 112 and 67; fp32 by elements,
// hidden = 4097, 200 and 122, gradient 296 and 130; calls of one row a group are
// up to 0.8 us slower ahead, fp32 M = 400, hidden = 1001: 2.6 and 3.4.)  In a stage
// the slots of neighbouring threads are next to one another: copies and reads
// of a warp are whole lines.  (Slots by thread, 112 bytes apart, took the
// gradient at M = 10007, hidden = 4096 from 56 to 85 us.)
template <typename T, int IN, int CH, int A>
struct RowFeed {
  using TB = typename T::bits;
  static constexpr int N = kPer16<T>;
  static constexpr bool kAhead = kCopied<sizeof(TB), A>;
  const TB *in[IN];
  int64_t stride[IN];
  int H, depth;
  uint32_t at, first, last;   // this thread's slots: of the current stage, the ring's bounds

  __device__ __forceinline__ uint32_t unit() const { return blockDim.x * blockDim.y * 16; }
  __device__ __forceinline__ uint32_t stage_bytes() const {
    return unit() * IN * CH;
  }
  __device__ __forceinline__ void init(uint4 *ring) {
    const int flat = threadIdx.y * blockDim.x + threadIdx.x;
    first = at = (uint32_t)__cvta_generic_to_shared(ring) + flat * 16;
    last = first + depth * stage_bytes();
  }
  __device__ __forceinline__ bool used() const { return in[IN - 1] != nullptr; }
  __device__ __forceinline__ bool on(int i) const {
    return in_row<N, A>(threadIdx.x + i * blockDim.x, H);
  }
  // Starts the copies of a row into the current stage (one group of copies,
  // empty if !live) and moves on to the next stage.
  __device__ __forceinline__ void start(int64_t row, bool live) {
    if constexpr (kAhead) {
      if (live) {
#pragma unroll
        for (int a = 0; a < IN; ++a) {
          if (a == IN - 1 && !used()) continue;
          const TB *p = in[a] + row * stride[a];
#pragma unroll
          for (int i = 0; i < CH; ++i)
            if (on(i))
              copy_piece_async<sizeof(TB), A>(at + (a * CH + i) * unit(), p,
                                              threadIdx.x + i * blockDim.x, H);
        }
      }
      copies_commit();
      at += stage_bytes();
      if (at == last) at = first;
    }
  }
  __device__ __forceinline__ void wait() const {
    if constexpr (kAhead) copies_wait(depth);
  }
  // This thread's piece i (on(i)) of array a, row `row` in the current stage.
  __device__ __forceinline__ Raw<T, N> get(int64_t row, int a, int i) const {
    if constexpr (kAhead)
      return raw_load_shared<T>(at + (a * CH + i) * unit());
    else
      return raw_load<T, N, A>(in[a] + row * stride[a], threadIdx.x + i * blockDim.x, H);
  }
};

// The weights of a thread's pieces as fp32: in registers over all of its rows
// where they are few, else read again (from L1) for every row.
template <typename W, int N, int CH, int A>
struct Weights {
  static constexpr bool kHeld = CH * N <= 16;
  f32x2 held[kHeld ? CH : 1][N / 2];

  static __device__ __forceinline__ void read(const typename W::bits *w, int H, int i,
                                              f32x2 (&f)[N / 2]) {
    const int c = threadIdx.x + i * blockDim.x;
    raw_up<W, N>(in_row<N, A>(c, H) ? raw_load<W, N, A>(w, c, H) : raw_zero<W, N>(), f);
  }
  __device__ __forceinline__ void load(const typename W::bits *w, int H) {
    if constexpr (kHeld) {
#pragma unroll
      for (int i = 0; i < CH; ++i) read(w, H, i, held[i]);
    }
  }
  __device__ __forceinline__ void get(const typename W::bits *w, int H, int i,
                                      f32x2 (&f)[N / 2]) const {
    if constexpr (kHeld) {
#pragma unroll
      for (int e = 0; e < N / 2; ++e) f[e] = held[i][e];
    } else {
      read(w, H, i, f);
    }
  }
};

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
//
//   s = T(x + r);  rstd = 1 / sqrt(mean(s^2) + eps);  out = T(s * rstd * w)
// and, by blocks of 128 columns with m = max |s * w|:
//   scale = m * rstd / 448,  code = e4m3((s * w) * 448 / m).
// The code's quotient leaves rstd out: for 16-bit s and w the product s * w
// and its multiple by 448 = 7 * 64 are exact in fp32 (16 + 3 bits for bf16;
// 22 + 3 for fp16, rounded once), so the only rounding ahead of the code is
// the quotient's, and the codes do not depend on the order of the sum of
// squares.  Where the scale would be below 2^-126 it is 2^-126, so that no
// scale is zero or subnormal.  Bound by HBM: bf16 at M = 32768, hidden = 4096
// (1.07 GB) 165 us, 6.5 TB/s; with E4M3 output at M = 4096 (118 MB) 23.0 us,
// 5.1 TB/s, of which launch, first loads and the last rows take about 4.  72
// registers a thread with one or two pieces: rows of other widths spill up to 48
// bytes there.

// The sum of squares is kept in fp32, whose range it can leave while rstd does
// not.  Where mean + eps is below 2^-80 (squares lose bits under 2^-126; they
// are lost against eps otherwise) or overflows, a row is summed again times a
// power of two, which comes out of the root exactly: 2^90 takes a sum of squares
// below 2^-66 (16384 elements) to 2^114 at most, and the least element, 2^-149,
// to 2^-59, whose square is normal; 2^-80 takes the largest, 2^128, to 2^48, and
// 16384 of those squares are 2^110.  The test costs an ordinary row 0.2 us in 23
// (bf16 with E4M3 output at M = 4096, hidden = 4096), nothing at M = 32768.
constexpr float kMeanLow = 0x1p-80f, kMeanHigh = 3.402823466e38f;
constexpr float kScaleUp = 0x1p90f, kScaleDown = 0x1p-80f;

struct NormArgs {
  const void *x, *r, *w;
  int64_t xs, rs;
  int M, H, depth;
  float eps, inv_H;
  void *sum, *out;
  uint8_t *codes;
  float *scale, *rstd;
};

// 448 * p / m for |p| <= m: with y = 1 / m rounded once, q = 448 p * y and its
// residual 448 p - q m (one fma), q + residual * y is the quotient to within
// its own rounding, and exact where the quotient is a float (a tie of the
// code's rounding is); one division a block instead of one an element
// (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990).  For m in [2^-100, 2^100], where neither the
// residual nor y leaves the normal range.
__device__ __forceinline__ f32x2 code_quotient(f32x2 p, f32x2 minus_m, f32x2 y) {
  const f32x2 a = mul2(p, pair(kE4m3Max, kE4m3Max)), q = mul2(a, y);
  return fma2(fma2(q, minus_m, a), y, q);
}

template <typename T, typename W, int CH, int A>
__global__ void __launch_bounds__(CH <= 2 ? 448 : 512, CH <= 2 ? 2 : 1)
    add_rmsnorm_kernel(NormArgs a) {
  using TB = typename T::bits;
  using WB = typename W::bits;
  constexpr int N = kPer16<T>;
  extern __shared__ uint4 ring[];
  __shared__ __align__(16) float red[2][kRedFloats];
  pdl_wait();
  pdl_trigger();
  const int H = a.H, tid = threadIdx.x, tpr = blockDim.x;
  const WB *w = static_cast<const WB *>(a.w);
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  RowFeed<T, 2, CH, A> feed{{static_cast<const TB *>(a.x), static_cast<const TB *>(a.r)},
                              {a.xs, a.rs},
                              H,
                              a.depth};
  feed.init(ring);
  for (int d = 0; d < a.depth; ++d) feed.start(row + d * step, row + d * step < a.M);
  Weights<W, N, CH, A> weights;
  weights.load(w, H);
  clear_red(red);
  int turn = 0;
  for (; row < a.M; row += step) {
    const size_t out_at = (size_t)row * H;
    feed.wait();
    Raw<T, N> sr[CH];
    f32x2 sq = 0;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      sr[i] = raw_zero<T, N>();
      if (feed.on(i)) {
        sr[i] = feed.get(row, 0, i);
        // the sum as it is stored is what is normalised
        if (feed.used()) sr[i] = raw_add<T, N>(sr[i], feed.get(row, 1, i));
        if (a.sum)
          raw_store<T, N, A>(static_cast<TB *>(a.sum) + out_at, tid + i * tpr, H, sr[i]);
      }
      f32x2 f[N / 2];
      raw_up<T, N>(sr[i], f);
#pragma unroll
      for (int e = 0; e < N / 2; ++e) sq = fma2(f[e], f[e], sq);
    }
    const float2 sq2 = unpair(sq);
    const float mean = group_sum(sq2.x + sq2.y, red[turn]) * a.inv_H + a.eps;
    // the slots of this row have been read: the row `depth` turns on goes there
    feed.start(row + a.depth * step, row + a.depth * step < a.M);
    turn ^= 1;
    float rstd = 1.f / sqrtf(mean);
    if (!(mean >= kMeanLow && mean <= kMeanHigh)) {   // the same for a whole group
      const float c = mean < kMeanLow ? kScaleUp : kScaleDown;
      sq = 0;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        f32x2 f[N / 2];
        raw_up<T, N>(sr[i], f);
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
          f[e] = mul2(f[e], pair(c, c));
          sq = fma2(f[e], f[e], sq);
        }
      }
      const float2 q = unpair(sq);
      rstd = c / sqrtf(group_sum(q.x + q.y, red[turn]) * a.inv_H + a.eps * c * c);
      turn ^= 1;
    }
    if (a.rstd && tid == 0) a.rstd[row] = rstd;
    if (!a.out && !a.codes) continue;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = tid + i * tpr;
      const bool on = feed.on(i);
      f32x2 f[N / 2], wf[N / 2];
      raw_up<T, N>(sr[i], f);
      weights.get(w, H, i, wf);
      if (a.out && on) {
        f32x2 v[N / 2];
#pragma unroll
        for (int e = 0; e < N / 2; ++e) v[e] = mul2(mul2(f[e], pair(rstd, rstd)), wf[e]);
        raw_store<T, N, A>(static_cast<TB *>(a.out) + out_at, c, H, raw_down<T>(v));
      }
      if (a.codes) {
        // Blocks of 128 columns: 128 / N lanes hold one; dealt out, a lane has
        // four elements of each of N / 4 blocks.
        constexpr int B = A == kDealt ? N / 4 : 1, G = N / B;   // blocks of a piece, elements each
#pragma unroll
        for (int b = 0; b < B; ++b) {
          float m = 0.f;
#pragma unroll
          for (int e = b * G / 2; e < (b + 1) * G / 2; ++e) {
            f[e] = mul2(f[e], wf[e]);
            const float2 p = unpair(f[e]);
            m = max_abs_nan(m, p.x, p.y);
          }
#pragma unroll
          for (int d = 64 / G; d > 0; d >>= 1) m = max_nan(m, __shfl_xor_sync(kFull, m, d));
          float sc = m * rstd / kE4m3Max;
          if (sc >= kScaleMin && m >= 0x1p-100f && m <= 0x1p100f) {
            const float y = 1.f / m;
#pragma unroll
            for (int e = b * G / 2; e < (b + 1) * G / 2; ++e)
              f[e] = code_quotient(f[e], pair(-m, -m), pair(y, y));
          } else {   // scales at their floor, and extremes of s * w
            const bool low = sc < kScaleMin;
#pragma unroll
            for (int e = b * G / 2; e < (b + 1) * G / 2; ++e) {
              const float2 p = unpair(f[e]);
              f[e] = low ? pair(p.x * rstd / kScaleMin, p.y * rstd / kScaleMin)
                         : pair(p.x * kE4m3Max / m, p.y * kE4m3Max / m);
            }
            if (low) sc = kScaleMin;
          }
          // the lane that holds a block's first element
          if (const int x = place<N, A>(c, b * G); x < H && x % 128 == 0)
            a.scale[row * ((H + 127) / 128) + x / 128] = sc;
        }
        uint32_t q[N / 4];
#pragma unroll
        for (int e = 0; e < N / 4; ++e) {
          const float2 lo = unpair(f[2 * e]), hi = unpair(f[2 * e + 1]);
          q[e] = to_e4m3x2(lo.x, lo.y) | ((uint32_t)to_e4m3x2(hi.x, hi.y) << 16);
        }
        if (on) {
          uint8_t *dst = a.codes + out_at;
          if constexpr (A != kWhole) {
#pragma unroll
            for (int e = 0; e < N; ++e)
              if (const int x = place<N, A>(c, e); x < H)
                dst[x] = (uint8_t)(q[e / 4] >> (8 * (e & 3)));
          } else if constexpr (N == 8) {
            *reinterpret_cast<uint2 *>(dst + (size_t)c * N) = make_uint2(q[0], q[1]);
          } else {
            *reinterpret_cast<uint32_t *>(dst + (size_t)c * N) = q[0];
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------
//
// With xh = s * rstd and g = dout * w:
//   dx = T(rstd * (g - xh * mean(g * xh)) + dsum),  dw = sum_t dout[t] * xh[t].
// A group walks over its rows with their part of dw in registers; one CTA an
// SM adds its groups' parts in order, the CTAs' parts go to the workspace
// [CTAs][H] and a second kernel adds those in a fixed order, so the bits are
// the same every time.  80 registers a thread with two pieces (8 bytes of spills
// on whole pieces, up to 76 by elements).  Bound by HBM: bf16 at M = 10007,
// hidden = 4096 (328 MB) 53.9 us, 6.1 TB/s, of which the second kernel and its
// launch take about 3.

struct NormGradArgs {
  const void *dout, *sum, *dsum, *w;
  const float *rstd;
  int64_t ds, ss, es;
  int M, H, depth;
  float inv_H;
  void *dx;
  float *part;       // [gridDim.x][H], or NULL: no dw
};

// Threads of a CTA: as many as the registers of an SM hold.
constexpr int grad_threads(int ch) { return ch <= 2 ? 768 : 512; }

template <typename T, typename W, int CH, int A>
__global__ void __launch_bounds__(grad_threads(CH)) rmsnorm_grad_kernel(NormGradArgs a) {
  using TB = typename T::bits;
  using WB = typename W::bits;
  constexpr int N = kPer16<T>;
  extern __shared__ uint4 ring[];
  __shared__ __align__(16) float red[2][kRedFloats];
  pdl_wait();
  pdl_trigger();
  const int H = a.H, tid = threadIdx.x, tpr = blockDim.x;
  const WB *w = static_cast<const WB *>(a.w);
  f32x2 dw[CH][N / 2] = {};
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  RowFeed<T, 3, CH, A> feed{{static_cast<const TB *>(a.dout), static_cast<const TB *>(a.sum),
                               static_cast<const TB *>(a.dsum)},
                              {a.ds, a.ss, a.es},
                              H,
                              a.depth};
  feed.init(ring);
  for (int d = 0; d < a.depth; ++d) feed.start(row + d * step, row + d * step < a.M);
  Weights<W, N, CH, A> weights;
  weights.load(w, H);
  clear_red(red);
  int turn = 0;
  float next = row < a.M ? a.rstd[row] : 0.f;   // rstd, read a row ahead
  for (; row < a.M; row += step) {
    const size_t out_at = (size_t)row * H;
    const float rstd = next;
    next = row + step < a.M ? a.rstd[row + step] : 0.f;
    const f32x2 rstd2 = pair(rstd, rstd);
    feed.wait();
    Raw<T, N> dr[CH], sr[CH];
    f32x2 dot = 0;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (!feed.on(i)) continue;
      dr[i] = feed.get(row, 0, i);
      sr[i] = feed.get(row, 1, i);
      f32x2 d[N / 2], xh[N / 2], wf[N / 2];
      raw_up<T, N>(dr[i], d);
      raw_up<T, N>(sr[i], xh);
      weights.get(w, H, i, wf);
#pragma unroll
      for (int e = 0; e < N / 2; ++e) {
        xh[e] = mul2(xh[e], rstd2);
        dw[i][e] = fma2(d[e], xh[e], dw[i][e]);
        dot = fma2(mul2(d[e], wf[e]), xh[e], dot);
      }
    }
    const float2 dot2 = unpair(dot);
    const float mean = group_sum(dot2.x + dot2.y, red[turn]) * a.inv_H;
    // no product of two rstd, which leaves fp32's range long before dx does
    const f32x2 back = pair(-mean, -mean);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (!feed.on(i)) continue;
      f32x2 d[N / 2], s[N / 2], wf[N / 2], v[N / 2] = {};
      raw_up<T, N>(dr[i], d);
      raw_up<T, N>(sr[i], s);
      if (feed.used()) raw_up<T, N>(feed.get(row, 2, i), v);
      weights.get(w, H, i, wf);
#pragma unroll
      for (int e = 0; e < N / 2; ++e)
        v[e] = fma2(rstd2, fma2(mul2(s[e], rstd2), back, mul2(d[e], wf[e])), v[e]);
      raw_store<T, N, A>(static_cast<TB *>(a.dx) + out_at, tid + i * tpr, H, raw_down<T>(v));
    }
    // the slots of this row have been read: the row `depth` turns on goes there
    feed.start(row + a.depth * step, row + a.depth * step < a.M);
    turn ^= 1;
  }
  if (!a.part) return;
  float *part = a.part + (size_t)blockIdx.x * H;
  // the groups' parts are added in shared memory, in the ring's place
  const bool shared = blockDim.y > 1;
  float *parts = reinterpret_cast<float *>(ring);
  copies_wait(1);
  if (shared) __syncthreads();
  float *mine = shared ? parts + threadIdx.y * H : part;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int h = (tid + i * tpr) * N;
    if (A == kWhole) {
      if (h < H)
#pragma unroll
        for (int e = 0; e < N / 4; ++e)
          *reinterpret_cast<ulonglong2 *>(mine + h + 4 * e) =
              make_ulonglong2(dw[i][2 * e], dw[i][2 * e + 1]);
    } else {
#pragma unroll
      for (int e = 0; e < N / 2; ++e) {
        const float2 v = unpair(dw[i][e]);
        const int c = tid + i * tpr;
        const int x = place<N, A>(c, 2 * e), y = place<N, A>(c, 2 * e + 1);
        if (x < H) mine[x] = v.x;
        if (y < H) mine[y] = v.y;
      }
    }
  }
  if (!shared) return;
  __syncthreads();
  for (int h = threadIdx.y * tpr + tid; h < H; h += tpr * blockDim.y) {
    float v = parts[h];
    for (int y = 1; y < (int)blockDim.y; ++y) v += parts[y * H + h];
    part[h] = v;
  }
}

constexpr int kSms = 152;

// dw[h] = sum over the CTAs' parts, kSms at most: 32 columns a CTA, 32 threads a
// column that take every 32nd part (five at most, all loads ahead of the sums),
// then a butterfly over those.
__global__ void __launch_bounds__(1024) sum_parts_kernel(const float *part, int n, int H,
                                                         float *dw) {
  __shared__ float red[32][33];
  pdl_wait();
  pdl_trigger();
  const int x = threadIdx.x, y = threadIdx.y, h = blockIdx.x * 32 + x;
  constexpr int kEach = (kSms + 31) / 32;
  float q[kEach], v = 0.f;
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    const int i = y + 32 * u;
    q[u] = h < H && i < n ? __ldcg(part + (size_t)i * H + h) : 0.f;
  }
#pragma unroll
  for (int u = 0; u < kEach; ++u) v += q[u];
  red[y][x] = v;
  __syncthreads();
  v = red[x][y];   // column y of the CTA, its x-th sum
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  if (x == 0 && blockIdx.x * 32 + y < H) dw[blockIdx.x * 32 + y] = v;
}

// The walk of the gradient over M rows: one CTA an SM (a constant, not the
// device's count: dw's order depends on M, hidden and the type alone), as many
// groups in it as its threads allow and the rows need.
struct Walk {
  int ctas, groups;
};
Walk grad_walk(int M, const Split &s) {
  const int64_t want = ceil_div64(M, kSms);
  const int fit = grad_threads(s.ch) / s.tpr;
  const int groups = want < 1 ? 1 : want < fit ? (int)want : fit;
  const int64_t ctas = ceil_div64(M, groups);
  return Walk{ctas < kSms ? (int)ctas : kSms, groups};
}

template <typename F>
int with_norm_types(int dtype, int weight_dtype, F &&f) {
  if (dtype == MOE_DTYPE_BF16 && weight_dtype == MOE_DTYPE_BF16) return f(BF16{}, BF16{});
  if (dtype == MOE_DTYPE_BF16 && weight_dtype == MOE_DTYPE_F32) return f(BF16{}, F32{});
  if (dtype == MOE_DTYPE_F16 && weight_dtype == MOE_DTYPE_F16) return f(F16{}, F16{});
  if (dtype == MOE_DTYPE_F16 && weight_dtype == MOE_DTYPE_F32) return f(F16{}, F32{});
  if (dtype == MOE_DTYPE_F32 && weight_dtype == MOE_DTYPE_F32) return f(F32{}, F32{});
  return MOE_EUNSUPPORTED;
}

bool float_dtype(int d) {
  return d == MOE_DTYPE_BF16 || d == MOE_DTYPE_F16 || d == MOE_DTYPE_F32;
}

int norm_sizes(int dtype, int weight_dtype, int M, int H) {
  if (!float_dtype(dtype) || !float_dtype(weight_dtype) || M < 0 || H < 1) return MOE_EINVAL;
  if (H > MOE_MAX_ROW_HIDDEN) return MOE_EUNSUPPORTED;
  return with_norm_types(dtype, weight_dtype, [](auto, auto) { return MOE_OK; });
}

}  // namespace

int check_add_rmsnorm(const void *x, int64_t x_stride, const void *residual,
                      int64_t residual_stride, const void *weight, int dtype, int weight_dtype,
                      int M, int hidden, float eps, const void *sum_out, const void *out,
                      const uint8_t *out_codes, const float *out_scale, const float *rstd) {
  const int st = norm_sizes(dtype, weight_dtype, M, hidden);
  if (st) return st;
  if (!(eps >= 0.f) || isinf(eps) || x_stride < 0 || residual_stride < 0) return MOE_EINVAL;
  if (M == 0) return MOE_OK;
  if (!x || !weight || (!sum_out && !out && !out_codes && !rstd)) return MOE_EINVAL;
  if (!out_codes != !out_scale) return MOE_EINVAL;
  const int b = dtype_bytes(dtype);
  if (!elem_aligned(x, b) || !elem_aligned(residual, b) || !elem_aligned(sum_out, b) ||
      !elem_aligned(out, b) || !elem_aligned(weight, dtype_bytes(weight_dtype)) ||
      !elem_aligned(out_scale, 4) || !elem_aligned(rstd, 4))
    return MOE_EINVAL;
  if (sum_out && sum_out == out) return MOE_EINVAL;
  // an output may take an input's place only element for element
  if ((x_stride != hidden && (x == sum_out || x == out)) ||
      (residual && residual_stride != hidden && (residual == sum_out || residual == out)))
    return MOE_EINVAL;
  return MOE_OK;
}

}  // namespace moe

extern "C" int moe_add_rmsnorm(const void *x, int64_t x_stride, const void *residual,
                               int64_t residual_stride, const void *weight, int dtype,
                               int weight_dtype, int M, int hidden, float eps, void *sum_out,
                               void *out, uint8_t *out_codes, float *out_scale, float *rstd,
                               void *stream) {
  using namespace moe;
  const int st = check_add_rmsnorm(x, x_stride, residual, residual_stride, weight, dtype,
                                   weight_dtype, M, hidden, eps, sum_out, out, out_codes,
                                   out_scale, rstd);
  if (st || M == 0) return st;
  const int b = dtype_bytes(dtype), wb = dtype_bytes(weight_dtype);
  const int n = 16 / b;   // elements of a piece
  int align = rows_alignment(x, x_stride, hidden, b);
  for (const int k : {rows_alignment(residual, residual_stride, hidden, b),
                      rows_alignment(sum_out, hidden, hidden, b),
                      rows_alignment(out, hidden, hidden, b),
                      rows_alignment(weight, hidden, hidden, wb)})
    if (k < align) align = k;
  if ((uintptr_t)out_codes % n && align == kWhole) align = kHalves;
  // CTAs of about 256 threads, as many as an SM's registers hold (72 a thread,
  // 128 with four pieces and more)
  const Split s = split_row(hidden, n, kTwoForward);
  const int rows = s.tpr >= 256 ? 1 : 256 / s.tpr;
  const int resident = (s.ch <= 2 ? 896 : 512) / (s.tpr * rows);
  const int sms = sm_count();
  if (!sms) return MOE_ECUDA;
  const int64_t turns = ceil_div64(M, rows), most = (int64_t)sms * resident;
  const int64_t ctas = turns < most ? turns : most;
  // 64 KB in flight an SM: at M = 32768, hidden = 4096 in bf16 165 us, but 175
  // with 96 or 128 KB (the reads crowd out the writes); at M = 16384, hidden =
  // 1024 23.3, with 32 KB 27.4, with 128 KB 25.6
  const size_t stage = (size_t)2 * s.ch * s.tpr * rows * 16;
  const int depth = plan_depth(stage, resident, ceil_div64(turns, ctas), 64 * 1024);
  const NormArgs a{x,   residual, weight,    x_stride,  residual_stride, M, hidden, depth,
                   eps, 1.f / hidden, sum_out, out, out_codes, out_scale, rstd};
  const dim3 grid((unsigned)ctas), block(s.tpr, rows);
  const size_t smem = can_copy(align, b) ? depth * stage : 0;
  return with_norm_types(dtype, weight_dtype, [&](auto t, auto w) {
    using T = decltype(t);
    using W = decltype(w);
    auto go = [&](auto kernel) {
      const int rc = ensure_smem_limit((const void *)kernel, smem + kStaticBytes);
      return rc ? rc : launch_pdl(kernel, grid, block, smem, stream, a);
    };
    auto with = [&](auto ch) {
      return by_align(align, hidden, b, [&](auto al) {
        return go(add_rmsnorm_kernel<T, W, decltype(ch)::value, decltype(al)::value>);
      });
    };
    if (s.ch == 1) return with(std::integral_constant<int, 1>{});
    if (s.ch == 2) return with(std::integral_constant<int, 2>{});
    if (s.ch == 4) return with(std::integral_constant<int, 4>{});
    if constexpr (sizeof(typename T::bits) == 4)   // fp32 rows above 8192
      return with(std::integral_constant<int, 8>{});
    return MOE_EUNSUPPORTED;
  });
}

extern "C" size_t moe_add_rmsnorm_backward_workspace_bytes(int M, int hidden) {
  if (M < 0 || hidden < 1 || hidden > MOE_MAX_ROW_HIDDEN) return 0;
  // of the most CTAs that M rows or fewer take
  const int ctas = M < 1 ? 1 : M < moe::kSms ? M : moe::kSms;
  return (size_t)ctas * hidden * sizeof(float);
}

extern "C" int moe_add_rmsnorm_backward(const void *dout, int64_t dout_stride, const void *sum,
                                        int64_t sum_stride, const void *weight, const float *rstd,
                                        const void *dsum, int64_t dsum_stride, int dtype,
                                        int weight_dtype, int M, int hidden, void *dx,
                                        float *dweight, void *workspace, size_t workspace_bytes,
                                        void *stream) {
  using namespace moe;
  const int st = norm_sizes(dtype, weight_dtype, M, hidden);
  if (st) return st;
  if (dout_stride < 0 || sum_stride < 0 || dsum_stride < 0) return MOE_EINVAL;
  if (M > 0 && (!dout || !sum || !weight || !rstd || !dx)) return MOE_EINVAL;
  const int b = dtype_bytes(dtype), wb = dtype_bytes(weight_dtype);
  if (!elem_aligned(dout, b) || !elem_aligned(sum, b) || !elem_aligned(dsum, b) ||
      !elem_aligned(dx, b) || !elem_aligned(weight, wb) || !elem_aligned(rstd, 4) ||
      !elem_aligned(dweight, 4))
    return MOE_EINVAL;
  if (dweight && (!workspace || ((uintptr_t)workspace & 15) ||
                  workspace_bytes < moe_add_rmsnorm_backward_workspace_bytes(M, hidden)))
    return MOE_EINVAL;
  if ((dout_stride != hidden && dout == dx) || (sum_stride != hidden && sum == dx) ||
      (dsum && dsum_stride != hidden && dsum == dx))
    return MOE_EINVAL;
  const int n = 16 / b;
  const Split s = split_row(hidden, n, hidden * b % 8 ? kTwoForward : kTwoGradient);
  int align = rows_alignment(dout, dout_stride, hidden, b);
  for (const int k : {rows_alignment(sum, sum_stride, hidden, b),
                      rows_alignment(dsum, dsum_stride, hidden, b),
                      rows_alignment(dx, hidden, hidden, b),
                      rows_alignment(weight, hidden, hidden, wb)})
    if (k < align) align = k;
  const Walk walk = grad_walk(M, s);
  float *part = dweight ? static_cast<float *>(workspace) : nullptr;
  if (M > 0) {
    const size_t stage = (size_t)3 * s.ch * s.tpr * walk.groups * 16;
    const int64_t turns = ceil_div64(M, (int64_t)walk.ctas * walk.groups);
    // 144 KB: two stages of the widest rows that are split in two a thread (72 KB,
    // 16-bit rows of 4096): at M = 10007 55.7 us, with one stage 64.1, with three
    // 56.6.  Narrower rows have up to four stages, of which 72 KB would do (M =
    // 16384, hidden = 1024: 26.7 us, with 72 KB 25.8); wider ones have one stage
    // of up to 192 KB, and a second where it would fit
    // gains 1 to 4 % (M = 4096, hidden = 7168 51.8 and 51.4; fp32 4096 47.6 and
    // 45.5, but bf16 16384 60.0 and 61.1).
    const int depth = plan_depth(stage, 1, turns, 144 * 1024);
    const size_t ring = can_copy(align, b) ? depth * stage : 0;
    const size_t parts = walk.groups > 1 ? (size_t)walk.groups * hidden * sizeof(float) : 0;
    const size_t smem = ring > parts ? ring : parts;
    const NormGradArgs a{dout, sum,    dsum,  weight, rstd, dout_stride, sum_stride, dsum_stride,
                         M,    hidden, depth, 1.f / hidden, dx, part};
    const dim3 grid(walk.ctas), block(s.tpr, walk.groups);
    const int rc = with_norm_types(dtype, weight_dtype, [&](auto t, auto w) {
      using T = decltype(t);
      using W = decltype(w);
      auto go = [&](auto kernel) {
        const int r = ensure_smem_limit((const void *)kernel, smem + kStaticBytes);
        return r ? r : launch_pdl(kernel, grid, block, smem, stream, a);
      };
      auto with = [&](auto ch) {
        return by_align(align, hidden, b, [&](auto al) {
          return go(rmsnorm_grad_kernel<T, W, decltype(ch)::value, decltype(al)::value>);
        });
      };
      if (s.ch == 1) return with(std::integral_constant<int, 1>{});
      if (s.ch == 2) return with(std::integral_constant<int, 2>{});
      if (s.ch == 4) return with(std::integral_constant<int, 4>{});
      if constexpr (sizeof(typename T::bits) == 4)   // fp32 rows above 8192
        return with(std::integral_constant<int, 8>{});
      return MOE_EUNSUPPORTED;
    });
    if (rc) return rc;
  }
  if (!dweight) return MOE_OK;
  if (const int r = ensure_max_carveout((const void *)sum_parts_kernel)) return r;
  return launch_pdl(sum_parts_kernel, dim3((hidden + 31) / 32), dim3(32, 32), 0, stream,
                    (const float *)part, M > 0 ? walk.ctas : 0, hidden, dweight);
}
