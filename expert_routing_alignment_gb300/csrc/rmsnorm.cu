// rmsnorm.cu -- residual addition with root-mean-square norm in front of the
// router (moe_add_rmsnorm), its 8-bit output, and its gradient
// (moe_add_rmsnorm_backward).
#include <math.h>

#include "common.cuh"
#include "rows.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kMaxWarps = 16;         // warps of a CTA
constexpr float kE4m3Max = 448.f;
constexpr float kScaleMin = 1.17549435e-38f;   // 2^-126, the smallest normal

// max that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Two floats to E4M3, saturating, ties to even; the first in the low byte.
__device__ __forceinline__ uint16_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Sum over the threads of a row group (blockDim.x threads, whole warps):
// butterfly in the warp, then the warps in order.  `red` has kMaxWarps floats
// per call in flight; one barrier.
__device__ __forceinline__ float group_sum(float v, float *red) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return v;
  const int base = threadIdx.y * nw;
  if ((threadIdx.x & 31) == 0) red[base + (threadIdx.x >> 5)] = v;
  __syncthreads();
  v = red[base];
  for (int i = 1; i < nw; ++i) v += red[base + i];
  return v;
}

// How a row of H elements is split: TPR threads (whole warps) of CH chunks
// each, thread i taking the chunks i, i + TPR, ...; a function of H alone, so
// that a row's bits do not depend on the batch.  Narrow rows share a CTA.
struct Split {
  int ch, tpr, rows;
};
Split split_row(int H, int cta_threads) {
  const int chunks = (H + kChunk - 1) / kChunk;
  const int ch = chunks <= 256 ? 1 : chunks <= 512 ? 2 : 4;
  const int tpr = ((chunks + ch - 1) / ch + 31) / 32 * 32;
  return Split{ch, tpr, tpr >= cta_threads ? 1 : cta_threads / tpr};
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
//
//   s = T(x + r);  rstd = 1 / sqrt(mean(s^2) + eps);  out = T(s * rstd * w)
// and, by blocks of 128 columns with a = max |s * w|:
//   scale = a * rstd / 448,  code = e4m3((s * w) * 448 / a).
// The code's quotient leaves rstd out: for 16-bit s and w the product s * w
// and its multiple by 448 = 7 * 64 are exact in fp32 (16 + 3 bits for bf16;
// 22 + 3 for fp16, rounded once), so the only rounding ahead of the code is
// the division's, and the codes do not depend on the order of the sum of
// squares.  Where the scale would be below 2^-126 it is 2^-126, so that no
// scale is zero or subnormal.  A row is read once and kept in registers.

struct NormArgs {
  const void *x, *r, *w;
  int64_t xs, rs;
  int M, H;
  float eps;
  void *sum, *out;
  uint8_t *codes;
  float *scale, *rstd;
};

template <typename T, typename W, int CH, bool VEC>
__global__ void __launch_bounds__(512) add_rmsnorm_kernel(NormArgs a) {
  using TB = typename T::bits;
  using WB = typename W::bits;
  __shared__ float red[kMaxWarps];
  pdl_wait();
  pdl_trigger();
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < a.M;
  const int H = a.H, chunks = (H + kChunk - 1) / kChunk, tid = threadIdx.x, tpr = blockDim.x;
  const TB *x = static_cast<const TB *>(a.x) + row * a.xs;
  const TB *r = static_cast<const TB *>(a.r) + row * a.rs;
  const WB *w = static_cast<const WB *>(a.w);
  Raw<T> xr[CH], rr[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = tid + i * tpr;
    const bool on = live && c < chunks;
    xr[i] = on ? raw_load<T, VEC>(x, c, H) : raw_zero<T>();
    rr[i] = on && a.r ? raw_load<T, VEC>(r, c, H) : raw_zero<T>();
  }
  float s[CH][kChunk];
  float sq = 0.f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = tid + i * tpr;
    raw_up<T>(xr[i], s[i]);
    if (a.r) {
      float f[kChunk];
      raw_up<T>(rr[i], f);
#pragma unroll
      for (int e = 0; e < kChunk; ++e) f[e] += s[i][e];
      xr[i] = raw_down<T>(f);   // the sum as it is stored is what is normalised
      raw_up<T>(xr[i], s[i]);
    }
    if (a.sum && live && c < chunks)
      raw_store<T, VEC>(static_cast<TB *>(a.sum) + row * H, c, H, xr[i]);
#pragma unroll
    for (int e = 0; e < kChunk; ++e) sq = fmaf(s[i][e], s[i][e], sq);
  }
  const float ms = group_sum(sq, red) / (float)H;
  const float rstd = 1.f / sqrtf(ms + a.eps);
  if (a.rstd && live && tid == 0) a.rstd[row] = rstd;
  if (!a.out && !a.codes) return;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = tid + i * tpr;
    const bool on = live && c < chunks;
    float wf[kChunk];
    raw_up<W>(c < chunks ? raw_load<W, VEC>(w, c, H) : raw_zero<W>(), wf);
    if (a.out && on) {
      float v[kChunk];
#pragma unroll
      for (int e = 0; e < kChunk; ++e) v[e] = s[i][e] * rstd * wf[e];
      raw_store<T, VEC>(static_cast<TB *>(a.out) + row * H, c, H, raw_down<T>(v));
    }
    if (a.codes) {
      float m = 0.f;
#pragma unroll
      for (int e = 0; e < kChunk; ++e) {
        s[i][e] *= wf[e];
        m = max_nan(m, fabsf(s[i][e]));
      }
      // the sixteen threads of a block of 128 columns
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) m = max_nan(m, __shfl_xor_sync(kFull, m, d));
      const float sc = m * rstd / kE4m3Max;
      const bool low = sc < kScaleMin;
      uint16_t q[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v0 = s[i][2 * e], v1 = s[i][2 * e + 1];
        v0 = low ? v0 * rstd / kScaleMin : v0 * kE4m3Max / m;
        v1 = low ? v1 * rstd / kScaleMin : v1 * kE4m3Max / m;
        q[e] = to_e4m3x2(v0, v1);
      }
      if (on) {
        uint8_t *dst = a.codes + row * H + (size_t)c * kChunk;
        const uint2 v = make_uint2(q[0] | ((uint32_t)q[1] << 16), q[2] | ((uint32_t)q[3] << 16));
        if (VEC) {
          *reinterpret_cast<uint2 *>(dst) = v;
        } else {
          const int left = H - c * kChunk;
#pragma unroll
          for (int e = 0; e < kChunk; ++e)
            if (e < left) dst[e] = (uint8_t)((e < 4 ? v.x : v.y) >> (8 * (e & 3)));
        }
        if ((tid & 15) == 0) a.scale[row * ((H + 127) / 128) + c / 16] = low ? kScaleMin : sc;
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
// A row group walks over its rows with their part of dw in registers; the
// CTAs' parts go to the workspace [CTAs][H] and a second kernel adds them in
// CTA order, so the bits are the same every time.

struct NormGradArgs {
  const void *dout, *sum, *w, *dsum;
  const float *rstd;
  int64_t ds, ss, dss;
  int M, H;
  void *dx;
  float *part;   // [gridDim.x][H], or NULL: no dw
};

template <typename T, typename W, int CH, bool VEC>
__global__ void __launch_bounds__(512) rmsnorm_grad_kernel(NormGradArgs a) {
  using TB = typename T::bits;
  using WB = typename W::bits;
  __shared__ float red[2][kMaxWarps];
  extern __shared__ float parts[];   // [blockDim.y][H] when rows share a CTA
  pdl_wait();
  pdl_trigger();
  const int H = a.H, chunks = (H + kChunk - 1) / kChunk, tid = threadIdx.x, tpr = blockDim.x;
  const WB *w = static_cast<const WB *>(a.w);
  float dw[CH][kChunk] = {};
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int turn = 0;
  // every group of the CTA makes the same number of turns: they share barriers
  for (int64_t r0 = (int64_t)blockIdx.x * blockDim.y; r0 < a.M; r0 += step, turn ^= 1) {
    const int64_t row = r0 + threadIdx.y;
    const bool live = row < a.M;
    const TB *d = static_cast<const TB *>(a.dout) + row * a.ds;
    const TB *s = static_cast<const TB *>(a.sum) + row * a.ss;
    const TB *ex = static_cast<const TB *>(a.dsum) + row * a.dss;
    Raw<T> dr[CH], sr[CH], er[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = tid + i * tpr;
      const bool on = live && c < chunks;
      dr[i] = on ? raw_load<T, VEC>(d, c, H) : raw_zero<T>();
      sr[i] = on ? raw_load<T, VEC>(s, c, H) : raw_zero<T>();
      er[i] = on && a.dsum ? raw_load<T, VEC>(ex, c, H) : raw_zero<T>();
    }
    const float rstd = live ? a.rstd[row] : 0.f;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = tid + i * tpr;
      float df[kChunk], xh[kChunk], wf[kChunk];
      raw_up<T>(dr[i], df);
      raw_up<T>(sr[i], xh);
      raw_up<W>(c < chunks ? raw_load<W, VEC>(w, c, H) : raw_zero<W>(), wf);
#pragma unroll
      for (int e = 0; e < kChunk; ++e) {
        xh[e] *= rstd;
        dw[i][e] = fmaf(df[e], xh[e], dw[i][e]);
        dot = fmaf(df[e] * wf[e], xh[e], dot);
      }
    }
    const float mean = group_sum(dot, red[turn]) / (float)H;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = tid + i * tpr;
      if (!live || c >= chunks) continue;
      float df[kChunk], xh[kChunk], wf[kChunk], ef[kChunk];
      raw_up<T>(dr[i], df);
      raw_up<T>(sr[i], xh);
      raw_up<T>(er[i], ef);
      raw_up<W>(raw_load<W, VEC>(w, c, H), wf);
#pragma unroll
      for (int e = 0; e < kChunk; ++e)
        ef[e] = fmaf(rstd, df[e] * wf[e] - xh[e] * rstd * mean, ef[e]);
      raw_store<T, VEC>(static_cast<TB *>(a.dx) + row * H, c, H, raw_down<T>(ef));
    }
  }
  if (!a.part) return;
  float *part = a.part + (size_t)blockIdx.x * H;
  if (blockDim.y == 1) {
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int e = 0; e < kChunk; ++e) {
        const int h = (tid + i * tpr) * kChunk + e;
        if (h < H) part[h] = dw[i][e];
      }
    return;
  }
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int e = 0; e < kChunk; ++e) {
      const int h = (tid + i * tpr) * kChunk + e;
      if (h < H) parts[threadIdx.y * H + h] = dw[i][e];
    }
  __syncthreads();
  for (int h = threadIdx.y * tpr + tid; h < H; h += tpr * blockDim.y) {
    float v = parts[h];
    for (int y = 1; y < (int)blockDim.y; ++y) v += parts[y * H + h];
    part[h] = v;
  }
}

// dw[h] = sum over the CTAs' parts: 32 columns a CTA, 16 threads a column
// that take every sixteenth part, then those sixteen in order.
constexpr int kSumRows = 16;
__global__ void __launch_bounds__(32 * kSumRows) sum_parts_kernel(const float *part, int n, int H,
                                                                  float *dw) {
  __shared__ float red[kSumRows][32];
  pdl_wait();
  pdl_trigger();
  const int h = blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  if (h < H)
    for (int i = threadIdx.y; i < n; i += kSumRows) v += __ldcg(part + (size_t)i * H + h);
  red[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0 && h < H) {
    for (int i = 1; i < kSumRows; ++i) v += red[i][threadIdx.x];
    dw[h] = v;
  }
}

constexpr int kGradCtas = 456;   // most CTAs of the gradient: three for each of 152 SMs
constexpr int kGradThreads = 256;

// CTAs of the gradient for M rows.
int grad_ctas(int M, const Split &s) {
  const int64_t want = ceil_div64(M, s.rows);
  return want < kGradCtas ? (int)want : kGradCtas;
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
  if (H > MOE_MAX_NORM_HIDDEN) return MOE_EUNSUPPORTED;
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
  const bool vec = hidden % kChunk == 0 && rows_vector(x, x_stride, b) &&
                   rows_vector(residual, residual_stride, b) && rows_vector(sum_out, hidden, b) &&
                   rows_vector(out, hidden, b) && rows_vector(weight, hidden, wb) &&
                   ((uintptr_t)out_codes & 7) == 0;
  const Split s = split_row(hidden, 128);
  const NormArgs a{x,      residual, weight, x_stride, residual_stride, M,    hidden,
                   eps,    sum_out,  out,    out_codes, out_scale,      rstd};
  const dim3 grid((unsigned)ceil_div64(M, s.rows)), block(s.tpr, s.rows);
  return with_norm_types(dtype, weight_dtype, [&](auto t, auto w) {
    using T = decltype(t);
    using W = decltype(w);
    auto go = [&](auto kernel) { return launch_pdl(kernel, grid, block, 0, stream, a); };
    if (s.ch == 1) return vec ? go(add_rmsnorm_kernel<T, W, 1, true>) : go(add_rmsnorm_kernel<T, W, 1, false>);
    if (s.ch == 2) return vec ? go(add_rmsnorm_kernel<T, W, 2, true>) : go(add_rmsnorm_kernel<T, W, 2, false>);
    return vec ? go(add_rmsnorm_kernel<T, W, 4, true>) : go(add_rmsnorm_kernel<T, W, 4, false>);
  });
}

extern "C" size_t moe_add_rmsnorm_backward_workspace_bytes(int M, int hidden) {
  if (M < 0 || hidden < 1 || hidden > MOE_MAX_NORM_HIDDEN) return 0;
  const moe::Split s = moe::split_row(hidden, moe::kGradThreads);
  const int ctas = moe::grad_ctas(M, s);
  return (size_t)(ctas > 0 ? ctas : 1) * hidden * sizeof(float);
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
  const Split s = split_row(hidden, kGradThreads);
  const int ctas = grad_ctas(M, s);
  float *part = dweight ? static_cast<float *>(workspace) : nullptr;
  if (M > 0) {
    const bool vec = hidden % kChunk == 0 && rows_vector(dout, dout_stride, b) &&
                     rows_vector(sum, sum_stride, b) && rows_vector(dsum, dsum_stride, b) &&
                     rows_vector(dx, hidden, b) && rows_vector(weight, hidden, wb);
    const NormGradArgs a{dout,        sum, weight, dsum, rstd, dout_stride, sum_stride,
                         dsum_stride, M,   hidden, dx,   part};
    const dim3 grid(ctas), block(s.tpr, s.rows);
    const size_t smem = s.rows > 1 ? (size_t)s.rows * hidden * sizeof(float) : 0;
    const int rc = with_norm_types(dtype, weight_dtype, [&](auto t, auto w) {
      using T = decltype(t);
      using W = decltype(w);
      auto go = [&](auto kernel) { return launch_pdl(kernel, grid, block, smem, stream, a); };
      if (s.ch == 1) return vec ? go(rmsnorm_grad_kernel<T, W, 1, true>) : go(rmsnorm_grad_kernel<T, W, 1, false>);
      if (s.ch == 2) return vec ? go(rmsnorm_grad_kernel<T, W, 2, true>) : go(rmsnorm_grad_kernel<T, W, 2, false>);
      return vec ? go(rmsnorm_grad_kernel<T, W, 4, true>) : go(rmsnorm_grad_kernel<T, W, 4, false>);
    });
    if (rc) return rc;
  }
  if (!dweight) return MOE_OK;
  return launch_pdl(sum_parts_kernel, dim3((hidden + 31) / 32), dim3(32, kSumRows), 0, stream,
                    (const float *)part, ctas, hidden, dweight);
}
