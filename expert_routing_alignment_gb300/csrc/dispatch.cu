// dispatch.cu -- token rows into expert order (moe_dispatch) and back with
// the routing weights applied (moe_combine), and the gradients of both
// ("fp8_moe_grouped.rs": moe_fp8_grouped_sort's sorted order, which its
// grouped launchers read through, and moe_weighted_sum_blend_fp8_grouped).
//
// All four are token-major: one CTA owns a token, reads the token's row once
// and touches its top_k sorted rows.  A position-major gather would read
// every token row top_k times, from HBM once x is larger than the L2.
// Everything is a copy or a short sum, so HBM bandwidth bounds all of it
// (launch latency at decode sizes).
#include "common.cuh"
#include "rows.cuh"

namespace moe {
namespace {

constexpr int kMaxK = 32;        // top_k admitted, as moe_topk_softmax
constexpr int kPadRows = 8;      // positions whose padding one CTA looks after
constexpr unsigned kFull = 0xFFFFFFFFu;

struct SlotArgs {
  const int32_t *ttp;      // [M * k] sorted position of a slot, -1 skipped
  const int32_t *sti;      // [num_rows] slot of a sorted position, n in the padding
  const int32_t *total;    // [1] rows in use
  int M, k, num_rows;
  uint32_t *err;
};

// The token's slot positions into shared memory (-1: skipped, or outside the
// rows, which is reported); threads [0, k) of the CTA.
__device__ __forceinline__ void load_positions(const SlotArgs &a, int t, int *pos) {
  if (threadIdx.x < a.k) {
    int p = __ldcg(a.ttp + (size_t)t * a.k + threadIdx.x);
    if (p < -1 || p >= a.num_rows) {
      if (a.err) atomicOr(a.err, MOE_ERR_BAD_POSITION);
      p = -1;
    }
    pos[threadIdx.x] = p;
  }
}

// Of the kPadRows positions of this CTA, the bits of those that hold padding:
// positions below the total whose slot is none.  Called by whole warps; every
// warp gets the same bits.
__device__ __forceinline__ unsigned padding_mask(const SlotArgs &a) {
  const int lane = threadIdx.x & 31;
  const int64_t p = (int64_t)blockIdx.x * kPadRows + lane;
  bool pad = false;
  if (lane < kPadRows && p < a.num_rows) {
    const int s = __ldcg(a.sti + p);
    pad = p < __ldcg(a.total) && (s < 0 || s >= a.M * a.k);
  }
  return __ballot_sync(kFull, pad);
}

// ---------------------------------------------------------------------------
// dispatch: rows[token_to_perm[t][j]] = x[t]
// ---------------------------------------------------------------------------
//
// A copy of bytes in units U (16-byte where the rows allow it), so one kernel
// serves every type.

template <typename U>
__global__ void __launch_bounds__(256) dispatch_kernel(SlotArgs a, const U *x, int64_t x_stride,
                                                       const float *xs, int units, int scales,
                                                       U *rows, float *rs) {
  __shared__ int pos[kMaxK];
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x, nt = blockDim.x;
  const unsigned pads = padding_mask(a);
  if (t < a.M) {
    load_positions(a, t, pos);
    const U *src = x + t * x_stride;
    __syncthreads();
    for (int c = threadIdx.x; c < units; c += nt) {
      const U v = __ldg(src + c);
      for (int j = 0; j < a.k; ++j)
        if (pos[j] >= 0) rows[(size_t)pos[j] * units + c] = v;
    }
    for (int c = threadIdx.x; c < scales; c += nt) {
      const float v = __ldg(xs + (size_t)t * scales + c);
      for (int j = 0; j < a.k; ++j)
        if (pos[j] >= 0) rs[(size_t)pos[j] * scales + c] = v;
    }
  }
  for (unsigned m = pads; m; m &= m - 1) {
    const size_t p = (size_t)blockIdx.x * kPadRows + (__ffs(m) - 1);
    for (int c = threadIdx.x; c < units; c += nt) rows[p * units + c] = U{};
    for (int c = threadIdx.x; c < scales; c += nt) rs[p * scales + c] = 0.f;
  }
}

// ---------------------------------------------------------------------------
// combine: out[t] = sum_j w[t][j] * rows[token_to_perm[t][j]]
// ---------------------------------------------------------------------------
//
// fp32, j ascending, rounded once.  Without weights it is the gradient of
// the dispatch.  The loads of U slots' chunks are issued before any is used.

template <typename R, typename O, bool WEIGHTED, bool VEC>
__global__ void __launch_bounds__(256) combine_kernel(SlotArgs a, const typename R::bits *rows,
                                                      const float *w, int H,
                                                      typename O::bits *out) {
  constexpr int U = sizeof(typename R::bits) == 2 ? 8 : 4;
  __shared__ int pos[kMaxK];
  __shared__ float wt[kMaxK];
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x;
  load_positions(a, t, pos);
  if (WEIGHTED && threadIdx.x < a.k) wt[threadIdx.x] = __ldcg(w + (size_t)t * a.k + threadIdx.x);
  __syncthreads();
  const int chunks = (H + kChunk - 1) / kChunk;
  for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
    float acc[kChunk] = {};
    for (int j0 = 0; j0 < a.k; j0 += U) {
      Raw<R> v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (j0 + u < a.k && pos[j0 + u] >= 0)
          v[u] = raw_load<R, VEC>(rows + (size_t)pos[j0 + u] * H, c, H);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (j0 + u < a.k && pos[j0 + u] >= 0) {
          float f[kChunk];
          raw_up<R>(v[u], f);
          const float wj = WEIGHTED ? wt[j0 + u] : 1.f;
#pragma unroll
          for (int i = 0; i < kChunk; ++i) acc[i] = WEIGHTED ? fmaf(wj, f[i], acc[i]) : acc[i] + f[i];
        }
      }
    }
    raw_store<O, VEC>(out + (size_t)t * H, c, H, raw_down<O>(acc));
  }
}

// ---------------------------------------------------------------------------
// gradient of combine
// ---------------------------------------------------------------------------
//
//   drows[token_to_perm[t][j]] = w[t][j] * dout[t],
//   dw[t][j] = sum_c dout[t][c] * rows[token_to_perm[t][j]][c]   (fp32).
// Eight slots at a time: a thread keeps their eight partial dot products,
// a warp ends them with a reduce-scatter butterfly (16 -> 8 -> 4 lanes hold
// 4 -> 2 -> 1 sums), the warps' sums are added in warp order.  The order
// depends on hidden alone: a token's bits are the same in every batch.

template <typename R, typename O, bool DW, bool DR, bool VEC>
__global__ void __launch_bounds__(256) combine_grad_kernel(SlotArgs a,
                                                           const typename O::bits *dout,
                                                           int64_t dout_stride,
                                                           const typename R::bits *rows,
                                                           const float *w, int H,
                                                           typename R::bits *drows, float *dw) {
  constexpr int U = 8;
  __shared__ int pos[kMaxK];
  __shared__ float wt[kMaxK];
  __shared__ float red[8][U];
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nwarps = blockDim.x >> 5;
  const unsigned pads = DR ? padding_mask(a) : 0u;
  const int chunks = (H + kChunk - 1) / kChunk;
  if (t < a.M) {
    load_positions(a, t, pos);
    if (DR && tid < a.k) wt[tid] = __ldcg(w + (size_t)t * a.k + tid);
    __syncthreads();
    const typename O::bits *drow = dout + t * dout_stride;
    for (int j0 = 0; j0 < a.k; j0 += U) {
      float acc[U] = {};
      for (int c = tid; c < chunks; c += blockDim.x) {
        const Raw<O> dr = raw_load<O, VEC>(drow, c, H);
        Raw<R> v[U];
        if (DW) {
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (j0 + u < a.k && pos[j0 + u] >= 0)
              v[u] = raw_load<R, VEC>(rows + (size_t)pos[j0 + u] * H, c, H);
        }
        float d[kChunk];
        raw_up<O>(dr, d);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (j0 + u < a.k && pos[j0 + u] >= 0) {
            if (DR) {
              float g[kChunk];
              const float wj = wt[j0 + u];
#pragma unroll
              for (int i = 0; i < kChunk; ++i) g[i] = wj * d[i];
              raw_store<R, VEC>(drows + (size_t)pos[j0 + u] * H, c, H, raw_down<R>(g));
            }
            if (DW) {
              float f[kChunk];
              raw_up<R>(v[u], f);
#pragma unroll
              for (int i = 0; i < kChunk; ++i) acc[u] = fmaf(d[i], f[i], acc[u]);
            }
          }
        }
      }
      if (DW) {
        // lane bits 4, 3, 2 choose the sum a lane ends with
        float s4[4], s2[2], s1;
        const bool h4 = lane & 16, h3 = lane & 8, h2 = lane & 4;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          s4[i] = (h4 ? acc[i + 4] : acc[i]) +
                  __shfl_xor_sync(kFull, h4 ? acc[i] : acc[i + 4], 16);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          s2[i] = (h3 ? s4[i + 2] : s4[i]) + __shfl_xor_sync(kFull, h3 ? s4[i] : s4[i + 2], 8);
        s1 = (h2 ? s2[1] : s2[0]) + __shfl_xor_sync(kFull, h2 ? s2[0] : s2[1], 4);
        s1 += __shfl_xor_sync(kFull, s1, 2);
        s1 += __shfl_xor_sync(kFull, s1, 1);
        if ((lane & 3) == 0) red[warp][lane >> 2] = s1;
        __syncthreads();
        if (tid < U && j0 + tid < a.k) {
          float v = red[0][tid];
          for (int i = 1; i < nwarps; ++i) v += red[i][tid];
          dw[(size_t)t * a.k + j0 + tid] = pos[j0 + tid] >= 0 ? v : 0.f;
        }
        if (j0 + U < a.k) __syncthreads();   // red is written again
      }
    }
  }
  if (DR) {
    for (unsigned m = pads; m; m &= m - 1) {
      const size_t p = (size_t)blockIdx.x * kPadRows + (__ffs(m) - 1);
      for (int c = tid; c < chunks; c += blockDim.x)
        raw_store<R, VEC>(drows + p * H, c, H, raw_zero<R>());
    }
  }
}

// Threads of a CTA: one chunk of eight elements each, up to 256.
dim3 row_threads(int pieces) {
  const int t = (pieces + 31) / 32 * 32;
  return dim3(t > 256 ? 256 : t);
}

// CTAs of a kernel that also clears padding rows: one per token, and as many
// as look after every position.
dim3 token_grid(int M, int num_rows) {
  const int pads = (int)ceil_div64(num_rows, kPadRows);
  return dim3(M > pads ? M : pads);
}

template <typename R, typename O>
int launch_combine(const SlotArgs &a, const void *rows, const float *w, int H, void *out, bool vec,
                   void *stream) {
  const dim3 grid(a.M), block = row_threads((H + kChunk - 1) / kChunk);
  auto r = static_cast<const typename R::bits *>(rows);
  auto o = static_cast<typename O::bits *>(out);
  if (w)
    return vec ? launch_pdl(combine_kernel<R, O, true, true>, grid, block, 0, stream, a, r, w, H, o)
               : launch_pdl(combine_kernel<R, O, true, false>, grid, block, 0, stream, a, r, w, H, o);
  return vec ? launch_pdl(combine_kernel<R, O, false, true>, grid, block, 0, stream, a, r, w, H, o)
             : launch_pdl(combine_kernel<R, O, false, false>, grid, block, 0, stream, a, r, w, H, o);
}

template <typename R, typename O, bool DW, bool DR>
int launch_combine_grad(const SlotArgs &a, const void *dout, int64_t stride, const void *rows,
                        const float *w, int H, void *drows, float *dw, bool vec, void *stream) {
  const dim3 grid = DR ? token_grid(a.M, a.num_rows) : dim3(a.M);
  const dim3 block = row_threads((H + kChunk - 1) / kChunk);
  auto d = static_cast<const typename O::bits *>(dout);
  auto r = static_cast<const typename R::bits *>(rows);
  auto g = static_cast<typename R::bits *>(drows);
  return vec ? launch_pdl(combine_grad_kernel<R, O, DW, DR, true>, grid, block, 0, stream, a, d,
                          stride, r, w, H, g, dw)
             : launch_pdl(combine_grad_kernel<R, O, DW, DR, false>, grid, block, 0, stream, a, d,
                          stride, r, w, H, g, dw);
}

template <typename R, typename O>
int launch_combine_grad(const SlotArgs &a, const void *dout, int64_t stride, const void *rows,
                        const float *w, int H, void *drows, float *dw, bool vec, void *stream) {
  if (drows && dw)
    return launch_combine_grad<R, O, true, true>(a, dout, stride, rows, w, H, drows, dw, vec, stream);
  if (dw)
    return launch_combine_grad<R, O, true, false>(a, dout, stride, rows, w, H, drows, dw, vec, stream);
  return launch_combine_grad<R, O, false, true>(a, dout, stride, rows, w, H, drows, dw, vec, stream);
}

// Host checks shared by the four entry points; MOE_OK with *a filled.
int slot_args(SlotArgs *a, int M, int top_k, int hidden, int num_rows,
              const int32_t *token_to_perm, const int32_t *sorted_token_ids,
              const int32_t *num_tokens_post_padded, uint32_t *err_word) {
  if (M < 0 || top_k < 1 || hidden < 1 || num_rows < 0) return MOE_EINVAL;
  if (top_k > kMaxK || (int64_t)M * top_k > MOE_MAX_SLOTS) return MOE_EUNSUPPORTED;
  if (M > 0 && !token_to_perm) return MOE_EINVAL;
  *a = SlotArgs{token_to_perm, sorted_token_ids, num_tokens_post_padded, M, top_k, num_rows,
                err_word};
  return MOE_OK;
}

// The pairs of row type and token type that combine and its gradient take.
template <typename F>
int with_types(int rows_dtype, int out_dtype, F &&f) {
  if (rows_dtype == MOE_DTYPE_BF16 && out_dtype == MOE_DTYPE_BF16) return f(BF16{}, BF16{});
  if (rows_dtype == MOE_DTYPE_F16 && out_dtype == MOE_DTYPE_F16) return f(F16{}, F16{});
  if (rows_dtype == MOE_DTYPE_F32 && out_dtype == MOE_DTYPE_F32) return f(F32{}, F32{});
  if (rows_dtype == MOE_DTYPE_F32 && out_dtype == MOE_DTYPE_BF16) return f(F32{}, BF16{});
  if (rows_dtype == MOE_DTYPE_F32 && out_dtype == MOE_DTYPE_F16) return f(F32{}, F16{});
  return MOE_EUNSUPPORTED;
}

bool float_dtype(int d) {
  return d == MOE_DTYPE_BF16 || d == MOE_DTYPE_F16 || d == MOE_DTYPE_F32;
}

int combine(const void *rows, int rows_dtype, const float *topk_w, const int32_t *token_to_perm,
            int M, int top_k, int hidden, int num_rows, int out_dtype, void *out,
            uint32_t *err_word, void *stream) {
  if (!float_dtype(rows_dtype) || !float_dtype(out_dtype)) return MOE_EINVAL;
  SlotArgs a;
  const int st = slot_args(&a, M, top_k, hidden, num_rows, token_to_perm, nullptr, nullptr,
                           err_word);
  if (st) return st;
  const int rb = dtype_bytes(rows_dtype), ob = dtype_bytes(out_dtype);
  if ((M > 0 && !out) || (num_rows > 0 && !rows)) return MOE_EINVAL;
  if (!elem_aligned(rows, rb) || !elem_aligned(out, ob)) return MOE_EINVAL;
  const bool vec = hidden % kChunk == 0 && rows_vector(rows, hidden, rb) &&
                   rows_vector(out, hidden, ob);
  return with_types(rows_dtype, out_dtype, [&](auto R, auto O) {
    if (M == 0) return MOE_OK;
    return launch_combine<decltype(R), decltype(O)>(a, rows, topk_w, hidden, out, vec, stream);
  });
}

}  // namespace
}  // namespace moe

extern "C" int moe_dispatch(const void *x, int64_t x_stride, const float *x_scale, int dtype, int M,
                            int top_k, int hidden, const int32_t *token_to_perm,
                            const int32_t *sorted_token_ids,
                            const int32_t *num_tokens_post_padded, int num_rows, void *rows,
                            float *rows_scale, uint32_t *err_word, void *stream) {
  using namespace moe;
  const int eb = dtype_bytes(dtype);
  if (!eb || x_stride < 0) return MOE_EINVAL;
  SlotArgs a;
  const int st = slot_args(&a, M, top_k, hidden, num_rows, token_to_perm, sorted_token_ids,
                           num_tokens_post_padded, err_word);
  if (st) return st;
  if ((dtype == MOE_DTYPE_E4M3) != (x_scale != nullptr) && M > 0) return MOE_EINVAL;
  if (num_rows > 0 && (!rows || !sorted_token_ids || !num_tokens_post_padded)) return MOE_EINVAL;
  if (num_rows > 0 && (dtype == MOE_DTYPE_E4M3) != (rows_scale != nullptr)) return MOE_EINVAL;
  if (M > 0 && !x) return MOE_EINVAL;
  if (!elem_aligned(x, eb) || !elem_aligned(rows, eb) || !elem_aligned(x_scale, 4) ||
      !elem_aligned(rows_scale, 4))
    return MOE_EINVAL;
  const dim3 grid = token_grid(M, num_rows);
  if (grid.x == 0) return MOE_OK;
  const int scales = dtype == MOE_DTYPE_E4M3 ? (hidden + 127) / 128 : 0;
  // the widest unit that every row's start and length are multiples of
  const uint64_t bits = (uint64_t)(uintptr_t)x | (uint64_t)(uintptr_t)rows |
                        (uint64_t)hidden * eb | (uint64_t)x_stride * eb;
  auto go = [&](auto unit) {
    using U = decltype(unit);
    const int64_t per = sizeof(U);
    const int units = (int)((int64_t)hidden * eb / per);
    return launch_pdl(dispatch_kernel<U>, grid, row_threads(units), 0, stream, a,
                      static_cast<const U *>(x), x_stride * eb / per, x_scale, units, scales,
                      static_cast<U *>(rows), rows_scale);
  };
  if (bits % 16 == 0) return go(uint4{});
  if (bits % 8 == 0) return go(uint2{});
  if (bits % 4 == 0) return go(uint32_t{});
  if (bits % 2 == 0) return go(uint16_t{});
  return go(uint8_t{});
}

extern "C" int moe_dispatch_backward(const void *drows, int dtype, int M, int top_k, int hidden,
                                     const int32_t *token_to_perm, int num_rows, void *dx,
                                     uint32_t *err_word, void *stream) {
  return moe::combine(drows, dtype, nullptr, token_to_perm, M, top_k, hidden, num_rows, dtype, dx,
                      err_word, stream);
}

extern "C" int moe_combine(const void *rows, int rows_dtype, const float *topk_w,
                           const int32_t *token_to_perm, int M, int top_k, int hidden,
                           int num_rows, int out_dtype, void *out, uint32_t *err_word,
                           void *stream) {
  if (M > 0 && !topk_w) return MOE_EINVAL;
  return moe::combine(rows, rows_dtype, topk_w, token_to_perm, M, top_k, hidden, num_rows,
                      out_dtype, out, err_word, stream);
}

extern "C" int moe_combine_backward(const void *dout, int64_t dout_stride, int out_dtype,
                                    const void *rows, int rows_dtype, const float *topk_w,
                                    const int32_t *token_to_perm,
                                    const int32_t *sorted_token_ids,
                                    const int32_t *num_tokens_post_padded, int M, int top_k,
                                    int hidden, int num_rows, void *drows, float *dtopk_w,
                                    uint32_t *err_word, void *stream) {
  using namespace moe;
  if (!float_dtype(rows_dtype) || !float_dtype(out_dtype) || dout_stride < 0) return MOE_EINVAL;
  SlotArgs a;
  const int st = slot_args(&a, M, top_k, hidden, num_rows, token_to_perm, sorted_token_ids,
                           num_tokens_post_padded, err_word);
  if (st) return st;
  const int rb = dtype_bytes(rows_dtype), ob = dtype_bytes(out_dtype);
  if (!drows && !dtopk_w && M > 0) return MOE_EINVAL;
  if (M > 0 && !dout) return MOE_EINVAL;
  if (M > 0 && num_rows > 0 && ((drows && !topk_w) || (dtopk_w && !rows))) return MOE_EINVAL;
  if (drows && num_rows > 0 && (!sorted_token_ids || !num_tokens_post_padded)) return MOE_EINVAL;
  if (!elem_aligned(dout, ob) || !elem_aligned(rows, rb) || !elem_aligned(drows, rb))
    return MOE_EINVAL;
  const bool vec = hidden % kChunk == 0 && rows_vector(dout, dout_stride, ob) &&
                   rows_vector(rows, hidden, rb) && rows_vector(drows, hidden, rb);
  return with_types(rows_dtype, out_dtype, [&](auto R, auto O) {
    if (M == 0 && (!drows || num_rows == 0)) return MOE_OK;
    return launch_combine_grad<decltype(R), decltype(O)>(a, dout, dout_stride, rows, topk_w,
                                                         hidden, drows, dtopk_w, vec, stream);
  });
}
