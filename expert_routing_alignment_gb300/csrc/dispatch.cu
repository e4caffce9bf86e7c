// dispatch.cu -- token rows into expert order (moe_dispatch) and back with
// the routing weights applied (moe_combine), and the gradients of both
// ("fp8_moe_grouped.rs": moe_fp8_grouped_sort's sorted order, which its
// grouped launchers read through, and moe_weighted_sum_blend_fp8_grouped).
//
// All four are token-major: a CTA has one token or a few, reads each token's
// row once and touches its top_k sorted rows.  A position-major gather
// would read every token row top_k times, from HBM once x is larger than the
// L2.  Everything is a copy or a short sum, so HBM bandwidth bounds all of it
// (launch latency at decode sizes).
#include <type_traits>

#include "common.cuh"
#include "rows.cuh"

namespace moe {
namespace {

constexpr int kMaxK = 32;        // top_k admitted, as moe_topk_softmax
constexpr int kPadRows = 8;      // positions that are looked through for padding together
constexpr unsigned kFull = 0xFFFFFFFFu;

struct SlotArgs {
  const int32_t *ttp;      // [M * k] sorted position of a slot, -1 skipped
  const int32_t *sti;      // [num_rows] slot of a sorted position, n in the padding
  const int32_t *total;    // [1] rows in use
  int M, k, num_rows;
  uint32_t *err;
};

// The sorted position of a slot; -1: skipped, or outside the rows, which is
// reported.
__device__ __forceinline__ int position(const SlotArgs &a, size_t slot) {
  int p = __ldcg(a.ttp + slot);
  if (p < -1 || p >= a.num_rows) {
    if (a.err) atomicOr(a.err, MOE_ERR_BAD_POSITION);
    p = -1;
  }
  return p;
}

// The padding rows (positions below the total whose slot is none) of a CTA's
// share: groups of eight positions, dealt to the CTAs in turn, since an
// expert's padding is one run and would be one CTA's otherwise.  look() reads
// four groups' slots, early in the kernel, so that their latency passes with
// the tokens' own; clear() calls f(p) for each padding row, the whole CTA at
// it.  Whole warps; every warp sees the same.
struct Padding {
  int64_t group;
  int total, slot;   // rows in use; the slot at this lane's position

  __device__ __forceinline__ int64_t at() const {
    const int lane = threadIdx.x & 31;
    return (group + (lane >> 3) * (int64_t)gridDim.x) * kPadRows + (lane & 7);
  }
  __device__ __forceinline__ void look(const SlotArgs &a) {
    group = blockIdx.x;
    total = 0;
    if (a.num_rows > 0) total = __ldcg(a.total);
    if (at() < a.num_rows) slot = __ldcg(a.sti + at());
  }
  template <typename F>
  __device__ __forceinline__ void clear(const SlotArgs &a, F &&f) {
    const int64_t stride = gridDim.x;
    total = min(total, a.num_rows);
    while (group * kPadRows < total) {
      const bool pad = at() < total && (slot < 0 || slot >= a.M * a.k);
      for (unsigned m = __ballot_sync(kFull, pad); m; m &= m - 1) {
        const int b = __ffs(m) - 1;
        f((group + (b >> 3) * stride) * kPadRows + (b & 7));
      }
      group += 4 * stride;
      if (at() < total) slot = __ldcg(a.sti + at());
    }
  }
};

// ---------------------------------------------------------------------------
// dispatch: rows[token_to_perm[t][j]] = x[t]
// ---------------------------------------------------------------------------
//
// A copy, so one kernel serves every type (H elements of ES bytes; whole pieces
// and halves are the same for all, and H then counts bytes).  A CTA takes TOK tokens and, in
// grid.y, a part of the row, one 16-byte piece a thread.  Bound by the writes:
// E4M3 rows at M = 4096, hidden = 4096, top_k = 8 over 256 experts (190 MB, 150
// of it written) 32 us, 5.9 TB/s; a plain fill writes 3.9 TB/s to this HBM, the
// L2 takes the rest.  Eight tokens (M = 8, hidden = 2048, 3.3 MB with the
// padding) take 2.8 us, a launch and two round trips.

template <int ES, int TOK, int A>
__global__ void __launch_bounds__(256) dispatch_kernel(SlotArgs a, const char *x, int64_t x_stride,
                                                       const float *xs, int H, int scales,
                                                       char *rows, float *rs) {
  __shared__ int pos[kMaxK];   // TOK * k <= kMaxK
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, c = blockIdx.y * blockDim.x + tid;
  const bool on = in_row<16 / ES, A>(c, H);
  const int64_t t0 = (int64_t)blockIdx.x * TOK;
  auto put = [&](int64_t p, const uint4 &v) {
    if (on) store16<ES, A>(rows + p * H * ES, c, H, v);
  };
  Padding padding;
  padding.look(a);
  if (t0 < a.M) {
    uint4 v[TOK];
#pragma unroll
    for (int i = 0; i < TOK; ++i) {
      v[i] = make_uint4(0, 0, 0, 0);
      if (on && t0 + i < a.M) v[i] = load16<ES, A>(x + (t0 + i) * x_stride, c, H);
    }
    const int n = (int)min((int64_t)TOK, a.M - t0) * a.k;
    if (tid < n) pos[tid] = position(a, t0 * a.k + tid);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TOK; ++i) {
      if (t0 + i >= a.M) break;
      for (int j = 0; j < a.k; ++j)
        if (const int p = pos[i * a.k + j]; p >= 0) put(p, v[i]);
    }
    if (blockIdx.y == 0)
      for (int i = tid; i < n / a.k * scales; i += blockDim.x) {
        const int t = i / scales, col = i - t * scales;
        const float q = xs[(t0 + t) * scales + col];
        for (int j = 0; j < a.k; ++j)
          if (pos[t * a.k + j] >= 0) rs[(size_t)pos[t * a.k + j] * scales + col] = q;
      }
  }
  padding.clear(a, [&](int64_t p) {
    put(p, make_uint4(0, 0, 0, 0));
    if (blockIdx.y == 0)
      for (int i = tid; i < scales; i += blockDim.x) rs[(size_t)p * scales + i] = 0.f;
  });
}

// ---------------------------------------------------------------------------
// combine: out[t] = sum_j w[t][j] * rows[token_to_perm[t][j]]
// ---------------------------------------------------------------------------
//
// fp32, j ascending, rounded once.  Without weights it is the gradient of
// the dispatch.  A CTA takes the `slots` of some tokens (at most 32) and, in
// grid.y, a part of the row, one 16-byte piece a thread.  Its first warp
// lists the slots that are there; eight loads are issued before any is used,
// so that as much is in flight with few slots a token, or many skipped, as
// with top_k = 8.  Bound by HBM: bf16 without weights at M = 8192,
// hidden = 2048, top_k = 8 (302 MB) 47.8 us, 6.3 TB/s; fp16 at M = 5003,
// hidden = 2880, top_k = 4 with half of the slots skipped (87 MB) 17.8 us,
// 4.9 TB/s, where two waves of CTAs end unevenly.

constexpr int kBatch = 8;

template <typename R, typename O, bool WEIGHTED, int A>
__global__ void __launch_bounds__(256) combine_kernel(SlotArgs a, const typename R::bits *rows,
                                                      const float *w, int H, int tok,
                                                      typename O::bits *out) {
  constexpr int N = kPer16<R>;
  __shared__ int pos[kMaxK];    // of the listed slots; -1: a token without any
  __shared__ float wt[kMaxK];
  __shared__ int ends[kMaxK];   // the token that a listed slot is the last of, or -1
  __shared__ int count;
  pdl_wait();
  pdl_trigger();
  const int64_t t0 = (int64_t)blockIdx.x * tok;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x, t = lane / a.k, j = lane - t * a.k;
    const bool slot = t < tok && t0 + t < a.M;
    int p = -1;
    float wj = 0.f;
    if (slot) {
      p = position(a, (t0 + t) * a.k + j);
      if (WEIGHTED) wj = __ldcg(w + (t0 + t) * a.k + j);
    }
    const unsigned there = __ballot_sync(kFull, p >= 0);
    const unsigned mine = (a.k == 32 ? kFull : ((1u << a.k) - 1) << (t * a.k));   // of the token
    const unsigned listed =
        __ballot_sync(kFull, p >= 0 || (slot && j == 0 && (there & mine) == 0));
    if (listed >> lane & 1) {
      const int at = __popc(listed & lanemask_lt());
      pos[at] = p;
      wt[at] = wj;
      ends[at] = (listed & mine) >> lane == 1 ? t : -1;
    }
    if (lane == 0) count = __popc(listed);
  }
  __syncthreads();
  const int c = blockIdx.y * blockDim.x + threadIdx.x;
  // halves keep their idle lanes: fp16 at M = 3000, top_k = 4, hidden = 2884
  // 19.1 us, and 27.6 when these return here
  const bool on = in_row<N, A>(c, H);
  if (A != kHalves && !on) return;
  const int n = count;
  f32x2 acc[N / 2] = {};
  for (int s0 = 0; s0 < n; s0 += kBatch) {
    Raw<R, N> v[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if ((A != kHalves || on) && s0 + u < n && pos[s0 + u] >= 0)
        v[u] = raw_load<R, N, A>(rows + (size_t)pos[s0 + u] * H, c, H);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (s0 + u >= n) break;
      if ((A != kHalves || on) && pos[s0 + u] >= 0) {
        f32x2 f[N / 2];
        raw_up<R, N>(v[u], f);
        const float wj = WEIGHTED ? wt[s0 + u] : 1.f;
#pragma unroll
        for (int e = 0; e < N / 2; ++e) acc[e] = fma2(pair(wj, wj), f[e], acc[e]);
      }
      if (const int t = ends[s0 + u]; t >= 0) {
        if (A != kHalves || on)
          raw_store<O, N, A>(out + (t0 + t) * H, c, H, raw_down<O>(acc));
#pragma unroll
        for (int e = 0; e < N / 2; ++e) acc[e] = 0;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// gradient of combine
// ---------------------------------------------------------------------------
//
//   drows[token_to_perm[t][j]] = w[t][j] * dout[t],
//   dw[t][j] = sum_c dout[t][c] * rows[token_to_perm[t][j]][c]   (fp32).
// A CTA takes TOK tokens and U = 8 / TOK slots of each at a time; its threads
// walk over the row in 16-byte pieces, all eight slots' loads issued before
// any is used.  A thread keeps the eight partial dot products, a warp ends
// them with a reduce-scatter butterfly (16 -> 8 -> 4 lanes hold 4 -> 2 -> 1
// sums), the warps' sums are added in warp order.  A sum's order depends on
// hidden and the type alone: a token's bits are the same in every batch.
// Bound by HBM: bf16 at M = 16384, hidden = 4096, top_k = 8 (2.42 GB, half of
// it written) 365 us, 6.6 TB/s; three CTAs an SM (80 registers; four tokens a CTA
// spill 16 to 64 bytes there, 16-bit rows of whole pieces none), since 96
// registers and two CTAs took 408 us.  Weights alone (fp32 rows, M = 512,
// hidden = 4096: 71 MB) 14 us, 5.1 TB/s, one wave of four CTAs an SM.  Skipped
// slots leave their loads unissued and their CTA's time with little in flight:
// bf16 at M = 4000, top_k = 6, hidden = 2880 with three of four skipped 38.5 us,
// 2.6 TB/s, weights alone 27.2.

template <typename R, typename O, int TOK, bool DW, bool DR, int A>
__global__ void __launch_bounds__(256, DR ? 3 : TOK > 1 ? 3 : 4) combine_grad_kernel(
    SlotArgs a, const typename O::bits *dout, int64_t dout_stride, const typename R::bits *rows,
    const float *w, int H, typename R::bits *drows, float *dw) {
  constexpr int N = kPer16<R>, U = 8 / TOK;
  __shared__ int pos[kMaxK];   // TOK * k <= kMaxK
  __shared__ float wt[kMaxK];
  __shared__ float red[8][8];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nwarps = blockDim.x >> 5;
  const int64_t t0 = (int64_t)blockIdx.x * TOK;
  Padding padding;
  if (DR) padding.look(a);
  if (t0 < a.M) {
    const int n = (int)min((int64_t)TOK, a.M - t0) * a.k;
    if (tid < TOK * a.k) {
      pos[tid] = tid < n ? position(a, t0 * a.k + tid) : -1;
      if (DR) wt[tid] = tid < n ? __ldcg(w + t0 * a.k + tid) : 0.f;
    }
    __syncthreads();
    for (int j0 = 0; j0 < a.k; j0 += U) {
      float acc[8] = {};   // slot u of token i at i * U + u
      for (int c = tid; in_row<N, A>(c, H); c += blockDim.x) {
        Raw<O, N> dr[TOK];
        Raw<R, N> v[TOK][U];
#pragma unroll
        for (int i = 0; i < TOK; ++i)
          dr[i] = TOK == 1 || t0 + i < a.M
                      ? raw_load<O, N, A>(dout + (t0 + i) * dout_stride, c, H)
                      : raw_zero<O, N>();
        if (DW) {
#pragma unroll
          for (int i = 0; i < TOK; ++i)
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const int s = i * a.k + j0 + u;
              if (j0 + u < a.k && pos[s] >= 0)
                v[i][u] = raw_load<R, N, A>(rows + (size_t)pos[s] * H, c, H);
            }
        }
#pragma unroll
        for (int i = 0; i < TOK; ++i) {
          float d[N];
          raw_up<O, N>(dr[i], d);
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int s = i * a.k + j0 + u;
            if (j0 + u < a.k && pos[s] >= 0) {
              if (DR) {
                float g[N];
                const float wj = wt[s];
#pragma unroll
                for (int e = 0; e < N; ++e) g[e] = wj * d[e];
                raw_store<R, N, A>(drows + (size_t)pos[s] * H, c, H, raw_down<R, N>(g));
              }
              if (DW) {
                float f[N];
                raw_up<R, N>(v[i][u], f);
#pragma unroll
                for (int e = 0; e < N; ++e) acc[i * U + u] = fmaf(d[e], f[e], acc[i * U + u]);
              }
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
        if (tid < 8) {
          const int i = tid / U, j = j0 + tid % U;
          if (t0 + i < a.M && j < a.k) {
            float v = red[0][tid];
            for (int x = 1; x < nwarps; ++x) v += red[x][tid];
            dw[(t0 + i) * a.k + j] = pos[i * a.k + j] >= 0 ? v : 0.f;
          }
        }
        if (j0 + U < a.k) __syncthreads();   // red is written again
      }
    }
  }
  if (DR)
    padding.clear(a, [&](int64_t p) {
      for (int c = tid; in_row<N, A>(c, H); c += blockDim.x)
        raw_store<R, N, A>(drows + p * H, c, H, raw_zero<R, N>());
    });
}

// The row in equal parts of at most 256 pieces, one a thread.
struct Parts {
  int parts, threads;
};
Parts split_parts(int pieces) {
  const int parts = (pieces + 255) / 256;
  return Parts{parts, ((pieces + parts - 1) / parts + 31) / 32 * 32};
}

// CTAs of a kernel that clears padding besides its tokens: with few tokens, up
// to one for every eight positions, eight an SM at most (bf16 dispatch at
// M = 512, hidden = 2048 over 128 experts in blocks of 64: 11.5 us with one an
// SM, 10.7 with four, 8.6 with eight, 8.3 with sixteen, more than are resident).
int64_t pad_ctas(int64_t ctas, int num_rows) {
  const int64_t pads = ceil_div64(num_rows, kPadRows);
  const int64_t most = 8 * (int64_t)sm_count();
  return pads <= ctas || ctas >= most ? ctas : pads < most ? pads : most;
}

template <typename R, typename O, bool WEIGHTED>
int launch_combine(const SlotArgs &a, const void *rows, const float *w, int H, void *out, int align,
                   void *stream) {
  const Parts s = split_parts((H + kPer16<R> - 1) / kPer16<R>);
  // Up to eight tokens and 32 slots a CTA while eight CTAs an SM remain: bf16
  // at M = 4000, top_k = 6, hidden = 2880 with three of four slots skipped
  // 23.4 us with one token a CTA and 13.9 with five; at M = 4096, top_k = 8,
  // hidden = 7168 with none skipped 87.2 with one and 85.2 with four.  With two,
  // four or eight CTAs an SM 13.6 and 84.8, with sixteen 14.2 and 84.8, with 32
  // 23.1 and 85.5.
  const int sms = sm_count();
  if (!sms) return MOE_ECUDA;
  const int64_t room = (int64_t)a.M * s.parts / (8 * sms);
  const int fit = 32 / a.k < 8 ? 32 / a.k : 8;
  const int tok = room < 1 ? 1 : room < fit ? (int)room : fit;
  const dim3 grid((unsigned)ceil_div64(a.M, tok), s.parts), block(s.threads);
  auto r = static_cast<const typename R::bits *>(rows);
  auto o = static_cast<typename O::bits *>(out);
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, block, 0, stream, a, r, w, H, tok, o);
  };
  return by_align<!std::is_same_v<R, O>>(align, H, sizeof(typename R::bits), [&](auto al) {
    return go(combine_kernel<R, O, WEIGHTED, decltype(al)::value>);
  });
}

template <typename R, typename O, int TOK, bool DW, bool DR>
int launch_combine_grad(const SlotArgs &a, const void *dout, int64_t stride, const void *rows,
                        const float *w, int H, void *drows, float *dw, int align, void *stream) {
  const int pieces = (H + kPer16<R> - 1) / kPer16<R>;
  const int threads = pieces >= 256 ? 256 : (pieces + 31) / 32 * 32;
  int64_t ctas = ceil_div64(a.M, TOK);
  if (DR) ctas = pad_ctas(ctas, a.num_rows);
  const dim3 grid((unsigned)ctas), block(threads);
  auto d = static_cast<const typename O::bits *>(dout);
  auto r = static_cast<const typename R::bits *>(rows);
  auto g = static_cast<typename R::bits *>(drows);
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, block, 0, stream, a, d, stride, r, w, H, g, dw);
  };
  return by_align<!std::is_same_v<R, O>>(align, H, sizeof(typename R::bits), [&](auto al) {
    return go(combine_grad_kernel<R, O, TOK, DW, DR, decltype(al)::value>);
  });
}

template <typename R, typename O, bool DW, bool DR>
int launch_combine_grad(const SlotArgs &a, const void *dout, int64_t stride, const void *rows,
                        const float *w, int H, void *drows, float *dw, int align, void *stream) {
  // Eight slots a CTA in flight when there are tokens enough: bf16 at
  // M = 16384, top_k = 1, hidden = 1024 44.6 us with one token a CTA and 22.3
  // with four; at M = 8192, top_k = 4, hidden = 2048 with half of the slots
  // skipped 57.0 with one and 41.4 with two.
  const int tok = a.M < 1024 || a.k > 4 ? 1 : a.k > 2 ? 2 : 4;
  auto go = [&](auto t) {
    return launch_combine_grad<R, O, decltype(t)::value, DW, DR>(a, dout, stride, rows, w, H, drows,
                                                                 dw, align, stream);
  };
  if (tok == 4) return go(std::integral_constant<int, 4>{});
  if (tok == 2) return go(std::integral_constant<int, 2>{});
  return go(std::integral_constant<int, 1>{});
}

template <typename R, typename O>
int launch_combine_grad(const SlotArgs &a, const void *dout, int64_t stride, const void *rows,
                        const float *w, int H, void *drows, float *dw, int align, void *stream) {
  auto go = [&](auto d, auto r) {
    return launch_combine_grad<R, O, decltype(d)::value, decltype(r)::value>(
        a, dout, stride, rows, w, H, drows, dw, align, stream);
  };
  if (drows && dw) return go(std::true_type{}, std::true_type{});
  if (dw) return go(std::true_type{}, std::false_type{});
  return go(std::false_type{}, std::true_type{});
}

// Host checks shared by the four entry points; MOE_OK with *a filled.
int slot_args(SlotArgs *a, int M, int top_k, int hidden, int num_rows,
              const int32_t *token_to_perm, const int32_t *sorted_token_ids,
              const int32_t *num_tokens_post_padded, uint32_t *err_word) {
  if (M < 0 || top_k < 1 || hidden < 1 || num_rows < 0) return MOE_EINVAL;
  if (hidden > MOE_MAX_ROW_HIDDEN || top_k > kMaxK || (int64_t)M * top_k > MOE_MAX_SLOTS)
    return MOE_EUNSUPPORTED;
  if (M > 0 && !token_to_perm) return MOE_EINVAL;
  if (!elem_aligned(token_to_perm, 4) || !elem_aligned(sorted_token_ids, 4) ||
      !elem_aligned(num_tokens_post_padded, 4) || !elem_aligned(err_word, 4))
    return MOE_EINVAL;
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

// The alignment of a call from its expert rows' and its token rows' own: of a
// mixed pair, 16 bytes of fp32 meet 8 of the 16-bit type, whole or by elements.
int pair_alignment(int rows, int tokens, int rb, int ob) {
  if (rb == ob) return rows < tokens ? rows : tokens;
  return rows == 16 && tokens >= 8 ? kWhole : kElems;
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
  if (!elem_aligned(rows, rb) || !elem_aligned(out, ob) || !elem_aligned(topk_w, 4))
    return MOE_EINVAL;
  const int align = pair_alignment(rows_alignment(rows, hidden, hidden, rb),
                                   rows_alignment(out, hidden, hidden, ob), rb, ob);
  return with_types(rows_dtype, out_dtype, [&](auto R, auto O) {
    if (M == 0) return MOE_OK;
    using RT = decltype(R);
    using OT = decltype(O);
    // without weights (the gradient of the dispatch) both types are one
    if constexpr (std::is_same_v<RT, OT>)
      if (!topk_w)
        return launch_combine<RT, OT, false>(a, rows, topk_w, hidden, out, align, stream);
    return launch_combine<RT, OT, true>(a, rows, topk_w, hidden, out, align, stream);
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
  if (M == 0 && num_rows == 0) return MOE_OK;
  const int scales = dtype == MOE_DTYPE_E4M3 ? (hidden + 127) / 128 : 0;
  const int len = hidden * eb;
  int align = rows_alignment(x, x_stride, hidden, eb);
  if (const int k = rows_alignment(rows, hidden, hidden, eb); k < align) align = k;
  const Parts s = split_parts((len + 15) / 16);
  // Two tokens a CTA when there are many of few slots: bf16 at M = 16384,
  // top_k = 1, hidden = 1024 19.2 us with one and 13.2 with two (13.0 with
  // eight); at M = 4000, top_k = 6, hidden = 2880 16.0 and 12.1; at top_k = 8
  // (M = 4096, hidden = 7168) 103.7 and 104.3.
  const int tok = M < 1024 || top_k > 6 ? 1 : 2;
  const dim3 grid((unsigned)pad_ctas(ceil_div64(M, tok), num_rows), s.parts), block(s.threads);
  auto go = [&](auto es, auto al) {
    constexpr int ES = decltype(es)::value, A = decltype(al)::value;
    auto launch = [&](auto kernel) {
      return launch_pdl(kernel, grid, block, 0, stream, a, static_cast<const char *>(x),
                        x_stride * eb, x_scale, len / ES, scales, static_cast<char *>(rows),
                        rows_scale);
    };
    return tok == 2 ? launch(dispatch_kernel<ES, 2, A>) : launch(dispatch_kernel<ES, 1, A>);
  };
  return by_align(align, hidden, eb, [&](auto al) {
    if constexpr (decltype(al)::value == kElems || decltype(al)::value == kDealt) {
      if (eb == 4) return go(std::integral_constant<int, 4>{}, al);
      if (eb == 2) return go(std::integral_constant<int, 2>{}, al);
    }
    return go(std::integral_constant<int, 1>{}, al);
  });
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
  // the weights of every slot are read, those of skipped ones too
  if (M > 0 && ((drows && !topk_w) || (num_rows > 0 && dtopk_w && !rows))) return MOE_EINVAL;
  if (drows && num_rows > 0 && (!sorted_token_ids || !num_tokens_post_padded)) return MOE_EINVAL;
  if (!elem_aligned(dout, ob) || !elem_aligned(rows, rb) || !elem_aligned(drows, rb) ||
      !elem_aligned(topk_w, 4) || !elem_aligned(dtopk_w, 4))
    return MOE_EINVAL;
  const int ar = rows_alignment(rows, hidden, hidden, rb);
  const int ag = rows_alignment(drows, hidden, hidden, rb);
  const int align = pair_alignment(ar < ag ? ar : ag,
                                   rows_alignment(dout, dout_stride, hidden, ob), rb, ob);
  return with_types(rows_dtype, out_dtype, [&](auto R, auto O) {
    if (M == 0 && (!drows || num_rows == 0)) return MOE_OK;
    return launch_combine_grad<decltype(R), decltype(O)>(a, dout, dout_stride, rows, topk_w,
                                                         hidden, drows, dtopk_w, align, stream);
  });
}
