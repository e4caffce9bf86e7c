// nvfp4_pack.cu -- token rows and expert weights into NVFP4 and back
// (moe_quantize_nvfp4, moe_dequantize_nvfp4).
//
// A group of elements (a row, or an expert's matrix) has a global scale g, each
// 16 of a row's elements a block scale s and a step t = s * g:
//   g = max(max|x| / 2688, 2^-80),  s = e4m3(max|block| / (6 g)),
//   code = e2m1(x / t),  value = code * t.
// A thread holds a whole block: its maximum, quotients and codes need no
// exchange.  Bound by the bytes in and out.
#include "nvfp4.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kThreads = 256;
constexpr int kMostParts = 128;   // parts of a group's maximum

struct PackArgs {
  const void *x;
  int64_t stride;         // of x's rows, in elements
  int64_t rows;           // of all groups
  int blocks;             // of a row
  int H;
  const float *given;     // [groups] or NULL
  const int32_t *sti;     // the rows' slots, or NULL
  int n;
  uint8_t *codes, *scale;
  float *global;
  void *values;
};

// Encodes block b of row `row` (m: its maximum) under g and writes what is wanted.
template <typename T, int A>
__device__ __forceinline__ void put_block(const PackArgs &a, int64_t row, int b,
                                          const RawBlock<T> &r, float m, float g) {
  const uint32_t sb = block_scale(m, g);
  const float s = e4m3_to_float(sb), t = s * g;
  f32x2 f[8];
  block_up<T>(r, f);
  const uint2 c = block_codes(f, s, t, m);
  const int64_t at = row * a.blocks + b;
  if (a.codes) reinterpret_cast<uint2 *>(a.codes)[at] = c;
  if (a.scale) a.scale[at] = (uint8_t)sb;
  if (a.values) {
    block_values(c, t, f);
    block_store<T, A>(static_cast<typename T::bits *>(a.values) + row * a.H, b, a.H, f);
  }
}

// Rows with a global scale each: `tpr` threads a row (a power of two, up to a
// warp, or whole warps), NB blocks a thread, in registers between the row's
// maximum and the codes.
template <typename T, int NB, int A>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(PackArgs a, int tpr) {
  using TB = typename T::bits;
  __shared__ float red[kThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int in_row = threadIdx.x % tpr;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr;
  const bool live = row < a.rows && !(a.sti && (unsigned)a.sti[row] >= (unsigned)a.n);
  const TB *x = static_cast<const TB *>(a.x) + row * a.stride;
  RawBlock<T> r[NB];
  float m[NB], top = 0.f;
#pragma unroll
  for (int i = 0; i < NB; ++i)
    if (const int b = in_row + i * tpr; live && b < a.blocks) r[i] = block_load<T, A>(x, b, a.H);
#pragma unroll
  for (int i = 0; i < NB; ++i)
    if (const int b = in_row + i * tpr; live && b < a.blocks) {
      f32x2 f[8];
      block_up<T>(r[i], f);
      m[i] = block_max(f);
      top = fmaxf(top, finite_max(m[i]));
    }
  float g;
  if (a.given) {
    g = live ? a.given[row] : 0.f;
  } else {
    for (int d = min(tpr, 32) >> 1; d > 0; d >>= 1)
      top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
    if (tpr > 32) {
      if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = top;
      __syncthreads();
      const int first = threadIdx.x / tpr * (tpr / 32);
      for (int w = 0; w < tpr / 32; ++w) top = fmaxf(top, red[first + w]);
    }
    g = global_of(top);
  }
  if (!live) return;
  if (in_row == 0 && a.global) a.global[row] = g;
#pragma unroll
  for (int i = 0; i < NB; ++i)
    if (const int b = in_row + i * tpr; b < a.blocks) put_block<T, A>(a, row, b, r[i], m[i], g);
}

// A matrix a group.  The blocks of a group are dealt out over gridDim.x CTAs;
// dense rows are one row of all its blocks.
struct Blocks {
  int64_t first;   // the group's first row
  uint32_t total;  // its blocks
  __device__ __forceinline__ int64_t row(uint32_t i, const PackArgs &a, int &b) const {
    const uint32_t q = i / (uint32_t)a.blocks;
    b = (int)(i - q * (uint32_t)a.blocks);
    return first + q;
  }
};

__device__ __forceinline__ float cta_max(float top) {
  __shared__ float red[kThreads / 32];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = top;
  __syncthreads();
  for (int w = 0; w < kThreads / 32; ++w) top = fmaxf(top, red[w]);
  return top;
}

// part[group][gridDim.x]: the maximum over a CTA's blocks.
template <typename T, int A>
__global__ void __launch_bounds__(kThreads) group_max_kernel(PackArgs a, int rows, float *part) {
  using TB = typename T::bits;
  pdl_wait();
  pdl_trigger();
  const Blocks g{(int64_t)blockIdx.y * rows, (uint32_t)rows * a.blocks};
  float top = 0.f;
  for (uint32_t i = blockIdx.x * kThreads + threadIdx.x; i < g.total; i += gridDim.x * kThreads) {
    int b;
    const int64_t row = g.row(i, a, b);
    f32x2 f[8];
    block_up<T>(block_load<T, A>(static_cast<const TB *>(a.x) + row * a.stride, b, a.H), f);
    top = fmaxf(top, finite_max(block_max(f)));
  }
  top = cta_max(top);
  if (threadIdx.x == 0) part[blockIdx.y * gridDim.x + blockIdx.x] = top;
}

template <typename T, int A>
__global__ void __launch_bounds__(kThreads)
    quantize_groups_kernel(PackArgs a, int rows, const float *part, int parts) {
  using TB = typename T::bits;
  pdl_wait();
  pdl_trigger();
  const Blocks gr{(int64_t)blockIdx.y * rows, (uint32_t)rows * a.blocks};
  float g;
  if (a.given) {
    g = a.given[blockIdx.y];
  } else {
    float top = 0.f;
    if ((int)threadIdx.x < parts) top = part[blockIdx.y * parts + threadIdx.x];
    g = global_of(cta_max(top));
  }
  if (a.global && blockIdx.x == 0 && threadIdx.x == 0) a.global[blockIdx.y] = g;
  for (uint32_t i = blockIdx.x * kThreads + threadIdx.x; i < gr.total;
       i += gridDim.x * kThreads) {
    int b;
    const int64_t row = gr.row(i, a, b);
    const RawBlock<T> r =
        block_load<T, A>(static_cast<const TB *>(a.x) + row * a.stride, b, a.H);
    f32x2 f[8];
    block_up<T>(r, f);
    put_block<T, A>(a, row, b, r, block_max(f), g);
  }
}

template <typename T, int A>
__global__ void __launch_bounds__(kThreads)
    dequantize_kernel(const uint8_t *codes, const uint8_t *scale, const float *global,
                      int64_t total, int64_t per_group, void *out) {
  using TB = typename T::bits;
  pdl_wait();
  pdl_trigger();
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * kThreads) {
    const float t = e4m3_to_float(scale[i]) * global[i / per_group];
    f32x2 f[8];
    block_values(reinterpret_cast<const uint2 *>(codes)[i], t, f);
    block_store<T, A>(static_cast<TB *>(out) + i * kBlock16, 0, kBlock16, f);
  }
}

template <typename F>
int with_float(int dtype, F &&f) {
  switch (dtype) {
    case MOE_DTYPE_BF16: return f(BF16{});
    case MOE_DTYPE_F16: return f(F16{});
    case MOE_DTYPE_F32: return f(F32{});
    default: return MOE_EINVAL;
  }
}
// f(integral_constant kWhole or kElems).
template <typename F>
int whole_or_elems(int align, F &&f) {
  if (align == 16) return f(std::integral_constant<int, kWhole>{});
  return f(std::integral_constant<int, kElems>{});
}

// What every call of a packed shape has to meet.
int pack_sizes(int groups, int rows, int cols) {
  if (groups < 0 || rows < 1 || cols < 1) return MOE_EINVAL;
  if (cols % kBlock16 || cols > MOE_MAX_ROW_HIDDEN ||
      (int64_t)groups * rows > 0x7FFFFFFF || (int64_t)rows * (cols / kBlock16) > 0x7FFFFFFF)
    return MOE_EUNSUPPORTED;
  return MOE_OK;
}

// CTAs of a group, so that all of them are a few for each SM.
int group_parts(int groups, int rows, int cols) {
  const int64_t most = ceil_div64((int64_t)rows * (cols / kBlock16), kThreads);
  int64_t parts = ceil_div64((int64_t)sm_count() * 8, groups);
  if (parts > most) parts = most;
  return (int)(parts < 1 ? 1 : parts > kMostParts ? kMostParts : parts);
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_quantize_nvfp4_workspace_bytes(int groups, int rows, int cols) {
  using namespace moe;
  if (pack_sizes(groups, rows, cols)) return 0;
  return rows == 1 ? 16 : ((size_t)groups * kMostParts * 4 + 15) / 16 * 16 + 16;
}

extern "C" int moe_quantize_nvfp4(const void *x, int64_t x_stride, int dtype, int groups, int rows,
                                  int cols, const float *given_scale,
                                  const int32_t *sorted_token_ids, int num_slots, uint8_t *codes,
                                  uint8_t *scale, float *global_scale, void *values,
                                  void *workspace, size_t workspace_bytes, void *stream) {
  using namespace moe;
  const int eb = dtype_bytes(dtype);
  if (eb < 2 || x_stride < 0 || num_slots < 0) return MOE_EINVAL;
  if (const int st = pack_sizes(groups, rows, cols)) return st;
  if (sorted_token_ids && rows != 1) return MOE_EUNSUPPORTED;
  if (groups == 0) return MOE_OK;
  if (!x || (!codes && !scale && !global_scale && !values)) return MOE_EINVAL;
  if (!elem_aligned(x, eb) || !elem_aligned(values, eb) || !elem_aligned(given_scale, 4) ||
      !elem_aligned(global_scale, 4) || !elem_aligned(sorted_token_ids, 4) ||
      ((uintptr_t)codes & 7))
    return MOE_EINVAL;
  if (values == x && rows * (int64_t)groups > 1 && x_stride != cols) return MOE_EINVAL;
  const bool parts_needed = rows > 1 && !given_scale;
  if (parts_needed && (!workspace || ((uintptr_t)workspace & 15) ||
                       workspace_bytes < moe_quantize_nvfp4_workspace_bytes(groups, rows, cols)))
    return MOE_EINVAL;
  const PackArgs a{x,     x_stride, (int64_t)groups * rows, cols / kBlock16, cols,  given_scale,
                   sorted_token_ids, num_slots, codes, scale, global_scale, values};
  int align = rows_alignment(x, x_stride, cols, eb);
  if (const int k = rows_alignment(values, cols, cols, eb); k < align) align = k;
  return with_float(dtype, [&](auto t) {
    using T = decltype(t);
    return whole_or_elems(align, [&](auto al) {
      constexpr int A = decltype(al)::value;
      if (rows == 1) {
        int tpr = 1;
        while (tpr < a.blocks && tpr < kThreads) tpr *= 2;
        const int threads = tpr > 128 ? kThreads : 128;
        const dim3 grid((unsigned)ceil_div64(groups, threads / tpr));
        if (a.blocks <= tpr)
          return launch_pdl(quantize_rows_kernel<T, 1, A>, grid, dim3(threads), 0, stream, a, tpr);
        if (a.blocks <= 2 * tpr)
          return launch_pdl(quantize_rows_kernel<T, 2, A>, grid, dim3(threads), 0, stream, a, tpr);
        return launch_pdl(quantize_rows_kernel<T, 4, A>, grid, dim3(threads), 0, stream, a, tpr);
      }
      if (!sm_count()) return MOE_ECUDA;
      const int parts = group_parts(groups, rows, cols);
      // one launch for every 65535 groups, the most a grid has in y
      for (int g0 = 0; g0 < groups; g0 += 65535) {
        const int gn = groups - g0 < 65535 ? groups - g0 : 65535;
        PackArgs b = a;
        const int64_t r0 = (int64_t)g0 * rows;
        b.x = static_cast<const char *>(x) + r0 * x_stride * eb;
        if (codes) b.codes = codes + r0 * (cols / 2);
        if (scale) b.scale = scale + r0 * (cols / 16);
        if (values) b.values = static_cast<char *>(values) + r0 * cols * eb;
        if (global_scale) b.global = global_scale + g0;
        if (given_scale) b.given = given_scale + g0;
        float *part = static_cast<float *>(workspace) + (int64_t)g0 * kMostParts;
        if (!given_scale)
          if (const int st = launch_pdl(group_max_kernel<T, A>, dim3(parts, gn), dim3(kThreads), 0,
                                        stream, b, rows, part))
            return st;
        if (const int st = launch_pdl(quantize_groups_kernel<T, A>, dim3(parts, gn),
                                      dim3(kThreads), 0, stream, b, rows, (const float *)part,
                                      parts))
          return st;
      }
      return MOE_OK;
    });
  });
}

extern "C" int moe_dequantize_nvfp4(const uint8_t *codes, const uint8_t *scale,
                                    const float *global_scale, int groups, int rows, int cols,
                                    int dtype, void *out, void *stream) {
  using namespace moe;
  const int eb = dtype_bytes(dtype);
  if (eb < 2) return MOE_EINVAL;
  if (const int st = pack_sizes(groups, rows, cols)) return st;
  if (groups == 0) return MOE_OK;
  if (!codes || !scale || !global_scale || !out) return MOE_EINVAL;
  if (((uintptr_t)codes & 7) || !elem_aligned(global_scale, 4) || !elem_aligned(out, eb))
    return MOE_EINVAL;
  if (!sm_count()) return MOE_ECUDA;
  const int64_t per = (int64_t)rows * (cols / kBlock16), total = per * groups;
  int64_t ctas = ceil_div64(total, kThreads);
  if (ctas > (int64_t)sm_count() * 32) ctas = (int64_t)sm_count() * 32;
  return with_float(dtype, [&](auto t) {
    return whole_or_elems(rows_alignment(out, cols, cols, eb), [&](auto al) {
      return launch_pdl(dequantize_kernel<decltype(t), decltype(al)::value>, dim3((unsigned)ctas),
                        dim3(kThreads), 0, stream, codes, scale, global_scale, total, per, out);
    });
  });
}
