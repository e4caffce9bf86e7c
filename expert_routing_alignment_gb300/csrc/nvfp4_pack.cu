// nvfp4_pack.cu -- token rows and expert weights into NVFP4 and back
// (moe_quantize_nvfp4, moe_dequantize_nvfp4).
//
// A group of elements (a row, or an expert's matrix) has a global scale g, each
// 16 of a row's elements a block scale s and a step t = s * g:
//   g = max(max|x| / 2688, 2^-80),  s = e4m3(max|block| / (6 g)),
//   code = e2m1(x / t),  value = code * t.
// Quantisation: a thread has a whole block, 32 bytes of a 16-bit type, which it
// loads and stores as a sector; its scale and step are computed once.  (By pieces
// of 16 bytes a lane, whose scale two lanes compute, 8192 x 4096 bf16 rows with
// values took 32.4 us.)  The inverse has pieces of 16 bytes a lane, so that a
// warp's loads and stores are runs of neighbours.
// Rows: x is read once; 8192 x 4096 bf16 with values (153 MB) 24.0 us, 6.4 TB/s,
// bound by HBM and, nearly, by issue; without values (86 MB) 15.8, 5.5 TB/s, as the
// codes' arithmetic is the same.  Matrices: read twice, for the maximum and for the
// codes; 32 x 1536 x 2048 bf16 with values (459 MB, 660 with the second read, which
// finds nothing of x in L2) 104 us, without 75.  (Read once, held in the shared memory
// of CTAs that meet at the maximum: 143 us with values, each meeting 4.5; in turns
// that find x in L2: 111 to 135.)  The inverse: 64 x 768 x 2048 to bf16 (258 MB)
// 39.7 us, 6.5 TB/s.
#include "nvfp4.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kThreads = 256;

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

// Encodes block b of row `row` (m: its maximum) and writes what is wanted.
template <typename T, int A>
__device__ __forceinline__ void put_block(const PackArgs &a, int64_t row, int b,
                                          const RawBlock<T> &r, float m, const GlobalScale &g) {
  const uint32_t sb = block_scale(m, g);
  const float s = e4m3_to_float(sb), t = s * g.g;
  const uint2 c = block_codes<T>(r, s, t, m);
  const int64_t at = row * a.blocks + b;
  if (a.codes) reinterpret_cast<uint2 *>(a.codes)[at] = c;
  if (a.scale) a.scale[at] = (uint8_t)sb;
  if (a.values) {
    f32x2 f[8];
    code_values<8>(c.x, t, f);
    code_values<8>(c.y, t, f + 4);
    block_store<T, A>(static_cast<typename T::bits *>(a.values) + row * a.H, b, raw_down<T>(f));
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
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int b = in_row + i * tpr;
    r[i] = live && b < a.blocks ? block_load<T, A>(x, b) : raw_zero<T, kBlock16>();
  }
  float m[NB], top = 0.f;
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    m[i] = block_max<T>(r[i]);
    top = fmaxf(top, finite_max(m[i]));
  }
  float g;
  if (a.given) {
    g = live ? a.given[row] : 1.f;
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
  const GlobalScale gs(g);
#pragma unroll
  for (int i = 0; i < NB; ++i)
    if (const int b = in_row + i * tpr; b < a.blocks) put_block<T, A>(a, row, b, r[i], m[i], gs);
}

// A matrix a group.  The blocks of a group are dealt out over gridDim.x CTAs.
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
    top = fmaxf(top, finite_max(block_max<T>(
                         block_load<T, A>(static_cast<const TB *>(a.x) + row * a.stride, b))));
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
    for (int i = threadIdx.x; i < parts; i += kThreads) top = fmaxf(top, part[blockIdx.y * parts + i]);
    g = global_of(cta_max(top));
  }
  if (a.global && blockIdx.x == 0 && threadIdx.x == 0) a.global[blockIdx.y] = g;
  const GlobalScale gs(g);
  for (uint32_t i = blockIdx.x * kThreads + threadIdx.x; i < gr.total;
       i += gridDim.x * kThreads) {
    int b;
    const int64_t row = gr.row(i, a, b);
    const RawBlock<T> r = block_load<T, A>(static_cast<const TB *>(a.x) + row * a.stride, b);
    put_block<T, A>(a, row, b, r, block_max<T>(r), gs);
  }
}

// U rows of pieces at a time for each thread column, so that their loads are in
// flight together.
constexpr int kRowsAhead = 4;
template <typename T, int A>
__global__ void __launch_bounds__(kThreads)
    dequantize_kernel(const uint8_t *codes, const uint8_t *scale, const float *global,
                      int64_t rows, int group_rows, int pieces, void *out) {
  using TB = typename T::bits;
  constexpr int N = kPer16<T>, L = kPieces16<T>;
  using P = typename PackedCodes<N>::type;
  pdl_wait();
  pdl_trigger();
  const int H = pieces * N;
  for (int64_t r0 = ((int64_t)blockIdx.x * blockDim.y + threadIdx.y) * kRowsAhead; r0 < rows;
       r0 += (int64_t)gridDim.x * blockDim.y * kRowsAhead) {
    float g[kRowsAhead];
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u)
      g[u] = r0 + u < rows ? global[(uint32_t)(r0 + u) / (uint32_t)group_rows] : 0.f;
    for (int c = threadIdx.x; c < pieces; c += blockDim.x) {
      uint32_t v[kRowsAhead], s[kRowsAhead];
#pragma unroll
      for (int u = 0; u < kRowsAhead; ++u) {
        const int64_t at = (r0 + u) * pieces + c;
        v[u] = r0 + u < rows ? reinterpret_cast<const P *>(codes)[at] : 0;
        s[u] = r0 + u < rows ? scale[at / L] : 0;
      }
#pragma unroll
      for (int u = 0; u < kRowsAhead; ++u) {
        if (r0 + u >= rows) break;
        f32x2 f[N / 2];
        code_values<N>(v[u], e4m3_to_float(s[u]) * g[u], f);
        raw_store<T, N, A>(static_cast<TB *>(out) + (r0 + u) * H, c, H, raw_down<T>(f));
      }
    }
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
// f(integral_constant of how blocks are moved) for rows aligned to `align` bytes.
template <typename F>
int by_block_align(int align, F &&f) {
  if (align == 32) return f(std::integral_constant<int, kSectors>{});
  if (align == 16) return f(std::integral_constant<int, kWhole>{});
  return f(std::integral_constant<int, kElems>{});
}
// The alignment, up to 32 bytes, of rows at p that are `stride` bytes apart (NULL: not used).
int block_alignment(const void *p, int64_t stride) {
  if (!p) return 32;
  const uint64_t v = (uint64_t)(uintptr_t)p | (uint64_t)stride | 32;
  return (int)(v & (~v + 1));
}

// What every call of a packed shape has to meet.
int pack_sizes(int groups, int rows, int cols) {
  if (groups < 0 || rows < 1 || cols < 1) return MOE_EINVAL;
  if (cols % kBlock16 || cols > MOE_MAX_ROW_HIDDEN ||
      (int64_t)groups * rows > 0x7FFFFFFF || (int64_t)rows * (cols / 4) > 0x7FFFFFFF)
    return MOE_EUNSUPPORTED;
  return MOE_OK;
}

// Parts of a group's maximum at most, a bound on the CTAs of a group.
int most_parts(int groups) {
  const int parts = groups > 0 ? 4096 / groups : 1;
  return parts < 1 ? 1 : parts > 1024 ? 1024 : parts;
}
// CTAs of a group: 24 for each SM in all, several times what is resident (8 of the
// maximum's, 6 of the codes'), so that the last ones are short.  bf16 with values, us by
// 6, 8, 12, 24 and 48 an SM: 32 x 1536 x 2048 110, 111, 108, 104, 104; 256 x 512 x 768
// 114, 118, 108, 105, 105; 128 x 2048 x 1536 439, 469, 422, 408, 397.  One matrix has
// most_parts at most: 16384 x 16384 293 by 912, and 326 by 1024, which is no whole
// number of waves.
int group_parts(int groups, int rows, int cols) {
  const int64_t most = ceil_div64((int64_t)rows * (cols / kBlock16), kThreads);
  int64_t parts = (int64_t)sm_count() * 24 / groups;
  if (parts > most) parts = most;
  if (parts > most_parts(groups)) parts = most_parts(groups);
  return (int)(parts < 1 ? 1 : parts);
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_quantize_nvfp4_workspace_bytes(int groups, int rows, int cols) {
  using namespace moe;
  if (pack_sizes(groups, rows, cols)) return 0;
  return rows == 1 ? 16 : ((size_t)groups * most_parts(groups) * 4 + 15) / 16 * 16 + 16;
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
  const PackArgs a{x,         x_stride, (int64_t)groups * rows, cols / kBlock16, cols,  given_scale,
                   sorted_token_ids, num_slots, codes, scale, global_scale, values};
  int align = block_alignment(x, (int64_t)groups * rows > 1 ? x_stride * eb : 0);
  if (const int k = block_alignment(values, (int64_t)cols * eb); k < align) align = k;
  return with_float(dtype, [&](auto t) {
    using T = decltype(t);
    return by_block_align(align, [&](auto al) {
      constexpr int A = decltype(al)::value;
      if (rows == 1) {
        // Two blocks a thread where there are more than the device has threads: the
        // row's scale and its reciprocal are each thread's own work.  bf16 with values,
        // us with one and with two: 512 x 2048 2.3 and 2.4, 1024 x 4096 4.8 and 4.5,
        // 2048 x 4096 7.3 and 5.9, 16384 x 2048 26.8 and 23.9; 8192 x 4096 27.8 and 24.0
        // (23.7 with four).
        const int want = (int64_t)groups * a.blocks > (int64_t)sm_count() * 2048 ? 2 : 1;
        int tpr = 1;
        while (want * tpr < a.blocks && tpr < kThreads) tpr *= 2;
        const int threads = tpr > 128 ? kThreads : 128;
        const dim3 grid((unsigned)ceil_div64(groups, threads / tpr));
        auto go = [&](auto kernel) {
          return launch_pdl(kernel, grid, dim3(threads), 0, stream, a, tpr);
        };
        if (a.blocks <= tpr) return go(quantize_rows_kernel<T, 1, A>);
        if (a.blocks <= 2 * tpr) return go(quantize_rows_kernel<T, 2, A>);
        return go(quantize_rows_kernel<T, 4, A>);
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
        float *part = static_cast<float *>(workspace) + (int64_t)g0 * most_parts(groups);
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
  const int pieces = cols * eb / 16;
  int tx = 8;
  while (tx < pieces && tx < kThreads) tx *= 2;
  const dim3 block(tx, kThreads / tx);
  int64_t ctas = ceil_div64((int64_t)groups * rows, (int64_t)block.y * kRowsAhead);
  if (ctas > (int64_t)sm_count() * 64) ctas = (int64_t)sm_count() * 64;
  return with_float(dtype, [&](auto t) {
    auto go = [&](auto kernel) {
      return launch_pdl(kernel, dim3((unsigned)ctas), block, 0, stream, codes, scale, global_scale,
                        (int64_t)groups * rows, rows, pieces, out);
    };
    using T = decltype(t);
    return rows_alignment(out, cols, cols, eb) == 16 ? go(dequantize_kernel<T, kWhole>)
                                                     : go(dequantize_kernel<T, kElems>);
  });
}
