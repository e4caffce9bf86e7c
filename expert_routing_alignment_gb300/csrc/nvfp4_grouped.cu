// nvfp4_grouped.cu -- grouped products of NVFP4 rows and NVFP4 expert weights
// on the block-scaled tensor cores (moe_grouped_product_nvfp4,
// moe_grouped_gate_up_nvfp4), any number of rows.
//
// For every real sorted position p of expert e's run, r the row it reads (its
// token's, or p itself):
//   y[p][o] = sum_k W_e[o][k] * x[r][k]
//   h[p][o] = silu(G_e[o] . x[r]) * (U_e[o] . x[r])
// Both operands are E2M1 codes under an E4M3 scale per 16 elements of k; the
// tensor cores multiply the codes, apply both blocks' scales and sum in fp32
// (tcgen05.mma kind::mxf4nvf4, scale_vec::4X); the global scales of the expert
// and of the row are factors of the whole sum.
//
// How, on sm_103a:
//  * The weights are the MMA's M side, 128 output features a tile, two tiles
//    (gate and up, or two neighbours of one matrix) over the same rows, which
//    are its N side: a run of few rows costs few columns, and each weight tile
//    is read once for up to 128 rows.
//  * A stage is 256 k: 128 bytes a row, the width of the swizzle.  Weight
//    tiles come by TMA boxes, rows by TMA gathers of four at a time, which
//    take any rows: tokens need not be copied into expert order first.
//  * Scales stay row-major as the format has them.  Four warps copy a stage's
//    16 bytes a row to shared memory ahead (cp.async) and write them to tensor
//    memory as the MMA reads them: lane = row % 32, column = row / 32, a
//    column's four bytes the four blocks of one 64-k step, the same in all
//    four quarters of the lanes.
//  * A persistent CTA an SM walks over (expert, feature tile, row tile), the
//    row tiles innermost: CTAs next to one another share weights, and an
//    expert's rows stay in L2.
//  * Roles: warp 0 copies, warp 1 issues MMAs, warps 4-7 bring the scales,
//    warps 8-15 the epilogue.  Every wait gives up after about two seconds
//    with MOE_ERR_TIMEOUT.
#include <cstring>

#include "nvfp4.cuh"
#include "tc_common.cuh"

namespace moe {
namespace {

using namespace tc;

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kStages = 4;
constexpr int kTileRows = 128;             // rows of a row tile, features of a feature tile
constexpr int kOperand = 128 * 128;        // bytes of a stage's codes of 128 rows
constexpr int kScales = 128 * 16;          // and of their scales
constexpr int kStageBytes = 3 * kOperand;  // two weight tiles, the rows
constexpr int kScaleWarp0 = 4, kEpi0 = 8;
constexpr int kWarps = 16, kThreads = kWarps * 32;
constexpr int kEpiThreads = (kWarps - kEpi0) * 32;
// Tensor memory: two accumulators of 128 columns, then a ring of the stages'
// scales, 16 columns for each operand (4 steps x 128 rows / 32).
constexpr uint32_t kAccCols = 128, kScaleBase = 2 * kAccCols, kScaleCols = 48;

struct ProductArgs {
  int E, R, K;               // experts, output features, input features
  int by_token, top_k, n;    // n slots
  int num_rows;              // of the expert-order buffers
  int feature_tiles;         // pairs of tiles (or gate and up tiles) of an expert
  const int32_t *offsets, *sti;
  const uint8_t *wscale[2];  // [E][R][K / 16] of the two tiles' matrices
  const float *wglobal[2];   // [E]
  const uint8_t *xscale;     // [rows][K / 16]
  const float *xglobal;      // [rows]
  void *out;                 // [num_rows][R]
  uint32_t *err;
};

// Codes {K / 2 bytes, E * R rows} box {128, 128}; rows {K / 2, rows} box {128, 1}.
struct ProductMaps {
  CUtensorMap w[2], x;
};

struct Smem {
  alignas(1024) uint8_t codes[kStages][kStageBytes];
  alignas(16) uint8_t scales[kStages][3 * kScales];
  float xg[kTileRows];         // the rows' global scales
  int valid[kTileRows];
  uint64_t full[kStages], empty[kStages], acc_full, acc_empty, drain;
  int failed;
  uint32_t tmem;
  int warp_sum[kWarps];
  int tiles[MOE_MAX_EXPERTS + 1];   // row tiles ahead of each expert's
};

// ---------------------------------------------------------------------------
// tcgen05, block-scaled
// ---------------------------------------------------------------------------

// Instruction descriptor: E2M1 x E2M1 under UE4M3 scales -> f32, both K-major,
// M = 128, N = n, K = 64.
__device__ __forceinline__ uint32_t idesc_nvf4(int n) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 7) << 27);
}
__device__ __forceinline__ void mma_nvf4(uint32_t d, uint64_t ad, uint64_t bd, uint32_t id,
                                         uint32_t sa, uint32_t sb, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X"
      " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(id), "r"(sa), "r"(sb), "r"(acc));
}
// 16 consecutive 32-bit columns of this warp's 32 TMEM lanes, from registers.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}
// Rows r0..r3 (from column x) of a two-dimensional map, 128 bytes each, to dst.
__device__ __forceinline__ void tma_gather4(void *dst, const CUtensorMap *map, int x, int r0,
                                            int r1, int r2, int r3, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(r0), "r"(r1), "r"(r2), "r"(r3),
      "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void tma_2d(void *dst, const CUtensorMap *map, int x, int y,
                                       uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}

// ---------------------------------------------------------------------------
// tiles
// ---------------------------------------------------------------------------

struct Tile {
  int e, m, p0, len;   // expert, feature tile, first position, positions to the run's end (<= 128)
};

__device__ __forceinline__ int clamp_to(int v, int hi) { return v < 0 ? 0 : v > hi ? hi : v; }

__device__ __forceinline__ Tile tile_of(const ProductArgs &a, const Smem &S, int idx) {
  const int mt = a.feature_tiles;
  int lo = 0, hi = a.E - 1;   // the last expert whose tiles begin at or ahead of idx
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (S.tiles[mid] * mt <= idx)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int rt = S.tiles[lo + 1] - S.tiles[lo], r = idx - S.tiles[lo] * mt;
  const int begin = clamp_to(a.offsets[lo], a.num_rows);
  const int end = clamp_to(a.offsets[lo + 1], a.num_rows);
  Tile t;
  t.e = lo;
  t.m = r / rt;
  t.p0 = begin + (r - t.m * rt) * kTileRows;
  t.len = min(kTileRows, end - t.p0);
  return t;
}

// The row that position p0 + i of a tile reads, or -1 where there is none.
__device__ __forceinline__ int row_at(const ProductArgs &a, const Tile &t, int i) {
  if (i >= t.len) return -1;
  const int s = a.sti[t.p0 + i];
  if ((unsigned)s >= (unsigned)a.n) return -1;
  return a.by_token ? s / a.top_k : t.p0 + i;
}
// Rows i = 4 * lane + 0..3 of a tile; returns the tile's rows (the last real
// one's place + 1), the same in every lane.
__device__ __forceinline__ int tile_rows(const ProductArgs &a, const Tile &t, int lane,
                                         int (&r)[4]) {
  int last = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    r[j] = row_at(a, t, 4 * lane + j);
    if (r[j] >= 0) last = 4 * lane + j + 1;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) last = max(last, __shfl_xor_sync(kFull, last, d));
  return last;
}

__device__ __forceinline__ void fail(Smem &S, const ProductArgs &a) {
  *(volatile int *)&S.failed = 1;
  if (a.err) atomicOr(a.err, MOE_ERR_TIMEOUT);
}
__device__ __forceinline__ bool wait_all(Smem &S, uint64_t *bar, uint32_t parity) {
  return __all_sync(kFull, wait_phase(&S.failed, bar, parity));
}

// ---------------------------------------------------------------------------
// roles
// ---------------------------------------------------------------------------

template <bool kPair>
__device__ __forceinline__ bool second_tile(const ProductArgs &a, const Tile &t) {
  return kPair || t.m * 256 + 128 < a.R;
}
// The first feature of tile j of a pair.
template <bool kPair>
__device__ __forceinline__ int feature_of(const Tile &t, int j) {
  return kPair ? t.m * 128 : t.m * 256 + j * 128;
}

template <bool kPair>
__device__ void producer(const ProductArgs &a, const ProductMaps &maps, Smem &S, int total) {
  const int lane = threadIdx.x & 31, kbs = (a.K + 255) / 256;
  uint32_t s = 0;
  bool ok = true;
  for (int idx = blockIdx.x; idx < total && ok; idx += gridDim.x) {
    const Tile t = tile_of(a, S, idx);
    int r[4];
    const int rows = tile_rows(a, t, lane, r);
    if (!rows) continue;
    const bool two = second_tile<kPair>(a, t);
    const uint32_t bytes = (two ? 2 : 1) * kOperand + (rows + 3) / 4 * 512;
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = max(r[j], 0);
    for (int kb = 0; kb < kbs; ++kb, ++s) {
      const int slot = s % kStages;
      uint64_t *bar = &S.full[slot];
      if (s >= kStages && !wait_all(S, &S.empty[slot], (s / kStages - 1) & 1)) {
        ok = false;
        break;
      }
      uint8_t *dst = S.codes[slot];
      if (lane == 0) {
        mbar_expect_tx(bar, bytes);
        tma_2d(dst, &maps.w[0], kb * 128, t.e * a.R + feature_of<kPair>(t, 0), bar);
        if (two)
          tma_2d(dst + kOperand, &maps.w[1], kb * 128, t.e * a.R + feature_of<kPair>(t, 1), bar);
      }
      __syncwarp();
      if (4 * lane < rows)
        tma_gather4(dst + 2 * kOperand + lane * 512, &maps.x, kb * 128, r[0], r[1], r[2], r[3],
                    bar);
    }
  }
  if (!ok && lane == 0) fail(S, a);
  // no copy may be in flight when the CTA ends
  for (uint32_t j = s < kStages ? 0 : s - kStages; j < s; ++j) {
    const uint64_t t0 = gtime();
    while (!mbar_poll(&S.full[j % kStages], (j / kStages) & 1))
      if (gtime() - t0 > kWaitNs) break;
  }
}

template <bool kPair>
__device__ void mma_issuer(const ProductArgs &a, Smem &S, int total, uint32_t tmem) {
  const int lane = threadIdx.x & 31, kbs = (a.K + 255) / 256;
  uint32_t s = 0, n = 0;
  bool ok = true;
  for (int idx = blockIdx.x; idx < total && ok; idx += gridDim.x) {
    const Tile t = tile_of(a, S, idx);
    int r[4];
    const int rows = tile_rows(a, t, lane, r);
    if (!rows) continue;
    const bool two = second_tile<kPair>(a, t);
    const uint32_t id = idesc_nvf4((rows + 15) / 16 * 16);
    if (n && !wait_all(S, &S.acc_empty, (n - 1) & 1)) {
      ok = false;
      break;
    }
    tc_fence_after();
    for (int kb = 0; kb < kbs; ++kb, ++s) {
      const int slot = s % kStages;
      if (!wait_all(S, &S.full[slot], (s / kStages) & 1)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (lane == 0) {
        const int steps = min(4, (a.K - kb * 256 + 63) / 64);
        const uint32_t codes = smem_addr(S.codes[slot]);
        const uint64_t bd = sdesc(codes + 2 * kOperand);
        const uint32_t sc = tmem + kScaleBase + slot * kScaleCols;
        for (int j = 0; j < (two ? 2 : 1); ++j) {
          const uint64_t ad = sdesc(codes + j * kOperand);
          for (int i = 0; i < steps; ++i)   // 64 k: 32 bytes on in the swizzled row
            mma_nvf4(tmem + j * kAccCols, ad + 2 * i, bd + 2 * i, id, sc + j * 16 + 4 * i,
                     sc + 32 + 4 * i, (kb | i) != 0);
        }
        mma_commit(&S.empty[slot]);
        if (kb == kbs - 1) mma_commit(&S.acc_full);
      }
      __syncwarp();
    }
    ++n;
  }
  if (!ok && lane == 0) fail(S, a);
  // tensor memory is given back only after the last MMA
  if (lane == 0) {
    mma_commit(&S.drain);
    const uint64_t t0 = gtime();
    while (!mbar_poll(&S.drain, 0))
      if (gtime() - t0 > kWaitNs) break;
  }
  __syncwarp();
}

// Copies the scales of 16 blocks (those ahead of K) of one row to shared
// memory, zeros for the rest: by 16 or 4 bytes asynchronously (ALIGN: of the
// rows' scales), else by two through registers.
template <int ALIGN>
__device__ __forceinline__ void copy_scales(uint8_t *dst, const uint8_t *row, int first, int have) {
  // have: blocks of the row behind `first`, <= 0 for no row
  if constexpr (ALIGN == 16) {
    const bool there = have > 0;   // whole pieces: K is a multiple of 256
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)),
                 "l"(there ? row + first : row), "r"(there ? 16 : 0)
                 : "memory");
  } else if constexpr (ALIGN == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      copy_async<4>(smem_addr(dst + 4 * i), 4 * i < have ? row + first + 4 * i : row,
                    4 * i < have);
  } else {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (2 * i < have)
        w[i / 2] |= (uint32_t)*reinterpret_cast<const uint16_t *>(row + first + 2 * i)
                    << (16 * (i & 1));
    *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Walks over the stages of a CTA's tiles, one copy of scales at a time.
template <bool kPair, int ALIGN>
struct ScaleWalk {
  const ProductArgs &a;
  Smem &S;
  int total, idx, kb, kbs, thread;
  uint32_t issued;
  const uint8_t *row[3];   // this thread's rows of the tile's operands, NULL: none

  __device__ ScaleWalk(const ProductArgs &args, Smem &sm, int tot)
      : a(args), S(sm), total(tot), idx((int)blockIdx.x - (int)gridDim.x), kb(0),
        kbs((args.K + 255) / 256), thread((int)threadIdx.x - kScaleWarp0 * 32), issued(0) {
    kb = kbs;
  }
  // The next stage's copies (one group, empty behind the end).
  __device__ __forceinline__ void next() {
    while (kb == kbs) {
      idx += gridDim.x;
      if (idx >= total) {
        idx = total;
        break;
      }
      const Tile t = tile_of(a, S, idx);
      int r[4];
      if (!tile_rows(a, t, thread & 31, r)) continue;
      const int pitch = a.K / 16;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int f = feature_of<kPair>(t, j) + thread;
        row[j] = f < a.R ? a.wscale[j] + ((int64_t)t.e * a.R + f) * pitch : nullptr;
      }
      const int x = row_at(a, t, thread);
      row[2] = x >= 0 ? a.xscale + (int64_t)x * pitch : nullptr;
      kb = 0;
    }
    if (kb < kbs) {
      uint8_t *dst = S.scales[issued % kStages] + thread * 16;
#pragma unroll
      for (int j = 0; j < 3; ++j)
        copy_scales<ALIGN>(dst + j * kScales, row[j] ? row[j] : a.wscale[0], row[j] ? kb * 16 : 0,
                           row[j] ? a.K / 16 - kb * 16 : 0);
      ++kb;
      ++issued;
    }
    copies_commit();
  }
};

// Warps 4-7.  Shared memory is a ring that these warps alone use: a slot is
// written again by the copies of stage s + 3, which are started after the
// barrier of stage s, when all have read stage s - 1.
template <bool kPair, int ALIGN>
__device__ void scale_role(const ProductArgs &a, Smem &S, int total, uint32_t tmem) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = tmem + ((uint32_t)((warp & 3) * 32) << 16) + kScaleBase;
  ScaleWalk<kPair, ALIGN> walk(a, S, total);
  for (int d = 0; d < kStages - 1; ++d) walk.next();
  bool ok = true;
  for (uint32_t s = 0; s < walk.issued; ++s) {
    const int slot = s % kStages;
    copies_wait(kStages - 1);
    asm volatile("bar.sync 1, 128;" ::: "memory");
    uint32_t v[3][16];
#pragma unroll
    for (int j = 0; j < 3; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint4 w = *reinterpret_cast<const uint4 *>(S.scales[slot] + j * kScales +
                                                         (q * 32 + lane) * 16);
        v[j][q] = w.x;
        v[j][4 + q] = w.y;
        v[j][8 + q] = w.z;
        v[j][12 + q] = w.w;
      }
    walk.next();
    // after a failure the walk goes on, so that the four warps' barriers match
    if (ok && s >= kStages && !wait_all(S, &S.empty[slot], (s / kStages - 1) & 1)) ok = false;
    if (ok) {
      tc_fence_after();
#pragma unroll
      for (int j = 0; j < 3; ++j) tmem_st16(base + slot * kScaleCols + j * 16, v[j]);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.full[slot]);
    }
  }
  if (!ok && lane == 0) fail(S, a);
}

template <typename T>
__device__ __forceinline__ void store_one(void *out, int64_t at, float v) {
  using TB = typename T::bits;
  if constexpr (sizeof(TB) == 2)
    static_cast<uint16_t *>(out)[at] = (uint16_t)(T::down2(v, 0.f) & 0xFFFFu);
  else
    static_cast<float *>(out)[at] = v;
}

__device__ __forceinline__ void epi_sync() {
  asm volatile("bar.sync 2, %0;" ::"n"(kEpiThreads) : "memory");
}

template <typename T, bool kPair>
__device__ void epilogue(const ProductArgs &a, Smem &S, int total, uint32_t tmem) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = warp & 3;
  const int half = (warp - kEpi0) >> 2, thread = (int)threadIdx.x - kEpi0 * 32;
  const uint32_t base = tmem + ((uint32_t)(q * 32) << 16);
  uint32_t n = 0;
  bool ok = true;
  for (int idx = blockIdx.x; idx < total; idx += gridDim.x) {
    const Tile t = tile_of(a, S, idx);
    int r[4];
    const int rows = tile_rows(a, t, lane, r);
    if (!rows) continue;
    epi_sync();   // the tile before has been read
    if (thread < kTileRows) {
      const int x = row_at(a, t, thread);
      S.valid[thread] = x >= 0;
      S.xg[thread] = x >= 0 ? a.xglobal[x] : 0.f;
      if (thread < t.len) {
        const int slot = a.sti[t.p0 + thread];
        if ((slot < 0 || slot > a.n) && a.err) atomicOr(a.err, MOE_ERR_BAD_POSITION);
      }
    }
    epi_sync();
    if (ok && !wait_all(S, &S.acc_full, n & 1)) ok = false;
    ++n;
    if (!ok) continue;   // the others' barriers match
    tc_fence_after();
    const float g0 = a.wglobal[0][t.e], g1 = a.wglobal[1][t.e];
    const int f0 = feature_of<kPair>(t, 0) + q * 32 + lane;
    const int f1 = feature_of<kPair>(t, 1) + q * 32 + lane;
    for (int c0 = half * 64; c0 < min(rows, half * 64 + 64); c0 += 16) {
      uint32_t v0[16], v1[16];
      tmem_ld16(base + c0, v0);
      tmem_ld16(base + kAccCols + c0, v1);
      tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        if (!S.valid[c0 + c]) continue;
        const float xg = S.xg[c0 + c];
        const int64_t at = (int64_t)(t.p0 + c0 + c) * a.R;
        const float y0 = __uint_as_float(v0[c]) * xg * g0, y1 = __uint_as_float(v1[c]) * xg * g1;
        if constexpr (kPair) {
          if (f0 < a.R) store_one<T>(a.out, at + f0, silu_f32(y0) * y1);
        } else {
          if (f0 < a.R) store_one<T>(a.out, at + f0, y0);
          if (f1 < a.R) store_one<T>(a.out, at + f1, y1);
        }
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.acc_empty);
  }
  if (!ok && lane == 0) fail(S, a);
}

template <typename T, bool kPair, int ALIGN>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_nvfp4_kernel(const __grid_constant__ ProductArgs a,
                         const __grid_constant__ ProductMaps maps) {
  extern __shared__ uint8_t raw[];
  Smem &S = *reinterpret_cast<Smem *>(raw + ((1024 - (smem_addr(raw) & 1023)) & 1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&S.full[i], 5);    // the copies, and each scale warp
      mbar_init(&S.empty[i], 1);
    }
    mbar_init(&S.acc_full, 1);
    mbar_init(&S.acc_empty, kWarps - kEpi0);
    mbar_init(&S.drain, 1);
    S.failed = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&S.tmem)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 0 && lane < 3) prefetch_tensormap(lane == 2 ? &maps.x : &maps.w[lane]);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem;
  pdl_wait();
  pdl_trigger();

  // S.tiles: the row tiles ahead of each expert's, two experts a thread
  int run[2], bad = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = 2 * threadIdx.x + i;
    run[i] = 0;
    if (e < a.E) {
      const int b = a.offsets[e], d = a.offsets[e + 1];
      bad |= b < 0 || d < b || d > a.num_rows;
      const int len = clamp_to(d, a.num_rows) - clamp_to(b, a.num_rows);
      run[i] = len > 0 ? (len + kTileRows - 1) / kTileRows : 0;
    }
  }
  // tables that are none: nothing is computed (their tiles could be any number)
  const bool refused = __syncthreads_or(bad);
  if (refused && a.err && threadIdx.x == 0) atomicOr(a.err, MOE_ERR_BAD_POSITION);
  int inc = run[0] + run[1];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(kFull, inc, d);
    if (lane >= d) inc += v;
  }
  if (lane == 31) S.warp_sum[warp] = inc;
  __syncthreads();
  for (int w = 0; w < warp; ++w) inc += S.warp_sum[w];
  if (2 * (int)threadIdx.x < a.E) {
    S.tiles[2 * threadIdx.x + 1] = inc - run[1];
    if (2 * (int)threadIdx.x + 1 < a.E) S.tiles[2 * threadIdx.x + 2] = inc;
  }
  if (threadIdx.x == 0) S.tiles[0] = 0;
  __syncthreads();
  const int total = refused ? 0 : S.tiles[a.E] * a.feature_tiles;

  if (warp == 0)
    producer<kPair>(a, maps, S, total);
  else if (warp == 1)
    mma_issuer<kPair>(a, S, total, tmem);
  else if (warp >= kEpi0)
    epilogue<T, kPair>(a, S, total, tmem);
  else if (warp >= kScaleWarp0)
    scale_role<kPair, ALIGN>(a, S, total, tmem);

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

constexpr size_t kSmemBytes = sizeof(Smem) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory of a CTA");

bool misaligned(const void *p, uintptr_t bytes) { return ((uintptr_t)p & (bytes - 1)) != 0; }

int grouped(const moe_proj *w0, const moe_proj *w1, int E, int R, int K, const uint8_t *codes,
            const uint8_t *scale, const float *global, int by_token, int M, int top_k,
            const int32_t *offsets, const int32_t *sti, int num_rows, int dtype, void *out,
            uint32_t *err, void *stream) {
  const int eb = dtype_bytes(dtype);
  if (E < 1 || R < 1 || K < 1 || M < 0 || top_k < 1 || num_rows < 0 || eb < 2) return MOE_EINVAL;
  if (E > MOE_MAX_EXPERTS || K % 32 || K > MOE_MAX_ROW_HIDDEN || R > 4 * MOE_MAX_ROW_HIDDEN ||
      top_k > 32 || (int64_t)M * top_k > MOE_MAX_SLOTS || (int64_t)E * R > 0x7FFFFFFF)
    return MOE_EUNSUPPORTED;
  if (M == 0 || num_rows == 0) return MOE_OK;
  const moe_proj *w[2] = {w0, w1 ? w1 : w0};
  for (int j = 0; j < 2; ++j) {
    if (!w[j] || !w[j]->codes || !w[j]->scale || !w[j]->global_scale) return MOE_EINVAL;
    if (misaligned(w[j]->codes, 16) || misaligned(w[j]->scale, 16) ||
        misaligned(w[j]->global_scale, 4))
      return MOE_EINVAL;
  }
  if (!codes || !scale || !global || !offsets || !sti || !out) return MOE_EINVAL;
  if (misaligned(codes, 16) || misaligned(scale, 16) || misaligned(global, 4) ||
      misaligned(offsets, 4) || misaligned(sti, 4) || misaligned(out, eb) || misaligned(err, 4))
    return MOE_EINVAL;
  const int sms = sm_count();
  if (!sms) return MOE_ECUDA;

  ProductArgs a = {};
  a.E = E;
  a.R = R;
  a.K = K;
  a.by_token = by_token;
  a.top_k = top_k;
  a.n = M * top_k;
  a.num_rows = num_rows;
  a.feature_tiles = w1 ? (R + 127) / 128 : (R + 255) / 256;
  a.offsets = offsets;
  a.sti = sti;
  for (int j = 0; j < 2; ++j) {
    a.wscale[j] = static_cast<const uint8_t *>(w[j]->scale);
    a.wglobal[j] = w[j]->global_scale;
  }
  a.xscale = scale;
  a.xglobal = global;
  a.out = out;
  a.err = err;
  ProductMaps maps;
  memset(&maps, 0, sizeof(maps));
  const cuuint64_t pitch[1] = {(cuuint64_t)K / 2};
  const cuuint64_t wd[2] = {(cuuint64_t)K / 2, (cuuint64_t)E * R};
  const cuuint64_t xd[2] = {(cuuint64_t)K / 2, (cuuint64_t)(by_token ? M : num_rows)};
  const cuuint32_t wbox[2] = {128, 128}, xbox[2] = {128, 1};
  for (int j = 0; j < 2; ++j)
    if (const int st = encode_u8_sw128(&maps.w[j], w[j]->codes, 2, wd, pitch, wbox)) return st;
  if (const int st = encode_u8_sw128(&maps.x, codes, 2, xd, pitch, xbox)) return st;

  // an upper bound of the tiles: experts have at most a tile more than whole ones
  const int64_t slots = a.n < E ? a.n : E;
  const int64_t most = (num_rows / kTileRows + slots) * a.feature_tiles;
  const dim3 grid((unsigned)(most < sms ? most : sms));
  auto go = [&](auto t, auto pair) {
    using T = decltype(t);
    constexpr bool P = decltype(pair)::value;
    auto launch = [&](auto kernel) {
      if (const int st = ensure_smem_limit((const void *)kernel, kSmemBytes)) return st;
      return launch_pdl(kernel, grid, dim3(kThreads), kSmemBytes, stream, a, maps);
    };
    if (K % 256 == 0) return launch(grouped_nvfp4_kernel<T, P, 16>);
    if (K % 64 == 0) return launch(grouped_nvfp4_kernel<T, P, 4>);
    return launch(grouped_nvfp4_kernel<T, P, 2>);
  };
  auto typed = [&](auto pair) {
    switch (dtype) {
      case MOE_DTYPE_BF16: return go(BF16{}, pair);
      case MOE_DTYPE_F16: return go(F16{}, pair);
      default: return go(F32{}, pair);
    }
  };
  return w1 ? typed(std::true_type{}) : typed(std::false_type{});
}

}  // namespace
}  // namespace moe

extern "C" int moe_grouped_product_nvfp4(const moe_proj *weight, int num_experts, int out_dim,
                                         int in_dim, const uint8_t *codes, const uint8_t *scale,
                                         const float *global_scale, int by_token, int M, int top_k,
                                         const int32_t *expert_offsets,
                                         const int32_t *sorted_token_ids, int num_rows,
                                         int out_dtype, void *out, uint32_t *err_word,
                                         void *stream) {
  return moe::grouped(weight, nullptr, num_experts, out_dim, in_dim, codes, scale, global_scale,
                      by_token, M, top_k, expert_offsets, sorted_token_ids, num_rows, out_dtype,
                      out, err_word, stream);
}

extern "C" int moe_grouped_gate_up_nvfp4(const moe_proj *gate, const moe_proj *up, int num_experts,
                                         int out_dim, int in_dim, const uint8_t *codes,
                                         const uint8_t *scale, const float *global_scale,
                                         int by_token, int M, int top_k,
                                         const int32_t *expert_offsets,
                                         const int32_t *sorted_token_ids, int num_rows,
                                         int out_dtype, void *out, uint32_t *err_word,
                                         void *stream) {
  if (!up) return MOE_EINVAL;
  return moe::grouped(gate, up, num_experts, out_dim, in_dim, codes, scale, global_scale, by_token,
                      M, top_k, expert_offsets, sorted_token_ids, num_rows, out_dtype, out,
                      err_word, stream);
}
