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
//  * A tile is up to 128 rows by 256 weight rows: 128 features of gate and of
//    up, or 256 neighbours of one matrix.  With many rows the tokens are the
//    MMA's 128 lanes and the weights its 256 columns, so that a thread of the
//    epilogue has neighbouring features of one row.  With few (32 or fewer) the
//    weights are the lanes and the tokens the columns: the epilogue is as short
//    as the rows are few.  Both read the same shared memory and the same scales.
//  * A stage is 256 k: 128 bytes a row, the width of the swizzle.  Weight tiles
//    come by TMA boxes, and so do rows in expert order; the tokens' own rows,
//    which can be any, by 16-byte copies (cp.async) that place them as the
//    swizzle would, so that tokens need not be copied into expert order first.
//    (TMA gathers of four rows each took the gate and up of 4096 rows from 91 to
//    150 us.)
//  * Scales stay row-major as the format has them.  TMA brings a stage's 16
//    bytes a row, and four warps turn them by words of 4 blocks (64 k) to where
//    the tensor cores' own copy to tensor memory takes them (tcgen05.cp 32x128b,
//    issued ahead of the stage's MMAs): for each 64 k and 128 rows 32 x 16 bytes,
//    line = row % 32, word = row / 32.  Rows of scales that TMA does not take (k
//    no multiple of 256) the four warps copy there themselves.
//  * A persistent CTA an SM walks over (expert, feature tile, row tile), the
//    row tiles innermost: CTAs next to one another share weights, and an
//    expert's rows stay in L2.
//  * Roles: warp 0 starts the copies of codes and warp 3 those of scales, which
//    run further ahead, warp 1 issues MMAs, warp 2 looks the tiles up ahead of
//    all others, warps 4-7 turn the scales and copy tokens' rows, warps 8-15 are
//    the epilogue, which takes the accumulators into registers first, so that
//    the next tile's MMAs run beside its arithmetic and stores.  The roles meet
//    at mbarriers alone; every wait gives up after about two seconds with
//    MOE_ERR_TIMEOUT.
//
// Measured and bounds (one GB300; E experts, k an expert's input width):
//  * Few rows an expert: HBM.  128 tokens, 199 of 256 experts active, 4096 x 1536
//    gate and up (1.41 GB read): 205-216 us, 6.6-6.9 TB/s.
//  * Many: no path's rate, but the ring of three stages (all that fits) and the MMAs'
//    issue.  Of about 1450 clocks a stage (clock() in the issuing warp; 4096 tokens'
//    gate and up, and down of 64 experts) 790-890 go by while the stage's copies of
//    scales and MMAs are given out, whose own time is 512; 350-480 are waited for its
//    bytes, which are there 2800-3200 clocks after their copies began; 160-290 lie
//    between tiles (the next tile's rows, the epilogue's taking of the accumulators).
//    Meanwhile (ncu) L2 to SM carries 10 TB/s, 27 % of what it can, L2 is at 37-44 %,
//    shared memory's banks at 31-36 %, HBM at 39-49 %, the tensor pipe at 28 %.  Gate
//    and up of 4096 tokens (128 experts, 2048 x 768, 206 GFLOP) 80 us, 2.6 PFLOP/s;
//    down of 8192 (256 experts, 1536 x 4096, 825 GFLOP, 1.5 GB) 304-311 us, 2.7.  Two
//    stages take 359 us there; tiles of 192 columns, whose accumulators tensor memory
//    holds twice, 365; codes brought to L2 ahead, 333.
//  * One token: its chain of latencies, 8.3 us (8 experts, 14 MB): 1 us to the
//    first tile's place, 1 to its first copies, eight stages of 0.45, which the
//    MMAs' issue bounds, the epilogue.
#include <atomic>
#include <cstring>

#include "nvfp4.cuh"
#include "tc_common.cuh"

namespace moe {
namespace {

using namespace tc;

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kStages = 3;
constexpr int kTileRows = 128;             // rows of a row tile, features of a feature tile
constexpr int kOperand = 128 * 128;        // bytes of a stage's codes of 128 rows
constexpr int kStageBytes = 3 * kOperand;  // two weight tiles, the rows
// The scales of a stage in shared memory: 512 bytes for each 64 k and 128 rows,
// set apart so that a warp's words of 8 rows x 4 steps, or pieces of 2 x 4, lie in
// 32 banks.
constexpr int kHalfPitch = 528, kWeightPitch = 2 * kHalfPitch, kRowPitch = 544;
constexpr int kScaleBytes = 4 * kWeightPitch + 4 * kRowPitch;
constexpr int kRawScales = 128 * 16;   // of 128 rows, row by row
constexpr int kCopyWarp0 = 4, kEpi0 = 8, kEpiWarps = 8;
constexpr int kWarps = kEpi0 + kEpiWarps, kThreads = kWarps * 32;
// Registers a thread, of the kLaunchRegs that the block starts with: the
// epilogue holds 128 accumulators.  Shares of a warpgroup each (of four warps),
// and no more in all than the block has.
constexpr int kLaunchRegs = 128, kIssueRegs = 40, kCopyRegs = 72, kEpiRegs = 200;
static_assert((kIssueRegs + kCopyRegs) * 128 + kEpiRegs * 256 <= kLaunchRegs * kThreads,
              "registers");
constexpr int kInfos = 4;                  // tiles looked up ahead
constexpr int kFewRows = 32;               // rows that are columns
// Tensor memory: the accumulators of 256 columns, then a ring of the stages'
// scales: for each of 4 steps of 64 k, 8 columns of the weights' 256 rows; for
// each, 4 columns of the tile's 128 rows.
constexpr uint32_t kTileCols = 128, kScaleBase = 256, kScaleCols = 48, kRowScales = 32;

struct ProductArgs {
  int E, R, K;               // experts, output features, input features
  int by_token, n;           // n slots
  uint32_t per_k;            // 2^32 / top_k, rounded up (0: top_k 1): slots are below 2^20
  int num_rows;              // of the expert-order buffers
  int x_rows;                // of the rows' codes and scales
  int align;                 // of the output's rows, in bytes: 16 or less
  int feature_tiles;         // pairs of tiles (or gate and up tiles) of an expert
  const int32_t *offsets, *sti;
  const uint8_t *wscale[2];  // [E][R][K / 16] of the two tiles' matrices
  const float *wglobal[2];   // [E]
  const uint8_t *xcodes, *xscale;   // [rows][K / 2], [rows][K / 16]
  const float *xglobal;      // [rows]
  void *out;                 // [num_rows][R]
  uint32_t *err;
};

// Codes {K / 2 bytes, E * R rows} box {128, 128} (pairs of matrices) or {128, 256};
// rows {K / 2, rows} box {128, 32} and {128, 128}; scales {K / 16 bytes, E * R rows}
// and {K / 16, rows} with 16 bytes of as many rows.
struct ProductMaps {
  CUtensorMap w[2], x[2], ws[2], xs;
};

// A tile as every role reads it: its place first, then its rows.
struct TileInfo {
  int e, m, p0, len;        // expert (< 0: no more tiles), feature tile, first position, positions
  int rows;                 // rows up to the last real one; 0 of padding alone
  alignas(16) int row[kTileRows];   // the row that each position reads, -1: none
};

struct Smem {
  alignas(1024) uint8_t codes[kStages][kStageBytes];
  alignas(128) uint8_t raw[kStages][3 * kRawScales];   // scales by row, as TMA brings them
  alignas(16) uint8_t scales[kStages][kScaleBytes];
  alignas(128) uint8_t staged[kEpiWarps][32 * 128];    // output on its way out, a warp's own
  alignas(16) TileInfo info[kInfos];
  uint64_t full[kStages], empty[kStages], raw_full[kStages], raw_empty[kStages];
  uint64_t info_place[kInfos], info_rows[kInfos], info_empty[kInfos];
  uint64_t acc_full, acc_empty, drain;
  int failed;
  uint32_t tmem;
  int tiles[MOE_MAX_EXPERTS + 1];   // row tiles ahead of each expert's
  int begin[MOE_MAX_EXPERTS + 1];   // the runs' first positions
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
// 32 consecutive fp32 columns of this warp's 32 TMEM lanes.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
      "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31"
      "}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr));
}
// One lane of a converged warp, the same one every time.  MMAs and copies are
// issued under it and unrolled: the compiler knows of it that one lane is
// active.  (In a rolled loop under lane == 0 an MMA took 180 to 190 clocks to issue,
// under this 150; unrolled one of 256 columns takes the tensor cores' own 128, and
// a copy of scales beside it none.)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
// 32 lines of 16 bytes in shared memory (8 lines of 128 bytes together) to four
// columns of tensor memory, the same in all four quarters of the lanes.
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint32_t smem) {
  const uint64_t desc = (uint64_t)((smem & 0x3FFFF) >> 4) | ((uint64_t)(128 >> 4) << 32) |
                        ((uint64_t)1 << 46);
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc));
}
// Arrives at a barrier, which counts it, when this thread's copies so far have
// landed.
__device__ __forceinline__ void copies_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar))
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

__device__ __forceinline__ void fail(Smem &S, const ProductArgs &a) {
  *(volatile int *)&S.failed = 1;
  if (a.err) atomicOr(a.err, MOE_ERR_TIMEOUT);
}
// A whole warp's wait for a phase.  The barrier's own waiting test parks the warp
// for a while; the clock and the other roles' failure are looked at now and then.
__device__ __forceinline__ bool wait_all(Smem &S, uint64_t *bar, uint32_t parity) {
  bool ok = mbar_try(bar, parity);
  if (!ok) {
    const uint64_t t0 = gtime();
    for (uint32_t i = 1; i < (1u << 28); ++i) {
      ok = mbar_try(bar, parity);
      if (ok || ((i & 63) == 0 && (*(volatile int *)&S.failed || gtime() - t0 > kWaitNs))) break;
    }
  }
  return __all_sync(kFull, ok);
}

// Warp 2 alone looks at the tables: S.tiles, the row tiles ahead of each expert's, and
// the runs' first positions; returns the number of tiles, 0 for tables that are
// none (their tiles could be any number).
__device__ __forceinline__ int lay_out_tiles(const ProductArgs &a, Smem &S) {
  constexpr int U = 4;   // neighbouring experts of a lane
  const int lane = threadIdx.x & 31;
  int ahead = 0, bad = 0;
#pragma unroll 1
  for (int e = lane * U; e - lane * U < a.E; e += 32 * U) {
    int at[U + 1], before[U + 1];
#pragma unroll
    for (int u = 0; u <= U; ++u) at[u] = a.offsets[min(e + u, a.E)];
    before[0] = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int wrong = at[u] < 0 || at[u + 1] < at[u] || at[u + 1] > a.num_rows;
      bad |= wrong;
      before[u + 1] =
          before[u] + (wrong ? 0 : (at[u + 1] - at[u] + kTileRows - 1) / kTileRows);
    }
    int inc = before[U];
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const int v = __shfl_up_sync(kFull, inc, k);
      if (lane >= k) inc += v;
    }
    const int first = ahead + inc - before[U];
#pragma unroll
    for (int u = 0; u <= U; ++u)
      if (e + u <= a.E) {   // the entry behind the last too; a neighbour writes the same
        S.tiles[e + u] = first + before[u];
        S.begin[e + u] = at[u];
      }
    ahead += __shfl_sync(kFull, inc, 31);
  }
  __syncwarp();
  bad = __reduce_or_sync(kFull, bad);
  if (bad && a.err && lane == 0) atomicOr(a.err, MOE_ERR_BAD_POSITION);
  return bad ? 0 : ahead * a.feature_tiles;
}

// The CTA's tiles in order.  A run's first tile is published as soon as its place
// is known, which is all that the weights' copies need, and again with its rows;
// later ones, of which those of padding alone are left out, with their rows.
__device__ __forceinline__ void scheduler(const ProductArgs &a, Smem &S, int total) {
  const int lane = threadIdx.x & 31, mt = a.feature_tiles;
  uint32_t n = 0;
  for (int idx = blockIdx.x;; idx += gridDim.x) {
    int e = -1, m = 0, p0 = 0, len = 0, rows = 0, r[4];
    bool looked = false;
    auto look = [&] {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = 4 * lane + j;
        const int s = i < len ? a.sti[p0 + i] : a.n;
        r[j] = (unsigned)s >= (unsigned)a.n ? -1
               : !a.by_token                ? p0 + i
               : a.per_k                    ? (int)__umulhi(s, a.per_k)
                                            : s;
        if (r[j] >= 0) rows = i + 1;
        if ((s < 0 || s > a.n) && a.err) atomicOr(a.err, MOE_ERR_BAD_POSITION);
      }
      rows = __reduce_max_sync(kFull, rows);
    };
    if (idx < total) {
      // the last expert whose tiles begin at or ahead of idx
      int ahead = 0;
      for (int i = lane; i < a.E; i += 32) ahead += S.tiles[i] * mt <= idx;
      e = __reduce_add_sync(kFull, ahead) - 1;
      const int rt = S.tiles[e + 1] - S.tiles[e], at = idx - S.tiles[e] * mt;
      m = at / rt;
      p0 = S.begin[e] + (at - m * rt) * kTileRows;
      len = min(kTileRows, S.begin[e + 1] - p0);
      looked = at != m * rt;
      if (looked) {
        look();
        if (!rows) continue;
      }
    }
    const int slot = n % kInfos;
    if (n >= kInfos && !wait_all(S, &S.info_empty[slot], (n / kInfos - 1) & 1)) {
      if (lane == 0) fail(S, a);
      return;
    }
    TileInfo &t = S.info[slot];
    if (lane == 0) {
      *reinterpret_cast<int4 *>(&t.e) = make_int4(e, m, p0, len);
      mbar_arrive(&S.info_place[slot]);
    }
    if (e >= 0) {
      if (!looked) look();
      *reinterpret_cast<int4 *>(&t.row[4 * lane]) = make_int4(r[0], r[1], r[2], r[3]);
    }
    if (lane == 0) t.rows = rows;
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.info_rows[slot]);
    if (e < 0) return;
    ++n;
  }
}

// A role's view of the tiles: next() gives the next one (NULL at the end, or
// after a failure, which sets ok = false), its place alone or with its rows;
// done() lets go of it.  Whole warps.
struct Tiles {
  Smem &S;
  uint64_t *known;
  uint32_t n = 0;
  bool ok = true;
  __device__ __forceinline__ Tiles(Smem &s, bool rows) : S(s), known(rows ? s.info_rows : s.info_place) {}
  __device__ __forceinline__ const TileInfo *next() {
    const TileInfo *t = &S.info[n % kInfos];
    if (!wait_all(S, &known[n % kInfos], (n / kInfos) & 1)) {
      ok = false;
      return nullptr;
    }
    return t->e < 0 ? nullptr : t;
  }
  __device__ __forceinline__ void done() {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&S.info_empty[n % kInfos]);
    ++n;
  }
};

// ---------------------------------------------------------------------------
// roles
// ---------------------------------------------------------------------------

// Whether a tile has its second 128 features, and the first feature of half j.
template <bool kPair>
__device__ __forceinline__ bool second_half(const ProductArgs &a, int m) {
  return kPair || m * 256 + 128 < a.R;
}
template <bool kPair>
__device__ __forceinline__ int feature_of(int m, int j) {
  return kPair ? m * 128 : m * 256 + j * 128;
}

// Waits until the copies counted by the last stages of a ring of barriers have
// landed: none may be in flight when the CTA ends.
__device__ __forceinline__ void copies_drain(uint64_t *bars, uint32_t s) {
  for (uint32_t j = s < kStages ? 0 : s - kStages; j < s; ++j) {
    const uint64_t t0 = gtime();
    while (!mbar_poll(&bars[j % kStages], (j / kStages) & 1))
      if (gtime() - t0 > kWaitNs) break;
  }
}

// Warp 0: codes of the weights, and of rows in expert order.
template <bool kPair>
__device__ void producer(const ProductArgs &a, const ProductMaps &maps, Smem &S) {
  const int kbs = (a.K + 255) / 256;
  uint32_t s = 0;
  Tiles tiles(S, false);
  while (const TileInfo *t = tiles.next()) {
    const int rows = a.by_token ? 0 : t->len <= 32 ? 32 : 128, p0 = t->p0;
    const int w0 = t->e * a.R + feature_of<kPair>(t->m, 0);
    tiles.done();
    const uint32_t bytes = 2 * kOperand + rows * 128;
    const CUtensorMap *x = &maps.x[rows == 128];
    for (int kb = 0; kb < kbs; ++kb, ++s) {
      const int slot = s % kStages;
      if (s >= kStages && !wait_all(S, &S.empty[slot], (s / kStages - 1) & 1)) {
        tiles.ok = false;
        break;
      }
      if (elect_one()) {
        uint64_t *bar = &S.full[slot];
        uint8_t *dst = S.codes[slot];
        mbar_expect_tx(bar, bytes);
        tma_2d(dst, &maps.w[0], kb * 128, w0, bar);
        if constexpr (kPair) tma_2d(dst + kOperand, &maps.w[1], kb * 128, w0, bar);
        if (rows) tma_2d(dst + 2 * kOperand, x, kb * 128, p0, bar);
      }
      __syncwarp();
    }
    if (!tiles.ok) break;
  }
  if (!tiles.ok && (threadIdx.x & 31) == 0) fail(S, a);
  copies_drain(S.full, s);
}

// Warp 3: their scales, row by row.
template <bool kPair>
__device__ void scale_producer(const ProductArgs &a, const ProductMaps &maps, Smem &S) {
  const int kbs = a.K / 256;
  const uint32_t bytes = (a.by_token ? 2 : 3) * kRawScales;
  uint32_t s = 0;
  Tiles tiles(S, false);
  while (const TileInfo *t = tiles.next()) {
    const int w0 = t->e * a.R + feature_of<kPair>(t->m, 0), p0 = t->p0;
    tiles.done();
    for (int kb = 0; kb < kbs; ++kb, ++s) {
      const int slot = s % kStages;
      if (s >= kStages && !wait_all(S, &S.raw_empty[slot], (s / kStages - 1) & 1)) {
        tiles.ok = false;
        break;
      }
      if (elect_one()) {
        uint64_t *bar = &S.raw_full[slot];
        uint8_t *dst = S.raw[slot];
        mbar_expect_tx(bar, bytes);
        tma_2d(dst, &maps.ws[0], kb * 16, w0, bar);
        if constexpr (kPair) tma_2d(dst + kRawScales, &maps.ws[1], kb * 16, w0, bar);
        if (!a.by_token) tma_2d(dst + 2 * kRawScales, &maps.xs, kb * 16, p0, bar);
      }
      __syncwarp();
    }
    if (!tiles.ok) break;
  }
  if (!tiles.ok && (threadIdx.x & 31) == 0) fail(S, a);
  copies_drain(S.raw_full, s);
}

// The tensor cores' work on a stage: its scales to tensor memory, then a step of
// 64 k (32 bytes of the swizzled rows) at a time.  kFew: the weights' halves are
// the lanes and the tile's rows the columns; else the other way round.
template <bool kFew, bool kTwo>
__device__ __forceinline__ void issue_step(int i, uint32_t tmem, uint32_t sc, uint64_t w,
                                           uint64_t x, uint32_t id, uint32_t acc) {
  const uint32_t sw = sc + 8 * i, sx = sc + kRowScales + 4 * i;
  if constexpr (kFew) {
    mma_nvf4(tmem, w + 2 * i, x + 2 * i, id, sw, sx, acc);
    if constexpr (kTwo)
      mma_nvf4(tmem + kTileCols, w + (kOperand >> 4) + 2 * i, x + 2 * i, id, sw + 4, sx, acc);
  } else {
    mma_nvf4(tmem, x + 2 * i, w + 2 * i, id, sx, sw, acc);
  }
}
template <bool kTwo>
__device__ __forceinline__ void copy_step(int i, uint32_t sc, uint32_t scales) {
  tmem_copy_scales(sc + 8 * i, scales + i * kWeightPitch);
  if constexpr (kTwo) tmem_copy_scales(sc + 8 * i + 4, scales + i * kWeightPitch + kHalfPitch);
  tmem_copy_scales(sc + kRowScales + 4 * i, scales + 4 * kWeightPitch + i * kRowPitch);
}
template <bool kFew, bool kTwo>
__device__ __forceinline__ void issue_stage(Smem &S, int slot, uint32_t tmem, uint32_t id,
                                            int steps, bool first) {
  const uint32_t codes = smem_addr(S.codes[slot]), scales = smem_addr(S.scales[slot]);
  const uint64_t w = sdesc(codes), x = sdesc(codes + 2 * kOperand);
  const uint32_t sc = tmem + kScaleBase + slot * kScaleCols;
  if (steps == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) copy_step<kTwo>(i, sc, scales);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      issue_step<kFew, kTwo>(i, tmem, sc, w, x, id, i || !first);
  } else {
    for (int i = 0; i < steps; ++i) {
      copy_step<kTwo>(i, sc, scales);
      issue_step<kFew, kTwo>(i, tmem, sc, w, x, id, i || !first);
    }
  }
}

template <bool kPair>
__device__ void mma_issuer(const ProductArgs &a, Smem &S, uint32_t tmem) {
  const int lane = threadIdx.x & 31, kbs = (a.K + 255) / 256;
  uint32_t s = 0;
  Tiles tiles(S, true);
  while (const TileInfo *t = tiles.next()) {
    const int rows = t->rows;
    const bool two = second_half<kPair>(a, t->m), few = rows <= kFewRows;
    tiles.done();
    // of padding alone: as a few rows that nothing reads
    const uint32_t id = idesc_nvf4(few ? max(rows + 15, 16) / 16 * 16 : two ? 256 : 128);
    if (tiles.n > 1 && !wait_all(S, &S.acc_empty, tiles.n & 1)) {
      tiles.ok = false;
      break;
    }
    tc_fence_after();
    for (int kb = 0; kb < kbs; ++kb, ++s) {
      const int slot = s % kStages;
      if (!wait_all(S, &S.full[slot], (s / kStages) & 1)) {
        tiles.ok = false;
        break;
      }
      tc_fence_after();
      const int steps = min(4, (a.K - kb * 256 + 63) / 64);
      if (elect_one()) {
        // what other threads' cp.async wrote, ahead of the tensor cores' reads
        fence_proxy_async_smem();
        if (few && two)
          issue_stage<true, true>(S, slot, tmem, id, steps, kb == 0);
        else if (few)
          issue_stage<true, false>(S, slot, tmem, id, steps, kb == 0);
        else if (two)
          issue_stage<false, true>(S, slot, tmem, id, steps, kb == 0);
        else
          issue_stage<false, false>(S, slot, tmem, id, steps, kb == 0);
        mma_commit(&S.empty[slot]);
        if (kb == kbs - 1) mma_commit(&S.acc_full);
      }
      __syncwarp();
    }
    if (!tiles.ok) break;
  }
  if (!tiles.ok && lane == 0) fail(S, a);
  // tensor memory is given back only after the last MMA
  if (elect_one()) {
    mma_commit(&S.drain);
    const uint64_t t0 = gtime();
    while (!mbar_poll(&S.drain, 0))
      if (gtime() - t0 > kWaitNs) break;
  }
  __syncwarp();
}

// Tokens' rows of a stage: eight lanes have a row's 128 bytes; the 16-byte piece c
// of row r goes to c ^ (r % 8), as the swizzle has it.  places: of the rows 4 warp
// + lane / 8 + 16 i, in pieces from the codes' beginning; ~0: none.
__device__ __forceinline__ void row_places(const ProductArgs &a, const TileInfo &t, int row0,
                                           uint32_t (&places)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int x = t.row[row0 + 16 * i];
    places[i] = x >= 0 ? (uint32_t)x * (uint32_t)(a.K / 32) : ~0u;
  }
}
__device__ __forceinline__ void copy_rows(const ProductArgs &a, uint8_t *dst, int row0, int kb,
                                          const uint32_t (&places)[8]) {
  const int piece = threadIdx.x & 7, from = kb * 128 + piece * 16, len = a.K / 2;
  const uint8_t *src = a.xcodes + (from < len ? from : 0);
  const uint32_t to = smem_addr(dst) + row0 * 128 + ((piece ^ (row0 & 7)) << 4);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (places[i] != ~0u)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + i * 2048),
                   "l"(src + (uint64_t)places[i] * 16), "r"(from < len ? 16 : 0)
                   : "memory");
}

// Warps 4-7 with scales by TMA: a thread turns line = 8 warp + lane / 4 of step
// lane % 4, the words of the rows line, line + 32, + 64, + 96, of each operand.
// Tokens' scales come by a load for each row, a stage ahead.
template <bool kPair>
__device__ void turner(const ProductArgs &a, Smem &S) {
  const int warp = (threadIdx.x >> 5) - kCopyWarp0, lane = threadIdx.x & 31;
  const int line = 8 * warp + (lane >> 2), step = lane & 3;
  const int row0 = 4 * warp + (lane >> 3);
  const int pitch = a.K / 16, kbs = a.K / 256;
  uint32_t s = 0;
  Tiles tiles(S, true);
  while (const TileInfo *t = tiles.next()) {
    const int words = (t->rows + 31) / 32;
    uint32_t places[8];
    const uint8_t *own = nullptr;   // the scales of row line + 32 step: words `step` of its line
    uint4 ahead = make_uint4(0, 0, 0, 0);
    if (a.by_token) {
      row_places(a, *t, row0, places);
      const int x = t->row[line + 32 * step];
      if (x >= 0) {
        own = a.xscale + (int64_t)x * pitch;
        ahead = *reinterpret_cast<const uint4 *>(own);
      }
    }
    tiles.done();
    for (int kb = 0; kb < kbs; ++kb, ++s) {
      const int slot = s % kStages;
      const uint4 x = ahead;
      if (own && kb + 1 < kbs) ahead = *reinterpret_cast<const uint4 *>(own + 16 * kb + 16);
      if (s >= kStages && !wait_all(S, &S.empty[slot], (s / kStages - 1) & 1)) {
        tiles.ok = false;
        break;
      }
      if (a.by_token) {
        copy_rows(a, S.codes[slot] + 2 * kOperand, row0, kb, places);
        copies_arrive(&S.full[slot]);
      }
      if (!wait_all(S, &S.raw_full[slot], (s / kStages) & 1)) {
        tiles.ok = false;
        break;
      }
      const uint8_t *from = S.raw[slot] + line * 16 + step * 4;
      uint8_t *to = S.scales[slot] + line * 16;
      auto turn = [&](const uint8_t *p, uint8_t *q) {
        uint4 v;
        v.x = *reinterpret_cast<const uint32_t *>(p);
        v.y = *reinterpret_cast<const uint32_t *>(p + 512);
        v.z = *reinterpret_cast<const uint32_t *>(p + 1024);
        v.w = *reinterpret_cast<const uint32_t *>(p + 1536);
        *reinterpret_cast<uint4 *>(q) = v;
      };
      turn(from, to + step * kWeightPitch);
      turn(from + kRawScales, to + step * kWeightPitch + kHalfPitch);
      uint8_t *xto = to + 4 * kWeightPitch;
      if (!a.by_token) {
        turn(from + 2 * kRawScales, xto + step * kRowPitch);
      } else if (step < words) {
        *reinterpret_cast<uint32_t *>(xto + 4 * step) = x.x;
        *reinterpret_cast<uint32_t *>(xto + 4 * step + kRowPitch) = x.y;
        *reinterpret_cast<uint32_t *>(xto + 4 * step + 2 * kRowPitch) = x.z;
        *reinterpret_cast<uint32_t *>(xto + 4 * step + 3 * kRowPitch) = x.w;
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&S.full[slot]);
        mbar_arrive(&S.raw_empty[slot]);
      }
    }
    if (!tiles.ok) break;
  }
  if (!tiles.ok && lane == 0) fail(S, a);
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// The 16 bytes of a row's scales from byte `at` (even) of an array of `total` on,
// `have` of them in the row (0 or less: none) and zeros behind, out of the two
// aligned pieces around them.
__device__ __forceinline__ uint4 load_scales(const uint8_t *base, int64_t at, int have,
                                             int64_t total) {
  const int64_t piece = at & ~(int64_t)15;
  const int off = (int)(at & 15), need = off + min(have, 16);
  uint32_t w[8];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    uint4 v = make_uint4(0, 0, 0, 0);
    const int64_t p = piece + 16 * q;
    if (have > 0 && 16 * q < need) {
      if (p + 16 <= total) {
        v = *reinterpret_cast<const uint4 *>(base + p);
      } else {   // the array's last bytes
        uint32_t b[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (p + 2 * i < total)
            b[i / 2] |= (uint32_t)*reinterpret_cast<const uint16_t *>(base + p + 2 * i)
                        << (16 * (i & 1));
        v = make_uint4(b[0], b[1], b[2], b[3]);
      }
    }
    w[4 * q] = v.x;
    w[4 * q + 1] = v.y;
    w[4 * q + 2] = v.z;
    w[4 * q + 3] = v.w;
  }
#pragma unroll
  for (int d = 2; d > 0; d >>= 1) {
    const bool down = off & (4 * d);
#pragma unroll
    for (int i = 0; i + d < 8; ++i) w[i] = down ? w[i + d] : w[i];
  }
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = __funnelshift_r(w[i], w[i + 1], (off & 2) * 8);
    const int left = have - 4 * i;
    v[i] = left >= 4 ? x : left < 2 ? 0 : x & 0xFFFFu;
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// Warps 4-7 with scales of other widths.  Whole words (k a multiple of 64): a
// thread copies those of one step of 64 k (its lane % 4), so that four lanes read
// 16 neighbouring bytes of a row, of 4 rows of each operand's 128.  Else a thread
// loads the 16 bytes of a row of each operand.
template <bool kPair>
__device__ void copier(const ProductArgs &a, Smem &S) {
  const int warp = (threadIdx.x >> 5) - kCopyWarp0, lane = threadIdx.x & 31;
  const bool words = a.K % 64 == 0;
  // the step, word and line of what is stored first
  const int step = words ? lane & 3 : 0, j = words ? (lane >> 2) & 3 : lane & 3;
  const int line = words ? (lane >> 4) + 8 * warp : 8 * warp + (lane >> 2);
  const int first = 32 * j + line, row0 = 4 * warp + (lane >> 3);
  const int pitch = a.K / 16, kbs = (a.K + 255) / 256;
  uint32_t s = 0;
  Tiles tiles(S, true);
  while (const TileInfo *t = tiles.next()) {
    const int rows = t->rows;
    int64_t w[2];
    int left[2], xs[4];
    uint32_t places[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int f = feature_of<kPair>(t->m, h) + first;
      w[h] = ((int64_t)t->e * a.R + f) * pitch + 4 * step;
      left[h] = a.R - f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) xs[i] = i == 0 || words ? t->row[first + 2 * i] : -1;
    if (a.by_token) row_places(a, *t, row0, places);
    tiles.done();
    for (int kb = 0; kb < kbs; ++kb, ++s) {
      const int slot = s % kStages, have = pitch - 16 * kb - 4 * step;
      uint4 v[3];
      if (!words) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          v[h] = load_scales(a.wscale[h], w[h] + 16 * kb, left[h] > 0 ? have : 0,
                             (int64_t)a.E * a.R * pitch);
        v[2] = load_scales(a.xscale, (int64_t)xs[0] * pitch + 16 * kb, xs[0] >= 0 ? have : 0,
                           (int64_t)a.x_rows * pitch);
      }
      if (s >= kStages && !wait_all(S, &S.empty[slot], (s / kStages - 1) & 1)) {
        tiles.ok = false;
        break;
      }
      if (a.by_token) copy_rows(a, S.codes[slot] + 2 * kOperand, row0, kb, places);
      uint8_t *dst = S.scales[slot] + line * 16 + j * 4;
      if (words) {
        auto copy = [&](uint8_t *to, const uint8_t *p, bool there) {
          copy_async<4>(smem_addr(to), there ? p : a.wscale[0], there);
        };
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            copy(dst + step * kWeightPitch + h * kHalfPitch + i * 32,
                 a.wscale[h] + w[h] + (int64_t)(2 * i) * pitch + 16 * kb,
                 2 * i < left[h] && have > 0);
        if (32 * j < rows) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            copy(dst + 4 * kWeightPitch + step * kRowPitch + i * 32,
                 a.xscale + (int64_t)xs[i] * pitch + 4 * step + 16 * kb, xs[i] >= 0 && have > 0);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 3; ++h) {
          uint8_t *to = dst + (h < 2 ? h * kHalfPitch : 4 * kWeightPitch);
          const int next = h < 2 ? kWeightPitch : kRowPitch;
          *reinterpret_cast<uint32_t *>(to) = v[h].x;
          *reinterpret_cast<uint32_t *>(to + next) = v[h].y;
          *reinterpret_cast<uint32_t *>(to + 2 * next) = v[h].z;
          *reinterpret_cast<uint32_t *>(to + 3 * next) = v[h].w;
        }
      }
      // the copies' own arrival, and this thread's for what it stored itself
      copies_arrive(&S.full[slot]);
      mbar_arrive(&S.full[slot]);
    }
    if (!tiles.ok) break;
  }
  if (!tiles.ok && lane == 0) fail(S, a);
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// silu(g) * u, from e = e^-|g|: the denominator 1 + e is in [1, 2], where the fast
// reciprocal is right to a unit, and gates far below zero end where fp32's exponential
// does.  (g / (1 + e^-g) by the fast division is 0 from -87.3 on, and took the gate and
// up of 4096 rows 81.0 us instead of 80.1; with e^-64 taken out of far gates 97.)
__device__ __forceinline__ float silu_times(float g, float u) {
  const float e = expf(-fabsf(g));
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return (g < 0.f ? g * e : g) * r * u;
}

template <typename T>
__device__ __forceinline__ void store_one(void *out, int64_t at, float v) {
  using TB = typename T::bits;
  if constexpr (sizeof(TB) == 2)
    static_cast<uint16_t *>(out)[at] = (uint16_t)(T::down2(v, 0.f) & 0xFFFFu);
  else
    static_cast<float *>(out)[at] = v;
}

// A lane's 32 neighbouring outputs of its row (in floats) to the warp's staging
// rows of 128 bytes, `half` saying which half of a row of 16-bit ones; piece c
// of row r goes to c ^ (r % 8), so that neither side of the exchange has bank
// conflicts.  (Straight to global memory, a warp's store is 32 rows of 32 bytes:
// that took the stores' pipe 125 clocks and held up every other copy; down of
// 8192 rows 390 us, staged 310.)
template <typename T>
__device__ __forceinline__ void stage_outputs(uint8_t *rows, int lane, int half,
                                              const uint32_t (&v)[32]) {
  constexpr int ES = sizeof(typename T::bits), PIECES = 32 * ES / 16;
#pragma unroll
  for (int c = 0; c < PIECES; ++c) {
    uint4 q;
    if constexpr (ES == 2) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = T::down2(__uint_as_float(v[8 * c + 2 * j]), __uint_as_float(v[8 * c + 2 * j + 1]));
      q = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      q = make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
    }
    *reinterpret_cast<uint4 *>(rows + lane * 128 +
                               (((half * PIECES + c) ^ (lane & 7)) << 4)) = q;
  }
}
// The staged rows (those of `real`) to positions p.. of the output from feature
// f on: whole lines of 128 bytes where rows allow 16-byte pieces.
template <typename T>
__device__ __forceinline__ void store_staged(const ProductArgs &a, const uint8_t *rows, int lane,
                                             uint32_t real, int p, int f) {
  using TB = typename T::bits;
  constexpr int ES = sizeof(TB), N = 128 / ES, PER = 16 / ES;
  __syncwarp();
  if (a.align >= 16) {
    const int c = lane & 7, first = f + c * PER;
    TB *dst = static_cast<TB *>(a.out) + (int64_t)p * a.R + first;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + (lane >> 3);
      const uint4 q = *reinterpret_cast<const uint4 *>(rows + r * 128 + ((c ^ (r & 7)) << 4));
      if ((real >> r & 1) && first < a.R)
        *reinterpret_cast<uint4 *>(dst + (int64_t)r * a.R) = q;
    }
  } else {
    for (int r = 0; r < 32; ++r) {
      if (!(real >> r & 1)) continue;
      for (int e = lane; e < N && f + e < a.R; e += 32)
        static_cast<TB *>(a.out)[(int64_t)(p + r) * a.R + f + e] = *reinterpret_cast<const TB *>(
            rows + r * 128 + (((e / PER) ^ (r & 7)) << 4) + e % PER * ES);
    }
  }
  __syncwarp();
}

template <typename T, bool kPair>
__device__ void epilogue(const ProductArgs &a, Smem &S, uint32_t tmem) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = warp & 3;
  const int group = (warp - kEpi0) >> 2;
  const uint32_t base = tmem + ((uint32_t)(q * 32) << 16);
  Tiles tiles(S, true);
  while (const TileInfo *t = tiles.next()) {
    const int rows = t->rows, m = t->m, p0 = t->p0;
    const bool few = rows <= kFewRows;
    const float g0 = a.wglobal[0][t->e], g1 = a.wglobal[1][t->e];
    // this lane's row (of few: of the group's columns), its global scale
    const int i = few ? group * 16 + (lane & 15) : q * 32 + lane, x = t->row[i];
    const float xg = x >= 0 ? a.xglobal[x] : 0.f;
    const uint32_t real = __ballot_sync(kFull, x >= 0);
    if (!wait_all(S, &S.acc_full, tiles.n & 1)) {
      tiles.ok = false;
      break;
    }
    tc_fence_after();
    if (few) {
      // lanes are features, columns rows: 16 of them for each group
      const int c0 = group * 16;
      uint32_t v0[16], v1[16];
      if (c0 < rows) {
        tmem_ld16(base + c0, v0);
        tmem_ld16(base + kTileCols + c0, v1);
        tmem_wait_ld();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.acc_empty);
      const int f0 = feature_of<kPair>(m, 0) + q * 32 + lane;
      const int f1 = feature_of<kPair>(m, 1) + q * 32 + lane;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const float xc = __shfl_sync(kFull, xg, c);
        if (!(real >> c & 1)) continue;
        const int64_t at = (int64_t)(p0 + c0 + c) * a.R;
        const float y0 = __uint_as_float(v0[c]) * xc * g0, y1 = __uint_as_float(v1[c]) * xc * g1;
        if constexpr (kPair) {
          if (f0 < a.R) store_one<T>(a.out, at + f0, silu_times(y0, y1));
        } else {
          if (f0 < a.R) store_one<T>(a.out, at + f0, y0);
          if (f1 < a.R) store_one<T>(a.out, at + f1, y1);
        }
      }
      tiles.done();
      continue;
    }
    // lanes are rows, columns features: 128 for each group (64 of gate and of up)
    tiles.done();
    uint32_t v[4][32];
    if (q * 32 < rows) {
#pragma unroll
      for (int h = 0; h < 4; ++h)
        tmem_ld32(base + (kPair ? (h >> 1) * kTileCols + group * 64 + (h & 1) * 32
                                : group * kTileCols + h * 32),
                  v[h]);
      tmem_wait_ld();
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.acc_empty);
    if (!real) continue;   // none of the warp's rows
    uint8_t *staged = S.staged[warp - kEpi0];
    constexpr int H = sizeof(typename T::bits) == 2 ? 2 : 1;   // parts of 32 in 128 bytes
#pragma unroll
    for (int h = 0; h < (kPair ? 2 : 4); ++h) {
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        const float y = __uint_as_float(v[h][c]) * xg * g0;
        if constexpr (kPair)
          v[h][c] = __float_as_uint(silu_times(y, __uint_as_float(v[2 + h][c]) * xg * g1));
        else
          v[h][c] = __float_as_uint(y);
      }
      stage_outputs<T>(staged, lane, h % H, v[h]);
      if (h % H == H - 1)
        store_staged<T>(a, staged, lane, real, p0 + q * 32,
                        (kPair ? m * 128 + group * 64 : m * 256 + group * 128) +
                            (h - h % H) * 32);
    }
  }
  if (!tiles.ok && lane == 0) fail(S, a);
}

template <typename T, bool kPair, bool kTmaScales>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_nvfp4_kernel(const __grid_constant__ ProductArgs a,
                         const __grid_constant__ ProductMaps maps) {
  extern __shared__ uint8_t raw[];
  Smem &S = *reinterpret_cast<Smem *>(raw + ((1024 - (smem_addr(raw) & 1023)) & 1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      // the TMA copies; scales by TMA: each warp that turns them, and each thread
      // that copies tokens' rows; else every copying thread, twice (copier)
      mbar_init(&S.full[i], kTmaScales ? 1 + 4 + (a.by_token ? 128 : 0) : 1 + 256);
      mbar_init(&S.empty[i], 1);
      mbar_init(&S.raw_full[i], 1);
      mbar_init(&S.raw_empty[i], 4);
    }
    for (int i = 0; i < kInfos; ++i) {
      mbar_init(&S.info_place[i], 1);
      mbar_init(&S.info_rows[i], 1);
      mbar_init(&S.info_empty[i], 2 + kTmaScales + 4 + kEpiWarps);
    }
    mbar_init(&S.acc_full, 1);
    mbar_init(&S.acc_empty, kEpiWarps);
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
  if (warp == 0 && lane < (kPair ? 2 : 1)) prefetch_tensormap(&maps.w[lane]);
  if (warp == 3 && kTmaScales && lane < (kPair ? 2 : 1)) prefetch_tensormap(&maps.ws[lane]);
  if (warp == 3 && !a.by_token && lane >= 8 && lane < 10) prefetch_tensormap(&maps.x[lane - 8]);
  if (warp == 3 && !a.by_token && kTmaScales && lane == 10) prefetch_tensormap(&maps.xs);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem;
  pdl_wait();
  pdl_trigger();

  if (warp >= kEpi0) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    epilogue<T, kPair>(a, S, tmem);
  } else if (warp >= kCopyWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCopyRegs));
    if constexpr (kTmaScales)
      turner<kPair>(a, S);
    else
      copier<kPair>(a, S);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (warp == 0)
      producer<kPair>(a, maps, S);
    else if (warp == 1)
      mma_issuer<kPair>(a, S, tmem);
    else if (warp == 2)
      scheduler(a, S, lay_out_tiles(a, S));
    else if (kTmaScales)
      scale_producer<kPair>(a, maps, S);
  }

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

constexpr size_t kSmemBytes = sizeof(Smem) + 1024;   // with its alignment
static_assert(kSmemBytes <= 227 * 1024, "shared memory of a CTA");

template <typename T, bool kPair, bool kTmaScales>
int launch_grouped(const ProductArgs &a, const ProductMaps &maps, dim3 grid, void *stream) {
  const auto kernel = grouped_nvfp4_kernel<T, kPair, kTmaScales>;
  if (const int st = ensure_smem_limit((const void *)kernel, kSmemBytes)) return st;
  // A warpgroup that asks for registers waits until the others have given up
  // theirs: a kernel that was built with fewer at launch must not run.  (Looked
  // up until known: a property of the program, the same on every device.)
  static std::atomic<int> regs{0};
  if (regs.load(std::memory_order_relaxed) != kLaunchRegs) {
    cudaFuncAttributes attr;
    const cudaError_t e = cudaFuncGetAttributes(&attr, (const void *)kernel);
    if (e != cudaSuccess) {
      set_last_cuda_error(e);
      return MOE_ECUDA;
    }
    if (attr.numRegs != kLaunchRegs) return MOE_EUNSUPPORTED;
    regs.store(attr.numRegs, std::memory_order_relaxed);
  }
  return launch_pdl(kernel, grid, dim3(kThreads), kSmemBytes, stream, a, maps);
}

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
  a.per_k = top_k == 1 ? 0 : (uint32_t)(((uint64_t)1 << 32) / top_k + ((((uint64_t)1 << 32) % top_k) != 0));
  a.n = M * top_k;
  a.num_rows = num_rows;
  a.x_rows = by_token ? M : num_rows;
  a.feature_tiles = w1 ? (R + 127) / 128 : (R + 255) / 256;
  a.offsets = offsets;
  a.sti = sti;
  for (int j = 0; j < 2; ++j) {
    a.wscale[j] = static_cast<const uint8_t *>(w[j]->scale);
    a.wglobal[j] = w[j]->global_scale;
  }
  a.xcodes = codes;
  a.xscale = scale;
  a.xglobal = global;
  a.out = out;
  const uint64_t v = (uint64_t)(uintptr_t)out | (uint64_t)R * eb | 16;
  a.align = (int)(v & (~v + 1));
  a.err = err;
  ProductMaps maps;
  memset(&maps, 0, sizeof(maps));
  const cuuint64_t pitch[1] = {(cuuint64_t)K / 2};
  const cuuint64_t wd[2] = {(cuuint64_t)K / 2, (cuuint64_t)E * R};
  const cuuint64_t xd[2] = {(cuuint64_t)K / 2, (cuuint64_t)a.x_rows};
  const cuuint32_t half = w1 ? 128 : 256;   // weight rows of a copy
  const cuuint32_t wbox[2] = {128, half}, xbox[2][2] = {{128, 32}, {128, 128}};
  const cuuint64_t spitch[1] = {(cuuint64_t)K / 16};
  const cuuint64_t wsd[2] = {(cuuint64_t)K / 16, wd[1]}, xsd[2] = {(cuuint64_t)K / 16, xd[1]};
  const cuuint32_t wsbox[2] = {16, half}, xsbox[2] = {16, 128};
  const bool tma_scales = K % 256 == 0;
  for (int j = 0; j < (w1 ? 2 : 1); ++j) {
    if (const int st = encode_u8_sw128(&maps.w[j], w[j]->codes, 2, wd, pitch, wbox)) return st;
    if (tma_scales)
      if (const int st = encode_u8_plain(&maps.ws[j], w[j]->scale, 2, wsd, spitch, wsbox))
        return st;
  }
  if (!by_token) {   // tokens' rows are copied by threads
    for (int j = 0; j < 2; ++j)
      if (const int st = encode_u8_sw128(&maps.x[j], codes, 2, xd, pitch, xbox[j])) return st;
    if (tma_scales)
      if (const int st = encode_u8_plain(&maps.xs, scale, 2, xsd, spitch, xsbox)) return st;
  }

  // an upper bound of the tiles: experts have at most a tile more than whole ones
  const int64_t slots = a.n < E ? a.n : E;
  const int64_t most = (num_rows / kTileRows + slots) * a.feature_tiles;
  const dim3 grid((unsigned)(most < sms ? most : sms));
  auto go = [&](auto t, auto pair) {
    using T = decltype(t);
    constexpr bool P = decltype(pair)::value;
    return tma_scales ? launch_grouped<T, P, true>(a, maps, grid, stream)
                      : launch_grouped<T, P, false>(a, maps, grid, stream);
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
