// route_grad.cu -- the gradient of the per-row top-k softmax
// (moe_topk_softmax_backward).
#include "common.cuh"

namespace moe {
namespace {

// The weights of a row are w_j = exp(l_j) / sum_i exp(l_i) over its k selected
// logits, so dl_j = w_j * (dw_j - sum_i w_i * dw_i), and every other logit's
// gradient is zero.  A warp takes 32 / G rows of G lanes, G the power of two
// from k up: lane j of a row owns slot j, a butterfly over the row's lanes
// sums w * dw.  The warp's rows are one run of floats: it clears the run in
// 16-byte pieces and then writes the k values of each row.  An id that stands
// twice in a row gets the sum of its slots' values, slots ascending.
// M = 32768, E = 256, k = 8 (37 MB) takes 7.9 us where a plain fill of the M * E
// floats takes 6.0: the writes, which stay in the L2, and on top of them the
// rows' shuffles and matches and the values written over the zeros (the largest
// stall is MIO throttle).  M = 8, E = 128: a launch, 1.6 us.
constexpr int kWarps = 4;

__global__ void __launch_bounds__(32 * kWarps) topk_softmax_grad_kernel(
    const int32_t *ids, const float *w, const float *dw, int M, int E, int k, int lanes,
    float *dlogits, uint32_t *err) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, rows = 32 / lanes, slot = lane % lanes, sub = lane / lanes;
  const int64_t row0 = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * rows;
  if (row0 >= M) return;
  const int64_t row = row0 + sub;
  const bool on = row < M && slot < k;
  int id = -1;
  float wv = 0.f, dv = 0.f;
  if (on) {
    const size_t at = (size_t)row * k + slot;
    id = __ldcg(ids + at);
    wv = __ldcg(w + at);
    dv = __ldcg(dw + at);
  }
  {
    float *p = dlogits + row0 * E;
    const int64_t n = (M - row0 < rows ? M - row0 : rows) * E;
    const int64_t ahead = (-(int64_t)((uintptr_t)p >> 2)) & 3;   // floats to a 16-byte boundary
    const int64_t head = ahead < n ? ahead : n, quads = (n - head) / 4;
    if (lane < head) p[lane] = 0.f;
    for (int64_t i = lane; i < quads; i += 32)
      reinterpret_cast<float4 *>(p + head)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    const int64_t tail = head + 4 * quads + lane;
    if (tail < n) p[tail] = 0.f;
  }
  if (on && (id < 0 || id >= E)) {
    // a slot that went to no expert: its weight counts in the sum, its logit
    // is none of the row's
    if (err) atomicOr(err, MOE_ERR_BAD_ID);
    id = -1;
  }
  float dot = on ? wv * dv : 0.f;
  for (int d = lanes >> 1; d > 0; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
  const float g = wv * (dv - dot);
  // lanes of the same row (E <= 1024 leaves the low 16 bits to the id)
  const unsigned same = __match_any_sync(0xffffffffu, (unsigned)sub << 16 | (id & 0xffff));
  float sum = g;
  if (__any_sync(0xffffffffu, id >= 0 && (same & (same - 1)))) {   // rare: an id stands twice
    const int first = sub * lanes;
    sum = 0.f;
    for (int j = 0; j < k; ++j) {
      const float v = __shfl_sync(0xffffffffu, g, first + j);
      if ((same >> (first + j)) & 1u) sum += v;
    }
  }
  __syncwarp();   // orders the zeros ahead of the values
  if (id >= 0 && lane == __ffs(same) - 1) dlogits[row * E + id] = sum;
}

}  // namespace
}  // namespace moe

extern "C" int moe_topk_softmax_backward(const int32_t *topk_ids, const float *topk_w,
                                         const float *dtopk_w, int M, int num_experts, int top_k,
                                         float *dlogits, uint32_t *err_word, void *stream) {
  if (M < 0 || num_experts < 1 || top_k < 1 || top_k > num_experts) return MOE_EINVAL;
  if (num_experts > MOE_MAX_EXPERTS || top_k > 32) return MOE_EUNSUPPORTED;
  if (M == 0) return MOE_OK;
  if (!topk_ids || !topk_w || !dtopk_w || !dlogits) return MOE_EINVAL;
  if (((uintptr_t)topk_ids | (uintptr_t)topk_w | (uintptr_t)dtopk_w | (uintptr_t)dlogits |
       (uintptr_t)err_word) & 3)
    return MOE_EINVAL;
  using namespace moe;
  int lanes = 1;
  while (lanes < top_k) lanes *= 2;
  return launch_pdl(topk_softmax_grad_kernel, dim3((unsigned)ceil_div64(M, kWarps * (32 / lanes))),
                    dim3(32 * kWarps), 0, stream, topk_ids, topk_w, dtopk_w, M, num_experts, top_k,
                    lanes, dlogits, err_word);
}
