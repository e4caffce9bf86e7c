// route_grad.cu -- the gradient of the per-row top-k softmax
// (moe_topk_softmax_backward).
#include "common.cuh"

namespace moe {
namespace {

// The weights of a row are w_j = exp(l_j) / sum_i exp(l_i) over its k selected
// logits, so dl_j = w_j * (dw_j - sum_i w_i * dw_i), and every other logit's
// gradient is zero.  One warp per row: lane j owns slot j, an xor butterfly
// sums w * dw, the warp writes the row's zeros and then its k values.  An id
// that stands twice in a row gets the sum of its slots' values, slots
// ascending.  Bound by the M * E floats it writes.
constexpr int kRowsPerCta = 4;

__global__ void __launch_bounds__(32 * kRowsPerCta) topk_softmax_grad_kernel(
    const int32_t *ids, const float *w, const float *dw, int M, int E, int k, float *dlogits,
    uint32_t *err) {
  pdl_wait();
  pdl_trigger();
  const int row = blockIdx.x * kRowsPerCta + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= M) return;
  const size_t at = (size_t)row * k + lane;
  int id = -1;
  float wv = 0.f, dv = 0.f;
  if (lane < k) {
    id = __ldcg(ids + at);
    wv = __ldcg(w + at);
    dv = __ldcg(dw + at);
    if (id < 0 || id >= E) {
      // a slot that went to no expert: its weight counts in the sum, its
      // logit is none of the row's
      if (err) atomicOr(err, MOE_ERR_BAD_ID);
      id = -1;
    }
  }
  float dot = lane < k ? wv * dv : 0.f;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
  const float g = wv * (dv - dot);
  const unsigned same = __match_any_sync(0xffffffffu, id);
  float sum = 0.f;
  for (int j = 0; j < k; ++j) {
    const float v = __shfl_sync(0xffffffffu, g, j);
    if ((same >> j) & 1u) sum += v;
  }
  float *out = dlogits + (size_t)row * E;
  for (int e = lane; e < E; e += 32) out[e] = 0.f;
  __syncwarp();   // orders the zeros ahead of the values
  if (id >= 0 && lane == __ffs(same) - 1) out[id] = sum;
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
  if (((uintptr_t)topk_ids | (uintptr_t)topk_w | (uintptr_t)dtopk_w | (uintptr_t)dlogits) & 3)
    return MOE_EINVAL;
  using namespace moe;
  return launch_pdl(topk_softmax_grad_kernel, dim3((unsigned)ceil_div64(M, kRowsPerCta)), dim3(32 * kRowsPerCta), 0, stream, topk_ids, topk_w, dtopk_w, M, num_experts,
                    top_k, dlogits, err_word);
}
