// block.cu -- the expert half of a transformer block in one call: residual
// addition and norm, then the decode layer on the normed rows.
#include "common.cuh"

namespace moe {
int check_layer_call(const moe_layer_desc *layer, const uint16_t *x, int M,
                     const float *router_logits, const int32_t *topk_ids, const float *topk_w,
                     const uint16_t *out, moe_workspace_view *v);
int check_add_rmsnorm(const void *x, int64_t x_stride, const void *residual,
                      int64_t residual_stride, const void *weight, int dtype, int weight_dtype,
                      int M, int hidden, float eps, const void *sum_out, const void *out,
                      const uint8_t *out_codes, const float *out_scale, const float *rstd);
}  // namespace moe

extern "C" int moe_decode_block(const moe_layer_desc *layer, const uint16_t *x,
                                const uint16_t *residual, const uint16_t *norm_weight, float eps,
                                int M, uint16_t *sum_out, uint16_t *normed, uint16_t *out,
                                void *workspace, size_t workspace_bytes, uint32_t *err_word,
                                void *stream) {
  // every host check of both halves first: a rejected call enqueues nothing
  moe_workspace_view v;
  int st = moe::check_layer_call(layer, normed, M, nullptr, nullptr, nullptr, out, &v);
  if (st) return st;
  if (!workspace || workspace_bytes < v.total_bytes || ((uintptr_t)workspace & 255))
    return MOE_EINVAL;
  if (!sum_out || normed == out || normed == sum_out || out == sum_out) return MOE_EINVAL;
  const int H = layer->routed.hidden;
  st = moe::check_add_rmsnorm(x, H, residual, H, norm_weight, MOE_DTYPE_BF16, MOE_DTYPE_BF16, M, H,
                              eps, sum_out, normed, nullptr, nullptr, nullptr);
  if (st) return st;
  st = moe_add_rmsnorm(x, H, residual, H, norm_weight, MOE_DTYPE_BF16, MOE_DTYPE_BF16, M, H, eps,
                       sum_out, normed, nullptr, nullptr, nullptr, stream);
  if (st) return st;
  return moe_decode_layer(layer, normed, M, nullptr, nullptr, nullptr, out, workspace,
                          workspace_bytes, err_word, stream);
}
