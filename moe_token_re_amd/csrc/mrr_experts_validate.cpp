// mrr_experts_validate.cpp -- the host-side argument checks of the experts'
// operators (4-bit quantisation, grouped product, few-token layer). No HIP
// header and no HIP call: every check runs, and is tested, without a GPU.
// Pointers are compared and tested for alignment, never dereferenced.
#include "mrr_checks.h"
#include "mrr_experts.h"

namespace mrr {

mrr_status check_mx(const mrr_mx_args* a, bool quantize) {
  if (a == nullptr) return MRR_ERROR_INVALID_VALUE;
  const int w = wide_bytes(a->wide_dtype);
  if (w == 0) return MRR_ERROR_UNSUPPORTED_DTYPE;
  if (a->rows < 0 || a->H <= 0 || a->H >= (int64_t(1) << 24) || a->H % 2 != 0 || !fits(a->rows, a->H, w))
    return MRR_ERROR_INVALID_SHAPE;
  if (a->rows == 0) return MRR_SUCCESS;
  if (a->wide == nullptr || a->packed == nullptr || a->scales == nullptr) return MRR_ERROR_INVALID_VALUE;
  if (!aligned(a->wide, w)) return MRR_ERROR_MISALIGNED;
  Buffers b;
  b.add(a->wide, a->rows * a->H * w, !quantize);
  b.add(a->packed, a->rows * (a->H / 2), quantize);
  b.add(a->scales, a->rows * mx_scale_bytes(a->H), quantize);
  return b.clash() ? MRR_ERROR_INVALID_VALUE : MRR_SUCCESS;
}

mrr_status check_grouped_mm(const mrr_grouped_mm_args* a, const void* ws, size_t ws_bytes) {
  if (a == nullptr) return MRR_ERROR_INVALID_VALUE;
  const int w = wide_bytes(a->out_dtype);
  if (w == 0 || (a->counts_dtype != MRR_I32 && a->counts_dtype != MRR_I64)) return MRR_ERROR_UNSUPPORTED_DTYPE;
  const int cb = a->counts_dtype == MRR_I64 ? 8 : 4;
  if (a->expert_token_num_type != 0 && a->expert_token_num_type != 1) return MRR_ERROR_INVALID_VALUE;
  if (a->gated != 0 && a->gated != 1) return MRR_ERROR_INVALID_VALUE;
  const int64_t most = int64_t(1) << 20;
  if (a->A < 0 || a->A > INT32_MAX || a->K <= 0 || a->K >= most || a->K % 32 != 0 || a->N <= 0 || a->N >= most ||
      (a->gated == 1 && a->N % 2 != 0) || a->E < 0 || a->E > 4096 || (a->E == 0 && a->A != 0))
    return MRR_ERROR_INVALID_SHAPE;
  if (a->E > 0 && a->expert_token_num == nullptr) return MRR_ERROR_INVALID_VALUE;
  if (a->A > 0 && (a->tokens == nullptr || a->token_scales == nullptr || a->weight == nullptr ||
                   a->weight_scales == nullptr || a->out == nullptr))
    return MRR_ERROR_INVALID_VALUE;
  if ((ws == nullptr) != (ws_bytes == 0)) return MRR_ERROR_INVALID_VALUE;
  if (!aligned(a->tokens, 16) || !aligned(a->weight, 16) || !aligned(a->expert_token_num, cb) ||
      !aligned(a->row_weight, 4) || !aligned(a->out, w) || !aligned(ws, 16))
    return MRR_ERROR_MISALIGNED;
  if (ws != nullptr && ws_bytes < MRR_GROUPED_MM_WORKSPACE_BYTES) return MRR_ERROR_WORKSPACE_TOO_SMALL;
  const int64_t sb = mx_scale_bytes(a->K);
  Buffers b;
  b.add(a->tokens, a->A * (a->K / 2), false);
  b.add(a->token_scales, a->A * sb, false);
  if (a->A > 0) b.add(a->weight, a->E * a->N * (a->K / 2), false);
  if (a->A > 0) b.add(a->weight_scales, a->E * a->N * sb, false);
  b.add(a->expert_token_num, a->E * cb, false);
  b.add(a->row_weight, a->A * 4, false);
  b.add(a->out, a->A * (a->gated ? a->N / 2 : a->N) * w, true);
  b.add(ws, static_cast<int64_t>(MRR_GROUPED_MM_WORKSPACE_BYTES), true);
  return b.clash() ? MRR_ERROR_INVALID_VALUE : MRR_SUCCESS;
}

mrr_status check_few_tokens(const mrr_few_tokens_args* a, const void* ws, size_t ws_bytes) {
  if (a == nullptr) return MRR_ERROR_INVALID_VALUE;
  if (a->dtype != MRR_F16 && a->dtype != MRR_BF16) return MRR_ERROR_UNSUPPORTED_DTYPE;
  const bool mx = a->weights_dtype == MRR_F4_E2M1;
  // 4-bit values times their scale are exact in bf16 (of the two largest scales an
  // eighth of them is), and beyond the range of fp16
  if (mx ? a->dtype != MRR_BF16 : a->weights_dtype != a->dtype) return MRR_ERROR_UNSUPPORTED_DTYPE;
  if (a->renormalize != 0 && a->renormalize != 1) return MRR_ERROR_INVALID_VALUE;
  if (a->T < 0 || a->T > MRR_FEW_TOKENS_MAX || a->H <= 0 || a->H > 65536 || a->H % 32 != 0 || a->I <= 0 ||
      a->I > 65536 || a->I % 32 != 0 || a->E <= 0 || a->E > kFewMaxExperts || a->top_k < 1 ||
      a->top_k > kFewMaxTopK)
    return MRR_ERROR_INVALID_SHAPE;
  // logits choose among these experts; ids may name other ranks' as well
  if (a->router_logits != nullptr && a->top_k > a->E) return MRR_ERROR_INVALID_SHAPE;
  if ((a->router_logits == nullptr) == (a->expert_ids == nullptr) && a->T > 0) return MRR_ERROR_INVALID_VALUE;
  if ((a->expert_ids == nullptr) != (a->expert_weight == nullptr)) return MRR_ERROR_INVALID_VALUE;
  if (a->gate_up == nullptr || a->down == nullptr) return MRR_ERROR_INVALID_VALUE;
  if (mx != (a->gate_up_scales != nullptr) || mx != (a->down_scales != nullptr)) return MRR_ERROR_INVALID_VALUE;
  if (a->T > 0 && (a->x == nullptr || a->y == nullptr || ws == nullptr)) return MRR_ERROR_INVALID_VALUE;
  if (!aligned(a->x, 16) || !aligned(a->gate_up, 16) || !aligned(a->down, 16) || !aligned(a->router_logits, 4) ||
      !aligned(a->expert_ids, 4) || !aligned(a->expert_weight, 4) || !aligned(a->y, 2) || !aligned(ws, 16))
    return MRR_ERROR_MISALIGNED;
  if (a->T > 0 && ws_bytes < mrr_few_tokens_workspace_size(a->T, a->top_k, a->I)) return MRR_ERROR_WORKSPACE_TOO_SMALL;
  Buffers b;
  b.add(a->x, a->T * a->H * 2, false);
  b.add(a->router_logits, a->T * a->E * 4, false);
  b.add(a->expert_ids, a->T * a->top_k * 4, false);
  b.add(a->expert_weight, a->T * a->top_k * 4, false);
  b.add(a->gate_up, mx ? a->E * a->I * a->H : a->E * a->I * a->H * 4, false);
  b.add(a->down, mx ? a->E * a->I * a->H / 2 : a->E * a->I * a->H * 2, false);
  b.add(a->gate_up_scales, a->E * a->I * 2 * mx_scale_bytes(a->H), false);
  b.add(a->down_scales, a->E * a->H * mx_scale_bytes(a->I), false);
  b.add(a->y, a->T * a->H * 2, true);
  if (a->T > 0) b.add(ws, static_cast<int64_t>(mrr_few_tokens_workspace_size(a->T, a->top_k, a->I)), true);
  return b.clash() ? MRR_ERROR_INVALID_VALUE : MRR_SUCCESS;
}

}  // namespace mrr

extern "C" mrr_status mrr_grouped_mm_validate(const mrr_grouped_mm_args* args, const void* workspace,
                                              size_t workspace_bytes) {
  return mrr::check_grouped_mm(args, workspace, workspace_bytes);
}

extern "C" mrr_status mrr_few_tokens_validate(const mrr_few_tokens_args* args, const void* workspace,
                                              size_t workspace_bytes) {
  return mrr::check_few_tokens(args, workspace, workspace_bytes);
}

extern "C" size_t mrr_few_tokens_workspace_size(int64_t T, int64_t top_k, int64_t I) {
  if (T < 0 || T > MRR_FEW_TOKENS_MAX || top_k < 1 || top_k > mrr::kFewMaxTopK || I <= 0 || I > 65536) return 0;
  return mrr::few_layout(T, top_k, I).bytes;
}
