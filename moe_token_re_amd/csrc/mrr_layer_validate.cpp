// mrr_layer_validate.cpp -- the host-side argument checks of the operators
// around an expert layer (norm, router, rows by expert and back). No HIP header
// and no HIP call: every check runs, and is tested, without a GPU. Pointers are
// compared and tested for alignment, never dereferenced.
#include "mrr_layer.h"

#include "mrr_checks.h"

namespace mrr {
namespace {

constexpr int64_t kMostRows = INT32_MAX;

bool norm_sizes(int64_t rows, int64_t H) { return rows >= 0 && rows <= kMostRows && H > 0 && H <= kNormMaxH; }

// eps as a normal number of 32 bits: the norm's reciprocal stays in their range.
bool norm_eps(double eps) { return eps >= 0x1p-126 && eps < 0x1p127; }

bool router_sizes(int64_t T, int64_t E, int64_t top_k) {
  return T >= 0 && T <= kMostRows && E > 0 && E <= kRouterMaxExperts && top_k >= 1 && top_k <= kLayerMaxTopK &&
         top_k <= E;
}

bool choice_sizes(int64_t T, int64_t top_k) {
  return T >= 0 && top_k >= 1 && top_k <= kLayerMaxTopK && T <= (kMostRows - 1) / top_k;
}

int token_bits(int32_t dt) {
  switch (dt) {
    case MRR_F32: return 32;
    case MRR_F16:
    case MRR_BF16: return 16;
    case MRR_I8:
    case MRR_F8_E5M2:
    case MRR_F8_E4M3FN:
    case MRR_HIF8: return 8;
    case MRR_F4_E2M1:
    case MRR_F4_E1M2: return 4;
    default: return 0;
  }
}

}  // namespace

mrr_status check_rms_norm(const mrr_rms_norm_args* a) {
  if (a == nullptr) return MRR_ERROR_INVALID_VALUE;
  const int b = wide_bytes(a->dtype), w = wide_bytes(a->weight_dtype);
  if (b == 0 || (a->weight_dtype != a->dtype && a->weight_dtype != MRR_F32)) return MRR_ERROR_UNSUPPORTED_DTYPE;
  const bool wide = a->y_dtype == a->dtype;
  if (!wide) {
    const bool row = a->scales_dtype == MRR_F32 && (a->y_dtype == MRR_I8 || a->y_dtype == MRR_F8_E4M3FN);
    const bool mx = a->scales_dtype == MRR_F8_E8M0 && (a->y_dtype == MRR_F8_E4M3FN || a->y_dtype == MRR_F4_E2M1);
    if (!row && !mx) return MRR_ERROR_UNSUPPORTED_DTYPE;
  }
  const bool fp4 = a->y_dtype == MRR_F4_E2M1;
  if (!norm_sizes(a->rows, a->H) || (fp4 && a->H % 2 != 0)) return MRR_ERROR_INVALID_SHAPE;
  if (!norm_eps(a->eps)) return MRR_ERROR_INVALID_VALUE;
  if (a->rows == 0) return MRR_SUCCESS;
  if (a->x == nullptr || a->weight == nullptr || a->y == nullptr) return MRR_ERROR_INVALID_VALUE;
  if (wide != (a->scales == nullptr) || (a->residual == nullptr) != (a->sum == nullptr)) return MRR_ERROR_INVALID_VALUE;
  const bool f32_scales = !wide && a->scales_dtype == MRR_F32;
  if (!aligned(a->x, b) || !aligned(a->residual, b) || !aligned(a->weight, w) || !aligned(a->sum, b) ||
      !aligned(a->y, wide ? b : 1) || !aligned(a->scales, f32_scales ? 4 : 1))
    return MRR_ERROR_MISALIGNED;
  const int64_t n = a->rows * a->H;
  Buffers s;
  s.add(a->x, n * b, false);
  s.add(a->residual, n * b, false);
  s.add(a->weight, a->H * w, false);
  s.add(a->y, wide ? n * b : fp4 ? n / 2 : n, true);
  s.add(a->scales, a->rows * (f32_scales ? 4 : 2 * ((a->H + 63) / 64)), true);
  s.add(a->sum, n * b, true);
  return s.clash() ? MRR_ERROR_INVALID_VALUE : MRR_SUCCESS;
}

mrr_status check_rms_norm_backward(const mrr_rms_norm_backward_args* a, const void* ws, size_t ws_bytes) {
  if (a == nullptr) return MRR_ERROR_INVALID_VALUE;
  const int b = wide_bytes(a->dtype), w = wide_bytes(a->weight_dtype);
  if (b == 0 || (a->weight_dtype != a->dtype && a->weight_dtype != MRR_F32)) return MRR_ERROR_UNSUPPORTED_DTYPE;
  if (!norm_sizes(a->rows, a->H)) return MRR_ERROR_INVALID_SHAPE;
  if (!norm_eps(a->eps)) return MRR_ERROR_INVALID_VALUE;
  if (a->weight == nullptr || a->grad_weight == nullptr) return MRR_ERROR_INVALID_VALUE;
  if (a->rows > 0 && (a->grad == nullptr || a->x == nullptr || a->grad_x == nullptr || ws == nullptr))
    return MRR_ERROR_INVALID_VALUE;
  if (!aligned(a->grad, b) || !aligned(a->x, b) || !aligned(a->grad_sum, b) || !aligned(a->grad_x, b) ||
      !aligned(a->weight, w) || !aligned(a->grad_weight, w) || !aligned(ws, 16))
    return MRR_ERROR_MISALIGNED;
  const size_t need = mrr_rms_norm_backward_workspace_size(a->rows, a->H);
  if (a->rows > 0 && ws_bytes < need) return MRR_ERROR_WORKSPACE_TOO_SMALL;
  const int64_t n = a->rows * a->H;
  Buffers s;
  s.add(a->grad, n * b, false);
  s.add(a->x, n * b, false);
  s.add(a->weight, a->H * w, false);
  s.add(a->grad_sum, n * b, false);
  s.add(a->grad_x, n * b, true);
  s.add(a->grad_weight, a->H * w, true);
  if (a->rows > 0) s.add(ws, static_cast<int64_t>(need), true);
  return s.clash() ? MRR_ERROR_INVALID_VALUE : MRR_SUCCESS;
}

mrr_status check_router(const mrr_router_args* a) {
  if (a == nullptr) return MRR_ERROR_INVALID_VALUE;
  const int b = wide_bytes(a->dtype);
  if (b == 0) return MRR_ERROR_UNSUPPORTED_DTYPE;
  if (!router_sizes(a->T, a->E, a->top_k)) return MRR_ERROR_INVALID_SHAPE;
  if (a->renormalize != 0 && a->renormalize != 1) return MRR_ERROR_INVALID_VALUE;
  if (a->T == 0) return MRR_SUCCESS;
  if (a->logits == nullptr || a->expert_weight == nullptr || a->expert_ids == nullptr) return MRR_ERROR_INVALID_VALUE;
  if (!aligned(a->logits, b) || !aligned(a->expert_weight, 4) || !aligned(a->expert_ids, 4)) return MRR_ERROR_MISALIGNED;
  Buffers s;
  s.add(a->logits, a->T * a->E * b, false);
  s.add(a->expert_weight, a->T * a->top_k * 4, true);
  s.add(a->expert_ids, a->T * a->top_k * 4, true);
  return s.clash() ? MRR_ERROR_INVALID_VALUE : MRR_SUCCESS;
}

mrr_status check_router_backward(const mrr_router_backward_args* a) {
  if (a == nullptr) return MRR_ERROR_INVALID_VALUE;
  const int b = wide_bytes(a->dtype);
  if (b == 0) return MRR_ERROR_UNSUPPORTED_DTYPE;
  if (!router_sizes(a->T, a->E, a->top_k)) return MRR_ERROR_INVALID_SHAPE;
  if (a->renormalize != 0 && a->renormalize != 1) return MRR_ERROR_INVALID_VALUE;
  if (a->T == 0) return MRR_SUCCESS;
  if (a->grad_weight == nullptr || (a->logits == nullptr && a->renormalize == 0) || a->expert_weight == nullptr ||
      a->expert_ids == nullptr || a->grad_logits == nullptr)
    return MRR_ERROR_INVALID_VALUE;
  if (!aligned(a->logits, b) || !aligned(a->grad_logits, b) || !aligned(a->grad_weight, 4) ||
      !aligned(a->expert_weight, 4) || !aligned(a->expert_ids, 4))
    return MRR_ERROR_MISALIGNED;
  Buffers s;
  s.add(a->logits, a->T * a->E * b, false);
  s.add(a->grad_weight, a->T * a->top_k * 4, false);
  s.add(a->expert_weight, a->T * a->top_k * 4, false);
  s.add(a->expert_ids, a->T * a->top_k * 4, false);
  s.add(a->grad_logits, a->T * a->E * b, true);
  return s.clash() ? MRR_ERROR_INVALID_VALUE : MRR_SUCCESS;
}

int64_t permute_row_bytes(const mrr_token_permute_args* a) { return a->H * token_bits(a->tokens_dtype) / 8; }

int64_t permute_scale_bytes(const mrr_token_permute_args* a) {
  if (a->per_token_scales == nullptr && a->permute_per_token_scales == nullptr) return 0;
  if (a->scales_dtype == MRR_F8_E8M0) return 2 * ((a->H + 63) / 64);
  return 4 * (a->scales_ndim == 2 ? a->scales_dims[1] : 1);
}

mrr_status check_token_permute(const mrr_token_permute_args* a, const void* ws, size_t ws_bytes) {
  if (a == nullptr) return MRR_ERROR_INVALID_VALUE;
  const int bits = token_bits(a->tokens_dtype);
  if (bits == 0) return MRR_ERROR_UNSUPPORTED_DTYPE;
  if (!choice_sizes(a->T, a->top_k) || a->H <= 0 || a->H > kPermuteMaxH || (bits == 4 && a->H % 2 != 0) || a->E <= 0 ||
      a->E > kPermuteMaxExperts)
    return MRR_ERROR_INVALID_SHAPE;
  if (a->expert_token_num_type != 0 && a->expert_token_num_type != 1) return MRR_ERROR_INVALID_VALUE;
  const bool scales = a->per_token_scales != nullptr || a->permute_per_token_scales != nullptr;
  if (scales) {
    const int64_t* d = a->scales_dims;
    if (a->scales_dtype == MRR_F32) {
      if (a->scales_ndim < 1 || a->scales_ndim > 2 || d[0] != a->T) return MRR_ERROR_INVALID_SHAPE;
      if (a->scales_ndim == 2 && (d[1] < 1 || d[1] > kPermuteMaxH)) return MRR_ERROR_INVALID_SHAPE;
    } else if (a->scales_dtype == MRR_F8_E8M0) {
      if (a->scales_ndim != 3 || d[0] != a->T || d[1] != (a->H + 63) / 64 || d[2] != 2) return MRR_ERROR_INVALID_SHAPE;
    } else {
      return MRR_ERROR_UNSUPPORTED_DTYPE;
    }
  }
  if (a->expert_token_num == nullptr) return MRR_ERROR_INVALID_VALUE;
  const int64_t n = a->T * a->top_k;
  if (n > 0 && (a->tokens == nullptr || a->expert_ids == nullptr || a->permute_tokens == nullptr ||
                a->permute_token_idx == nullptr || (ws == nullptr && n > kPermuteSelfChoices) ||
                (a->per_token_scales == nullptr) != (a->permute_per_token_scales == nullptr) ||
                (a->expert_weight == nullptr) != (a->permute_topk_weight == nullptr)))
    return MRR_ERROR_INVALID_VALUE;
  const int b = bits < 8 ? 1 : bits / 8;
  if (!aligned(a->tokens, b) || !aligned(a->permute_tokens, b) || !aligned(a->expert_ids, 4) ||
      !aligned(a->expert_weight, 4) || !aligned(a->permute_token_idx, 4) || !aligned(a->expert_token_num, 4) ||
      !aligned(a->permute_topk_weight, 4) || !aligned(ws, 16))
    return MRR_ERROR_MISALIGNED;
  if (scales && a->scales_dtype == MRR_F32 && (!aligned(a->per_token_scales, 4) || !aligned(a->permute_per_token_scales, 4)))
    return MRR_ERROR_MISALIGNED;
  const size_t need = n > kPermuteSelfChoices ? mrr_token_permute_workspace_size(a->T, a->top_k, a->E) : 0;
  if (ws_bytes < need) return MRR_ERROR_WORKSPACE_TOO_SMALL;
  const int64_t row = permute_row_bytes(a), srow = permute_scale_bytes(a);
  Buffers s;
  s.add(a->tokens, a->T * row, false);
  s.add(a->expert_ids, n * 4, false);
  s.add(a->per_token_scales, a->T * srow, false);
  s.add(a->expert_weight, n * 4, false);
  s.add(a->permute_tokens, n * row, true);
  s.add(a->permute_per_token_scales, n * srow, true);
  s.add(a->permute_token_idx, n * 4, true);
  s.add(a->expert_token_num, a->E * 4, true);
  s.add(a->permute_topk_weight, n * 4, true);
  s.add(ws, static_cast<int64_t>(need), true);
  return s.clash() ? MRR_ERROR_INVALID_VALUE : MRR_SUCCESS;
}

mrr_status check_token_unpermute(const mrr_token_unpermute_args* a) {
  if (a == nullptr) return MRR_ERROR_INVALID_VALUE;
  const int b = wide_bytes(a->dtype);
  if (b == 0) return MRR_ERROR_UNSUPPORTED_DTYPE;
  if (!choice_sizes(a->T, a->top_k) || a->R < 0 || a->R > kMostRows || a->H <= 0 || a->H > kPermuteMaxH)
    return MRR_ERROR_INVALID_SHAPE;
  if (a->T == 0) return MRR_SUCCESS;
  if ((a->rows == nullptr && a->R > 0) || a->permute_token_idx == nullptr || a->y == nullptr ||
      (a->row_values == nullptr && a->choice_values != nullptr && a->R > 0) ||
      (a->row_values != nullptr && a->choice_values == nullptr))
    return MRR_ERROR_INVALID_VALUE;
  if (!aligned(a->rows, b) || !aligned(a->permute_token_idx, 4) || !aligned(a->expert_weight, 4) || !aligned(a->y, b) ||
      !aligned(a->row_values, 4) || !aligned(a->choice_values, 4))
    return MRR_ERROR_MISALIGNED;
  const int64_t n = a->T * a->top_k;
  Buffers s;
  s.add(a->rows, a->R * a->H * b, false);
  s.add(a->permute_token_idx, n * 4, false);
  s.add(a->expert_weight, n * 4, false);
  s.add(a->row_values, a->R * 4, false);
  s.add(a->y, a->T * a->H * b, true);
  s.add(a->choice_values, n * 4, true);
  return s.clash() ? MRR_ERROR_INVALID_VALUE : MRR_SUCCESS;
}

mrr_status check_token_unpermute_backward(const mrr_token_unpermute_backward_args* a) {
  if (a == nullptr) return MRR_ERROR_INVALID_VALUE;
  const int b = wide_bytes(a->dtype);
  if (b == 0) return MRR_ERROR_UNSUPPORTED_DTYPE;
  if (!choice_sizes(a->T, a->top_k) || a->R < 0 || a->R > kMostRows || a->H <= 0 || a->H > kPermuteMaxH)
    return MRR_ERROR_INVALID_SHAPE;
  if (a->T == 0) return MRR_SUCCESS;
  if (a->grad == nullptr || a->permute_token_idx == nullptr ||
      (a->expert_weight == nullptr) != (a->grad_weight == nullptr) ||
      (a->R > 0 && (a->grad_rows == nullptr || (a->rows == nullptr && a->expert_weight != nullptr))))
    return MRR_ERROR_INVALID_VALUE;
  if (!aligned(a->grad, b) || !aligned(a->rows, b) || !aligned(a->permute_token_idx, 4) ||
      !aligned(a->expert_weight, 4) || !aligned(a->grad_rows, b) || !aligned(a->grad_weight, 4))
    return MRR_ERROR_MISALIGNED;
  const int64_t n = a->T * a->top_k;
  Buffers s;
  s.add(a->grad, a->T * a->H * b, false);
  s.add(a->rows, a->R * a->H * b, false);
  s.add(a->permute_token_idx, n * 4, false);
  s.add(a->expert_weight, n * 4, false);
  s.add(a->grad_rows, a->R * a->H * b, true);
  s.add(a->grad_weight, n * 4, true);
  return s.clash() ? MRR_ERROR_INVALID_VALUE : MRR_SUCCESS;
}

}  // namespace mrr

extern "C" {

mrr_status mrr_rms_norm_validate(const mrr_rms_norm_args* args) { return mrr::check_rms_norm(args); }

size_t mrr_rms_norm_backward_workspace_size(int64_t rows, int64_t H) {
  if (!mrr::norm_sizes(rows, H)) return 0;
  return 256 + mrr::round_up(4 * static_cast<size_t>(mrr::norm_backward_groups(rows, H) * H), 256);
}

mrr_status mrr_rms_norm_backward_validate(const mrr_rms_norm_backward_args* args, const void* workspace,
                                          size_t workspace_bytes) {
  return mrr::check_rms_norm_backward(args, workspace, workspace_bytes);
}

mrr_status mrr_router_validate(const mrr_router_args* args) { return mrr::check_router(args); }

mrr_status mrr_router_backward_validate(const mrr_router_backward_args* args) {
  return mrr::check_router_backward(args);
}

size_t mrr_token_permute_workspace_size(int64_t T, int64_t top_k, int64_t E) {
  if (!mrr::choice_sizes(T, top_k) || E <= 0 || E > mrr::kPermuteMaxExperts) return 0;
  const int64_t n = T * top_k;
  return 256 + mrr::round_up(4 * static_cast<size_t>(mrr::permute_blocks(n, E) * (E + 1)), 256);
}

mrr_status mrr_token_permute_validate(const mrr_token_permute_args* args, const void* workspace,
                                      size_t workspace_bytes) {
  return mrr::check_token_permute(args, workspace, workspace_bytes);
}

mrr_status mrr_token_unpermute_validate(const mrr_token_unpermute_args* args) {
  return mrr::check_token_unpermute(args);
}

mrr_status mrr_token_unpermute_backward_validate(const mrr_token_unpermute_backward_args* args) {
  return mrr::check_token_unpermute_backward(args);
}

}  // extern "C"
