// mrr_experts.h -- shared between the host checks of the experts' operators
// (mrr_experts_validate.cpp, which includes no HIP header) and their kernels
// (mrr_mx_quant.hip, mrr_grouped_mm.hip, mrr_few_tokens.hip). Not part of the
// public ABI.
#pragma once

#include "mrr_internal.h"

namespace mrr {

// Bytes of the scales of a row of n values.
inline int64_t mx_scale_bytes(int64_t n) { return 2 * ((n + 63) / 64); }

constexpr int64_t kFewMaxTopK = 16;
constexpr int64_t kFewMaxExperts = 1024;

// Most runs of 16 or 32 output rows, over all parts of the experts, that the
// few-token layer's second kernel computes at once.
constexpr int64_t kFewMostRuns = 512;

// Workspace of the few-token layer: the routing [T, k] (int32 expert, or -1, float
// weight, and in 32 bits where its h lies), a count for each run, 32
// partial sums in fp32 for each run and token, and h [T k, I] of 4 bytes a value;
// each part rounded up to 256 bytes.
struct FewLayout {
  size_t ids, weight, between, arrived, part, h, bytes;
};
inline FewLayout few_layout(int64_t T, int64_t k, int64_t I) {
  FewLayout l{};
  l.ids = 0;
  l.weight = round_up(4 * static_cast<size_t>(T * k), 256);
  l.between = 2 * l.weight;
  l.arrived = 3 * l.weight;
  l.part = l.arrived + 4 * static_cast<size_t>(kFewMostRuns);
  l.h = l.part + static_cast<size_t>(kFewMostRuns * 32 * 4 * T);
  l.bytes = l.h + round_up(4 * static_cast<size_t>(T * k * I), 256) + 256;
  return l;
}

// The host checks; `quantize` says which side of a conversion is written.
mrr_status check_mx(const mrr_mx_args* args, bool quantize);
mrr_status check_grouped_mm(const mrr_grouped_mm_args* args, const void* ws, size_t ws_bytes);
mrr_status check_few_tokens(const mrr_few_tokens_args* args, const void* ws, size_t ws_bytes);

}  // namespace mrr
