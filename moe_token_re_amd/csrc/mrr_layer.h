// mrr_layer.h -- shared between the host checks of the operators around an
// expert layer (mrr_layer_validate.cpp, which includes no HIP header) and their
// kernels (mrr_rms_norm.hip, mrr_rms_norm_backward.hip, mrr_router.hip,
// mrr_token_permute.hip, mrr_token_unpermute.hip). Not part of the public ABI.
#pragma once

#include "mrr_internal.h"

namespace mrr {

constexpr int64_t kNormMaxH = 16384;
constexpr int64_t kLayerMaxTopK = 16;
constexpr int64_t kRouterMaxExperts = 1024;
constexpr int64_t kPermuteMaxExperts = 4096;
constexpr int64_t kPermuteMaxH = 65536;

// How rows of H values lie on the lanes of the norm's kernels: 8 neighbouring
// values a lane and unit, `lanes` lanes and `units` units a lane a row.
struct NormShape {
  int lanes, units;
};
// Rows up to this many take more lanes a row: they leave most of the chip empty. (bf16 with
// their sum, to fp8 rows, us of the kernel with these lanes and with those below: 256 rows of
// 7168 5.3 and 7.4, of 4096 4.5 and 4.9, one row of 7168 3.6 and 5.3; 512 of 4096 6.2 and
// 6.0, of 7168 7.9 and 9.0; 16384 of 4096 107 and 71, of 7168 143 and 123.)
constexpr int64_t kNormFewRows = 256;
inline NormShape norm_shape(int64_t rows, int64_t H) {
  if (H <= 512) return {64, 1};
  if (rows <= kNormFewRows) return H <= 2048 ? NormShape{256, 1} : H <= 8192 ? NormShape{1024, 1} : NormShape{1024, 2};
  if (H <= 1024) return {64, 2};
  if (H <= 2048) return {256, 1};
  if (H <= 4096) return {256, 2};
  if (H <= 8192) return {256, 4};
  return {1024, 2};
}

// The same for the gradient, which keeps three rows, the next ones, and a sum of each
// column in registers. (8192 rows with the sum's gradient: bf16 of 7168 by 1024 lanes 85.8 us
// and by 512 of two units 84.7, of 8192 93.4 and 96.0, fp32 of 8192 195 and 214; bf16 of 16384
// by 512 lanes of four units 243 and by 1024 of two 285.)
inline NormShape norm_backward_shape(int64_t H) {
  if (H <= 512) return {64, 1};
  if (H <= 1024) return {128, 1};
  if (H <= 2048) return {256, 1};
  if (H <= 4096) return {512, 1};
  if (H <= 8192) return {1024, 1};
  return {512, 4};
}
// Workgroups that each take every so-manieth row and keep a partial sum of the weight's
// gradient for each of their rows that run at once: eight waves a CU, which have the next
// row under way (8192 x 4096 bf16: 256 workgroups of 512 threads 49 us, 512 of them 54).
inline int64_t norm_backward_groups(int64_t rows, int64_t H) {
  const NormShape s = norm_backward_shape(H);
  const int64_t at_once = s.lanes == 64 ? 4 : 1, most = s.lanes >= 512 ? 256 : s.lanes == 128 ? 1024 : 512;
  const int64_t groups = (rows + at_once - 1) / at_once;
  return at_once * (groups < most ? groups : most);
}

// Few choices are sorted by every workgroup of one kernel by itself; more in blocks,
// whose counts by expert [blocks, E + 1] lie in the workspace. Every block reads all
// counts, so the blocks stay few.
// (8 choices a token: 512 tokens of 4 KiB by the one kernel 11.1 us and by blocks 10.7, of
// 128 bytes 9.6 and 11.2; 1024 of 4 KiB 23.0 and 13.9.)
constexpr int64_t kPermuteFewChoices = 4096;
// Up to so many choices the blocks are small and count all choices by themselves (rows of
// 128 bytes, us so and by the counts: 8192 choices 11.7 and 15.2, 16384 13.2 and 15.6, 32768
// 16.6 and 16.3).
constexpr int64_t kPermuteSelfChoices = MRR_TOKEN_PERMUTE_ALONE, kPermuteSelfBlock = 1024;
constexpr int64_t kPermuteMostBlocks = 64;
// With more experts than this fewer waves of a block place its choices: smaller blocks
// (32768 choices of 1024 experts 18.0 us so and 23.9 with the larger, of 4096 experts 34.8 and
// 60; 131072 choices of 512 experts 22.0 so and 20.5 with the larger).
constexpr int64_t kPermuteManyExperts = 512;
constexpr int64_t kPermuteBlockChoices = 1024;
inline int64_t permute_block(int64_t choices, int64_t E) {
  const int64_t least = E <= kPermuteManyExperts ? 4 * kPermuteBlockChoices : kPermuteBlockChoices;
  const int64_t each = static_cast<int64_t>(
      round_up(static_cast<size_t>((choices + kPermuteMostBlocks - 1) / kPermuteMostBlocks), kPermuteBlockChoices));
  return each > least ? each : least;
}
inline int64_t permute_blocks(int64_t choices, int64_t E) {
  const int64_t block = permute_block(choices, E);
  return (choices + block - 1) / block;
}

// The gradient of the rows' sums: a token's row by a wave, or by four past so many bytes (64 tokens
// of 6 rows, forward and back, us by a wave and by four: of 3 KiB 8.8 and 7.0, of 8 KiB 15.9 and
// 9.5; 4096 tokens of 6 rows of 1 KiB 20.0 and 24.9, of 4 KiB 61.5 and 60.2).
constexpr int64_t kGradWideRow = 2048;
// And by eight past so many (us by four, eight and sixteen: one token of 15 rows of 57 KiB 63,
// 24 and 19; 64 tokens of 8 rows of 14 KiB 10.9, 9.8 and 9.7; 8192 tokens of 8 rows of 8 KiB
// 329, 323 and 316, of 6 rows of 5 KiB 140, 138 and 174).
constexpr int64_t kGradWiderRow = 4096;
constexpr int grad_waves(int64_t row_bytes) { return row_bytes > kGradWiderRow ? 8 : row_bytes > kGradWideRow ? 4 : 1; }
// Choices of a token that one workgroup takes: above 8 two do.
constexpr int grad_choices_at_once(int64_t top_k) {
  return top_k <= 2 ? static_cast<int>(top_k) : top_k <= 4 ? 4 : top_k <= 6 ? 6 : 8;
}
// Tokens of one launch, whose grid holds less than 2^32 threads.
constexpr int64_t grad_launch_tokens(int64_t row_bytes, int64_t top_k) {
  const int64_t groups = (top_k + grad_choices_at_once(top_k) - 1) / grad_choices_at_once(top_k);
  return (int64_t(1) << 31) / (64 * grad_waves(row_bytes) * groups);
}

mrr_status check_rms_norm(const mrr_rms_norm_args* a);
mrr_status check_rms_norm_backward(const mrr_rms_norm_backward_args* a, const void* ws, size_t ws_bytes);
mrr_status check_router(const mrr_router_args* a);
mrr_status check_router_backward(const mrr_router_backward_args* a);
mrr_status check_token_permute(const mrr_token_permute_args* a, const void* ws, size_t ws_bytes);
mrr_status check_token_unpermute(const mrr_token_unpermute_args* a);
mrr_status check_token_unpermute_backward(const mrr_token_unpermute_backward_args* a);

// Bytes of a token's row and of its scales' (0: none), of checked arguments.
int64_t permute_row_bytes(const mrr_token_permute_args* a);
int64_t permute_scale_bytes(const mrr_token_permute_args* a);

}  // namespace mrr
