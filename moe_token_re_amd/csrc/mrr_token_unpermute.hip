// mrr_token_unpermute.hip -- the experts' rows summed back by token, with the choices'
// weights, and the gradients of the rows and the weights.
//
//   y[t] = sum over j of weight[t, j] rows[idx[t, j]]
//   grad_rows[idx[t, j]] = weight[t, j] grad[t];  grad_weight[t, j] = <grad[t], rows[idx[t, j]]>
//
// Bound by memory: every row is read once (and its gradient written once). A lane holds
// 16 bytes of a token's row, all of its choices' loads are under way at once, and sums are
// fp32 in the order of j. For the gradient a workgroup takes a token, and its lanes keep a
// part of each choice's product, which are added across lanes at the end; of more than eight
// choices two workgroups take a token.
// 8192 tokens of 8 rows of 14 KiB: 177 us, 6.0 TB/s of 1.06 GB (reading as many bytes in
// their order takes 137; two KiB a wave, workgroups of 2 to 14 KiB and a token's pieces on
// one die change nothing). 8192 of 6 rows of 4 KiB: 43 us, and the gradient 69, 6.3 TB/s.
#include "mrr_rows.h"

namespace mrr {
namespace {

// How rows are read and written: of any alignment; or in whole units, written past the
// caches; and read past them as well.
enum { kAny = 0, kWhole = 1, kPast = 2 };

struct SumArgs {
  const uint8_t* rows;
  const int32_t* idx;
  const float* weight;  // or null
  uint8_t* y;
  const float* row_values;  // or null
  float* choice_values;     // or null
  uint32_t T, k, R, H;
};

// One unit's sum over choices [first, first + kK) of a token, of which those below k exist.
template <int kDtype, int kK, bool kAll, int kHow>
__device__ __forceinline__ void add_choices(const SumArgs& a, size_t token, uint32_t first, uint32_t col,
                                            float (&sum)[16 / Unit16<kDtype>::kBytes]) {
  using U = Unit16<kDtype>;
  constexpr int kN = 16 / U::kBytes;
  U v[kK];
  float w[kK];
#pragma unroll
  for (int j = 0; j < kK; ++j) {
    const bool exists = kAll || first + j < a.k;
    const size_t at = token * a.k + first + j;
    const uint32_t row = exists ? static_cast<uint32_t>(a.idx[at]) : 0xffffffffu;
    const bool here = row < a.R;
    w[j] = !here ? 0.0f : a.weight != nullptr ? a.weight[at] : 1.0f;
    if constexpr (kHow != kAny) {
      const size_t from = here ? static_cast<size_t>(row) * a.H * U::kBytes : 0;
      v[j].load_whole(WholeRow<kHow == kPast>(a.rows + from, here ? a.H * U::kBytes : 0), col);
    } else {
#pragma unroll
      for (int i = 0; i < U::kWords; ++i) v[j].w[i] = 0;
      if (here) v[j].load(a.rows + static_cast<size_t>(row) * a.H * U::kBytes, col, a.H);
    }
  }
#pragma unroll
  for (int j = 0; j < kK; ++j)
#pragma unroll
    for (int i = 0; i < kN; ++i) sum[i] = __builtin_fmaf(w[j], v[j].get(i), sum[i]);
}

// kK: so many choices, or 0: more than 8.
template <int kDtype, int kK, int kHow>
__device__ __forceinline__ void sum_unit(const SumArgs& a, size_t token, uint32_t col) {
  using U = Unit16<kDtype>;
  constexpr int kN = 16 / U::kBytes;
  float sum[kN] = {};
  if constexpr (kK > 0) {
    add_choices<kDtype, kK, true, kHow>(a, token, 0, col, sum);
  } else {
    add_choices<kDtype, 8, true, kHow>(a, token, 0, col, sum);
    add_choices<kDtype, 8, false, kHow>(a, token, 8, col, sum);
  }
  U out;
#pragma unroll
  for (int i = 0; i < kN; i += 2) out.put(i / 2, sum[i], sum[i + 1]);
  if constexpr (kHow != kAny)
    out.store_whole(WholeRow<kHow == kPast>(a.y + token * a.H * U::kBytes, a.H * U::kBytes), col);
  else
    out.store(a.y + token * a.H * U::kBytes, col, a.H);
}

__device__ __forceinline__ void choice_value(const SumArgs& a, size_t token, uint32_t j) {
  const size_t at = token * a.k + j;
  const uint32_t row = static_cast<uint32_t>(a.idx[at]);
  a.choice_values[at] = row < a.R ? a.row_values[row] : 0.0f;
}

// Rows of more than 64 units: a wave takes 1 KiB of a token's.
template <int kDtype, int kK, int kHow>
__global__ __launch_bounds__(64) void sum_rows_kernel(SumArgs a) {
  constexpr uint32_t kN = 16 / Unit16<kDtype>::kBytes;
  const uint32_t token = blockIdx.y, col = (blockIdx.x * 64 + threadIdx.x) * kN;
  if (a.choice_values != nullptr && blockIdx.x == 0 && threadIdx.x < a.k) choice_value(a, token, threadIdx.x);
  if (col < a.H) sum_unit<kDtype, kK, kHow>(a, token, col);
}

// Shorter ones: as many tokens a wave as fit.
template <int kDtype, int kK>
__global__ __launch_bounds__(256) void sum_short_rows_kernel(SumArgs a) {
  constexpr uint32_t kN = 16 / Unit16<kDtype>::kBytes;
  const uint32_t units = (a.H + kN - 1) / kN;
  const uint32_t lane = threadIdx.x % 64, tokens = 64 / units, in_wave = lane / units;
  const size_t token = (static_cast<size_t>(blockIdx.x) * 4 + threadIdx.x / 64) * tokens + in_wave;
  if (in_wave >= tokens || token >= a.T) return;
  const uint32_t unit = lane - in_wave * units;
  if (a.choice_values != nullptr)
    for (uint32_t j = unit; j < a.k; j += units) choice_value(a, token, j);
  sum_unit<kDtype, kK, kAny>(a, token, unit * kN);
}

struct GradArgs {
  const uint8_t* grad;
  const uint8_t* rows;
  const int32_t* idx;
  const float* weight;
  uint8_t* grad_rows;
  float* grad_weight;
  uint32_t T, k, R, H;
};

// Choices [first, first + kK) of a token, of which those below k exist.
template <int kDtype, int kK, int kWaves, int kHow>
__device__ __forceinline__ void grad_choices(const GradArgs& a, size_t token, uint32_t first, float (&sh)[kWaves][kK]) {
  // two products of fp16 values are not to become one instruction, which has another
  // rounding and no subnormal numbers
#pragma clang fp contract(off)
  using U = Unit16<kDtype>;
  constexpr uint32_t kN = 16 / U::kBytes;
  const uint32_t tid = threadIdx.x;
  const uint8_t* grad = a.grad + token * a.H * U::kBytes;
  const size_t at = token * a.k + first;
  float dot[kK], w[kK];
  int32_t idx[kK];  // read before any store: a load behind one would wait for it
#pragma unroll
  for (int j = 0; j < kK; ++j) {
    const bool exists = first + j < a.k;
    dot[j] = 0.0f;
    idx[j] = exists ? a.idx[at + j] : static_cast<int32_t>(0x80000000u);
    w[j] = exists ? a.weight[at + j] : 0.0f;
  }
  for (uint32_t col = tid * kN; col < a.H; col += 64 * kWaves * kN) {
    U g, v[kK];
    if constexpr (kHow != kAny)
      g.load_whole(WholeRow<kHow == kPast>(grad, a.H * U::kBytes), col);
    else
      g.load(grad, col, a.H);
#pragma unroll
    for (int j = 0; j < kK; ++j) {
      const uint32_t row = static_cast<uint32_t>(idx[j]);
      if constexpr (kHow != kAny) {
        const size_t from = row < a.R ? static_cast<size_t>(row) * a.H * U::kBytes : 0;
        v[j].load_whole(WholeRow<kHow == kPast>(a.rows + from, row < a.R ? a.H * U::kBytes : 0), col);
      } else {
#pragma unroll
        for (int i = 0; i < U::kWords; ++i) v[j].w[i] = 0;
        if (row < a.R) v[j].load(a.rows + static_cast<size_t>(row) * a.H * U::kBytes, col, a.H);
      }
    }
#pragma unroll
    for (int j = 0; j < kK; ++j) {
      const bool gone = idx[j] < 0;
      const uint32_t row = static_cast<uint32_t>(gone ? ~idx[j] : idx[j]);
      U out;
#pragma unroll
      for (uint32_t e = 0; e < kN; e += 2) {
        const float g0 = g.get(e), g1 = g.get(e + 1);
        dot[j] = __builtin_fmaf(g0, v[j].get(e), dot[j]);
        dot[j] = __builtin_fmaf(g1, v[j].get(e + 1), dot[j]);
        out.put(e / 2, gone ? 0.0f : w[j] * g0, gone ? 0.0f : w[j] * g1);
      }
      uint8_t* to = a.grad_rows + static_cast<size_t>(row) * a.H * U::kBytes;
      if constexpr (kHow != kAny)
        out.store_whole(WholeRow<kHow == kPast>(to, row < a.R ? a.H * U::kBytes : 0), col);
      else if (row < a.R)
        out.store(to, col, a.H);
    }
  }
#pragma unroll
  for (int j = 0; j < kK; ++j) {
    // without a row it is 0, whatever the gradient holds
    const float d = static_cast<uint32_t>(idx[j]) < a.R ? sum64_f32(dot[j]) : 0.0f;
    if (tid % 64 == 0) sh[tid / 64][j] = d;
  }
  __syncthreads();
  if (tid < kK && first + tid < a.k) {
    float d = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) d += sh[w][tid];
    a.grad_weight[at + tid] = d;
  }
}

template <int kDtype, int kK, int kWaves, int kHow>
__global__ __launch_bounds__(64 * kWaves) void sum_rows_backward_kernel(GradArgs a) {
  __shared__ float sh[kWaves][kK];
  grad_choices<kDtype, kK, kWaves, kHow>(a, blockIdx.x, blockIdx.y * kK, sh);
}

constexpr uint32_t kMostGridY = 65535;
constexpr uint32_t kMostTokens = 1u << 23;  // of a launch of short rows, at most a wave a token: less than 2^32 threads
// Sums and gradients of aligned rows are written past the caches (512 tokens of 8 rows of
// 14 KiB, forward and back: 32.6 us so and 38.6 through them; smaller ones take the same
// either way). From so many bytes on, which the last of the caches does not hold, the rows
// are read past them too (8192 tokens of 8 rows of 14 KiB, 940 MB: 178 us so and 193
// otherwise; of 6 rows of 4 KiB, 200 MB, forward and back: 120 us so and 114 otherwise).
constexpr int64_t kPastBytes = int64_t(256) << 20;
int how(int64_t bytes, bool whole) { return !whole ? kAny : bytes < kPastBytes ? kWhole : kPast; }

template <int kDtype, int kK, int kHow>
void launch_sum(const SumArgs& all, hipStream_t stream) {
  constexpr uint32_t kN = 16 / Unit16<kDtype>::kBytes, kBytes = Unit16<kDtype>::kBytes;
  const uint32_t units = (all.H + kN - 1) / kN, most = units > 64 ? kMostGridY : kMostTokens;
  for (uint32_t t = 0; t < all.T;) {
    SumArgs a = all;
    a.T = all.T - t < most ? all.T - t : most;
    a.idx += static_cast<size_t>(t) * a.k;
    if (a.weight != nullptr) a.weight += static_cast<size_t>(t) * a.k;
    if (a.choice_values != nullptr) a.choice_values += static_cast<size_t>(t) * a.k;
    a.y += static_cast<size_t>(t) * a.H * kBytes;
    if (units > 64) {
      sum_rows_kernel<kDtype, kK, kHow><<<dim3((units + 63) / 64, a.T), 64, 0, stream>>>(a);
    } else {
      const uint32_t each = 4 * (64 / units);
      sum_short_rows_kernel<kDtype, kK><<<(a.T + each - 1) / each, 256, 0, stream>>>(a);
    }
    if (hipPeekAtLastError() != hipSuccess) return;
    t += a.T;
  }
}

template <int kDtype, int kHow>
void launch_sum_k(const SumArgs& a, hipStream_t stream) {
  switch (a.k) {
    case 1: launch_sum<kDtype, 1, kHow>(a, stream); break;
    case 2: launch_sum<kDtype, 2, kHow>(a, stream); break;
    case 3: launch_sum<kDtype, 3, kHow>(a, stream); break;
    case 4: launch_sum<kDtype, 4, kHow>(a, stream); break;
    case 5: launch_sum<kDtype, 5, kHow>(a, stream); break;
    case 6: launch_sum<kDtype, 6, kHow>(a, stream); break;
    case 7: launch_sum<kDtype, 7, kHow>(a, stream); break;
    case 8: launch_sum<kDtype, 8, kHow>(a, stream); break;
    default: launch_sum<kDtype, 0, kHow>(a, stream); break;
  }
}

template <int kHow>
void launch_sum_how(const SumArgs& a, int32_t dtype, hipStream_t stream) {
  switch (dtype) {
    case MRR_F16: launch_sum_k<MRR_F16, kHow>(a, stream); break;
    case MRR_BF16: launch_sum_k<MRR_BF16, kHow>(a, stream); break;
    default: launch_sum_k<MRR_F32, kHow>(a, stream); break;
  }
}
void launch_sum_dtype(const SumArgs& a, int32_t dtype, int how, hipStream_t stream) {
  if (how == kAny)
    launch_sum_how<kAny>(a, dtype, stream);
  else if (how == kWhole)
    launch_sum_how<kWhole>(a, dtype, stream);
  else
    launch_sum_how<kPast>(a, dtype, stream);
}

template <int kDtype, int kK, int kHow>
void launch_grad(const GradArgs& all, hipStream_t stream) {
  constexpr uint32_t kBytes = Unit16<kDtype>::kBytes;
  const int64_t row = static_cast<int64_t>(all.H) * kBytes;
  const uint32_t most = static_cast<uint32_t>(grad_launch_tokens(row, all.k));
  for (uint32_t t = 0; t < all.T;) {
    GradArgs a = all;
    a.T = all.T - t < most ? all.T - t : most;
    a.idx += static_cast<size_t>(t) * a.k;
    a.weight += static_cast<size_t>(t) * a.k;
    a.grad_weight += static_cast<size_t>(t) * a.k;
    a.grad += static_cast<size_t>(t) * a.H * kBytes;
    const dim3 grid(a.T, (a.k + kK - 1) / kK);
    switch (grad_waves(row)) {
      case 8: sum_rows_backward_kernel<kDtype, kK, 8, kHow><<<grid, 512, 0, stream>>>(a); break;
      case 4: sum_rows_backward_kernel<kDtype, kK, 4, kHow><<<grid, 256, 0, stream>>>(a); break;
      default: sum_rows_backward_kernel<kDtype, kK, 1, kHow><<<grid, 64, 0, stream>>>(a); break;
    }
    if (hipPeekAtLastError() != hipSuccess) return;
    t += a.T;
  }
}

template <int kDtype, int kHow>
void launch_grad_k(const GradArgs& a, hipStream_t stream) {
  switch (grad_choices_at_once(a.k)) {
    case 1: launch_grad<kDtype, 1, kHow>(a, stream); break;
    case 2: launch_grad<kDtype, 2, kHow>(a, stream); break;
    case 4: launch_grad<kDtype, 4, kHow>(a, stream); break;
    case 6: launch_grad<kDtype, 6, kHow>(a, stream); break;
    default: launch_grad<kDtype, 8, kHow>(a, stream); break;
  }
}

template <int kHow>
void launch_grad_how(const GradArgs& a, int32_t dtype, hipStream_t stream) {
  switch (dtype) {
    case MRR_F16: launch_grad_k<MRR_F16, kHow>(a, stream); break;
    case MRR_BF16: launch_grad_k<MRR_BF16, kHow>(a, stream); break;
    default: launch_grad_k<MRR_F32, kHow>(a, stream); break;
  }
}
void launch_grad_dtype(const GradArgs& a, int32_t dtype, int how, hipStream_t stream) {
  if (how == kAny)
    launch_grad_how<kAny>(a, dtype, stream);
  else if (how == kWhole)
    launch_grad_how<kWhole>(a, dtype, stream);
  else
    launch_grad_how<kPast>(a, dtype, stream);
}

}  // namespace
}  // namespace mrr

extern "C" mrr_status mrr_token_unpermute(const mrr_token_unpermute_args* args, struct ihipStream_t* stream) {
  using namespace mrr;
  const mrr_status st = check_token_unpermute(args);
  if (st != MRR_SUCCESS || args->T == 0) return st;
  const SumArgs a{static_cast<const uint8_t*>(args->rows), args->permute_token_idx, args->expert_weight,
                  static_cast<uint8_t*>(args->y), args->row_values, args->choice_values, static_cast<uint32_t>(args->T),
                  static_cast<uint32_t>(args->top_k), static_cast<uint32_t>(args->R), static_cast<uint32_t>(args->H)};
  const int64_t b = args->dtype == MRR_F32 ? 4 : 2;
  launch_sum_dtype(a, args->dtype, how(args->T * args->top_k * args->H * b, whole_units(args->H * b, a.rows, a.y)), stream);
  return hipGetLastError() == hipSuccess ? MRR_SUCCESS : MRR_ERROR_HIP;
}

extern "C" mrr_status mrr_token_unpermute_backward(const mrr_token_unpermute_backward_args* args,
                                                   struct ihipStream_t* stream) {
  using namespace mrr;
  const mrr_status st = check_token_unpermute_backward(args);
  if (st != MRR_SUCCESS || args->T == 0) return st;
  const int64_t b = args->dtype == MRR_F32 ? 4 : 2;
  if (args->expert_weight == nullptr) {
    if (args->R > 0)
      move_rows(args->grad, args->grad_rows, args->H * b, args->permute_token_idx, args->T, args->top_k, args->R, stream);
    return hipGetLastError() == hipSuccess ? MRR_SUCCESS : MRR_ERROR_HIP;
  }
  const GradArgs a{static_cast<const uint8_t*>(args->grad), static_cast<const uint8_t*>(args->rows),
                   args->permute_token_idx, args->expert_weight, static_cast<uint8_t*>(args->grad_rows),
                   args->grad_weight, static_cast<uint32_t>(args->T), static_cast<uint32_t>(args->top_k),
                   static_cast<uint32_t>(args->R), static_cast<uint32_t>(args->H)};
  launch_grad_dtype(a, args->dtype,
                    how(args->T * args->top_k * args->H * b, whole_units(args->H * b, a.grad, a.rows, a.grad_rows)),
                    stream);
  return hipGetLastError() == hipSuccess ? MRR_SUCCESS : MRR_ERROR_HIP;
}
