// mrr_rms_norm_backward.hip -- the gradient of the root-mean-square norm:
//
//   n = x r, r = 1 / sqrt(mean(x^2) + eps)
//   grad_x = r (g w - n mean(g w n)) + grad_sum,  grad_weight = sum over rows of g n
//
// Bound by memory: three rows in (x, g, grad_sum), one out, two sums of a row (x^2 and
// g w x) in one barrier. A workgroup takes every so-manieth row and keeps its part of
// grad_weight in registers; the parts, fp32, go to the workspace, and a second kernel
// adds them in a fixed order, so that the result is the same each time. 8192 x 4096 bf16
// rows: 47 us and 4 of the second kernel, together 5.3 TB/s (a plain copy of 1 GiB: 6.7); without
// the next row under way 62.
#include "mrr_rows.h"

namespace mrr {
namespace {

struct BackArgs {
  const uint8_t* grad;
  const uint8_t* x;
  const uint8_t* weight;
  const uint8_t* grad_sum;  // or null
  uint8_t* grad_x;
  float* part;  // [groups, H]
  uint8_t* grad_weight;
  uint32_t rows, H, groups;
  float eps, inv_h;
};

// Rows of so many bytes are read and written past the caches (H 4096: 8192 rows of bf16
// 51.6 us so and 54.1 through them, 16384 93.5 and 100, 1024 14.6 and 14.3). Not 32-bit ones:
// a lane's 8 values are two units there, two requests to each line, which then comes twice
// (8192 rows 173 us past the caches and 99 through them).
constexpr int64_t kStreamBytes = int64_t(64) << 20;
// Between these sums of squares 32 bits do; a smaller one is nothing next to kLeastEps.
constexpr float kMostSum = 1e37f, kLeastSum = 1e-30f, kLeastEps = 1e-20f;

// The sum over a row's waves, by way of sh; all of them are here.
template <int kWaves>
__device__ __forceinline__ float sum_of_row(float v, float* sh) {
  v = sum64_f32(v);
  if constexpr (kWaves > 1) {
    __syncthreads();  // an earlier sum has been read
    if (threadIdx.x % 64 == 0) sh[threadIdx.x / 64] = v;
    __syncthreads();
    v = 0.0f;
    for (int i = 0; i < kWaves; ++i) v += sh[i];
  }
  return v;
}

// How rows are read: with a branch for a unit that the row's end cuts, or such a unit
// beginning earlier, so that it holds values of the one before again (they are left out of
// the sums, and written twice); or whole units past the caches.
enum { kCut = 0, kAgain = 1, kStreamed = 2 };

template <int kX, int kW, int kLanes, int kUnits, int kRead>
__global__ __launch_bounds__(kLanes == 64 ? 256 : kLanes) void rms_norm_backward_kernel(BackArgs a) {
  constexpr int kThreads = kLanes == 64 ? 256 : kLanes, kAtOnce = kThreads / kLanes, kWaves = kLanes / 64;
  using X = Eight<kX>;
  // the next row's values are under way during this one's sums, where registers allow it
  constexpr bool kAhead = kRead != kCut && kUnits * X::kBytes <= 4;
  // and grad_sum is read with the others, where they allow that
  constexpr bool kLate = kUnits * X::kBytes > 4;
  const uint32_t lane = threadIdx.x % kLanes;
  const uint32_t group = blockIdx.x * static_cast<uint32_t>(kAtOnce) + (kAtOnce > 1 ? threadIdx.x / kLanes : 0);
  if (kAtOnce > 1 && group >= a.groups) return;  // whole waves, which meet no barrier

  float part[kUnits][8];
  Eight<kW> w[kUnits];
  uint32_t at[kUnits];  // the unit's first column
  uint32_t skip[kUnits];  // and its values that are not its own
  X own[kUnits];          // ones where they are
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const uint32_t col = 8 * (i * kLanes + lane);
    at[i] = kRead == kAgain ? min(col, a.H - 8) : col;
    skip[i] = min(col - at[i], 8u);
#pragma unroll
    for (uint32_t k = 0; k < X::kWords; ++k) {
      if constexpr (X::kBytes == 4)
        own[i].w[k] = k >= skip[i] ? 0xffffffffu : 0;
      else
        own[i].w[k] = 2 * k >= skip[i] ? 0xffffffffu : 2 * k + 1 >= skip[i] ? 0xffff0000u : 0;
    }
    if constexpr (kLate) {
    } else if constexpr (kRead != kAgain)
      w[i].load(a.weight, col, a.H);
    else
      w[i].load_all(a.weight + static_cast<size_t>(at[i]) * Eight<kW>::kBytes);
#pragma unroll
    for (int k = 0; k < 8; ++k) part[i][k] = 0.0f;
  }

  // Of the longest rows the weight is read again with every row as well.
  const auto weight_of = [&](int i) {
    Eight<kW> v = w[i];
    if constexpr (kLate) {
      if constexpr (kRead == kAgain)
        v.load_all(a.weight + static_cast<size_t>(at[i]) * Eight<kW>::kBytes);
      else
        v.load(a.weight, at[i], a.H);
    }
    return v;
  };
  struct Row {
    X x[kUnits], g[kUnits], d[kUnits];
  };
  const bool has_sum = a.grad_sum != nullptr;
  const auto read = [&](Row& v, uint32_t row) {
    const size_t from = static_cast<size_t>(row) * a.H * X::kBytes;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      if constexpr (kRead == kCut) {
        v.x[i].load(a.x + from, at[i], a.H);
        v.g[i].load(a.grad + from, at[i], a.H);
        if (!kLate && has_sum) v.d[i].load(a.grad_sum + from, at[i], a.H);
      } else if constexpr (kRead == kAgain) {
        const size_t to = from + static_cast<size_t>(at[i]) * X::kBytes;
        v.x[i].load_all(a.x + to);
        v.g[i].load_all(a.grad + to);
        // without a grad_sum these are x's again, and not used
        if constexpr (!kLate) v.d[i].load_all((has_sum ? a.grad_sum : a.x) + to);
      } else {
        const uint32_t bytes = a.H * X::kBytes;
        v.x[i].load_whole(WholeRow<>(a.x + from, bytes), at[i]);
        v.g[i].load_whole(WholeRow<>(a.grad + from, bytes), at[i]);
        if constexpr (!kLate) v.d[i].load_whole(WholeRow<>((has_sum ? a.grad_sum : a.x) + from, has_sum ? bytes : 0), at[i]);
      }
    }
  };

  __shared__ f32x2 sh[2][kWaves];
  __shared__ float sh_again[kWaves];
  int turn = 0;
  const auto take = [&](Row& now, uint32_t row) {
    const size_t first = static_cast<size_t>(row) * a.H;
    X(&x)[kUnits] = now.x;
    X(&g)[kUnits] = now.g;
    const auto own_of = [&](int i) {
      X v = x[i];
#pragma unroll
      for (int k = 0; k < X::kWords; ++k) v.w[k] &= kRead == kAgain ? own[i].w[k] : 0xffffffffu;
      return v;
    };
    float sum = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const X own_x = own_of(i);
      const Eight<kW> weight = weight_of(i);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float v = own_x.get(k);
        sum = __builtin_fmaf(v, v, sum);
        dot = __builtin_fmaf(g[i].get(k) * weight.get(k), v, dot);
      }
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) x[i].keep_packed(), g[i].keep_packed(), w[i].keep_packed();
    sum = sum64_f32(sum);
    dot = sum64_f32(dot);
    if constexpr (kWaves > 1) {
      // two buffers in turn: a wave writes the next row's only when all have read this one's
      if (threadIdx.x % 64 == 0) sh[turn][threadIdx.x / 64] = f32x2{sum, dot};
      __syncthreads();
      sum = 0.0f, dot = 0.0f;
#pragma unroll
      for (int v = 0; v < kWaves; ++v) {
        sum += sh[turn][v][0];
        dot += sh[turn][v][1];
      }
    }
    // the same for all lanes of a row
    float up = 1.0f, r, mean;
    if (sum <= kMostSum && (sum >= kLeastSum || a.eps >= kLeastEps) && fabsf(dot) <= kMostSum) {
      r = 1.0f / __builtin_sqrtf(__builtin_fmaf(sum, a.inv_h, a.eps));
      mean = dot * r * a.inv_h;
    } else {
      // sums that leave the range of 32 bits, or are not finite: again of x times a power of
      // two (a row below kLeastSum has values under 2^-49, one above kMostSum some over 2^54),
      // and the second one of n
      up = sum < kLeastSum ? 0x1p60f : sum <= kMostSum ? 1.0f : 0x1p-80f;
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const X own_x = own_of(i);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float v = own_x.get(k) * up;
          sum = __builtin_fmaf(v, v, sum);
        }
      }
      sum = sum_of_row<kWaves>(sum, sh_again);
      r = 1.0f / __builtin_sqrtf(__builtin_fmaf(sum, a.inv_h, a.eps * up * up));
      dot = 0.0f;
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const X own_x = own_of(i);
        const Eight<kW> weight = weight_of(i);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          dot = __builtin_fmaf(g[i].get(k) * weight.get(k), own_x.get(k) * up * r, dot);
      }
      mean = sum_of_row<kWaves>(dot, sh_again) * a.inv_h;
    }
    const float norm = r * up;  // 1 / sqrt(mean(x^2) + eps), where r is that of x up
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      if constexpr (kLate) {
        if (has_sum) now.d[i].load(a.grad_sum + first * X::kBytes, at[i], a.H);
      }
      const X& d = now.d[i];
      const Eight<kW> weight = weight_of(i);
      X out;
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        float v[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float n = x[i].get(k + h) * up * r, gr = g[i].get(k + h);
          part[i][k + h] = __builtin_fmaf(gr, n, part[i][k + h]);
          v[h] = norm * __builtin_fmaf(-n, mean, gr * weight.get(k + h));
          v[h] = has_sum ? v[h] + d.get(k + h) : v[h];
        }
        out.put(k / 2, v[0], v[1]);
      }
      if constexpr (kRead == kCut)
        out.store(a.grad_x + first * X::kBytes, at[i], a.H);
      else if constexpr (kRead == kAgain)
        out.store_all(a.grad_x + (first + at[i]) * X::kBytes);
      else
        out.store_whole(WholeRow<>(a.grad_x + first * X::kBytes, a.H * X::kBytes), at[i]);
    }
    turn ^= 1;
  };
  if constexpr (kAhead) {
    // behind the last row that one once more
    Row one, two;
    uint32_t row = group;
    const auto after = [&](uint32_t r) { return r + a.groups < a.rows ? r + a.groups : r; };
    if (row < a.rows) read(one, row);
    while (row < a.rows) {
      read(two, after(row));
      take(one, row);
      row += a.groups;
      if (row >= a.rows) break;
      read(one, after(row));
      take(two, row);
      row += a.groups;
    }
  } else {
    for (uint32_t row = group; row < a.rows; row += a.groups) {
      Row one;
      read(one, row);
      take(one, row);
    }
  }
  float* mine = a.part + static_cast<size_t>(group) * a.H;
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k)
      if (k >= skip[i] && at[i] + k < a.H) mine[at[i] + k] = part[i][k];
  }
}

// grad_weight from the groups' parts: a workgroup takes 16 columns, each of its 64 rows of
// lanes every 64th group; they are added by lanes, then by waves, in a fixed order.
constexpr int kSumCols = 16, kSumWaves = 16, kSumRows = 64 * kSumWaves / kSumCols;
template <int kW>
__global__ __launch_bounds__(64 * kSumWaves) void rms_norm_weight_kernel(BackArgs a) {
  const uint32_t lane = threadIdx.x % kSumCols, row = threadIdx.x / kSumCols, col = blockIdx.x * kSumCols + lane;
  __shared__ float sh[kSumWaves][kSumCols];
  float sum = 0.0f;
  if (col < a.H) {
    const float* p = a.part + col;
    uint32_t at = row;
    for (; at + 7 * kSumRows < a.groups; at += 8 * kSumRows) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = p[static_cast<size_t>(at + i * kSumRows) * a.H];
      sum += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    }
    for (; at < a.groups; at += kSumRows) sum += p[static_cast<size_t>(at) * a.H];
  }
  sum += __shfl_xor(sum, 16);
  sum += __shfl_xor(sum, 32);
  if (threadIdx.x % 64 < kSumCols) sh[threadIdx.x / 64][lane] = sum;
  __syncthreads();
  if (threadIdx.x >= kSumCols || col >= a.H) return;
  sum = 0.0f;
#pragma unroll
  for (int v = 0; v < kSumWaves; ++v) sum += sh[v][lane];
  Eight<kW> out;
  out.put(0, sum, 0.0f);
  constexpr int kBytes = Eight<kW>::kBytes;
  __builtin_memcpy(a.grad_weight + static_cast<size_t>(col) * kBytes, &out.w[0], kBytes);
}

template <int kX, int kW, int kLanes, int kUnits>
void launch(const BackArgs& a, hipStream_t stream) {
  constexpr uint32_t kAtOnce = kLanes == 64 ? 4 : 1, kThreads = kLanes == 64 ? 256 : kLanes;
  const dim3 grid((a.groups + kAtOnce - 1) / kAtOnce);
  // 32-bit rows of the longest kind leave no registers for reading them another way
  constexpr bool kOneWay = kUnits > 1 && kX == MRR_F32;
  if constexpr (kOneWay || kLanes * kUnits == 64) {
    if (kOneWay || a.H < 8) {
      rms_norm_backward_kernel<kX, kW, kLanes, kUnits, kCut><<<grid, kThreads, 0, stream>>>(a);
      return;
    }
  }
  if constexpr (!kOneWay) {
    const int64_t row = static_cast<int64_t>(a.H) * Eight<kX>::kBytes;
    if constexpr (kX != MRR_F32) {
      if (a.rows * row >= kStreamBytes && whole_units(row, a.x, a.grad, a.grad_sum, a.grad_x)) {
        rms_norm_backward_kernel<kX, kW, kLanes, kUnits, kStreamed><<<grid, kThreads, 0, stream>>>(a);
        return;
      }
    }
    rms_norm_backward_kernel<kX, kW, kLanes, kUnits, kAgain><<<grid, kThreads, 0, stream>>>(a);
  }
}

template <int kX, int kW>
void launch_types(const BackArgs& a, NormShape s, hipStream_t stream) {
  if (a.rows > 0) {
    switch (s.lanes * 16 + s.units) {
      case 64 * 16 + 1: launch<kX, kW, 64, 1>(a, stream); break;
      case 128 * 16 + 1: launch<kX, kW, 128, 1>(a, stream); break;
      case 256 * 16 + 1: launch<kX, kW, 256, 1>(a, stream); break;
      case 512 * 16 + 1: launch<kX, kW, 512, 1>(a, stream); break;
      case 1024 * 16 + 1: launch<kX, kW, 1024, 1>(a, stream); break;
      default: launch<kX, kW, 512, 4>(a, stream); break;
    }
    if (hipPeekAtLastError() != hipSuccess) return;
  }
  rms_norm_weight_kernel<kW><<<(a.H + kSumCols - 1) / kSumCols, 64 * kSumWaves, 0, stream>>>(a);
}

}  // namespace
}  // namespace mrr

extern "C" mrr_status mrr_rms_norm_backward(const mrr_rms_norm_backward_args* args, void* workspace,
                                            size_t workspace_bytes, struct ihipStream_t* stream) {
  using namespace mrr;
  const mrr_status st = check_rms_norm_backward(args, workspace, workspace_bytes);
  if (st != MRR_SUCCESS) return st;
  const NormShape shape = norm_backward_shape(args->H);
  BackArgs a;
  a.grad = static_cast<const uint8_t*>(args->grad);
  a.x = static_cast<const uint8_t*>(args->x);
  a.weight = static_cast<const uint8_t*>(args->weight);
  a.grad_sum = static_cast<const uint8_t*>(args->grad_sum);
  a.grad_x = static_cast<uint8_t*>(args->grad_x);
  a.part = static_cast<float*>(workspace);
  a.grad_weight = static_cast<uint8_t*>(args->grad_weight);
  a.rows = static_cast<uint32_t>(args->rows);
  a.H = static_cast<uint32_t>(args->H);
  a.groups = static_cast<uint32_t>(norm_backward_groups(args->rows, args->H));
  a.eps = static_cast<float>(args->eps);
  a.inv_h = 1.0f / static_cast<float>(args->H);
  const bool same = args->weight_dtype == args->dtype;
  switch (args->dtype) {
    case MRR_F16: same ? launch_types<MRR_F16, MRR_F16>(a, shape, stream) : launch_types<MRR_F16, MRR_F32>(a, shape, stream); break;
    case MRR_BF16:
      same ? launch_types<MRR_BF16, MRR_BF16>(a, shape, stream) : launch_types<MRR_BF16, MRR_F32>(a, shape, stream);
      break;
    default: launch_types<MRR_F32, MRR_F32>(a, shape, stream); break;
  }
  return hipGetLastError() == hipSuccess ? MRR_SUCCESS : MRR_ERROR_HIP;
}
