// mrr_rms_norm_backward.hip -- the gradient of the root-mean-square norm:
//
//   n = x r, r = 1 / sqrt(mean(x^2) + eps)
//   grad_x = r (g w - n mean(g w n)) + grad_sum,  grad_weight = sum over rows of g n
//
// Bound by memory: three rows in (x, g, grad_sum), one out, two sums of a row (x^2 and
// g w x) in one barrier. A workgroup takes every so-manieth row and keeps its part of
// grad_weight in registers; the parts, fp32, go to the workspace, and a second kernel
// adds them in a fixed order, so that the result is the same each time.
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

template <int kX, int kW, int kLanes, int kUnits>
__global__ __launch_bounds__(kLanes < 256 ? 256 : kLanes) void rms_norm_backward_kernel(BackArgs a) {
  constexpr int kThreads = kLanes < 256 ? 256 : kLanes, kAtOnce = kThreads / kLanes, kWaves = kLanes / 64;
  using X = Eight<kX>;
  const uint32_t lane = threadIdx.x % kLanes;
  const uint32_t group = blockIdx.x * static_cast<uint32_t>(kAtOnce) + (kAtOnce > 1 ? threadIdx.x / kLanes : 0);
  if (kAtOnce > 1 && group >= a.groups) return;  // whole waves, which meet no barrier

  float part[kUnits][8];
  Eight<kW> w[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    w[i].template load<false>(a.weight, 8 * (i * kLanes + lane), a.H);
#pragma unroll
    for (int k = 0; k < 8; ++k) part[i][k] = 0.0f;
  }

  __shared__ f32x2 sh[2][kWaves];
  __shared__ float sh_again[kWaves];
  int turn = 0;
  for (uint32_t row = group; row < a.rows; row += a.groups, turn ^= 1) {
    const size_t first = static_cast<size_t>(row) * a.H;
    X x[kUnits], g[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const uint32_t col = 8 * (i * kLanes + lane);
      x[i].template load<false>(a.x + first * X::kBytes, col, a.H);
      g[i].template load<false>(a.grad + first * X::kBytes, col, a.H);
    }
    float sum = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float v = x[i].get(k);
        sum = __builtin_fmaf(v, v, sum);
        dot = __builtin_fmaf(g[i].get(k) * w[i].get(k), v, dot);
      }
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
      for (int i = 0; i < kUnits; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float v = x[i].get(k) * up;
          sum = __builtin_fmaf(v, v, sum);
        }
      sum = sum_of_row<kWaves>(sum, sh_again);
      r = 1.0f / __builtin_sqrtf(__builtin_fmaf(sum, a.inv_h, a.eps * up * up));
      dot = 0.0f;
#pragma unroll
      for (int i = 0; i < kUnits; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k)
          dot = __builtin_fmaf(g[i].get(k) * w[i].get(k), x[i].get(k) * up * r, dot);
      mean = sum_of_row<kWaves>(dot, sh_again) * a.inv_h;
    }
    const float norm = r * up;  // 1 / sqrt(mean(x^2) + eps), where r is that of x up
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const uint32_t col = 8 * (i * kLanes + lane);
      X d;
      if (a.grad_sum != nullptr) d.template load<false>(a.grad_sum + first * X::kBytes, col, a.H);
      X out;
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        float v[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float n = x[i].get(k + h) * up * r, gr = g[i].get(k + h);
          part[i][k + h] = __builtin_fmaf(gr, n, part[i][k + h]);
          v[h] = norm * __builtin_fmaf(-n, mean, gr * w[i].get(k + h));
          if (a.grad_sum != nullptr) v[h] += d.get(k + h);
        }
        out.put(k / 2, v[0], v[1]);
      }
      if (col < a.H) out.template store<false>(a.grad_x + first * X::kBytes, col, a.H);
    }
  }
  float* mine = a.part + static_cast<size_t>(group) * a.H;
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const uint32_t col = 8 * (i * kLanes + lane);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (col + k < a.H) mine[col + k] = part[i][k];
  }
}

// grad_weight from the groups' parts: a workgroup takes 64 columns, each of its 16
// waves every sixteenth group, and the first wave adds the waves' sums in their order.
constexpr int kSumWaves = 16;
template <int kW>
__global__ __launch_bounds__(64 * kSumWaves) void rms_norm_weight_kernel(BackArgs a) {
  const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64, col = blockIdx.x * 64 + lane;
  __shared__ float sh[kSumWaves][64];
  float sum = 0.0f;
  if (col < a.H) {
    const float* p = a.part + col;
    uint32_t at = wave;
    for (; at + 3 * kSumWaves < a.groups; at += 4 * kSumWaves) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = p[static_cast<size_t>(at + i * kSumWaves) * a.H];
      sum += (v[0] + v[1]) + (v[2] + v[3]);
    }
    for (; at < a.groups; at += kSumWaves) sum += p[static_cast<size_t>(at) * a.H];
  }
  sh[wave][lane] = sum;
  __syncthreads();
  if (wave != 0 || col >= a.H) return;
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
  constexpr uint32_t kAtOnce = kLanes == 64 ? 4 : 1;
  rms_norm_backward_kernel<kX, kW, kLanes, kUnits>
      <<<(a.groups + kAtOnce - 1) / kAtOnce, kLanes < 256 ? 256 : kLanes, 0, stream>>>(a);
}

template <int kX, int kW>
void launch_types(const BackArgs& a, NormShape s, hipStream_t stream) {
  if (a.rows > 0) {
    switch (s.lanes * 16 + s.units) {
      case 64 * 16 + 1: launch<kX, kW, 64, 1>(a, stream); break;
      case 64 * 16 + 2: launch<kX, kW, 64, 2>(a, stream); break;
      case 256 * 16 + 1: launch<kX, kW, 256, 1>(a, stream); break;
      case 256 * 16 + 2: launch<kX, kW, 256, 2>(a, stream); break;
      case 256 * 16 + 4: launch<kX, kW, 256, 4>(a, stream); break;
      case 512 * 16 + 2: launch<kX, kW, 512, 2>(a, stream); break;
      default: launch<kX, kW, 512, 4>(a, stream); break;
    }
  }
  rms_norm_weight_kernel<kW><<<(a.H + 63) / 64, 64 * kSumWaves, 0, stream>>>(a);
}

}  // namespace
}  // namespace mrr

extern "C" mrr_status mrr_rms_norm_backward(const mrr_rms_norm_backward_args* args, void* workspace,
                                            size_t workspace_bytes, struct ihipStream_t* stream) {
  using namespace mrr;
  const mrr_status st = check_rms_norm_backward(args, workspace, workspace_bytes);
  if (st != MRR_SUCCESS) return st;
  const NormShape shape = norm_backward_shape(args->rows, args->H);
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
