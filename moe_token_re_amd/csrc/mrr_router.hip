// mrr_router.hip -- the router's choice of experts from its logits, and its gradient.
//
// A token's logits lie on 16 lanes (up to 256 experts; on 64 above), four neighbouring
// ones a lane and load, as unsigned keys of their order. A round finds the largest key
// left and the lowest expert that has it by four DPP steps each (six with 64 lanes), and
// lane r of the token keeps round r's. Bound by the rounds' instructions: about 2 per
// value and round, which 16 lanes a token share among four tokens a wave.
#include "mrr_rows.h"

namespace mrr {
namespace {

constexpr int kThreads = 256;

// A logit as an unsigned key of the same order; 0 for -inf (never chosen), NaN above
// all, both zeros alike.
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t b = __float_as_uint(l + 0.0f);
  if (l != l) return 0xffffffffu;
  if (b == 0xff800000u) return 0;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  if (key == 0) return -INFINITY;
  return __uint_as_float(key & 0x80000000u ? key == 0xffffffffu ? 0x7fc00000u : key ^ 0x80000000u : ~key);
}

// e^x of x <= 0 (or NaN): 2^(x log2 e), the product's rounding made good to first order.
__device__ __forceinline__ float exp_of(float x) {
  constexpr double kLog2E = 1.4426950408889634, kLn2 = 0.6931471805599453;
  constexpr float kHi = static_cast<float>(kLog2E), kLo = static_cast<float>(kLog2E - static_cast<double>(kHi));
  const float hi = x * kHi, lo = __builtin_fmaf(x, kLo, __builtin_fmaf(x, kHi, -hi));
  const float e = __builtin_amdgcn_exp2f(hi);
  return x < -87.0f ? 0.0f : __builtin_fmaf(e, lo * static_cast<float>(kLn2), e);
}

template <int kLanes>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  return kLanes == 64 ? max64_u32(v) : max16_u32(v);
}
template <int kLanes>
__device__ __forceinline__ float group_sum(float v) {
  return kLanes == 64 ? sum64_f32(v) : sum16_f32(v);
}

// Four neighbouring logits of a row, -inf behind its end.
template <int kDtype>
__device__ __forceinline__ void load_four(float (&v)[4], const uint8_t* row, uint32_t col, uint32_t E) {
  constexpr int kBytes = kDtype == MRR_F32 ? 4 : 2;
  uint32_t w[4] = {};
  const uint8_t* p = row + col * kBytes;
  if (col + 4 <= E) {
    __builtin_memcpy(w, p, 4 * kBytes);
  } else {
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (col + k < E) {
        if constexpr (kBytes == 4) {
          __builtin_memcpy(&w[k], p + 4 * k, 4);
        } else {
          uint16_t h;
          __builtin_memcpy(&h, p + 2 * k, 2);
          w[k / 2] |= static_cast<uint32_t>(h) << (k % 2 * 16);
        }
      }
  }
  Eight<kDtype> e;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (kBytes == 4)
      e.w[k] = w[k];
    else
      e.w[k / 2] = w[k / 2];
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = col + k < E ? e.get(k) : -INFINITY;
}

struct RouterArgs {
  const uint8_t* logits;
  float* weight;
  int32_t* ids;
  uint32_t T, E, k;
  int32_t renormalize;
};

template <int kDtype, int kLanes, int kFours>
__global__ __launch_bounds__(kThreads) void router_kernel(RouterArgs a) {
  constexpr int kBytes = kDtype == MRR_F32 ? 4 : 2;
  const uint32_t lane = threadIdx.x % kLanes;
  const uint32_t token = blockIdx.x * static_cast<uint32_t>(kThreads / kLanes) + threadIdx.x / kLanes;
  if (token >= a.T) return;  // whole tokens' lanes, which only meet their own
  const uint8_t* row = a.logits + static_cast<size_t>(token) * a.E * kBytes;
  float l[kFours][4];
  uint32_t key[kFours][4], best = 0;
#pragma unroll
  for (int i = 0; i < kFours; ++i) load_four<kDtype>(l[i], row, 4 * (i * kLanes + lane), a.E);
#pragma unroll
  for (int i = 0; i < kFours; ++i)
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      key[i][b] = key_of(l[i][b]);
      best = max(best, key[i][b]);
    }
  best = group_max<kLanes>(best);
  const float top = value_of(best);
  uint32_t mine = 0, id = 0xffffffffu;  // lane r's: the key and expert of round r
  for (uint32_t r = 0; r < a.k; ++r) {
    if (r > 0) {
      best = 0;
#pragma unroll
      for (int i = 0; i < kFours; ++i)
#pragma unroll
        for (int b = 0; b < 4; ++b) best = max(best, key[i][b]);
      best = group_max<kLanes>(best);
    }
    uint32_t at = 0xffffffffu;
    const uint32_t first = 4 * lane;
#pragma unroll
    for (int i = kFours - 1; i >= 0; --i)
#pragma unroll
      for (int b = 3; b >= 0; --b)
        if (key[i][b] == best) at = first + 4 * i * kLanes + b;
    at = ~group_max<kLanes>(~at);  // the lowest
#pragma unroll
    for (int i = 0; i < kFours; ++i)
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (at == first + 4 * i * kLanes + b) key[i][b] = 0;
    if (lane == r && best != 0) mine = best, id = at;
  }
  const float p = id != 0xffffffffu ? exp_of(value_of(mine) - top) : 0.0f;
  float sum = p;
  if (!a.renormalize) {
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kFours; ++i)
#pragma unroll
      for (int b = 0; b < 4; ++b) sum += exp_of(l[i][b] - top);
  }
  sum = group_sum<kLanes>(sum);
  if (lane < a.k) {
    const size_t to = static_cast<size_t>(token) * a.k + lane;
    a.weight[to] = id != 0xffffffffu ? p / sum : 0.0f;
    a.ids[to] = static_cast<int32_t>(id);
  }
}

struct RouterBackArgs {
  const float* grad;
  const uint8_t* logits;
  const float* weight;
  const int32_t* ids;
  uint8_t* out;
  uint32_t T, E, k;
  int32_t renormalize;
};

// The chosen experts' gradients go to their lanes by way of LDS.
template <int kDtype, int kLanes, int kFours>
__global__ __launch_bounds__(kThreads) void router_backward_kernel(RouterBackArgs a) {
  constexpr int kBytes = kDtype == MRR_F32 ? 4 : 2, kTokens = kThreads / kLanes;
  __shared__ float4 sh[kTokens][kFours * kLanes];
  const uint32_t lane = threadIdx.x % kLanes, in_group = threadIdx.x / kLanes;
  const uint32_t token = blockIdx.x * static_cast<uint32_t>(kTokens) + in_group;
  const bool here = token < a.T;
  const uint8_t* row = a.logits + static_cast<size_t>(here ? token : 0) * a.E * kBytes;
  float l[kFours][4];
  if (!a.renormalize && here) {
#pragma unroll
    for (int i = 0; i < kFours; ++i) load_four<kDtype>(l[i], row, 4 * (i * kLanes + lane), a.E);
  }
  float g = 0.0f, p = 0.0f;
  uint32_t id = 0xffffffffu;
  if (here && lane < a.k) {
    const size_t at = static_cast<size_t>(token) * a.k + lane;
    id = static_cast<uint32_t>(a.ids[at]);
    if (id < a.E) g = a.grad[at], p = a.weight[at];
  }
#pragma unroll
  for (int i = 0; i < kFours; ++i) sh[in_group][i * kLanes + lane] = float4{0.0f, 0.0f, 0.0f, 0.0f};
  const float mean = group_sum<kLanes>(g * p);
  __syncthreads();
  if (id < a.E) reinterpret_cast<float*>(sh[in_group])[id] = a.renormalize ? p * (g - mean) : g;
  __syncthreads();
  if (!here) return;
  uint8_t* out = a.out + static_cast<size_t>(token) * a.E * kBytes;
  float sum = 0.0f;
  bool none = false;  // every logit is -inf
  if (!a.renormalize) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < kFours; ++i)
#pragma unroll
      for (int b = 0; b < 4; ++b) best = max(best, key_of(l[i][b]));
    best = group_max<kLanes>(best);
    const float top = value_of(best);
    none = best == 0;
#pragma unroll
    for (int i = 0; i < kFours; ++i)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        l[i][b] = exp_of(l[i][b] - top);
        sum += l[i][b];
      }
    sum = 1.0f / group_sum<kLanes>(sum);
  }
#pragma unroll
  for (int i = 0; i < kFours; ++i) {
    const uint32_t col = 4 * (i * kLanes + lane);
    const float4 v = sh[in_group][i * kLanes + lane];
    float d[4] = {v.x, v.y, v.z, v.w};
    if (!a.renormalize) {
#pragma unroll
      for (int b = 0; b < 4; ++b) d[b] = none ? 0.0f : l[i][b] * sum * (d[b] - mean);
    }
    Eight<kDtype> e;
    e.put(0, d[0], d[1]);
    e.put(1, d[2], d[3]);
    uint8_t* to = out + col * kBytes;
    if (col + 4 <= a.E) {
      __builtin_memcpy(to, e.w, 4 * kBytes);
    } else {
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (col + k < a.E) {
          if constexpr (kBytes == 4) {
            __builtin_memcpy(to + 4 * k, &e.w[k], 4);
          } else {
            const uint16_t h = static_cast<uint16_t>(e.w[k / 2] >> (k % 2 * 16));
            __builtin_memcpy(to + 2 * k, &h, 2);
          }
        }
    }
  }
}

template <int kDtype, int kLanes, int kFours>
void launch(const RouterArgs& a, hipStream_t stream) {
  constexpr uint32_t kTokens = kThreads / kLanes;
  router_kernel<kDtype, kLanes, kFours><<<(a.T + kTokens - 1) / kTokens, kThreads, 0, stream>>>(a);
}
template <int kDtype, int kLanes, int kFours>
void launch(const RouterBackArgs& a, hipStream_t stream) {
  constexpr uint32_t kTokens = kThreads / kLanes;
  router_backward_kernel<kDtype, kLanes, kFours><<<(a.T + kTokens - 1) / kTokens, kThreads, 0, stream>>>(a);
}

template <int kDtype, typename Args>
void launch_size(const Args& a, hipStream_t stream) {
  if (a.E <= 64)
    launch<kDtype, 16, 1>(a, stream);
  else if (a.E <= 128)
    launch<kDtype, 16, 2>(a, stream);
  else if (a.E <= 256)
    launch<kDtype, 16, 4>(a, stream);
  else if (a.E <= 512)
    launch<kDtype, 64, 2>(a, stream);
  else
    launch<kDtype, 64, 4>(a, stream);
}

template <typename Args>
mrr_status launch_dtype(const Args& a, int32_t dtype, hipStream_t stream) {
  switch (dtype) {
    case MRR_F16: launch_size<MRR_F16>(a, stream); break;
    case MRR_BF16: launch_size<MRR_BF16>(a, stream); break;
    default: launch_size<MRR_F32>(a, stream); break;
  }
  return hipGetLastError() == hipSuccess ? MRR_SUCCESS : MRR_ERROR_HIP;
}

// A launch holds less than 2^32 threads.
constexpr int64_t kTokensPerLaunch = int64_t(1) << 24;

}  // namespace
}  // namespace mrr

extern "C" mrr_status mrr_router(const mrr_router_args* args, struct ihipStream_t* stream) {
  using namespace mrr;
  mrr_status st = check_router(args);
  const int64_t b = st == MRR_SUCCESS && args->dtype == MRR_F32 ? 4 : 2;
  for (int64_t t = 0; st == MRR_SUCCESS && t < args->T; t += kTokensPerLaunch) {
    const int64_t n = args->T - t < kTokensPerLaunch ? args->T - t : kTokensPerLaunch;
    const RouterArgs a{static_cast<const uint8_t*>(args->logits) + t * args->E * b, args->expert_weight + t * args->top_k,
                       args->expert_ids + t * args->top_k, static_cast<uint32_t>(n), static_cast<uint32_t>(args->E),
                       static_cast<uint32_t>(args->top_k), static_cast<int32_t>(args->renormalize)};
    st = launch_dtype(a, args->dtype, stream);
  }
  return st;
}

extern "C" mrr_status mrr_router_backward(const mrr_router_backward_args* args, struct ihipStream_t* stream) {
  using namespace mrr;
  mrr_status st = check_router_backward(args);
  const int64_t b = st == MRR_SUCCESS && args->dtype == MRR_F32 ? 4 : 2;
  for (int64_t t = 0; st == MRR_SUCCESS && t < args->T; t += kTokensPerLaunch) {
    const int64_t n = args->T - t < kTokensPerLaunch ? args->T - t : kTokensPerLaunch;
    const uint8_t* logits = args->renormalize ? nullptr : static_cast<const uint8_t*>(args->logits) + t * args->E * b;
    const RouterBackArgs a{args->grad_weight + t * args->top_k, logits, args->expert_weight + t * args->top_k,
                           args->expert_ids + t * args->top_k, static_cast<uint8_t*>(args->grad_logits) + t * args->E * b,
                           static_cast<uint32_t>(n), static_cast<uint32_t>(args->E), static_cast<uint32_t>(args->top_k),
                           static_cast<int32_t>(args->renormalize)};
    st = launch_dtype(a, args->dtype, stream);
  }
  return st;
}
