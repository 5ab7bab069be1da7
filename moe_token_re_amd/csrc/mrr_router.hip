// mrr_router.hip -- the router's choice of experts from its logits, and its gradient.
//
// A token's logits lie on 16 lanes (up to 256 experts; on 64 above), four neighbouring
// ones a lane and load. Each becomes one number that has the logit's order and, among
// equal logits, the experts' falling one, so that no two are equal: of a 16-bit logit 32
// bits, of a 32-bit one a 64-bit float whose last bits, which the logit leaves zeros, hold
// the expert. A lane sorts its numbers, and in four steps (six of 64 lanes) pairs of lanes
// join their lists and keep the largest, until all have the token's. Every exchange is a
// maximum and a minimum, and none waits for a choice before it: top_k rounds that search
// the largest left and its place, and take it out, take twice the instructions (16384
// tokens, 8 of 256 experts: 12.9 us against 9.3; its 17 MB take 3).
#include "mrr_rows.h"

namespace mrr {
namespace {

constexpr int kThreads = 256;

// How lanes are paired in a step; lanes that were joined before hold the same.
constexpr int step_ctrl(int step) {
  return step == 0 ? kDppXor1 : step == 1 ? kDppXor2 : step == 2 ? kDppMirror8 : kDppMirror16;
}

// Numbers of a logit's order. None: -inf, which is never chosen, and what is no logit;
// NaN comes above all, and both zeros are alike.
template <int kDtype>
struct Ordered {  // of 16 bits: (order, expert) in 32
  using T = uint32_t;
  static constexpr T kNone = 0;
  static __device__ __forceinline__ T make(float l, uint32_t e) {
    uint32_t b;
    if constexpr (kDtype == MRR_BF16)
      b = __float_as_uint(l + 0.0f) >> 16;
    else
      b = __builtin_bit_cast(uint16_t, static_cast<_Float16>(l + 0.0f));
    const uint32_t order = l != l ? 0xffffu : b & 0x8000u ? ~b & 0xffffu : b | 0x8000u;
    return l == -INFINITY ? kNone : order << 16 | (0xffffu - e);
  }
  static __device__ __forceinline__ uint32_t expert(T v) { return 0xffffu - (v & 0xffffu); }
  static __device__ __forceinline__ float value(T v) {
    const uint32_t order = v >> 16, b = order & 0x8000u ? order & 0x7fffu : ~order & 0xffffu;
    if (v == kNone) return -INFINITY;
    if (order == 0xffffu) return __builtin_nanf("");
    if constexpr (kDtype == MRR_BF16) return __uint_as_float(b << 16);
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(b)));
  }
  static __device__ __forceinline__ void order(T& a, T& b) {
    const T hi = max(a, b);
    b = min(a, b);
    a = hi;
  }
  static __device__ __forceinline__ T larger(T a, T b) { return max(a, b); }
  template <int kStep>
  static __device__ __forceinline__ T of_lane(T v) {
    if constexpr (kStep < 4) return dpp_u32<step_ctrl(kStep)>(v);
    return static_cast<T>(__shfl_xor(static_cast<int>(v), 1 << kStep));
  }
};
template <>
struct Ordered<MRR_F32> {
  using T = uint64_t;  // a float of 64 bits, never a NaN
  static constexpr uint32_t kNoneHigh = 0xffe00000u, kInfHigh = 0x7fd00000u, kNanHigh = 0x7fe00000u;
  static constexpr T kNone = static_cast<T>(kNoneHigh) << 32;
  static constexpr uint32_t kExperts = 0x3ffu;
  static __device__ __forceinline__ T make(float l, uint32_t e) {
    const T wide = __builtin_bit_cast(T, static_cast<double>(l + 0.0f));
    const uint32_t high = static_cast<uint32_t>(wide >> 32);
    const uint32_t low = static_cast<uint32_t>(wide) | (high & 0x80000000u ? e : kExperts - e);
    const uint32_t odd = l != l ? kNanHigh : l > 0.0f ? kInfHigh : kNoneHigh;
    if (fabsf(l) < INFINITY) return static_cast<T>(high) << 32 | low;
    return static_cast<T>(odd) << 32 | (odd == kNoneHigh ? 0 : kExperts - e);
  }
  static __device__ __forceinline__ uint32_t expert(T v) {
    const uint32_t low = static_cast<uint32_t>(v) & kExperts;
    return v >> 63 ? low : kExperts - low;
  }
  static __device__ __forceinline__ float value(T v) {
    const uint32_t high = static_cast<uint32_t>(v >> 32);
    if (high == kNoneHigh) return -INFINITY;
    if (high == kNanHigh) return __builtin_nanf("");
    if (high == kInfHigh) return INFINITY;
    return static_cast<float>(__builtin_bit_cast(double, v & ~static_cast<T>(kExperts)));
  }
  // The instructions by name: the compiler would first make sure of each operand that it
  // is no signalling NaN.
  static __device__ __forceinline__ T larger(T a, T b) {
    T r;
    asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
  }
  static __device__ __forceinline__ T smaller(T a, T b) {
    T r;
    asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
  }
  static __device__ __forceinline__ void order(T& a, T& b) {
    const T hi = larger(a, b);
    b = smaller(a, b);
    a = hi;
  }
  template <int kStep>
  static __device__ __forceinline__ T of_lane(T v) {
    const uint32_t low = Ordered<MRR_BF16>::of_lane<kStep>(static_cast<uint32_t>(v));
    return static_cast<T>(Ordered<MRR_BF16>::of_lane<kStep>(static_cast<uint32_t>(v >> 32))) << 32 | low;
  }
};

// Sorts a lane's numbers, the largest first (odd-even merges).
template <typename O, int kN>
__device__ __forceinline__ void sort_list(typename O::T (&v)[kN]) {
#pragma unroll
  for (int p = 1; p < kN; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < kN; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < kN && (i + j) / (2 * p) == (i + j + k) / (2 * p)) O::order(v[i + j], v[i + j + k]);
}

// The kKeep largest of a lane's list and its partner's, by lists of twice the length
// until they are as long.
template <typename O, int kStep, int kSteps, int kKeep, int kN>
__device__ __forceinline__ void join_lists(const typename O::T (&v)[kN], typename O::T (&out)[kKeep]) {
  if constexpr (kStep == kSteps) {
#pragma unroll
    for (int i = 0; i < kKeep; ++i) out[i] = i < kN ? v[i] : O::kNone;
  } else {
    constexpr int kNext = kN >= kKeep ? kKeep : 2 * kN;
    typename O::T next[kNext];
    // a falling list and the other's, reversed: first rising, then falling, or the other way
    if constexpr (kN >= kKeep) {
#pragma unroll
      for (int i = 0; i < kKeep; ++i) next[i] = O::larger(v[i], O::template of_lane<kStep>(v[kKeep - 1 - i]));
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i) next[i] = v[i], next[2 * kN - 1 - i] = O::template of_lane<kStep>(v[i]);
    }
#pragma unroll
    for (int k = kNext / 2; k >= 1; k /= 2)
#pragma unroll
      for (int i = 0; i < kNext; ++i)
        if ((i & k) == 0) O::order(next[i], next[i + k]);
    join_lists<O, kStep + 1, kSteps, kKeep>(next, out);
  }
}

// e^x of x <= 0 (or NaN): 2^(x log2 e), the product's rounding made good to first order. 0 below
// e^-87, which is nothing in a sum that e^0 is part of; with kAll down to the smallest numbers
// of 32 bits, which the instruction would not give.
template <bool kAll = false>
__device__ __forceinline__ float exp_of(float x) {
  constexpr double kLog2E = 1.4426950408889634, kLn2 = 0.6931471805599453;
  constexpr float kHi = static_cast<float>(kLog2E), kLo = static_cast<float>(kLog2E - static_cast<double>(kHi));
  const float hi = x * kHi, lo = __builtin_fmaf(x, kLo, __builtin_fmaf(x, kHi, -hi));
  const bool below = kAll && hi < -125.0f;  // hi + 64 is exact there
  const float e = __builtin_amdgcn_exp2f(below ? hi + 64.0f : hi);
  const float r = __builtin_fmaf(e, lo * static_cast<float>(kLn2), e);
  return x < (kAll ? -104.0f : -87.0f) ? 0.0f : below ? r * 0x1p-64f : r;
}

template <int kLanes>
__device__ __forceinline__ float group_max(float v) {
  v = fmaxf(v, dpp_f32<kDppXor1>(v));
  v = fmaxf(v, dpp_f32<kDppXor2>(v));
  v = fmaxf(v, dpp_f32<kDppMirror8>(v));
  v = fmaxf(v, dpp_f32<kDppMirror16>(v));
  if constexpr (kLanes == 64) {
    v = fmaxf(v, __shfl_xor(v, 16));
    v = fmaxf(v, __shfl_xor(v, 32));
  }
  return v;
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

// kKeep: at least top_k.
template <int kDtype, int kLanes, int kFours, int kKeep>
__global__ __launch_bounds__(kThreads) void router_kernel(RouterArgs a) {
  using O = Ordered<kDtype>;
  constexpr int kBytes = kDtype == MRR_F32 ? 4 : 2, kSteps = kLanes == 64 ? 6 : 4;
  const uint32_t lane = threadIdx.x % kLanes;
  const uint32_t token = blockIdx.x * static_cast<uint32_t>(kThreads / kLanes) + threadIdx.x / kLanes;
  if (token >= a.T) return;  // whole tokens' lanes, which only meet their own
  const uint8_t* row = a.logits + static_cast<size_t>(token) * a.E * kBytes;
  float l[kFours][4];
  typename O::T list[4 * kFours], best[kKeep];
#pragma unroll
  for (int i = 0; i < kFours; ++i) load_four<kDtype>(l[i], row, 4 * (i * kLanes + lane), a.E);
#pragma unroll
  for (int i = 0; i < kFours; ++i)
#pragma unroll
    for (int b = 0; b < 4; ++b) list[4 * i + b] = O::make(l[i][b], 4 * (i * kLanes + lane) + b);
  sort_list<O>(list);
  join_lists<O, 0, kSteps, kKeep>(list, best);
  const float top = O::value(best[0]);
  typename O::T mine = O::kNone;  // lane r's: the r-th
#pragma unroll
  for (int r = 0; r < kKeep; ++r) mine = static_cast<int>(lane) == r ? best[r] : mine;
  const bool chosen = mine != O::kNone && lane < a.k;
  const float p = chosen ? exp_of<true>(O::value(mine) - top) : 0.0f;
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
    a.weight[to] = chosen ? p / sum : 0.0f;
    a.ids[to] = chosen ? static_cast<int32_t>(O::expert(mine)) : -1;
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
    float top = -INFINITY;  // of what is no NaN; one makes every value NaN by itself
#pragma unroll
    for (int i = 0; i < kFours; ++i)
#pragma unroll
      for (int b = 0; b < 4; ++b) top = fmaxf(top, l[i][b]);
    top = group_max<kLanes>(top);
    if (top == -INFINITY) {  // the same for all lanes of a token
      float odd = 0.0f;
#pragma unroll
      for (int i = 0; i < kFours; ++i)
#pragma unroll
        for (int b = 0; b < 4; ++b) odd = l[i][b] != l[i][b] ? 1.0f : odd;
      none = group_max<kLanes>(odd) == 0.0f;
    }
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
  const dim3 grid((a.T + kTokens - 1) / kTokens);
  if (a.k <= 4)
    router_kernel<kDtype, kLanes, kFours, 4><<<grid, kThreads, 0, stream>>>(a);
  else if (a.k <= 8)
    router_kernel<kDtype, kLanes, kFours, 8><<<grid, kThreads, 0, stream>>>(a);
  else
    router_kernel<kDtype, kLanes, kFours, 16><<<grid, kThreads, 0, stream>>>(a);
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
