// mrr_rms_norm.hip -- root-mean-square norm of rows with the residual's addition,
// to rows of the input's type, to int8 or e4m3 rows with a scale each, or to
// microscaled rows (e4m3 or e2m1 values, e8m0 scales of 32).
//
//   s = round(x + residual);  y = w s / sqrt(mean(s^2) + eps)
//
// Bound by memory: a row is read once, kept in registers as it lies there, and
// written once. Rows of 8-bit values with one scale need two numbers of a row,
// sum(s^2) and max |p|, p = w s; both are found in one pass over the registers and
// one barrier, since the norm cancels in the values: y / scale = 127 p / max |p|.
// Of bf16 weights and values p is exact in 32 bits, and so is 127 p (448 p); the
// quotient is q0 + (127 p - q0 max) / max with q0 = 127 p (1 / max), whose remainder is
// exact in one fma, so the rounding to 8 bits is that of the exact quotient, ties
// included, for three instructions a value instead of a division.
//
// Rows whose sum of squares or largest product leave the range of 32 bits (or
// are not finite) are taken again in 64 bits, which their workgroup alone pays for.
#include "mrr_rows.h"

namespace mrr {
namespace {

enum { kWide = 0, kRow = 1, kMx = 2 };  // what is written

struct NormArgs {
  const uint8_t* x;
  const uint8_t* residual;  // or null
  const uint8_t* weight;
  uint8_t* y;
  uint8_t* scales;
  uint8_t* sum;
  uint32_t rows, H;
  float eps;
  double eps64;
  float inv_h;
  int32_t stream;  // rows go past the caches
  int32_t narrow;  // y's type: I8 or F8_E4M3FN with kRow, F8_E4M3FN or F4_E2M1 with kMx
};

// The sums of squares between which 32 bits do for the norm, and the largest products
// from which on they do for a row's scale.
constexpr float kMostSum = 1e37f, kLeastSum = 1e-30f, kLeastTop = 1e-30f, kMostTop = 1e35f;
// A sum of squares below kLeastSum is nothing next to an eps from here on.
constexpr float kLeastEps = 1e-20f;

template <int kLanes>
struct Shared {
  static constexpr int kWaves = kLanes / 64;
  float sum[kWaves];
  uint32_t top[kWaves];
  double sum64[kWaves], top64[kWaves];
};

// 2^(s - 127), s < 255
__device__ __forceinline__ float two_to(uint32_t s) { return __uint_as_float(s == 0 ? 0x00400000u : s << 23); }

__device__ __forceinline__ uint32_t pack_i8(float a, float b, float c, float d) {
  const auto byte = [](float v) { return static_cast<uint32_t>(static_cast<int>(__builtin_rintf(v))) & 0xffu; };
  return byte(a) | byte(b) << 8 | byte(c) << 16 | byte(d) << 24;
}
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true));
}

// n <= 8 bytes of `v` to p
__device__ __forceinline__ void store_bytes(uint8_t* p, uint64_t v, int n) {
  if (n == 8) {
    __builtin_memcpy(p, &v, 8);
  } else {
    for (int k = 0; k < n; ++k) p[k] = static_cast<uint8_t>(v >> (8 * k));
  }
}

template <int kX, int kW, int kOut, int kLanes, int kUnits>
__global__ __launch_bounds__(kLanes < 256 ? 256 : kLanes) void rms_norm_kernel(NormArgs a) {
  constexpr int kThreads = kLanes < 256 ? 256 : kLanes, kAtOnce = kThreads / kLanes;
  const uint32_t lane = threadIdx.x % kLanes;
  const uint32_t row = blockIdx.x * static_cast<uint32_t>(kAtOnce) + (kAtOnce > 1 ? threadIdx.x / kLanes : 0);
  if (kAtOnce > 1 && row >= a.rows) return;  // whole waves, which meet no barrier
  const size_t first = static_cast<size_t>(row) * a.H;

  Eight<kX> s[kUnits];
  Eight<kW> w[kUnits];
  constexpr uint32_t kBytes = Eight<kX>::kBytes;
  const auto col_of = [&](int i) { return 8 * (i * kLanes + lane); };
  const auto load = [&](Eight<kX>(&v)[kUnits], const uint8_t* from) {
    if (a.stream) {
      const WholeRow<> r(from + first * kBytes, a.H * kBytes);
#pragma unroll
      for (int i = 0; i < kUnits; ++i) v[i].load_whole(r, col_of(i));
    } else {
#pragma unroll
      for (int i = 0; i < kUnits; ++i) v[i].load(from + first * kBytes, col_of(i), a.H);
    }
  };
  const auto store = [&](uint8_t* to, int i, const Eight<kX>& v) {
    if (a.stream)
      v.store_whole(WholeRow<>(to + first * kBytes, a.H * kBytes), col_of(i));
    else
      v.store(to + first * kBytes, col_of(i), a.H);
  };
  Eight<kX> add[kUnits];
  load(s, a.x);
  if (a.residual != nullptr) load(add, a.residual);
#pragma unroll
  for (int i = 0; i < kUnits; ++i) w[i].load(a.weight, col_of(i), a.H);
  if (a.residual != nullptr) {
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
#pragma unroll
      for (int k = 0; k < 8; k += 2)
        s[i].put(k / 2, s[i].get(k) + add[i].get(k), s[i].get(k + 1) + add[i].get(k + 1));
      store(a.sum, i, s[i]);
    }
  }

  float sum = 0.0f;
  uint32_t top = 0;  // |p| by its bits, so that infinities and NaN come above every number
#pragma unroll
  for (int i = 0; i < kUnits; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float v = s[i].get(k);
      sum = __builtin_fmaf(v, v, sum);
      if constexpr (kOut == kRow) top = max(top, __float_as_uint(v * w[i].get(k)) & 0x7fffffffu);
    }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) s[i].keep_packed(), w[i].keep_packed();
  sum = sum64_f32(sum);
  if constexpr (kOut == kRow) top = max64_u32(top);
  __shared__ Shared<kLanes> sh;
  if constexpr (kLanes > 64) {
    if (threadIdx.x % 64 == 0) {
      sh.sum[threadIdx.x / 64] = sum;
      if constexpr (kOut == kRow) sh.top[threadIdx.x / 64] = top;
    }
    __syncthreads();
    sum = 0.0f, top = 0;
#pragma unroll
    for (int v = 0; v < kLanes / 64; ++v) {
      sum += sh.sum[v];
      if constexpr (kOut == kRow) top = max(top, sh.top[v]);
    }
  }

  // the same for all lanes of a row
  float most = __uint_as_float(top);
  const bool plain = sum <= kMostSum && (sum >= kLeastSum || a.eps >= kLeastEps) &&
                     (kOut != kRow || top == 0 || (most >= kLeastTop && most <= kMostTop));
  float r = 1.0f / __builtin_sqrtf(__builtin_fmaf(sum, a.inv_h, a.eps));
  double r64 = 0.0, most64 = 0.0;
  bool bad = false;  // a row with one scale and a product that is not finite
  if (!plain) {
    double sum64 = 0.0;
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const double v = s[i].get(k);
        sum64 += v * v;
        if constexpr (kOut == kRow) {
          const double p = fabs(v * static_cast<double>(w[i].get(k)));
          most64 = p <= 1e300 ? fmax(most64, p) : 1e301;  // 32-bit numbers' products are below 1e78
        }
      }
    sum64 = sum64_f64(sum64);
    if constexpr (kOut == kRow) most64 = max64_f64(most64);
    if constexpr (kLanes > 64) {
      if (threadIdx.x % 64 == 0) {
        sh.sum64[threadIdx.x / 64] = sum64;
        sh.top64[threadIdx.x / 64] = most64;
      }
      __syncthreads();
      sum64 = 0.0;
#pragma unroll
      for (int v = 0; v < kLanes / 64; ++v) {
        sum64 += sh.sum64[v];
        most64 = fmax(most64, sh.top64[v]);
      }
    }
    r64 = 1.0 / sqrt(sum64 / a.H + a.eps64);
    bad = most64 > 1e300;
  }

  if constexpr (kOut == kRow) {
    const float full = a.narrow == MRR_I8 ? 127.0f : 448.0f;
    if (lane == 0) {
      const float scale = bad      ? __builtin_nanf("")
                          : !plain ? static_cast<float>(r64 * most64 / full)
                                   : r * (most / full);
      __builtin_memcpy(a.scales + static_cast<size_t>(row) * 4, &scale, 4);
    }
    const float over = top == 0 ? 0.0f : 1.0f / most;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const uint32_t col = col_of(i);
      if (col >= a.H) break;
      float q[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float p = full * (s[i].get(k) * w[i].get(k));
        const float q0 = p * over;
        q[k] = __builtin_fmaf(__builtin_fmaf(-q0, most, p), over, q0);
      }
      if (!plain) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const double p = static_cast<double>(s[i].get(k)) * static_cast<double>(w[i].get(k));
          q[k] = bad || most64 == 0.0 ? 0.0f : static_cast<float>(full * p / most64);
        }
      }
      const uint64_t lo = a.narrow == MRR_I8 ? pack_i8(q[0], q[1], q[2], q[3]) : pack_e4m3(q[0], q[1], q[2], q[3]);
      const uint64_t hi = a.narrow == MRR_I8 ? pack_i8(q[4], q[5], q[6], q[7]) : pack_e4m3(q[4], q[5], q[6], q[7]);
      store_bytes(a.y + first + col, lo | hi << 32, static_cast<int>(min(8u, a.H - col)));
    }
    return;
  }

#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const uint32_t col = col_of(i);
    float y[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = s[i].get(k) * r * w[i].get(k);
    if (!plain) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        y[k] = static_cast<float>(static_cast<double>(s[i].get(k)) * r64 * static_cast<double>(w[i].get(k)));
    }
    if constexpr (kOut == kWide) {
      Eight<kX> out;
#pragma unroll
      for (int k = 0; k < 8; k += 2) out.put(k / 2, y[k], y[k + 1]);
      store(a.y, i, out);
    } else {
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(y[k]) & 0x7fffffffu);
      m = max(m, dpp_u32<kDppXor1>(m));
      m = max(m, dpp_u32<kDppXor2>(m));  // of the block's four lanes
      const uint32_t e = m >> 23, least = a.narrow == MRR_F4_E2M1 ? 2 : 8;
      const uint32_t scale = e == 255 ? 255 : e > least ? e - least : 0;
      if (scale == 255) {
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = 0.0f;
      }
      const uint32_t scale_row = 2 * ((a.H + 63) / 64);
      if (lane % 4 == 0 && col / 32 < scale_row)
        a.scales[static_cast<size_t>(row) * scale_row + col / 32] = static_cast<uint8_t>(scale);
      if (col >= a.H) continue;
      const int n = static_cast<int>(min(8u, a.H - col));
      if (a.narrow == MRR_F4_E2M1) {
        const float by = two_to(scale == 255 ? 127 : scale);
        uint32_t c = 0;
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[0], y[1], by, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[2], y[3], by, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[4], y[5], by, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[6], y[7], by, 3);
        uint8_t* p = a.y + (first + col) / 2;
        if (n == 8) {
          __builtin_memcpy(p, &c, 4);
        } else {
          for (int k = 0; k < n / 2; ++k) p[k] = static_cast<uint8_t>(c >> (8 * k));
        }
      } else {
        // a block's values over its scale are below 512
        const float by = two_to(scale == 255 ? 127 : 254 - scale);
        float q[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) q[k] = __builtin_amdgcn_fmed3f(y[k] * by, -448.0f, 448.0f);
        const uint64_t lo = pack_e4m3(q[0], q[1], q[2], q[3]), hi = pack_e4m3(q[4], q[5], q[6], q[7]);
        store_bytes(a.y + first + col, lo | hi << 32, n);
      }
    }
  }
}

template <int kX, int kW, int kOut, int kLanes, int kUnits>
void launch(const NormArgs& a, hipStream_t stream) {
  constexpr uint32_t kAtOnce = kLanes == 64 ? 4 : 1;
  rms_norm_kernel<kX, kW, kOut, kLanes, kUnits>
      <<<(a.rows + kAtOnce - 1) / kAtOnce, kLanes < 256 ? 256 : kLanes, 0, stream>>>(a);
}

template <int kX, int kW, int kOut>
void launch_shape(const NormArgs& a, NormShape s, hipStream_t stream) {
  switch (s.lanes * 16 + s.units) {
    case 64 * 16 + 1: launch<kX, kW, kOut, 64, 1>(a, stream); break;
    case 64 * 16 + 2: launch<kX, kW, kOut, 64, 2>(a, stream); break;
    case 256 * 16 + 1: launch<kX, kW, kOut, 256, 1>(a, stream); break;
    case 256 * 16 + 2: launch<kX, kW, kOut, 256, 2>(a, stream); break;
    case 256 * 16 + 4: launch<kX, kW, kOut, 256, 4>(a, stream); break;
    case 1024 * 16 + 1: launch<kX, kW, kOut, 1024, 1>(a, stream); break;
    default: launch<kX, kW, kOut, 1024, 2>(a, stream); break;
  }
}

template <int kX, int kW>
void launch_types(const NormArgs& a, int out, NormShape s, hipStream_t stream) {
  if (out == kWide)
    launch_shape<kX, kW, kWide>(a, s, stream);
  else if (out == kRow)
    launch_shape<kX, kW, kRow>(a, s, stream);
  else
    launch_shape<kX, kW, kMx>(a, s, stream);
}

// A launch holds less than 2^32 threads.
constexpr int64_t kRowsPerLaunch = int64_t(1) << 21;
// From so many bytes of rows on they are read, and written, past the caches.
constexpr int64_t kStreamBytes = int64_t(64) << 20;

}  // namespace
}  // namespace mrr

extern "C" mrr_status mrr_rms_norm(const mrr_rms_norm_args* args, struct ihipStream_t* stream) {
  using namespace mrr;
  const mrr_status st = check_rms_norm(args);
  if (st != MRR_SUCCESS) return st;
  const NormShape shape = norm_shape(args->rows, args->H);
  const int out = args->y_dtype == args->dtype ? kWide : args->scales_dtype == MRR_F32 ? kRow : kMx;
  const bool same = args->weight_dtype == args->dtype;
  const int64_t b = args->dtype == MRR_F32 ? 4 : 2;
  const int64_t scale_row = out == kRow ? 4 : 2 * ((args->H + 63) / 64);
  for (int64_t row = 0; row < args->rows; row += kRowsPerLaunch) {
    const int64_t rows = args->rows - row < kRowsPerLaunch ? args->rows - row : kRowsPerLaunch;
    const int64_t at = row * args->H;
    NormArgs a;
    a.x = static_cast<const uint8_t*>(args->x) + at * b;
    a.residual = args->residual == nullptr ? nullptr : static_cast<const uint8_t*>(args->residual) + at * b;
    a.weight = static_cast<const uint8_t*>(args->weight);
    a.y = static_cast<uint8_t*>(args->y) + (out == kWide ? at * b : args->y_dtype == MRR_F4_E2M1 ? at / 2 : at);
    a.scales = out == kWide ? nullptr : static_cast<uint8_t*>(args->scales) + row * scale_row;
    a.sum = args->sum == nullptr ? nullptr : static_cast<uint8_t*>(args->sum) + at * b;
    a.rows = static_cast<uint32_t>(rows);
    a.H = static_cast<uint32_t>(args->H);
    a.eps = static_cast<float>(args->eps);
    a.eps64 = args->eps;
    a.inv_h = 1.0f / static_cast<float>(args->H);
    a.stream = args->rows * args->H * b >= kStreamBytes &&
               whole_units(args->H * b, a.x, a.residual, a.sum, out == kWide ? a.y : nullptr);
    a.narrow = args->y_dtype;
    switch (args->dtype) {
      case MRR_F16:
        same ? launch_types<MRR_F16, MRR_F16>(a, out, shape, stream) : launch_types<MRR_F16, MRR_F32>(a, out, shape, stream);
        break;
      case MRR_BF16:
        same ? launch_types<MRR_BF16, MRR_BF16>(a, out, shape, stream)
             : launch_types<MRR_BF16, MRR_F32>(a, out, shape, stream);
        break;
      default: launch_types<MRR_F32, MRR_F32>(a, out, shape, stream); break;
    }
    if (hipGetLastError() != hipSuccess) return MRR_ERROR_HIP;
  }
  return MRR_SUCCESS;
}
