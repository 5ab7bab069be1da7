// mrr_rms_norm.hip -- root-mean-square norm of rows with the residual's addition,
// to rows of the input's type, to int8 or e4m3 rows with a scale each, or to
// microscaled rows (e4m3 or e2m1 values, e8m0 scales of 32).
//
//   s = round(x + residual);  y = w s / sqrt(mean(s^2) + eps)
//
// Bound by memory: a row is read once, kept in registers as it lies there, and
// written once (16384 x 7168 bf16 with a residual to fp8 rows: 123 us, 6.7 TB/s of 823 MB,
// which is what a plain copy of 1 GiB by waves of 1 KiB reaches; with the values kept wide over
// the sums, and half as many waves, 138). Rows of 8-bit values with one scale need two numbers of a row,
// sum(s^2) and max |p|, p = w s; both are found in one pass over the registers and
// one barrier, since the norm cancels in the values: y / scale = 127 p / max |p|.
// Of bf16 weights and values p is exact in 32 bits, and so is 127 p (448 p); the
// quotient is q0 + (127 p - q0 max) / max with q0 = 127 p (1 / max), whose remainder is
// exact in one fma, so the rounding to 8 bits is that of the exact quotient, ties
// included, for three instructions a value instead of a division.
//
// Other values with few bits are rounded from 32-bit numbers that are off by less than
// kDoubt of themselves. Where a number so much smaller and one so much larger are rounded
// otherwise, which is in about one row of 7168 values of seven, the row is taken again in
// 64 bits, whose roundings to 32 on the way keep on which side of a border a number lay
// (mrr_quotient.h; a quotient's exact number, whatever the rows' type).
// So is a row whose sum of squares or largest product leaves the range of 32 bits, is not
// finite, or is nothing there though the row is not of zeros.
#include "mrr_quotient.h"
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

// What a 32-bit y (or a product over the largest) may be off by: the sum of squares has at
// most 4 additions a lane and column, 3 over the columns, 6 over a wave, 4 over waves, and
// half of that counts; the mean, root, reciprocal, two products and a quotient 6 more: 15
// roundings of 2^-24.
constexpr float kDoubt = 0x1p-20f;

// The sum, or the largest, of a row's waves.
template <int kWaves, typename T, typename F>
__device__ __forceinline__ T join(const T (&sh)[kWaves], F&& f) {
  T v[kWaves];
#pragma unroll
  for (int i = 0; i < kWaves; ++i) v[i] = sh[i];
#pragma unroll
  for (int d = kWaves / 2; d > 0; d /= 2)
#pragma unroll
    for (int i = 0; i < d; ++i) v[i] = f(v[i], v[i + d]);
  return v[0];
}

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
    if (kX != MRR_F32 && a.stream) {
      const WholeRow<> r(from + first * kBytes, a.H * kBytes);
#pragma unroll
      for (int i = 0; i < kUnits; ++i) v[i].load_whole(r, col_of(i));
    } else {
#pragma unroll
      for (int i = 0; i < kUnits; ++i) v[i].load(from + first * kBytes, col_of(i), a.H);
    }
  };
  const auto store = [&](uint8_t* to, int i, const Eight<kX>& v) {
    if (kX != MRR_F32 && a.stream)
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

  constexpr int kWaves = kLanes / 64;
  const auto add_f = [](auto x, auto y) { return x + y; };
  float column[8] = {};
  uint32_t top = 0;  // |p| by its bits, so that infinities and NaN come above every number
#pragma unroll
  for (int i = 0; i < kUnits; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float v = s[i].get(k);
      column[k] = __builtin_fmaf(v, v, column[k]);
      if constexpr (kOut == kRow) top = max(top, __float_as_uint(v * w[i].get(k)) & 0x7fffffffu);
    }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) s[i].keep_packed(), w[i].keep_packed();
  float sum = sum64_f32(((column[0] + column[1]) + (column[2] + column[3])) +
                        ((column[4] + column[5]) + (column[6] + column[7])));
  if constexpr (kOut == kRow) top = max64_u32(top);
  __shared__ Shared<kLanes> sh;
  if constexpr (kWaves > 1) {
    if (threadIdx.x % 64 == 0) {
      sh.sum[threadIdx.x / 64] = sum;
      if constexpr (kOut == kRow) sh.top[threadIdx.x / 64] = top;
    }
    __syncthreads();
    sum = join(sh.sum, add_f);
    if constexpr (kOut == kRow) top = join(sh.top, [](uint32_t x, uint32_t y) { return max(x, y); });
  }

  // Writes a row of values that value(i, k) gives: y, or with one scale y over it. Whether
  // one might be rounded otherwise than its exact number.
  const float full = a.narrow == MRR_I8 ? 127.0f : 448.0f;
  const auto write = [&](auto guarded, auto&& value) {
    constexpr bool kGuarded = decltype(guarded)::value;
    constexpr float kLess = kGuarded ? 1.0f - kDoubt : 1.0f, kMore = 1.0f + kDoubt;
    bool doubt = false;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const uint32_t col = col_of(i);
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = value(i, k);
      if constexpr (kOut == kWide) {
        Eight<kX> out;
#pragma unroll
        for (int k = 0; k < 8; k += 2) out.put(k / 2, v[k], v[k + 1]);
        store(a.y, i, out);
      } else {
        const auto bytes = [&](float by) {
          const bool i8 = kOut == kRow && a.narrow == MRR_I8;
          const uint64_t lo = i8 ? pack_i8(v[0] * by, v[1] * by, v[2] * by, v[3] * by)
                                 : pack_e4m3(v[0] * by, v[1] * by, v[2] * by, v[3] * by);
          const uint64_t hi = i8 ? pack_i8(v[4] * by, v[5] * by, v[6] * by, v[7] * by)
                                 : pack_e4m3(v[4] * by, v[5] * by, v[6] * by, v[7] * by);
          return lo | hi << 32;
        };
        if constexpr (kOut == kMx) {
          uint32_t m = 0;
#pragma unroll
          for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(v[k]) & 0x7fffffffu);
          m = max(m, dpp_u32<kDppXor1>(m));
          m = max(m, dpp_u32<kDppXor2>(m));  // of the block's four lanes
          const uint32_t e = __float_as_uint(__uint_as_float(m) * kLess) >> 23;
          if constexpr (kGuarded) doubt = doubt || e != __float_as_uint(__uint_as_float(m) * kMore) >> 23;
          const uint32_t least = a.narrow == MRR_F4_E2M1 ? 2 : 8;
          const uint32_t scale = e == 255 ? 255 : e > least ? e - least : 0;
          const uint32_t scale_row = 2 * ((a.H + 63) / 64);
          if (lane % 4 == 0 && col / 32 < scale_row)
            a.scales[static_cast<size_t>(row) * scale_row + col / 32] = static_cast<uint8_t>(scale);
          if (a.narrow == MRR_F4_E2M1) {
            const float unit = two_to(scale == 255 ? 127 : scale);
            const auto codes = [&](float by) {
              uint32_t c = 0;
              c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0] * by, v[1] * by, unit, 0);
              c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2] * by, v[3] * by, unit, 1);
              c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4] * by, v[5] * by, unit, 2);
              return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6] * by, v[7] * by, unit, 3);
            };
            if (scale == 255) {
#pragma unroll
              for (int k = 0; k < 8; ++k) v[k] = 0.0f;
            }
            const uint32_t c = codes(kLess);
            if constexpr (kGuarded) doubt = doubt || c != codes(kMore);
            uint8_t* p = a.y + (first + col) / 2;
            const int n = col < a.H ? static_cast<int>(min(8u, a.H - col)) : 0;
            if (n == 8) {
              __builtin_memcpy(p, &c, 4);
            } else {
              for (int k = 0; k < n / 2; ++k) p[k] = static_cast<uint8_t>(c >> (8 * k));
            }
            continue;
          }
          // a block's values over its scale are below 512, and those over 448 end there
          const float by = two_to(scale == 255 ? 127 : 254 - scale);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = scale == 255 ? 0.0f : __builtin_amdgcn_fmed3f(v[k] * by, -448.0f, 448.0f);
        }
        const uint64_t out = bytes(kLess);
        if constexpr (kGuarded) doubt = doubt || out != bytes(kMore);
        if (col < a.H) store_bytes(a.y + first + col, out, static_cast<int>(min(8u, a.H - col)));
      }
    }
    return doubt;
  };

  // the same for all lanes of a row
  const float most = __uint_as_float(top);
  const bool plain = sum <= kMostSum && (sum >= kLeastSum || a.eps >= kLeastEps) &&
                     (kOut != kRow || top == 0 || (most >= kLeastTop && most <= kMostTop));
  constexpr bool kExact = kOut == kWide || (kOut == kRow && kX == MRR_BF16 && kW == MRR_BF16);
  bool doubt = false;
  if (plain) {
    const float r = 1.0f / __builtin_sqrtf(__builtin_fmaf(sum, a.inv_h, a.eps));
    if constexpr (kOut == kRow) {
      if (lane == 0) {
        const float scale = r * (most / full);
        __builtin_memcpy(a.scales + static_cast<size_t>(row) * 4, &scale, 4);
      }
      const float over = top == 0 ? 0.0f : 1.0f / most;
      doubt = write(std::bool_constant<!kExact>{}, [&](int i, int k) {
        const float p = full * (s[i].get(k) * w[i].get(k)), q0 = p * over;
        return __builtin_fmaf(__builtin_fmaf(-q0, most, p), over, q0);
      });
    } else {
      doubt = write(std::bool_constant<!kExact>{}, [&](int i, int k) { return s[i].get(k) * r * w[i].get(k); });
    }
  }
  if constexpr (kOut == kRow) {
    if (top == 0) {  // of zeros, or products that are nothing in 32 bits
#pragma unroll
      for (int i = 0; i < kUnits; ++i) doubt = doubt || s[i].any() != 0;
    }
  }
  if (!kExact || (kOut == kRow && top == 0)) doubt = kWaves > 1 ? __syncthreads_or(doubt) != 0 : __any(doubt) != 0;
  if (plain && !doubt) return;

  double sum64 = 0.0, most64 = 0.0;
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
  if constexpr (kWaves > 1) {
    if (threadIdx.x % 64 == 0) {
      sh.sum64[threadIdx.x / 64] = sum64;
      sh.top64[threadIdx.x / 64] = most64;
    }
    __syncthreads();
    sum64 = join(sh.sum64, add_f);
    if constexpr (kOut == kRow) most64 = join(sh.top64, [](double x, double y) { return fmax(x, y); });
  }
  const double r64 = 1.0 / sqrt(sum64 / a.H + a.eps64);
  if constexpr (kOut == kRow) {
    const bool bad = most64 > 1e300;  // a product that is not finite
    if (lane == 0) {
      const float scale = bad ? __builtin_nanf("") : static_cast<float>(r64 * most64 / full);
      __builtin_memcpy(a.scales + static_cast<size_t>(row) * 4, &scale, 4);
    }
    const bool zeros = bad || most64 == 0.0;
    const double inverse = 1.0 / most64;
    const auto rounded = [&](auto&& quotient) {
      write(std::false_type{}, [&](int i, int k) {
        const double p = static_cast<double>(s[i].get(k)) * static_cast<double>(w[i].get(k));
        return zeros ? 0.0f : quotient(p, most64, inverse, full);
      });
    };
    if (kX == MRR_F32 && a.narrow == MRR_I8)
      rounded(quotient_to_odd);
    else
      rounded(short_quotient_to_odd);
  } else {
    write(std::false_type{}, [&](int i, int k) {
      const double y = static_cast<double>(s[i].get(k)) * r64 * static_cast<double>(w[i].get(k));
      return kOut == kMx ? to_odd(y) : static_cast<float>(y);
    });
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
// From so many bytes of rows on, with which the eight L2 are full, they are read, and
// written, past the caches. Rows of 14 KiB with their sum, to fp8 rows: 22 MB take 16.8 us
// through the caches and 17.6 past them, 34 MB 25.1 and 24.0, 50 MB 39.8 and 32.1. Not 32-bit
// ones: a lane's 8 values are two units there, two requests to each line, which then moves
// twice (8192 rows of 4096 with their sum, to e4m3 rows 155 us past the caches and 81
// through them, to 32-bit ones 272 and 95).
constexpr int64_t kStreamBytes = int64_t(24) << 20;

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
    a.stream = b == 2 && args->rows * args->H * b >= kStreamBytes &&
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
