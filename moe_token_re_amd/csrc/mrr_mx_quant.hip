// mrr_mx_quant.hip -- conversion between wide rows (fp16, bf16, fp32) and
// microscaled 4-bit rows (OCP MX v1.0: e2m1 values, e8m0 scales), in the layout
// the re-routing operator moves: [rows, H/2] bytes and [rows, ceil(H/64), 2]
// scales.
//
// Per block of 32 values: s = max(exponent field of max |x| - 2, 0), so that
// 2^(s - 127) = 2^(floor(log2 max |x|) - 2), and q = round(x / 2^(s - 127)) to
// e2m1. Bound by memory: a value costs its 2 or 4 bytes and 17/32 byte. A lane
// takes 16 bytes of a row, so that what a wave reads or writes of it at once is
// 1 KiB without gaps (with 8 fp32 values a lane 30000 x 3000 of them took 190 us
// there and back, with 4 they take 147); the 4 or 8 lanes of a block find its maximum by
// two or three DPP steps, and the conversions are the chip's scaled ones (division
// by the scale, round to nearest even, saturating).
#include "mrr_device.h"
#include "mrr_experts.h"

namespace mrr {
namespace {

using f16x2 = _Float16 __attribute__((ext_vector_type(2)));
using bf16x2 = __bf16 __attribute__((ext_vector_type(2)));
using f32x2 = float __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;

// The scale as the conversions take it: 2^(s - 127). They read the exponent
// alone; 2^-127 is the subnormal with its top mantissa bit set.
__device__ __forceinline__ float scale_float(uint32_t s) {
  return __uint_as_float(s == 0 ? 0x00400000u : s << 23);
}

// The largest of the lanes of a block: 4 or 8 neighbours.
template <int kLanes>
__device__ __forceinline__ uint32_t block_max(uint32_t v) {
  constexpr int kSwap1 = 0xB1, kSwap2 = 0x4E;  // quad_perm [1,0,3,2] and [2,3,0,1]
  constexpr int kMirror8 = 0x141;              // lane i of eight takes lane 7 - i's
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), kSwap1, 0xf, 0xf, false)));
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), kSwap2, 0xf, 0xf, false)));
  if constexpr (kLanes == 8)
    v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), kMirror8, 0xf, 0xf, false)));
  return v;
}

// A lane's values of one type, a unit: loading, the largest |x| as fp32 bits (so that
// infinities and NaN compare above every finite value), and both conversions.
template <int kDtype>
struct Unit;

template <>
struct Unit<MRR_BF16> {
  uint32_t w[4];
  static constexpr int kBytes = 2, kValues = 8;
  __device__ void set(int i, const uint8_t* p) {
    uint16_t v;
    __builtin_memcpy(&v, p, 2);
    w[i / 2] |= static_cast<uint32_t>(v) << (i % 2 * 16);
  }
  __device__ uint32_t top() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max((w[i] << 16) & 0x7fffffffu, w[i] & 0x7fff0000u));
    return m;
  }
  __device__ uint32_t pack(float s) const {
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, w[0]), s, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, w[1]), s, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, w[2]), s, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, w[3]), s, 3);
  }
  __device__ void unpack(uint32_t c, float s) {
    w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0));
    w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1));
    w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2));
    w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3));
  }
  __device__ void get(int i, uint8_t* p) const {
    const uint16_t v = static_cast<uint16_t>(w[i / 2] >> (i % 2 * 16));
    __builtin_memcpy(p, &v, 2);
  }
};

template <>
struct Unit<MRR_F16> : Unit<MRR_BF16> {
  __device__ uint32_t top() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f16x2 h = __builtin_bit_cast(f16x2, w[i]);
      m = max(m, max(__float_as_uint(static_cast<float>(h[0])) & 0x7fffffffu,
                     __float_as_uint(static_cast<float>(h[1])) & 0x7fffffffu));
    }
    return m;
  }
  __device__ uint32_t pack(float s) const {
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(f16x2, w[0]), s, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(f16x2, w[1]), s, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(f16x2, w[2]), s, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(f16x2, w[3]), s, 3);
  }
  __device__ void unpack(uint32_t c, float s) {
    w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 0));
    w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 1));
    w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 2));
    w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 3));
  }
};

template <>
struct Unit<MRR_F32> {
  float w[4];
  static constexpr int kBytes = 4, kValues = 4;
  __device__ void set(int i, const uint8_t* p) { __builtin_memcpy(&w[i], p, 4); }
  __device__ uint32_t top() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, __float_as_uint(w[i]) & 0x7fffffffu);
    return m;
  }
  __device__ uint32_t pack(float s) const {
    const uint32_t r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0, w[0], w[1], s, 0);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, w[2], w[3], s, 1);
  }
  __device__ void unpack(uint32_t c, float s) {
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1);
    w[0] = a[0], w[1] = a[1], w[2] = b[0], w[3] = b[1];
  }
  __device__ void get(int i, uint8_t* p) const { __builtin_memcpy(p, &w[i], 4); }
};

struct MxArgs {
  uint8_t* wide;
  uint8_t* packed;
  uint8_t* scales;
  uint32_t units;          // of this launch, padding included
  uint32_t units_per_row;  // unused when kFlat
  uint32_t H;              // unused when kFlat
};

// Where a unit lies. kFlat: H is a multiple of 64, so rows follow each other
// without padding and no row number is needed.
struct Place {
  uint64_t wide, packed, scale;  // element, byte and byte offsets
  int count;                     // values of the unit that exist, fewer at a row's end
};

template <bool kFlat, int kUnit>
__device__ __forceinline__ Place place_of(const MxArgs& a, uint32_t u) {
  Place p;
  p.scale = u / (32 / kUnit);
  if constexpr (kFlat) {
    p.wide = static_cast<uint64_t>(u) * kUnit;
    p.packed = static_cast<uint64_t>(u) * (kUnit / 2);
    p.count = kUnit;
  } else {
    const uint32_t row = u / a.units_per_row;
    const uint32_t col = (u - row * a.units_per_row) * kUnit;
    p.count = col >= a.H ? 0 : min(a.H - col, static_cast<uint32_t>(kUnit));
    p.wide = static_cast<uint64_t>(row) * a.H + col;
    p.packed = p.wide / 2;
  }
  return p;
}

using u32x4 = uint32_t __attribute__((ext_vector_type(4)));
using loose4 = u32x4 __attribute__((aligned(2)));

// A lane's wide values; kStream: past the caches.
template <bool kStream, typename W>
__device__ __forceinline__ void load_unit(W (&w)[4], const uint8_t* p) {
  u32x4 v;
  if constexpr (kStream)
    v = __builtin_nontemporal_load(reinterpret_cast<const loose4*>(p));
  else
    v = *reinterpret_cast<const loose4*>(p);
  __builtin_memcpy(w, &v, 16);
}
template <bool kStream, typename W>
__device__ __forceinline__ void store_unit(uint8_t* p, const W (&w)[4]) {
  u32x4 v;
  __builtin_memcpy(&v, w, 16);
  if constexpr (kStream)
    __builtin_nontemporal_store(v, reinterpret_cast<loose4*>(p));
  else
    *reinterpret_cast<loose4*>(p) = v;
}

template <int kDtype, bool kFlat, int kIter, bool kStream>
__global__ __launch_bounds__(kThreads) void mx_quantize_kernel(MxArgs a) {
  using V = Unit<kDtype>;
  constexpr int kUnit = V::kValues, kLanes = 32 / kUnit;  // lanes of a block
  using Packed = std::conditional_t<kUnit == 8, uint32_t, uint16_t>;
  const uint32_t u0 = blockIdx.x * static_cast<uint32_t>(kThreads * kIter) + threadIdx.x;
  V v[kIter];
  Place p[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const uint32_t u = u0 + i * kThreads;
    v[i] = V{};
    p[i] = place_of<kFlat, kUnit>(a, u);
    if (u >= a.units) p[i].count = 0;
    const uint8_t* src = a.wide + p[i].wide * V::kBytes;
    if (p[i].count == kUnit) {
      load_unit<kStream>(v[i].w, src);
    } else {
      for (int k = 0; k < kUnit; ++k)
        if (k < p[i].count) v[i].set(k, src + k * V::kBytes);
    }
  }
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    // units come in whole blocks, so the lanes of a block are in range together
    const uint32_t e = block_max<kLanes>(v[i].top()) >> 23;
    const uint32_t s = e == 255 ? 255 : e > 2 ? e - 2 : 0;
    const Packed c = static_cast<Packed>(s == 255 ? 0 : v[i].pack(scale_float(s)));
    uint8_t* dst = a.packed + p[i].packed;
    if (p[i].count == kUnit) {
      __builtin_memcpy(dst, &c, sizeof(c));
    } else {
      for (int k = 0; k < kUnit / 2; ++k)
        if (2 * k < p[i].count) dst[k] = static_cast<uint8_t>(c >> (8 * k));
    }
    if (threadIdx.x % kLanes == 0 && u0 + i * kThreads < a.units) a.scales[p[i].scale] = static_cast<uint8_t>(s);
  }
}

template <int kDtype, bool kFlat, int kIter, bool kStream>
__global__ __launch_bounds__(kThreads) void mx_dequantize_kernel(MxArgs a) {
  using V = Unit<kDtype>;
  constexpr int kUnit = V::kValues;
  using Packed = std::conditional_t<kUnit == 8, uint32_t, uint16_t>;
  const uint32_t u0 = blockIdx.x * static_cast<uint32_t>(kThreads * kIter) + threadIdx.x;
  Packed c[kIter];
  uint32_t s[kIter];
  Place p[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const uint32_t u = u0 + i * kThreads;
    p[i] = place_of<kFlat, kUnit>(a, u);
    if (u >= a.units) p[i].count = 0;
    c[i] = s[i] = 0;
    const uint8_t* src = a.packed + p[i].packed;
    if (p[i].count == kUnit) {
      __builtin_memcpy(&c[i], src, sizeof(c[i]));
    } else {
      for (int k = 0; k < kUnit / 2; ++k)
        if (2 * k < p[i].count) c[i] |= static_cast<Packed>(src[k] << (8 * k));
    }
    if (p[i].count > 0) s[i] = a.scales[p[i].scale];
  }
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    V v;
    v.unpack(c[i], scale_float(s[i]));  // s = 255: the scale is an infinity, every value a NaN
    uint8_t* dst = a.wide + p[i].wide * V::kBytes;
    if (p[i].count == kUnit) {
      store_unit<kStream>(dst, v.w);
    } else {
      for (int k = 0; k < kUnit; ++k)
        if (k < p[i].count) v.get(k, dst + k * V::kBytes);
    }
  }
}

// Units are numbered in 32 bits, so more rows than this take several launches.
constexpr int64_t kMaxUnits = int64_t(1) << 30;
// From this many units on a lane takes four of them.
constexpr int64_t kManyUnits = int64_t(kThreads) * 2048;
// From so many bytes of wide rows on they are read, and written, past the caches,
// which would not hold them for a reader anyway: 16384 x 7168 bf16 rows quantised
// and read back in 131 us by way of the caches and 89 past them; but 4096 x 2048 fp32 in
// 15.4 and 19. (There and back the 4-bit rows between are still in the last-level
// cache. From memory the first takes 46 us, 6.5 TB/s, and the way back 53, 5.6 TB/s.)
constexpr int64_t kStreamBytes = int64_t(64) << 20;

template <int kDtype, bool kFlat, int kIter, bool kStream>
void launch_kernel(const MxArgs& a, bool quantize, hipStream_t stream) {
  const dim3 grid((a.units + kThreads * kIter - 1) / (kThreads * kIter));
  if (quantize)
    mx_quantize_kernel<kDtype, kFlat, kIter, kStream><<<grid, kThreads, 0, stream>>>(a);
  else
    mx_dequantize_kernel<kDtype, kFlat, kIter, kStream><<<grid, kThreads, 0, stream>>>(a);
}

template <int kDtype, bool kFlat>
void launch_mx(const MxArgs& a, bool quantize, bool large, hipStream_t stream) {
  if (a.units < kManyUnits)
    launch_kernel<kDtype, kFlat, 1, false>(a, quantize, stream);
  else if (large)
    launch_kernel<kDtype, kFlat, 4, true>(a, quantize, stream);
  else
    launch_kernel<kDtype, kFlat, 4, false>(a, quantize, stream);
}

template <int kDtype>
void launch_dtype(const MxArgs& a, bool flat, bool quantize, bool large, hipStream_t stream) {
  if (flat)
    launch_mx<kDtype, true>(a, quantize, large, stream);
  else
    launch_mx<kDtype, false>(a, quantize, large, stream);
}

mrr_status run_mx(const mrr_mx_args* args, bool quantize, hipStream_t stream) {
  const mrr_status st = check_mx(args, quantize);
  if (st != MRR_SUCCESS || args->rows == 0) return st;
  const int64_t w = args->wide_dtype == MRR_F32 ? 4 : 2;
  const int64_t per_scale = args->wide_dtype == MRR_F32 ? 8 : 4;  // units
  const int64_t per_row = per_scale * mx_scale_bytes(args->H);
  const bool flat = args->H % 64 == 0, large = args->rows * args->H * w >= kStreamBytes;
  const int64_t step = kMaxUnits / per_row;  // rows of a launch
  for (int64_t row = 0; row < args->rows; row += step) {
    const int64_t rows = args->rows - row < step ? args->rows - row : step;
    MxArgs a;
    a.wide = static_cast<uint8_t*>(args->wide) + row * args->H * w;
    a.packed = static_cast<uint8_t*>(args->packed) + row * (args->H / 2);
    a.scales = static_cast<uint8_t*>(args->scales) + row * (per_row / per_scale);
    a.units = static_cast<uint32_t>(rows * per_row);
    a.units_per_row = static_cast<uint32_t>(per_row);
    a.H = static_cast<uint32_t>(args->H);
    switch (args->wide_dtype) {
      case MRR_F16: launch_dtype<MRR_F16>(a, flat, quantize, large, stream); break;
      case MRR_BF16: launch_dtype<MRR_BF16>(a, flat, quantize, large, stream); break;
      default: launch_dtype<MRR_F32>(a, flat, quantize, large, stream); break;
    }
    if (hipGetLastError() != hipSuccess) return MRR_ERROR_HIP;
  }
  return MRR_SUCCESS;
}

}  // namespace
}  // namespace mrr

extern "C" mrr_status mrr_mx_quantize(const mrr_mx_args* args, struct ihipStream_t* stream) {
  return mrr::run_mx(args, true, stream);
}

extern "C" mrr_status mrr_mx_dequantize(const mrr_mx_args* args, struct ihipStream_t* stream) {
  return mrr::run_mx(args, false, stream);
}
