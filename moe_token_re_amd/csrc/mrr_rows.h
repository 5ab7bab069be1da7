// mrr_rows.h -- rows of fp16, bf16 or fp32 values in a wave's registers, some
// neighbouring ones a lane, and sums over a wave or a workgroup. Device code
// of the norm and the row sums.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include <type_traits>

#include "mrr_layer.h"

namespace mrr {

using f32x2 = float __attribute__((ext_vector_type(2)));
using rows_u32x4 = uint32_t __attribute__((ext_vector_type(4)));

// 16 bytes at any alignment.
__device__ __forceinline__ rows_u32x4 load16(const uint8_t* p) {
  rows_u32x4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}
__device__ __forceinline__ void store16(uint8_t* p, rows_u32x4 v) { __builtin_memcpy(p, &v, 16); }

// A row that begins and ends at multiples of 16 bytes, as a buffer: what lies outside
// reads as zeros and is not written, without a branch. Its address is the same for all
// lanes. It is written past the caches, and read past them where kPast (16384 x 7168 bf16
// norm with residual: 124 us, with writes by way of the caches 143, reads as well 143).
template <bool kPast = true>
struct WholeRow {
  __amdgpu_buffer_rsrc_t r;
  __device__ __forceinline__ WholeRow(const uint8_t* p, uint32_t bytes) {
    constexpr int kRaw = 0x00027000;  // 32-bit data, no swizzle, no stride
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t low = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
    const uint32_t high = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
    r = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(static_cast<uint64_t>(high) << 32 | low), 0, bytes, kRaw);
  }
  static constexpr int kNt = 2, kSc1 = 16;
  __device__ __forceinline__ rows_u32x4 load(uint32_t at) const {
    return __builtin_bit_cast(rows_u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, kPast ? kNt : 0));
  }
  __device__ __forceinline__ void store(uint32_t at, rows_u32x4 v) const {
    __builtin_amdgcn_raw_buffer_store_b128(v, r, at, 0, kSc1 | kNt);
  }
};
// Whether rows of so many bytes from these addresses on are such.
template <typename... P>
inline bool whole_units(int64_t row_bytes, const P*... p) {
  return row_bytes % 16 == 0 && (... && (reinterpret_cast<uintptr_t>(p) % 16 == 0));
}

// kN neighbouring values of a row as they lie in memory, a multiple of 16 bytes; fewer
// at the row's end, zeros behind.
template <int kDtype, int kN>
struct Pack {
  static constexpr int kBytes = kDtype == MRR_F32 ? 4 : 2;
  static constexpr int kWords = kBytes * kN / 4;  // of 4 bytes
  uint32_t w[kWords];

  __device__ __forceinline__ void set(int i, rows_u32x4 v) {
    w[i] = v[0], w[i + 1] = v[1], w[i + 2] = v[2], w[i + 3] = v[3];
  }
  __device__ __forceinline__ rows_u32x4 four(int i) const { return rows_u32x4{w[i], w[i + 1], w[i + 2], w[i + 3]}; }

  __device__ __forceinline__ void load(const uint8_t* row, uint32_t col, uint32_t H) {
    const uint8_t* p = row + static_cast<size_t>(col) * kBytes;
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
    if (col + kN <= H) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) set(i, load16(p + 4 * i));
    } else {
#pragma unroll
      for (int k = 0; k < kN - 1; ++k)
        if (col + k < H) {
          if constexpr (kBytes == 4) {
            __builtin_memcpy(&w[k], p + 4 * k, 4);
          } else {
            uint16_t v;
            __builtin_memcpy(&v, p + 2 * k, 2);
            w[k / 2] |= static_cast<uint32_t>(v) << (k % 2 * 16);
          }
        }
    }
  }

  // All of them from p, without a branch, which would have later loads waited for with these.
  __device__ __forceinline__ void load_all(const uint8_t* p) {
#pragma unroll
    for (int i = 0; i < kWords; i += 4) set(i, load16(p + 4 * i));
  }
  __device__ __forceinline__ void store_all(uint8_t* p) const {
#pragma unroll
    for (int i = 0; i < kWords; i += 4) store16(p + 4 * i, four(i));
  }
  // From, or to, column col of a row that is a buffer.
  template <bool kPast>
  __device__ __forceinline__ void load_whole(const WholeRow<kPast>& row, uint32_t col) {
#pragma unroll
    for (int i = 0; i < kWords; i += 4) set(i, row.load(col * kBytes + 4 * i));
  }
  template <bool kPast>
  __device__ __forceinline__ void store_whole(const WholeRow<kPast>& row, uint32_t col) const {
#pragma unroll
    for (int i = 0; i < kWords; i += 4) row.store(col * kBytes + 4 * i, four(i));
  }

  __device__ __forceinline__ void store(uint8_t* row, uint32_t col, uint32_t H) const {
    uint8_t* p = row + static_cast<size_t>(col) * kBytes;
    if (col + kN <= H) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) store16(p + 4 * i, four(i));
    } else {
#pragma unroll
      for (int k = 0; k < kN - 1; ++k)
        if (col + k < H) {
          if constexpr (kBytes == 4) {
            __builtin_memcpy(p + 4 * k, &w[k], 4);
          } else {
            const uint16_t v = static_cast<uint16_t>(w[k / 2] >> (k % 2 * 16));
            __builtin_memcpy(p + 2 * k, &v, 2);
          }
        }
    }
  }

  __device__ __forceinline__ float get(int k) const {
    if constexpr (kDtype == MRR_F32) return __uint_as_float(w[k]);
    const uint32_t v = w[k / 2];
    if constexpr (kDtype == MRR_BF16) return __uint_as_float(k % 2 ? v & 0xffff0000u : v << 16);
    using f16x2 = _Float16 __attribute__((ext_vector_type(2)));
    return static_cast<float>(__builtin_bit_cast(f16x2, v)[k % 2]);
  }

  // Not 0 where one of the values is not.
  __device__ __forceinline__ uint32_t any() const {
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < kWords; ++i) bits |= w[i] & (kDtype == MRR_F32 ? 0x7fffffffu : 0x7fff7fffu);
    return bits;
  }

  // Has the values widened anew from here on, instead of kept wide in twice the registers.
  __device__ __forceinline__ void keep_packed() {
    if constexpr (kDtype != MRR_F32) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) asm volatile("" : "+v"(w[i]));
    }
  }

  // Values 2 i and 2 i + 1, rounded to nearest even.
  __device__ __forceinline__ void put(int i, float a, float b) {
    if constexpr (kDtype == MRR_F32) {
      w[2 * i] = __float_as_uint(a), w[2 * i + 1] = __float_as_uint(b);
    } else {
      using T = std::conditional_t<kDtype == MRR_BF16, __bf16, _Float16>;
      using T2 = T __attribute__((ext_vector_type(2)));
      w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, T2));
    }
  }
};
template <int kDtype>
using Eight = Pack<kDtype, 8>;
// 16 bytes of them.
template <int kDtype>
using Unit16 = Pack<kDtype, kDtype == MRR_F32 ? 4 : 8>;

// Lane i takes lane i ^ 1, i ^ 2's value of its four, 7 - i's of its eight, 15 - i's
// of its sixteen: sums and maxima over those many lanes, without LDS.
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppMirror8 = 0x141, kDppMirror16 = 0x140;
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), kCtrl, 0xf, 0xf, true));
}
template <int kCtrl>
__device__ __forceinline__ float dpp_f32(float v) {
  return __uint_as_float(dpp_u32<kCtrl>(__float_as_uint(v)));
}

// Sums over the 16 lanes of a row of lanes, every lane getting the result.
__device__ __forceinline__ float sum16_f32(float v) {
  v += dpp_f32<kDppXor1>(v);
  v += dpp_f32<kDppXor2>(v);
  v += dpp_f32<kDppMirror8>(v);
  return v + dpp_f32<kDppMirror16>(v);
}
__device__ __forceinline__ uint32_t max16_u32(uint32_t v) {
  v = max(v, dpp_u32<kDppXor1>(v));
  v = max(v, dpp_u32<kDppXor2>(v));
  v = max(v, dpp_u32<kDppMirror8>(v));
  return max(v, dpp_u32<kDppMirror16>(v));
}

// Over all 64 lanes.
__device__ __forceinline__ float sum64_f32(float v) {
  v = sum16_f32(v);
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}
__device__ __forceinline__ uint32_t max64_u32(uint32_t v) {
  v = max16_u32(v);
  v = max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), 16)));
  return max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), 32)));
}
__device__ __forceinline__ double sum64_f64(double v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ double max64_f64(double v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v = fmax(v, __shfl_xor(v, d));
  return v;
}

// Rows src [T] to rows dst [R] by an index [T, k], zeros for an index below 0, -1 - row
// (mrr_token_permute.hip).
void move_rows(const void* src, void* dst, int64_t row_bytes, const int32_t* idx, int64_t T, int64_t k, int64_t R,
               hipStream_t stream);

}  // namespace mrr
