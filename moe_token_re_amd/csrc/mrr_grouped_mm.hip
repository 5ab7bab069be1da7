// mrr_grouped_mm.hip -- the experts' product over expert-major rows of
// microscaled 4-bit values:
//     out[r, n] = row_weight[r] * sum over k of x[r, k] w[e(r), n, k],
// or, gated, silu of the first half of the n times the second half.
//
// One workgroup computes a tile of kBM rows of one expert by kBN of its weight
// rows with the scaled matrix instruction 32x32x64 (its two operands hold 32
// values of a row a lane, with their scale; sums in fp32). The row tiles of an
// expert are not known on the host: the grid covers the most there can be, and
// every workgroup scans the counts for its own.
#include "mrr_device.h"
#include "mrr_experts.h"

namespace mrr {
namespace {

using i32x8 = int __attribute__((ext_vector_type(8)));
using f32x16 = float __attribute__((ext_vector_type(16)));
using u32x4 = uint32_t __attribute__((ext_vector_type(4)));

constexpr int kMxFp4 = 4;        // the matrix instruction's operand format e2m1
constexpr int kTileBlocks = 8;   // blocks of a row in a K tile (256 values, 128 bytes)
constexpr int kRowBytes = 128;   // of a row in a K tile

struct GroupedArgs {
  const uint8_t* x;
  const uint8_t* x_scales;
  const uint8_t* w;
  const uint8_t* w_scales;
  const void* counts;
  const float* row_weight;
  void* out;
  WsHeader* hdr;
  int32_t A, N, E;
  int32_t blocks;          // K / 32
  int32_t scale_bytes;     // of a row
  int32_t n_tiles;
  int32_t wide_counts;     // int64 counts
  int32_t running;         // expert_token_num_type 0
  int32_t out_dtype;
};

// This workgroup's tile.
struct Tile {
  int expert, row, rows, n;  // row: its first row; rows: how many exist; n: the n tile
};

__device__ __forceinline__ int64_t raw_count(const GroupedArgs& a, int e) {
  return a.wide_counts ? static_cast<const int64_t*>(a.counts)[e]
                       : static_cast<int64_t>(static_cast<const int32_t*>(a.counts)[e]);
}

// Rows of expert e, or -1 when they cannot be right.
__device__ __forceinline__ int32_t count_of(const GroupedArgs& a, int e) {
  int64_t c = raw_count(a, e);
  if (a.running) {
    const int64_t before = e > 0 ? raw_count(a, e - 1) : 0;
    if (c < 0 || c > a.A || before < 0 || before > c) return -1;
    c -= before;
  }
  return c < 0 || c > a.A ? -1 : static_cast<int32_t>(c);
}

// Finds the workgroup's tile; false when it has none or the counts are bad.
// Every thread takes a run of experts; the runs' rows and tiles are scanned
// over the workgroup. The exact sum of the counts is kept in two 16-bit halves
// (4096 counts of at most 2^31).
template <int kBM, int kWgThreads>
__device__ bool find_tile(const GroupedArgs& a, Tile* t) {
  constexpr int kWaves = kWgThreads / 64;
  __shared__ uint32_t s_rows[kWaves], s_tiles[kWaves], s_low[kWaves], s_high[kWaves], s_bad[kWaves];
  __shared__ Tile s_tile;
  const int tid = threadIdx.x, wave = tid / 64;
  const int per = (a.E + kWgThreads - 1) / kWgThreads;
  const int e0 = tid * per, e1 = min(a.E, e0 + per);
  uint32_t rows = 0, tiles = 0, low = 0, high = 0, bad = 0;
  for (int e = e0; e < e1; ++e) {
    const int32_t c = count_of(a, e);
    if (c < 0) {
      bad = 1;
      continue;
    }
    rows += c;
    tiles += (static_cast<uint32_t>(c) + kBM - 1) / kBM;
    low += c & 0xffff;
    high += static_cast<uint32_t>(c) >> 16;
  }
  const uint32_t rows_in = wave_scan_u32(rows), tiles_in = wave_scan_u32(tiles);
  const uint32_t low_sum = wave_sum_u32(low), high_sum = wave_sum_u32(high);
  const bool any_bad = __any(bad != 0);
  if (tid % 64 == 63) {
    s_rows[wave] = rows_in;
    s_tiles[wave] = tiles_in;
    s_low[wave] = low_sum;
    s_high[wave] = high_sum;
    s_bad[wave] = any_bad;
  }
  __syncthreads();
  uint32_t row0 = rows_in - rows, tile0 = tiles_in - tiles, all_tiles = 0, is_bad = 0;
  uint64_t total = 0;
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) {
      row0 += s_rows[w];
      tile0 += s_tiles[w];
    }
    all_tiles += s_tiles[w];
    total += s_low[w] + (static_cast<uint64_t>(s_high[w]) << 16);
    is_bad |= s_bad[w];
  }
  const bool valid = is_bad == 0 && total == static_cast<uint64_t>(a.A);
  if (a.hdr != nullptr && blockIdx.x == 0 && tid == 0) {
    a.hdr->status = valid ? kCountsValid : kTablesBad;
    a.hdr->flags = is_bad ? kFlagNegative : valid ? 0 : kFlagSumMismatch;
    a.hdr->inverse = 0;
    a.hdr->A = a.A;
    a.hdr->N = 1;
    a.hdr->E = a.E;
    a.hdr->total = static_cast<int64_t>(total);
  }
  const uint32_t work = all_tiles * static_cast<uint32_t>(a.n_tiles);
  if (!valid || blockIdx.x >= work) return false;
  // The hardware deals workgroups to the 8 XCDs in turn; each XCD gets a run of
  // neighbouring tiles (n fastest), so that they share rows in its L2.
  const uint32_t xcd = blockIdx.x % 8, at = blockIdx.x / 8;
  const uint32_t base = work / 8, extra = work % 8;
  const uint32_t id = xcd * base + min(xcd, extra) + at;
  const uint32_t m = id / a.n_tiles;
  if (m >= tile0 && m < tile0 + tiles) {
    uint32_t first = tile0, r = row0;
    for (int e = e0; e < e1; ++e) {
      const uint32_t c = static_cast<uint32_t>(count_of(a, e)), n = (c + kBM - 1) / kBM;
      if (m < first + n) {
        const uint32_t k = m - first;
        s_tile.expert = e;
        s_tile.row = static_cast<int>(r + k * kBM);
        s_tile.rows = static_cast<int>(min(c - k * kBM, static_cast<uint32_t>(kBM)));
        s_tile.n = static_cast<int>(id - m * a.n_tiles);
        break;
      }
      first += n;
      r += c;
    }
  }
  __syncthreads();
  *t = s_tile;
  return true;
}

__device__ __forceinline__ void load_to_lds(const uint8_t* src, uint8_t* lds) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                   (__attribute__((address_space(3))) void*)lds, 16, 0, 0);
}

// The four scale bytes of blocks b .. b + 3 of a row; 127 (a factor of one)
// past its end.
__device__ __forceinline__ uint32_t load_scales(const uint8_t* row, int b, int n) {
  uint32_t v = 0x7f7f7f7fu;
  if (b + 4 <= n) {
    __builtin_memcpy(&v, row + b, 4);
  } else {
    for (int i = 0; i < 4; ++i)
      if (b + i < n) v = (v & ~(0xffu << (8 * i))) | static_cast<uint32_t>(row[b + i]) << (8 * i);
  }
  return v;
}

__device__ __forceinline__ float silu(float g) { return g / (1.0f + __expf(-g)); }

// Four neighbouring outputs of one row, of which `count` exist.
template <typename T>
__device__ __forceinline__ void store4(T* p, const float (&v)[4], int count) {
  T q[4] = {static_cast<T>(v[0]), static_cast<T>(v[1]), static_cast<T>(v[2]), static_cast<T>(v[3])};
  if (count >= 4) {
    __builtin_memcpy(p, q, sizeof(q));
  } else {
    for (int i = 0; i < 4; ++i)
      if (i < count) p[i] = q[i];
  }
}

// kFN x kFM fragments of 32 weight rows x 32 token rows a wave, kWN x kWM
// waves a workgroup. A K tile is 256 values: the halves of a wave take its
// first and last four blocks, so that the four scales a lane needs for the
// tile's four products are one dword. A row of the tile is 128 bytes of LDS,
// its 16-byte chunks permuted by the row's number so that eight neighbouring
// rows touch all banks; the tiles go from memory to LDS directly, the next one
// while this one is multiplied.
template <int kFM, int kFN, int kWM, int kWN, bool kGated>
__global__ __launch_bounds__(64 * kWM * kWN) void grouped_mm_kernel(GroupedArgs a) {
  constexpr int kWaves = kWM * kWN, kWgThreads = 64 * kWaves;
  constexpr int kBM = 32 * kFM * kWM, kBN = 32 * kFN * kWN;
  constexpr int kStage = (kBM + kBN) * kRowBytes;
  constexpr int kXLoads = kBM / 8 / kWaves, kWLoads = kBN / 8 / kWaves;
  static_assert(kXLoads * 8 * kWaves == kBM && kWLoads * 8 * kWaves == kBN, "whole loads");
  __shared__ __align__(1024) uint8_t lds[2 * kStage];

  Tile t;
  if (!find_tile<kBM, kWgThreads>(a, &t)) return;

  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int wm = wave % kWM, wn = wave / kWM;
  const int r32 = lane % 32, half = lane / 32;
  const int half_n = a.N / 2;                            // gated: the up projection's first row
  const int n0 = t.n * (kGated ? kBN / 2 : kBN);         // first output column of the tile
  const int n_end = kGated ? half_n : a.N;
  const int64_t row_bytes = static_cast<int64_t>(a.blocks) * 16;
  const int64_t w_row0 = static_cast<int64_t>(t.expert) * a.N;

  // The weight row in place j of the tile: within a wave's fragments, gated
  // ones are the gate's and then the same columns of the up projection.
  auto weight_row = [&](int j) {
    int col, part = 0;
    if constexpr (kGated) {
      constexpr int kHalf = 32 * kFN / 2;
      const int in_wave = j % (32 * kFN);
      part = in_wave / kHalf;
      col = n0 + j / (32 * kFN) * kHalf + in_wave % kHalf;
    } else {
      col = n0 + j;
    }
    return w_row0 + min(col, n_end - 1) + (part ? half_n : 0);
  };

  // What this lane stages: chunk lane % 8 (permuted) of a row of every eight.
  const uint8_t* src[kXLoads + kWLoads];
  int chunk[1];
  chunk[0] = (lane % 8) ^ (lane / 8);
#pragma unroll
  for (int i = 0; i < kXLoads; ++i) {
    const int j = (i * kWaves + wave) * 8 + lane / 8;
    src[i] = a.x + static_cast<int64_t>(t.row + min(j, t.rows - 1)) * row_bytes;
  }
#pragma unroll
  for (int i = 0; i < kWLoads; ++i) {
    const int j = (i * kWaves + wave) * 8 + lane / 8;
    src[kXLoads + i] = a.w + weight_row(j) * row_bytes;
  }
  auto stage = [&](int kt, int buf) {
    uint8_t* base = lds + buf * kStage + wave * 1024;
    const int b = min(kt * kTileBlocks + chunk[0], a.blocks - 1);  // past the row's end: any block of it
#pragma unroll
    for (int i = 0; i < kXLoads; ++i) load_to_lds(src[i] + b * 16, base + i * kWaves * 1024);
#pragma unroll
    for (int i = 0; i < kWLoads; ++i)
      load_to_lds(src[kXLoads + i] + b * 16, base + kBM * kRowBytes + i * kWaves * 1024);
  };

  const uint8_t* xs[kFM];
  const uint8_t* ws[kFN];
#pragma unroll
  for (int i = 0; i < kFM; ++i)
    xs[i] = a.x_scales + static_cast<int64_t>(t.row + min((wm * kFM + i) * 32 + r32, t.rows - 1)) * a.scale_bytes;
#pragma unroll
  for (int i = 0; i < kFN; ++i) ws[i] = a.w_scales + weight_row((wn * kFN + i) * 32 + r32) * a.scale_bytes;

  f32x16 acc[kFN][kFM];
#pragma unroll
  for (int i = 0; i < kFN; ++i)
#pragma unroll
    for (int j = 0; j < kFM; ++j)
#pragma unroll
      for (int k = 0; k < 16; ++k) acc[i][j][k] = 0.0f;

  uint32_t sx[kFM], sw[kFN];
  auto fetch_scales = [&](int kt) {
    const int b = kt * kTileBlocks + half * 4;
#pragma unroll
    for (int i = 0; i < kFM; ++i) sx[i] = load_scales(xs[i], b, a.blocks);
#pragma unroll
    for (int i = 0; i < kFN; ++i) sw[i] = load_scales(ws[i], b, a.blocks);
  };

  const int k_tiles = (a.blocks + kTileBlocks - 1) / kTileBlocks;
  stage(0, 0);
  fetch_scales(0);
  for (int kt = 0; kt < k_tiles; ++kt) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    uint32_t cx[kFM], cw[kFN];
#pragma unroll
    for (int i = 0; i < kFM; ++i) cx[i] = sx[i];
#pragma unroll
    for (int i = 0; i < kFN; ++i) cw[i] = sw[i];
    if (kt + 1 < k_tiles) {
      stage(kt + 1, (kt + 1) % 2);
      fetch_scales(kt + 1);
    }
    const uint8_t* xt = lds + kt % 2 * kStage + wm * kFM * 32 * kRowBytes;
    const uint8_t* wt = lds + kt % 2 * kStage + (kBM + wn * kFN * 32) * kRowBytes;
    const int left = a.blocks - kt * kTileBlocks;  // blocks of the rows in this tile
    auto step = [&](auto s_) {
      constexpr int s = decltype(s_)::value;
      const int block = half * 4 + s;
      const int at = r32 * kRowBytes + ((block ^ (r32 % 8)) * 16);
      i32x8 xf[kFM], wf[kFN];
#pragma unroll
      for (int j = 0; j < kFM; ++j) {
        u32x4 v = *reinterpret_cast<const u32x4*>(xt + j * 32 * kRowBytes + at);
        if (block >= left) v = u32x4{0, 0, 0, 0};
        xf[j] = i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < kFN; ++i) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(wt + i * 32 * kRowBytes + at);
        wf[i] = i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < kFN; ++i)
#pragma unroll
        for (int j = 0; j < kFM; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wf[i], xf[j], acc[i][j], kMxFp4, kMxFp4, s,
                                                                      (int)cw[i], s, (int)cx[j]);
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
  }

  // A lane holds one token row of each fragment and, of its 32 weight rows,
  // four times four neighbours.
  constexpr int kOutFN = kGated ? kFN / 2 : kFN;
#pragma unroll
  for (int j = 0; j < kFM; ++j) {
    const int m = (wm * kFM + j) * 32 + r32;
    if (m >= t.rows) continue;
    const int64_t row = t.row + m;
    const float rw = a.row_weight != nullptr ? a.row_weight[row] : 1.0f;
#pragma unroll
    for (int i = 0; i < kOutFN; ++i) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int col = n0 + (wn * kOutFN + i) * 32 + q * 8 + half * 4;
        if (col >= n_end) continue;
        float v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[k] = acc[i][j][q * 4 + k];
          if constexpr (kGated) v[k] = silu(v[k]) * acc[i + kOutFN][j][q * 4 + k];
          v[k] *= rw;
        }
        const int64_t o = row * n_end + col;
        if (a.out_dtype == MRR_BF16)
          store4(static_cast<__bf16*>(a.out) + o, v, n_end - col);
        else if (a.out_dtype == MRR_F16)
          store4(static_cast<_Float16*>(a.out) + o, v, n_end - col);
        else
          store4(static_cast<float*>(a.out) + o, v, n_end - col);
      }
    }
  }
}

// The counts alone, for a call without rows: their verdict.
__global__ void check_counts_kernel(GroupedArgs a) {
  Tile t;
  find_tile<256, 256>(a, &t);
}

template <int kFM, int kFN, int kWM, int kWN>
mrr_status launch_grouped(GroupedArgs a, bool gated, hipStream_t stream) {
  constexpr int kBM = 32 * kFM * kWM, kBN = 32 * kFN * kWN;
  a.n_tiles = gated ? (a.N / 2 + kBN / 2 - 1) / (kBN / 2) : (a.N + kBN - 1) / kBN;
  // the most row tiles there can be: every expert may end in a partial one
  const int64_t m_tiles = a.A / kBM + (a.E < a.A ? a.E : a.A);
  const int64_t grid = m_tiles * a.n_tiles;
  if (grid > max_launch_grid(64 * kWM * kWN)) return MRR_ERROR_INVALID_SHAPE;
  const dim3 g(static_cast<unsigned>(grid)), b(64 * kWM * kWN);
  if (gated)
    hipLaunchKernelGGL((grouped_mm_kernel<kFM, kFN, kWM, kWN, true>), g, b, 0, stream, a);
  else
    hipLaunchKernelGGL((grouped_mm_kernel<kFM, kFN, kWM, kWN, false>), g, b, 0, stream, a);
  return hipGetLastError() == hipSuccess ? MRR_SUCCESS : MRR_ERROR_HIP;
}

}  // namespace
}  // namespace mrr

extern "C" mrr_status mrr_mx_grouped_mm(const mrr_grouped_mm_args* args, void* workspace, size_t workspace_bytes,
                                        struct ihipStream_t* stream) {
  const mrr_status st = mrr::check_grouped_mm(args, workspace, workspace_bytes);
  if (st != MRR_SUCCESS) return st;
  mrr::GroupedArgs a{};
  a.x = static_cast<const uint8_t*>(args->tokens);
  a.x_scales = static_cast<const uint8_t*>(args->token_scales);
  a.w = static_cast<const uint8_t*>(args->weight);
  a.w_scales = static_cast<const uint8_t*>(args->weight_scales);
  a.counts = args->expert_token_num;
  a.row_weight = args->row_weight;
  a.out = args->out;
  a.hdr = static_cast<mrr::WsHeader*>(workspace);
  a.A = static_cast<int32_t>(args->A);
  a.N = static_cast<int32_t>(args->N);
  a.E = static_cast<int32_t>(args->E);
  a.blocks = static_cast<int32_t>(args->K / 32);
  a.scale_bytes = static_cast<int32_t>(mrr::mx_scale_bytes(args->K));
  a.wide_counts = args->counts_dtype == MRR_I64;
  a.running = args->expert_token_num_type == 0;
  a.out_dtype = args->out_dtype;
  if (args->A == 0) {
    if (workspace == nullptr) return MRR_SUCCESS;
    hipLaunchKernelGGL(mrr::check_counts_kernel, dim3(1), dim3(256), 0, stream, a);
    return hipGetLastError() == hipSuccess ? MRR_SUCCESS : MRR_ERROR_HIP;
  }
  return mrr::launch_grouped<2, 2, 2, 2>(a, args->gated == 1, stream);
}
