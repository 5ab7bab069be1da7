// mrr_grouped_mm.hip -- the experts' product over expert-major rows of
// microscaled 4-bit values:
//     out[r, n] = row_weight[r] * sum over k of x[r, k] w[e(r), n, k],
// or, gated, silu of the first half of the n times the second half.
//
// One workgroup computes a tile of kBM rows of one expert by kBN of its weight
// rows with the scaled matrix instruction 32x32x64 (its two operands hold 32
// values of a row a lane, with their scale; sums in fp32). The row tiles of an
// expert are not known on the host: every wave scans the counts for its own.
// What it measured: 16384 rows of 16 experts, gate and up (K 7168, N 4096) 298 us,
// 3.2 PFLOP/s, where the matrix instructions alone would take 163 (the counters show
// them in 40% of the active cycles; the rest are LDS reads, loads and barriers between
// them, and a last round of tiles that is half empty); down (K 2048, N 7168) 175 us, of
// which some 45 wait for 235 MB of results; 64 rows of 16 experts (K 2048, N 4096)
// 13.9 us, 5.1 TB/s of weights.
#include "mrr_device.h"
#include "mrr_experts.h"

namespace mrr {
namespace {

using i32x8 = int __attribute__((ext_vector_type(8)));
using f32x4 = float __attribute__((ext_vector_type(4)));
using f32x16 = float __attribute__((ext_vector_type(16)));
using u32x4 = uint32_t __attribute__((ext_vector_type(4)));

constexpr int kMxFp4 = 4;        // the matrix instruction's operand format e2m1
constexpr int kTileBlocks = 8;   // blocks of a row in a K tile (256 values)
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

// A tile of the output.
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

// The tiles of all experts, and which of them are this workgroup's. Every wave
// holds all of it for itself, without LDS or barriers: a lane has a run of
// experts, the runs' rows and tiles are scanned over the wave.
template <int kBM>
struct Tiles {
  int e0, e1;            // the lane's run of experts
  int32_t head;          // rows of the run's first expert
  uint32_t rows, tiles;  // first row and first row tile of the run
  uint32_t end;          // first row tile behind it
  uint32_t all;          // row tiles of all experts
  uint32_t first, count, step;  // this workgroup's tiles: first + i step, i < count

  // False when the counts are bad. Their exact sum is kept in two 16-bit
  // halves (4096 counts of at most 2^31).
  __device__ __forceinline__ bool scan(const GroupedArgs& a) {
    const int lane = threadIdx.x % 64;
    const int per = (a.E + 63) / 64;
    e0 = lane * per, e1 = min(a.E, e0 + per);
    uint32_t r = 0, n = 0, low = 0, high = 0, bad = 0;
    head = 0;
    for (int e = e0; e < e1; ++e) {
      const int32_t c = count_of(a, e);
      if (e == e0) head = c;
      if (c < 0) {
        bad = 1;
        continue;
      }
      r += c;
      n += (static_cast<uint32_t>(c) + kBM - 1) / kBM;
      low += c & 0xffff;
      high += static_cast<uint32_t>(c) >> 16;
    }
    end = wave_scan_u32(n);
    rows = wave_scan_u32(r) - r;
    tiles = end - n;
    all = __builtin_amdgcn_readlane(end, 63);
    const uint64_t total = wave_sum_u32(low) + (static_cast<uint64_t>(wave_sum_u32(high)) << 16);
    const bool is_bad = __any(bad != 0);
    const bool valid = !is_bad && total == static_cast<uint64_t>(a.A);
    if (a.hdr != nullptr && blockIdx.x == 0 && threadIdx.x == 0) {
      a.hdr->status = valid ? kCountsValid : kTablesBad;
      a.hdr->flags = is_bad ? kFlagNegative : valid ? 0 : kFlagSumMismatch;
      a.hdr->inverse = 0;
      a.hdr->A = a.A;
      a.hdr->N = 1;
      a.hdr->E = a.E;
      a.hdr->total = static_cast<int64_t>(total);
    }
    return valid;
  }

  // The hardware deals workgroups to the 8 XCDs in turn. Each XCD gets a run of
  // neighbouring tiles, which its workgroups take in turn, so that they share
  // rows in its L2.
  __device__ __forceinline__ void deal(const GroupedArgs& a) {
    const uint32_t work = all * static_cast<uint32_t>(a.n_tiles);
    const uint32_t xcd = blockIdx.x % 8, at = blockIdx.x / 8;
    const uint32_t run = work / 8 + (xcd < work % 8);
    step = (gridDim.x - xcd + 7) / 8;
    first = xcd * (work / 8) + min(xcd, work % 8) + at;
    count = at < run ? (run - at + step - 1) / step : 0;
  }

  // Tile i of this workgroup. Neighbours go down kGroup row tiles, then to the
  // next columns: a square of tiles shares the most rows.
  __device__ __forceinline__ Tile find(const GroupedArgs& a, uint32_t i) const {
    constexpr uint32_t kGroup = 4;
    const uint32_t id = first + i * step;
    const uint32_t band = id / (kGroup * a.n_tiles), in_band = id - band * kGroup * a.n_tiles;
    const uint32_t high = min(kGroup, all - band * kGroup);
    const uint32_t n = in_band / high;
    const uint32_t m = band * kGroup + in_band - n * high;
    const uint64_t mine = __ballot(m >= tiles && m < end);
    const int owner = __ffsll(static_cast<unsigned long long>(mine)) - 1;  // one lane's run holds tile m
    int expert = e0;
    uint32_t r = rows, exist = 0, before = tiles;
    if (static_cast<int>(threadIdx.x % 64) == owner)
      for (int e = e0; e < e1; ++e) {
        const uint32_t c = static_cast<uint32_t>(e == e0 ? head : count_of(a, e)), t = (c + kBM - 1) / kBM;
        if (m < before + t) {
          expert = e;
          exist = min(c - (m - before) * kBM, static_cast<uint32_t>(kBM));
          r += (m - before) * kBM;
          break;
        }
        before += t;
        r += c;
      }
    Tile t;
    t.expert = __builtin_amdgcn_readlane(expert, owner);
    t.row = static_cast<int>(__builtin_amdgcn_readlane(r, owner));
    t.rows = static_cast<int>(__builtin_amdgcn_readlane(exist, owner));
    t.n = static_cast<int>(__builtin_amdgcn_readfirstlane(n));
    return t;
  }
};

// 16 bytes of every lane, at `base` + its offset, to LDS from byte `lds` on in
// the order of the lanes. In assembly, as the compiler would wait for every
// such load before it lets any LDS read pass; the kernel waits by itself. (The
// compiler warns of m0, which it gives to no variable, but sets by itself elsewhere.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_to_lds(const uint8_t* base, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(offset), "s"(base)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// The four scale bytes of blocks b .. b + 3 of a row of n; 127 (a factor of
// one) past its end. b and n are the same for all lanes.
__device__ __forceinline__ uint32_t load_scales(const uint8_t* row, int b, int n) {
  constexpr uint32_t kOnes = 0x7f7f7f7fu;
  if (n >= 4) {  // the row's last four bytes hold what there is of them
    const int at = min(b, n - 4), over = b - at;
    uint32_t v;
    __builtin_memcpy(&v, row + at, 4);
    return over == 0 ? v : over >= 4 ? kOnes : v >> (8 * over) | kOnes << (32 - 8 * over);
  }
  uint32_t v = kOnes;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const uint32_t byte = row[min(b + i, n - 1)];
    if (b + i < n) v = (v & ~(0xffu << (8 * i))) | byte << (8 * i);
  }
  return v;
}

// A pointer that is the same for all lanes, in scalar registers.
__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t low = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t high = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return reinterpret_cast<const uint8_t*>(static_cast<uint64_t>(high) << 32 | low);
}

// How a row's 16-byte chunks are permuted: by bits of the row's number such that
// eight rows' same chunks fill 128 bytes of banks once, and sixteen rows' 256.
__device__ __forceinline__ int swizzle(int row) { return (row >> 1 & 3) | ((row ^ row >> 3) & 1) << 2; }

// Waits until at most kLeft of the wave's loads are on their way.
template <int kLeft>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLeft) : "memory");
}

// A barrier of LDS alone: loads from memory stay on their way.
__device__ __forceinline__ void workgroup_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// g / (1 + exp(-g)) with the chip's own exponential and reciprocal (an ulp each;
// a division would cost more than all else that is done to a result).
__device__ __forceinline__ float silu(float g) {
  constexpr float kLog2E = 1.44269504f;
  return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2E * g));
}

// A wave's results, kFM x kFN fragments, to rows m0 + ... of the tile's `rows`
// and columns col0 on of `cols`. A lane has one token row of each fragment and,
// of its 32 weight rows, four times four neighbours; by way of LDS (kLdsBytes of
// the wave alone, rows' 16-byte chunks permuted) it stores 16 bytes of a row, and
// its neighbours the next ones. kStream: past the caches, as the large tiles store,
// whatever the result's size: of bf16, 2048 x 7168 (29 MB) took 30.7 us so and 33.0 by
// way of the caches, 4096 x 2048 (17 MB, gated, K 7168) 65 and 69, 16384 x 7168 (235 MB)
// 139 and 159, and quantising them right behind does not turn it: 38.6 us for both and
// 40.2, 75 and 77, 179 and 196.
template <typename T, int kFM, int kFN, bool kGated, int kLdsBytes, bool kStream>
__device__ __forceinline__ void store_tile(const f32x16 (&acc)[kFN][kFM], uint8_t* lds, T* out, const float* row_weight,
                                           int64_t row0, int m0, int rows, int col0, int cols) {
  constexpr int kOutFN = kGated ? kFN / 2 : kFN;
  constexpr int kRowMost = kLdsBytes >= 32 * 256 ? 256 : 128;  // bytes of a row that a pass can take
  static_assert(kLdsBytes >= 32 * kRowMost, "32 rows");
  constexpr int kMost = kRowMost / 32 / static_cast<int>(sizeof(T));
  constexpr int kPerPass = kOutFN < kMost ? kOutFN : kMost;     // fragments of a pass
  constexpr int kChunks = kPerPass * 32 * sizeof(T) / 16;  // of a row
  constexpr int kValues = 16 / sizeof(T);
  constexpr int kLineRows = 64 / kChunks;                  // rows that the wave stores at a time
  using Out = T __attribute__((ext_vector_type(kValues)));
  using Loose = Out __attribute__((aligned(sizeof(T))));
  // opaque, or the compiler keeps the addresses below in registers that the
  // products need, spills them, and waits for the stores when it reloads them
  int lane = threadIdx.x % 64;
  asm volatile("" : "+v"(lane));
  const int r32 = lane % 32, half = lane / 32;
  constexpr int kWide = 4 * sizeof(T);  // bytes of four values
  const int chunk = lane % kChunks, line = lane / kChunks;
  // bits of the chunk are below those of the row, so the permutation is one xor
  const int write0 = r32 * kChunks * 16 + ((r32 % kChunks) * 16 ^ half * kWide / 16 * 16) + half * kWide % 16;
  const int read0 = line * kChunks * 16;
  const int64_t pitch = static_cast<int64_t>(cols) * sizeof(T);
#pragma unroll
  for (int j = 0; j < kFM; ++j) {
    const int left = rows - m0 - j * 32;  // rows of this fragment that exist
    if (left <= 0) return;
    const int64_t first = row0 + m0 + j * 32;
    const float rw = row_weight != nullptr ? row_weight[first + min(r32, left - 1)] : 1.0f;
#pragma unroll
    for (int i0 = 0; i0 < kOutFN; i0 += kPerPass) {
#pragma unroll
      for (int i = i0; i < i0 + kPerPass; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          T v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float y = acc[i][j][q * 4 + k];
            if constexpr (kGated) y = silu(y) * acc[i + kOutFN][j][q * 4 + k];
            v[k] = static_cast<T>(y * rw);
          }
          uint8_t* to = lds + (write0 ^ ((i - i0) * 32 + q * 8) * static_cast<int>(sizeof(T)));
          if constexpr (sizeof(T) == 4)
            *reinterpret_cast<f32x4*>(to) = f32x4{v[0], v[1], v[2], v[3]};
          else
            *reinterpret_cast<T __attribute__((ext_vector_type(4)))*>(to) = {v[0], v[1], v[2], v[3]};
        }
      const int col = col0 + i0 * 32 + chunk * kValues;
      uint8_t* p = reinterpret_cast<uint8_t*>(out + first * cols + col) + line * pitch;
#pragma unroll
      for (int l = 0; l < 32; l += kLineRows, p += kLineRows * pitch) {
        const int permuted = (chunk ^ ((l + line) % kChunks)) * 16;
        const Out v = *reinterpret_cast<const Out*>(lds + read0 + l * kChunks * 16 + permuted);
        if (l + line >= left) continue;
        if (col + kValues <= cols) {
          if constexpr (kStream)
            __builtin_nontemporal_store(v, reinterpret_cast<Loose*>(p));
          else
            *reinterpret_cast<Loose*>(p) = v;
        } else {
          for (int k = 0; k < kValues; ++k)
            if (col + k < cols) reinterpret_cast<T*>(p)[k] = v[k];
        }
      }
    }
  }
}

// kFN x kFM fragments of 32 weight rows x 32 token rows a wave, kWN x kWM
// waves a workgroup, which stays and takes tile after tile. A K tile is 256
// values, 128 bytes of a row, a whole line of the caches: the halves of a wave
// take its first and last four blocks, so that the four scales a lane needs for
// the tile's four products are one dword. The K tiles go from memory to LDS
// directly, kStages of them in turn: while one is multiplied, the next ones are
// on their way, those of the next output tile among them. The scales of two K
// tiles (16 bytes of a row) go through registers, as their rows have any alignment.
template <int kFM, int kFN, int kWM, int kWN, int kStages, bool kGated>
__global__ __launch_bounds__(64 * kWM * kWN, 2) void grouped_mm_kernel(GroupedArgs a) {
  constexpr int kWaves = kWM * kWN, kWgThreads = 64 * kWaves;
  constexpr int kBM = 32 * kFM * kWM, kBN = 32 * kFN * kWN, kRows = kBM + kBN;
  constexpr int kStage = kRows * kRowBytes;
  constexpr int kXLoads = kBM / 8 / kWaves, kWLoads = kBN / 8 / kWaves;
  static_assert(kXLoads * 8 * kWaves == kBM && kWLoads * 8 * kWaves == kBN, "whole loads");
  constexpr int kOwn = (kRows + kWgThreads - 1) / kWgThreads;  // rows whose scales a thread loads
  __shared__ __align__(1024) uint8_t lds[kStages * kStage];
  __shared__ uint32_t lds_scales[2 * 2 * 2 * kRows];  // two of [K tile of two][half][row]

  Tiles<kBM> tiles;
  if (!tiles.scan(a)) return;
  tiles.deal(a);
  if (tiles.count == 0) return;

  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  // waves of the same rows on different SIMDs: a tile of few rows then costs less
  const int wn = wave % kWN, wm = wave / kWN;
  const int r32 = lane % 32, half = lane / 32;
  const int half_n = a.N / 2;                      // gated: the up projection's first row
  const int n_end = kGated ? half_n : a.N;
  constexpr int kCols = kGated ? kBN / 2 : kBN;    // output columns of a tile
  const int64_t row_bytes = static_cast<int64_t>(a.blocks) * 16;
  const int k_tiles = (a.blocks + kTileBlocks - 1) / kTileBlocks;

  // The weight row in place j of a tile is column `col` of part `part`: gated,
  // a wave's fragments are the gate's and then the same columns of the up
  // projection.
  constexpr int kHalf = 32 * kFN / 2;
  auto part_of = [&](int j) { return kGated ? j % (32 * kFN) / kHalf : 0; };
  auto col_of = [&](int j, int n0) {
    const int col = n0 + (kGated ? j / (32 * kFN) * kHalf + j % kHalf : j);
    return min(col, n_end - 1);
  };

  // Staging: of every 8 rows a lane brings chunk lane % 8 (permuted) of one.
  const int chunk_even = (lane % 8) ^ swizzle(lane / 8);  // of rows with bit 3 clear
  uint32_t offset[kXLoads + kWLoads];
  const uint8_t* base[kXLoads + kWLoads];
  int stage_kt = 0, stage_slot = 0;
  uint32_t stage_tile = 0;
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)lds));
  // A wave's eight rows are number i * kWaves + wave of the operand's.
  auto chunk_of = [&](int i) { return chunk_even ^ ((i * kWaves + wave) % 2 * 4); };
  constexpr int kParity = kWaves % 2;  // whether a wave's loads alternate between the two permutations
  uint32_t back[2];  // past the row's end: its last block again, which does not count
  auto stage_begin = [&]() {
    const int left = a.blocks - stage_kt * kTileBlocks;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      back[i] = left < kTileBlocks && chunk_of(i) >= left ? (chunk_of(i) - left + 1) * 16 : 0;
    if (stage_tile >= tiles.count || stage_kt != 0) return;  // behind the last tile: its first K tile again
    const Tile t = tiles.find(a, stage_tile);
    const int n0 = t.n * kCols;
    int lane = threadIdx.x % 64;
    asm volatile("" : "+v"(lane));  // computed here, not kept in registers meanwhile
#pragma unroll
    for (int i = 0; i < kXLoads; ++i) {
      const int j = (i * kWaves + wave) * 8 + lane / 8;
      base[i] = uniform(a.x + t.row * row_bytes);
      offset[i] = static_cast<uint32_t>(min(j, t.rows - 1) * row_bytes) + chunk_of(i) * 16;
    }
#pragma unroll
    for (int i = 0; i < kWLoads; ++i) {
      const int j0 = (i * kWaves + wave) * 8;
      const int64_t row0 = static_cast<int64_t>(t.expert) * a.N + n0 + (part_of(j0) ? half_n : 0);
      base[kXLoads + i] = uniform(a.w + row0 * row_bytes);
      offset[kXLoads + i] = static_cast<uint32_t>((col_of(j0 + lane / 8, n0) - n0) * row_bytes) + chunk_of(i) * 16;
    }
  };
  auto stage_load = [&](int i) {  // load i of the K tile
    const int in_operand = i < kXLoads ? i : i - kXLoads;
    const uint32_t to = lds0 + stage_slot * kStage + (i < kXLoads ? 0 : kBM * kRowBytes) +
                        (in_operand * kWaves + wave) * 1024;
    load_to_lds(base[i] + stage_kt * kRowBytes, offset[i] - back[in_operand % 2 * kParity], to);
  };
  auto stage_end = [&]() {
    stage_slot = stage_slot + 1 == kStages ? 0 : stage_slot + 1;
    if (stage_tile < tiles.count && ++stage_kt == k_tiles) {
      stage_kt = 0;
      ++stage_tile;
    }
  };
  constexpr int kLoads = kXLoads + kWLoads;

  // The scales of this thread's rows for two K tiles.
  const uint8_t* s_row[kOwn];
  u32x4 held[kOwn];
  int scale_kt = 0;
  uint32_t scale_tile = 0;
  auto fetch_scales = [&]() {
    if (scale_tile >= tiles.count) return;
    if (scale_kt == 0) {
      const Tile t = tiles.find(a, scale_tile);
      const int n0 = t.n * kCols;
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const int j = threadIdx.x + i * kWgThreads, w = min(j, kRows - 1) - kBM;
        s_row[i] = j < kBM ? a.x_scales + static_cast<int64_t>(t.row + min(j, t.rows - 1)) * a.scale_bytes
                           : a.w_scales + (static_cast<int64_t>(t.expert) * a.N + col_of(w, n0) +
                                           (part_of(w) ? half_n : 0)) * a.scale_bytes;
      }
    }
    const int b = scale_kt * kTileBlocks;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      if (b + 16 <= a.blocks) {
        __builtin_memcpy(&held[i], s_row[i] + b, 16);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) held[i][c] = load_scales(s_row[i], b + 4 * c, a.blocks);
      }
    }
    scale_kt += 2;
    if (scale_kt >= k_tiles) {
      scale_kt = 0;
      ++scale_tile;
    }
  };
  int scale_slot = 0;
  auto keep_scales = [&]() {
    uint32_t* to = lds_scales + scale_slot * 4 * kRows;
    scale_slot ^= 1;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int j = threadIdx.x + i * kWgThreads;
      if (kRows % kWgThreads != 0 && j >= kRows) continue;
#pragma unroll
      for (int c = 0; c < 4; ++c) to[c * kRows + j] = held[i][c];
    }
  };

  f32x16 acc[kFN][kFM];
  const int at0 = r32 * kRowBytes + (((half * 4) ^ swizzle(r32)) * 16);
  // One K tile: a step's operands are read while the step before is multiplied,
  // and the next stage's loads are spread among the products.
  auto multiply = [&](int pair_tile, int scale_slot, int slot) {
    const uint8_t* xt = lds + slot * kStage + wm * kFM * 32 * kRowBytes;
    const uint8_t* wt = lds + slot * kStage + (kBM + wn * kFN * 32) * kRowBytes;
    const uint32_t* st = lds_scales + ((scale_slot * 2 + pair_tile) * 2 + half) * kRows + r32;
    int sx[kFM], sw[kFN];
    u32x4 xf[2][kFM], wf[2][kFN];
    auto read = [&](int s) {
      const int at = at0 ^ (s * 16);
#pragma unroll
      for (int i = 0; i < kFN; ++i) wf[s % 2][i] = *reinterpret_cast<const u32x4*>(wt + i * 32 * kRowBytes + at);
#pragma unroll
      for (int j = 0; j < kFM; ++j) xf[s % 2][j] = *reinterpret_cast<const u32x4*>(xt + j * 32 * kRowBytes + at);
    };
#pragma unroll
    for (int j = 0; j < kFM; ++j) sx[j] = static_cast<int>(st[(wm * kFM + j) * 32]);
#pragma unroll
    for (int i = 0; i < kFN; ++i) sw[i] = static_cast<int>(st[kBM + (wn * kFN + i) * 32]);
    read(0);
    constexpr int kProducts = kFN * kFM;
    auto step = [&](auto s_) {
      constexpr int s = decltype(s_)::value;
      if (s < 3) read(s + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int n = 0; n < kProducts; ++n) {
        const int i = n / kFM, j = n % kFM;
        const u32x4 w = wf[s % 2][i], x = xf[s % 2][j];
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            i32x8{(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0},
            i32x8{(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0}, acc[i][j], kMxFp4, kMxFp4, s, sw[i], s, sx[j]);
        // a load after each of the first products: the later ones are the time they have
#pragma unroll
        for (int l = 0; l < kLoads; ++l)
          if (l % (4 * kProducts) == s * kProducts + n) {
            __builtin_amdgcn_sched_barrier(0);
            stage_load(l);
            __builtin_amdgcn_sched_barrier(0);
          }
      }
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
  };

  fetch_scales();
  keep_scales();
  fetch_scales();
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    stage_begin();
#pragma unroll
    for (int l = 0; l < kLoads; ++l) stage_load(l);
    stage_end();
  }
  int slot = 0, read_slot = 1;
  for (uint32_t tile = 0; tile < tiles.count; ++tile) {
    const Tile t = tiles.find(a, tile);
    const bool works = wm * kFM * 32 < t.rows;  // a wave without rows only stages
#pragma unroll
    for (int i = 0; i < kFN; ++i)
#pragma unroll
      for (int j = 0; j < kFM; ++j)
#pragma unroll
        for (int k = 0; k < 16; ++k) acc[i][j][k] = 0.0f;
    for (int kt = 0; kt < k_tiles; ++kt) {
      // this K tile has arrived for the wave, and after the barrier for all of them
      if (kt > 0 || tile == 0) wait_loads<kLoads * (kStages - 2)>();
      workgroup_barrier();
      if (kt % 2 == 0) {  // the next two K tiles' scales, where no wave reads any more
        read_slot ^= 1;
        keep_scales();
        fetch_scales();
      }
      stage_begin();
      const int left = a.blocks - kt * kTileBlocks;
      if (left < kTileBlocks) {  // no products past the row's end: zeros for the tokens' values there
        for (int i = threadIdx.x; i < kBM * 8; i += kWgThreads)
          if (((i % 8) ^ swizzle(i / 8)) >= left)
            *reinterpret_cast<u32x4*>(lds + slot * kStage + i * 16) = u32x4{0, 0, 0, 0};
        workgroup_barrier();
      }
      if (works) {
        multiply(kt % 2, read_slot, slot);
      } else {
#pragma unroll
        for (int l = 0; l < kLoads; ++l) stage_load(l);
      }
      stage_end();
      slot = slot + 1 == kStages ? 0 : slot + 1;
    }
    // what the next tile begins with is here before the stores are on their way,
    // which it need not wait for
    wait_loads<0>();
    workgroup_barrier();
#pragma unroll
    for (int i = 0; i < kOwn; ++i) asm volatile("" : "+v"(held[i]));

    // The results go to memory by way of the K tile that was multiplied last, so
    // that a row's neighbouring columns are stored together.
    if (works) {
      auto store = [&](auto* type) {
        using T = std::remove_pointer_t<decltype(type)>;
        uint8_t* free_slot = lds + (slot == 0 ? kStages - 1 : slot - 1) * kStage;
        store_tile<T, kFM, kFN, kGated, kStage / kWaves, kBM * kBN >= 65536>(
            acc, free_slot + wave * (kStage / kWaves), static_cast<T*>(a.out), a.row_weight, t.row, wm * kFM * 32, t.rows,
            t.n * kCols + wn * (kCols / kWN), n_end);
      };
      if (a.out_dtype == MRR_BF16)
        store(static_cast<__bf16*>(nullptr));
      else if (a.out_dtype == MRR_F16)
        store(static_cast<_Float16*>(nullptr));
      else
        store(static_cast<float*>(nullptr));
    }
  }
}

// The counts alone, for a call without rows: their verdict.
__global__ void check_counts_kernel(GroupedArgs a) {
  Tiles<64> t;
  t.scan(a);
}

// A shape of tiles: kFN x kFM fragments a wave, kWN x kWM waves, and what it
// costs, in nanoseconds measured on the chip: a K tile of a workgroup that has
// its CU to itself, one beside as many others as the CU holds, and what comes
// on top for a tile of the output (its first loads, its stores).
template <int kFM_, int kFN_, int kWM_, int kWN_, int kAlone, int kFull, int kOutput>
struct Shape {
  static constexpr int kFM = kFM_, kFN = kFN_, kWM = kWM_, kWN = kWN_;
  static constexpr int kBM = 32 * kFM * kWM, kBN = 32 * kFN * kWN;
  static constexpr int kStages = 2;
  static constexpr int kLdsBytes = (kBM + kBN) * (kStages * kRowBytes + 32);
  static constexpr int kByLds = 160 * 1024 / kLdsBytes, kByWaves = 8 / (kWM * kWN);
  static constexpr int64_t kResident = 256 * (kByLds < kByWaves ? kByLds : kByWaves);  // workgroups the chip holds

  static int64_t n_tiles(const GroupedArgs& a, bool gated) {
    return gated ? (a.N / 2 + kBN / 2 - 1) / (kBN / 2) : (a.N + kBN - 1) / kBN;
  }

  // The call's time as far as the host can know it: rows spread evenly over
  // the experts, half a tile of each expert's rows empty.
  static int64_t cost(const GroupedArgs& a, bool gated) {
    const int64_t used = a.E < a.A ? a.E : a.A;
    const int64_t rows = a.A / kBM + (used + 1) / 2;
    const int64_t tiles = (rows > used ? rows : used) * n_tiles(a, gated);
    const int64_t rounds = (tiles + kResident - 1) / kResident;
    const int64_t k_tiles = (a.blocks + kTileBlocks - 1) / kTileBlocks;
    return rounds * (k_tiles * (tiles <= 256 ? kAlone : kFull) + kOutput);
  }

  static mrr_status launch(GroupedArgs a, bool gated, hipStream_t stream) {
    a.n_tiles = static_cast<int32_t>(n_tiles(a, gated));
    // the most row tiles there can be: every expert may end in a partial one
    const int64_t m_tiles = a.A / kBM + (a.E < a.A ? a.E : a.A);
    if (m_tiles * a.n_tiles > INT32_MAX) return MRR_ERROR_INVALID_SHAPE;  // tiles are numbered in 32 bits
    // as many workgroups as the chip holds at once, each taking its tiles in turn
    const int64_t grid = m_tiles * a.n_tiles < kResident ? m_tiles * a.n_tiles : kResident;
    const dim3 g(static_cast<unsigned>(grid)), b(64 * kWM * kWN);
    if (gated)
      hipLaunchKernelGGL((grouped_mm_kernel<kFM, kFN, kWM, kWN, kStages, true>), g, b, 0, stream, a);
    else
      hipLaunchKernelGGL((grouped_mm_kernel<kFM, kFN, kWM, kWN, kStages, false>), g, b, 0, stream, a);
    return hipGetLastError() == hipSuccess ? MRR_SUCCESS : MRR_ERROR_HIP;
  }
};

// Large tiles bring each operand row from L2 fewer times, small ones fill the
// chip with fewer rows. Measured (us) as 256 x 256, 128 x 128, 64 x 128 (rows x
// weight rows): 16384 rows of 16 experts, K 2048, N 7168: 171, 197, 272; 1024
// rows of 8 experts, K 4096, N 4096: 30, 24, 32; 64 rows of 16 experts, K 2048,
// N 4096: 18.1, 14.8, 14.4; 256 rows of one expert, K 7168, N 1024: 42, 20, 17.
using Large = Shape<2, 4, 4, 2, 1500, 2000, 6000>;
using Medium = Shape<2, 2, 2, 2, 720, 1400, 4000>;
using Small = Shape<1, 2, 2, 2, 610, 1100, 3000>;

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
    hipLaunchKernelGGL(mrr::check_counts_kernel, dim3(1), dim3(64), 0, stream, a);
    return hipGetLastError() == hipSuccess ? MRR_SUCCESS : MRR_ERROR_HIP;
  }
  const bool gated = args->gated == 1;
  const int64_t large = mrr::Large::cost(a, gated), medium = mrr::Medium::cost(a, gated);
  const int64_t small = mrr::Small::cost(a, gated);
  if (small <= medium && small <= large) return mrr::Small::launch(a, gated, stream);
  return medium <= large ? mrr::Medium::launch(a, gated, stream) : mrr::Large::launch(a, gated, stream);
}
