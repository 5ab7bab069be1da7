// mrr_token_permute.hip -- tokens sorted by expert: a stable counting sort of the
// choices (t, j) by expert, and the move of every token's row to the rows of its choices.
//
// Bound by memory: a row is read once and written top_k times. Few choices: one kernel,
// whose workgroups find their own token's rows, each the number of choices before it in
// the order of (expert, place), by comparing all choices with it (a ballot and a count
// for 64 of them). Many: blocks of choices are counted by expert, then placed (every
// block adds up the blocks before it), and the rows follow the index. In between blocks
// count all choices by themselves.
//
// Rows move in units of 16 bytes at any alignment; the last unit of a row that is no
// whole number of them begins earlier, so that two lanes write the same bytes twice. A
// wave holds 1 KiB of a token and writes it top_k times: 16384 tokens of 7168 bytes and
// their scales, 8 choices each, move in 205 to 211 us, 5.3 TB/s (a plain copy of 1 GiB: 6.7);
// waves that write an output row's 1 KiB each and read it anew take 258 to 390, workgroups
// of whole rows, two KiB a wave and waves that stay as long as this. With the sort 225 us;
// one token 3.5 us of kernel.
#include "mrr_rows.h"

namespace mrr {
namespace {

// One kind of rows: tokens', or their scales'.
struct Rows {
  const uint8_t* src;
  uint8_t* dst;
  uint32_t bytes;  // of a row
  uint32_t unit;   // 16, or what divides a shorter row: 4, 2 or 1
  uint32_t units;  // of a row
};

Rows rows_of(const void* src, void* dst, int64_t bytes) {
  Rows r{static_cast<const uint8_t*>(src), static_cast<uint8_t*>(dst), static_cast<uint32_t>(bytes), 16, 0};
  if (bytes < 16) r.unit = bytes % 4 == 0 ? 4 : bytes % 2 == 0 ? 2 : 1;
  r.units = static_cast<uint32_t>((bytes + r.unit - 1) / r.unit);
  return r;
}

// Moves one unit of a row of `r` in its lane: a load, then a store for each choice.
struct Unit {
  rows_u32x4 v;
  uint32_t at;
  __device__ __forceinline__ void load(const Rows& r, size_t row, uint32_t unit) {
    const uint8_t* p = r.src + row * r.bytes;
    at = unit * r.unit;
    if (r.unit == 16) {
      at = min(at, r.bytes - 16);
      v = load16(p + at);
    } else if (r.unit == 4) {
      uint32_t x;
      __builtin_memcpy(&x, p + at, 4);
      v[0] = x;
    } else if (r.unit == 2) {
      uint16_t x;
      __builtin_memcpy(&x, p + at, 2);
      v[0] = x;
    } else {
      v[0] = p[at];
    }
  }
  __device__ __forceinline__ void store(const Rows& r, size_t row, bool zero) const {
    uint8_t* p = r.dst + row * r.bytes + at;
    if (r.unit == 16) {
      store16(p, zero ? rows_u32x4{0, 0, 0, 0} : v);
    } else {
      const uint32_t x = zero ? 0 : v[0];
      if (r.unit == 4) {
        __builtin_memcpy(p, &x, 4);
      } else if (r.unit == 2) {
        const uint16_t h = static_cast<uint16_t>(x);
        __builtin_memcpy(p, &h, 2);
      } else {
        *p = static_cast<uint8_t>(x);
      }
    }
  }
};

struct SortArgs {
  const int32_t* ids;
  const float* weight;  // or null
  int32_t* idx;
  int32_t* num;
  float* out_weight;
  int32_t* counts;  // [blocks, E + 1]
  uint32_t n, T, k, E, block, blocks;
  int32_t cumsum;
};

// The expert of a choice, E for those that are not here.
__device__ __forceinline__ uint32_t expert_of(int32_t id, uint32_t E) {
  const uint32_t e = static_cast<uint32_t>(id);
  return e < E ? e : E;
}

// Inclusive sums over a workgroup's threads, by way of sh [threads / 64].
template <int kThreads>
__device__ __forceinline__ uint32_t scan_threads(uint32_t v, uint32_t* sh) {
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t o = static_cast<uint32_t>(__shfl_up(static_cast<int>(v), d));
    if (lane >= d) v += o;
  }
  if (lane == 63) sh[wave] = v;
  __syncthreads();
  for (int w = 0; w < wave; ++w) v += sh[w];
  return v;
}

// Writes expert_token_num from counts by expert in LDS; all threads of the workgroup.
template <int kThreads>
__device__ __forceinline__ void write_num(const uint32_t* count, const SortArgs& a, uint32_t* sh) {
  const uint32_t per = (a.E + kThreads - 1) / kThreads, first = threadIdx.x * per;
  uint32_t sum = 0;
  for (uint32_t i = 0; i < per; ++i)
    if (first + i < a.E) sum += count[first + i];
  uint32_t at = scan_threads<kThreads>(sum, sh) - sum;
  for (uint32_t i = 0; i < per; ++i) {
    if (first + i >= a.E) break;
    const uint32_t c = count[first + i];
    at += c;
    a.num[first + i] = static_cast<int32_t>(a.cumsum ? at : c);
  }
}

// ------------------------------------------------------------- few choices

constexpr int kFewThreads = 256;
constexpr int kFewWaves = kFewThreads / 64;
// A workgroup moves so many units of a token's row.
constexpr uint32_t kFewUnits = kFewThreads;

// kK: at least top_k.
template <int kK>
__global__ __launch_bounds__(kFewThreads) void permute_few_kernel(SortArgs a, Rows tokens, Rows scales) {
  __shared__ uint32_t sh[kPermuteMaxExperts];
  __shared__ uint32_t sh_before[kFewWaves][kK];  // and, of the last workgroup, sums of its waves
  const uint32_t tid = threadIdx.x, lane = tid % 64, wave = tid / 64, token = blockIdx.y;
  if (token == a.T) {  // the last workgroup counts
    if (blockIdx.x != 0) return;
    for (uint32_t e = tid; e < a.E; e += kFewThreads) sh[e] = 0;
    __syncthreads();
    for (uint32_t i = tid; i < a.n; i += kFewThreads) {
      const uint32_t e = expert_of(a.ids[i], a.E);
      if (e < a.E) atomicAdd(&sh[e], 1u);
    }
    __syncthreads();
    write_num<kFewThreads>(sh, a, &sh_before[0][0]);
    return;
  }
  const uint32_t unit = blockIdx.x * kFewUnits + tid, first = token * a.k;
  const bool moves = unit < tokens.units, moves_scales = blockIdx.x == 0 && tid < scales.units;
  const bool writes = blockIdx.x == 0 && tid < a.k;  // the index and the weight of choice tid
  Unit u, s;
  if (moves) u.load(tokens, token, unit);
  if (moves_scales) s.load(scales, token, tid);
  const float weight = writes && a.weight != nullptr ? a.weight[first + tid] : 0.0f;
  // (expert, place) as one number; a token's own are read by the lanes with all the rest
  const auto number = [&](int32_t id, uint32_t i) { return expert_of(id, a.E) * a.n + i; };
  uint32_t i = 64 * wave + lane;  // every wave compares its part of all choices with the token's own
  const int32_t own_id = lane < a.k ? a.ids[first + lane] : 0;
  int32_t id = i < a.n ? a.ids[i] : 0;
  const uint32_t own_number = lane < a.k ? number(own_id, first + lane) : 0;
  uint32_t own[kK], row[kK];
#pragma unroll
  for (uint32_t j = 0; j < kK; ++j) {
    own[j] = __builtin_amdgcn_readlane(own_number, j);
    row[j] = 0;
  }
  while (i - lane < a.n) {
    const uint32_t c = i < a.n ? number(id, i) : 0xffffffffu;
    i += kFewThreads;
    id = i < a.n ? a.ids[i] : 0;
#pragma unroll
    for (uint32_t j = 0; j < kK; ++j) row[j] += static_cast<uint32_t>(__popcll(__ballot(c < own[j])));
  }
  uint32_t mine = 0;  // lane j: the row of choice j
#pragma unroll
  for (uint32_t j = 0; j < kK; ++j) mine = lane == j ? row[j] : mine;
  if (lane < kK) sh_before[wave][lane] = mine;
  __syncthreads();
  mine = 0;
#pragma unroll
  for (int w = 0; w < kFewWaves; ++w) mine += sh_before[w][lane % kK];
  const uint64_t gone = __ballot(own_number >= a.E * a.n);
  if (writes) {
    const bool zero = gone >> tid & 1;
    a.idx[first + tid] = static_cast<int32_t>(zero ? ~mine : mine);
    if (a.weight != nullptr) a.out_weight[mine] = zero ? 0.0f : weight;
  }
#pragma unroll 1
  for (uint32_t j = 0; j < a.k; ++j) {
    const uint32_t to = __builtin_amdgcn_readlane(mine, j);
    const bool zero = gone >> j & 1;
    if (moves) u.store(tokens, to, zero);
    if (moves_scales) s.store(scales, to, zero);
  }
  if (blockIdx.x != 0) return;
  for (uint32_t more = tid + kFewThreads; more < scales.units; more += kFewThreads) {
    s.load(scales, token, more);
#pragma unroll 1
    for (uint32_t j = 0; j < a.k; ++j) {
      uint32_t to = 0;  // not read from lane j: it may have no more of them, and be out of the loop
#pragma unroll 1
      for (int w = 0; w < kFewWaves; ++w) to += sh_before[w][j];
      s.store(scales, to, gone >> j & 1);
    }
  }
}

// ------------------------------------------------------------ many choices

constexpr int kSortThreads = 1024;

// f(i, expert) of a lane's choices, from `first` (of lane 0) on every kStride-th, up to
// `end`, eight of them read at once. Choices that are not here are counted for the wave at
// once, by away(i, how many): they would all meet at one place.
template <uint32_t kStride, typename F, typename G>
__device__ __forceinline__ void each_choice(const SortArgs& a, uint32_t first, uint32_t end, F&& f, G&& away) {
  const uint32_t lane = threadIdx.x % 64;
  for (uint32_t i0 = first; i0 < end; i0 += 8 * kStride) {
    int32_t id[8];
#pragma unroll
    for (uint32_t x = 0; x < 8; ++x) id[x] = a.ids[min(i0 + x * kStride + lane, end - 1)];
#pragma unroll
    for (uint32_t x = 0; x < 8; ++x) {
      const uint32_t i = i0 + x * kStride + lane, e = expert_of(id[x], a.E);
      const uint64_t gone = __ballot(i < end && e == a.E);
      if (i < end && e < a.E) f(i, e);
      if (gone != 0 && lane == 0) away(i, static_cast<uint32_t>(__popcll(gone)));
    }
  }
}

__global__ __launch_bounds__(kSortThreads) void permute_count_kernel(SortArgs a) {
  __shared__ uint32_t count[kPermuteMaxExperts + 1];
  for (uint32_t e = threadIdx.x; e <= a.E; e += kSortThreads) count[e] = 0;
  __syncthreads();
  const uint32_t first = blockIdx.x * a.block;
  each_choice<kSortThreads>(a, first + threadIdx.x / 64 * 64, min(a.n, first + a.block), [&](uint32_t, uint32_t e) { atomicAdd(&count[e], 1u); },
              [&](uint32_t, uint32_t n) { atomicAdd(&count[a.E], n); });
  __syncthreads();
  for (uint32_t e = threadIdx.x; e <= a.E; e += kSortThreads)
    a.counts[static_cast<size_t>(blockIdx.x) * (a.E + 1) + e] = static_cast<int32_t>(count[e]);
}

// What the wave's lanes read and wrote in LDS before comes before what they do after: one
// instruction of a wave is done for all lanes before its next, and the compiler is told to keep it so.
__device__ __forceinline__ void in_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A block's choices take their rows. kRuns of its waves have a run of neighbouring choices
// each, counted by expert and placed in order, 64 at a time: the lanes of the same expert
// are found by its bits.
// kSelf: without the blocks' counts, of few blocks; each counts all choices by itself.
template <int kRuns, bool kSelf>
__global__ __launch_bounds__(kSortThreads) void permute_place_kernel(SortArgs a) {
  extern __shared__ uint32_t at[];  // [kRuns + 2, E + 1]
  __shared__ uint32_t sh[kSortThreads / 64];
  const uint32_t tid = threadIdx.x, lane = tid % 64, wave = tid / 64, width = a.E + 1;
  uint32_t* total = at + kRuns * width;
  uint32_t* start = total + width;
  for (uint32_t i = tid; i < width * (kRuns + 2); i += kSortThreads) at[i] = 0;
  __syncthreads();
  const uint32_t run = (kSelf ? static_cast<uint32_t>(kPermuteSelfBlock) : a.block) / kRuns;  // a multiple of 64
  const uint32_t from = blockIdx.x * a.block;
  // Of an expert: all its choices, those of the blocks before this one, and each run's.
  if constexpr (kSelf) {
    const uint32_t to = min(a.n, from + a.block);
    const auto count = [&](uint32_t i, uint32_t e, uint32_t n) {  // in total only those behind, for now
      uint32_t* counts = i < from ? start : i < to ? at + (i - from) / run * width : total;
      atomicAdd(&counts[e], n);
    };
    each_choice<kSortThreads>(a, wave * 64, a.n, [&](uint32_t i, uint32_t e) { count(i, e, 1); },
                              [&](uint32_t i, uint32_t n) { count(i, a.E, n); });  // 64 of them, in one run
    __syncthreads();
    for (uint32_t e = tid; e < width; e += kSortThreads) {
      uint32_t all = total[e] + start[e];
#pragma unroll
      for (uint32_t w = 0; w < kRuns; ++w) all += at[w * width + e];
      total[e] = all;
    }
  } else {
    constexpr uint32_t kShare = kSortThreads / 64 / kRuns;  // waves of a run
    const uint32_t begin = from + wave / kShare * run;
    uint32_t* counts = at + wave / kShare * width;
    each_choice<64 * kShare>(a, begin + wave % kShare * 64, min(a.n, begin + run),
                             [&](uint32_t, uint32_t e) { atomicAdd(&counts[e], 1u); },
                             [&](uint32_t, uint32_t n) { atomicAdd(&counts[a.E], n); });
    // threads share its column of the blocks' counts among them where there are enough
    const uint32_t slices = width >= kSortThreads ? 1 : kSortThreads / width;
    for (uint32_t i = tid; i < width * slices; i += kSortThreads) {
      const uint32_t e = i % width, slice = i / width;
      uint32_t all = 0, before = 0;
      const int32_t* c = a.counts + e;
      for (uint32_t b0 = slice; b0 < a.blocks; b0 += 16 * slices) {
        uint32_t v[16];
#pragma unroll
        for (uint32_t x = 0; x < 16; ++x)
          v[x] = static_cast<uint32_t>(c[static_cast<size_t>(min(b0 + x * slices, a.blocks - 1)) * width]);
#pragma unroll
        for (uint32_t x = 0; x < 16; ++x) {
          all += b0 + x * slices < a.blocks ? v[x] : 0;
          before += b0 + x * slices < blockIdx.x ? v[x] : 0;
        }
      }
      atomicAdd(&total[e], all);
      atomicAdd(&start[e], before);
    }
  }
  __syncthreads();
  // where its rows begin, where this block's of them do, then each wave's
  const uint32_t per = (width + kSortThreads - 1) / kSortThreads, e0 = tid * per;
  uint32_t sum = 0;
  for (uint32_t i = 0; i < per; ++i)
    if (e0 + i < width) sum += total[e0 + i];
  uint32_t begin = scan_threads<kSortThreads>(sum, sh) - sum;
  for (uint32_t i = 0; i < per; ++i) {
    const uint32_t e = e0 + i;
    if (e >= width) break;
    uint32_t place = begin + start[e];
    begin += total[e];
    if (blockIdx.x == 0 && e < a.E) a.num[e] = static_cast<int32_t>(a.cumsum ? begin : total[e]);
    for (int w = 0; w < kRuns; ++w) {
      const uint32_t c = at[w * width + e];
      at[w * width + e] = place;
      place += c;
    }
  }
  __syncthreads();
  if (wave >= kRuns) return;
  const uint32_t first = from + wave * run, end = min(a.n, first + run);
  uint32_t* mine = at + wave * width;
  const int bits = 32 - __builtin_clz(a.E);
  // four times 64 choices are read before the first is written: a load behind a store
  // would wait for it
  constexpr int kAhead = 4;
  for (uint32_t i0 = first; i0 < end; i0 += 64 * kAhead) {
    uint32_t expert[kAhead];
    float weight[kAhead];
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const uint32_t i = min(i0 + 64 * x + lane, end - 1);
      expert[x] = expert_of(a.ids[i], a.E);
      weight[x] = a.weight != nullptr ? a.weight[i] : 0.0f;
    }
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const uint32_t i = i0 + 64 * x + lane, e = expert[x];
      const bool here = i < end;
      uint64_t same = __ballot(here);
      for (int bit = 0; bit < bits; ++bit) {
        const bool set = e >> bit & 1;
        const uint64_t with = __ballot(set);
        same &= set ? with : ~with;
      }
      if (here) {
        const uint32_t rank = static_cast<uint32_t>(__popcll(same & ((uint64_t(1) << lane) - 1)));
        const uint32_t row = mine[e] + rank;
        in_order();  // all have read before the last of them writes
        if ((same >> lane) == 1) mine[e] = row + 1;
        in_order();  // and that is what the next 64 read
        a.idx[i] = static_cast<int32_t>(e < a.E ? row : ~row);
        if (a.weight != nullptr) a.out_weight[row] = e < a.E ? weight[x] : 0.0f;
      }
    }
  }
}

struct MoveArgs {
  const int32_t* idx;
  uint32_t T, k;
  uint32_t R;  // rows of the output
};

// Moves one unit of a token's row to its choices' rows. The index is read before the
// stores, eight choices at a time: a load behind a store would wait for it.
__device__ __forceinline__ void move_unit(const MoveArgs& a, const Rows& r, size_t token, uint32_t unit) {
  Unit u;
  u.load(r, token, unit);
  const int32_t* idx = a.idx + token * a.k;
  for (uint32_t j0 = 0; j0 < a.k; j0 += 8) {
    int32_t i[8];
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j) i[j] = idx[min(j0 + j, a.k - 1)];
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j) {
      const uint32_t row = static_cast<uint32_t>(i[j] < 0 ? ~i[j] : i[j]);
      if (j0 + j < a.k && row < a.R) u.store(r, row, i[j] < 0);
    }
  }
}

// Rows of more than 64 units: a wave moves 64 units of a token's row. Scales that are
// shorter go by the waves of the first workgroups, as many tokens each as fit.
// The token's index lies on the lanes, read once before the stores, and a row's address
// in scalar registers.
template <bool kStream>
__global__ __launch_bounds__(64) void move_rows_kernel(MoveArgs a, Rows r, Rows scales, uint32_t first) {
  if (blockIdx.y < first) {
    const uint32_t tokens = 64 / scales.units, in_wave = threadIdx.x / scales.units;
    const uint32_t t = (blockIdx.y * gridDim.x + blockIdx.x) * tokens + in_wave;
    if (in_wave < tokens && t < a.T) move_unit(a, scales, t, threadIdx.x - in_wave * scales.units);
    return;
  }
  const uint32_t token = blockIdx.y - first;
  const int32_t mine = a.idx[static_cast<size_t>(token) * a.k + min(threadIdx.x, a.k - 1)];
  // lanes behind the row's end move its last unit as well
  const uint32_t at = min((blockIdx.x * 64 + threadIdx.x) * 16, r.bytes - 16);
  const rows_u32x4 v = load16(r.src + static_cast<size_t>(token) * r.bytes + at);
  for (uint32_t j = 0; j < a.k; ++j) {
    const int32_t i = __builtin_amdgcn_readlane(mine, j);
    const uint32_t row = static_cast<uint32_t>(i < 0 ? ~i : i);
    if (row >= a.R) continue;
    uint8_t* to = r.dst + static_cast<size_t>(row) * r.bytes;
    const rows_u32x4 out = i >= 0 ? v : rows_u32x4{0, 0, 0, 0};
    if constexpr (kStream)
      WholeRow<>(to, r.bytes).store(at, out);
    else
      store16(to + at, out);
  }
}

// Shorter ones, scales included: as many tokens a wave as fit.
__global__ __launch_bounds__(256) void move_short_rows_kernel(MoveArgs a, Rows r, Rows scales) {
  const uint32_t units = r.units + scales.units;
  const uint32_t lane = threadIdx.x % 64, tokens = 64 / units, in_wave = lane / units;
  const size_t token = (static_cast<size_t>(blockIdx.x) * 4 + threadIdx.x / 64) * tokens + in_wave;
  if (in_wave >= tokens || token >= a.T) return;
  const uint32_t unit = lane - in_wave * units;
  if (unit < r.units)
    move_unit(a, r, token, unit);
  else
    move_unit(a, scales, token, unit - r.units);
}

// Tokens of a launch whose grid's second dimension they are, with the scales' rows of workgroups.
constexpr uint32_t kMostGridY = 32767;
template <bool kStream>
void move_all(const MoveArgs& all, Rows r, Rows scales, hipStream_t stream) {
  if (scales.units > 64 || (r.units <= 64 && r.units + scales.units > 64)) {  // each by itself
    move_all<false>(all, scales, Rows{}, stream);
    if (hipPeekAtLastError() != hipSuccess) return;
    scales = Rows{};
  }
  const bool wide = r.units > 64;
  constexpr uint32_t kMostTokens = 1u << 24;  // of a launch, which holds less than 2^32 threads
  MoveArgs a = all;
  for (uint32_t t = 0; t < all.T;) {
    const uint32_t most = wide ? kMostGridY : kMostTokens;
    a.T = all.T - t < most ? all.T - t : most;
    if (wide) {
      const uint32_t pieces = (r.units + 63) / 64;
      const uint32_t more = scales.units == 0 ? 0 : (a.T + pieces * (64 / scales.units) - 1) / (pieces * (64 / scales.units));
      move_rows_kernel<kStream><<<dim3(pieces, a.T + more), 64, 0, stream>>>(a, r, scales, more);
    } else {
      const uint32_t each = 4 * (64 / (r.units + scales.units));
      move_short_rows_kernel<<<(a.T + each - 1) / each, 256, 0, stream>>>(a, r, scales);
    }
    if (hipPeekAtLastError() != hipSuccess) return;
    t += a.T;
    a.idx += static_cast<size_t>(a.T) * a.k;
    r.src += static_cast<size_t>(a.T) * r.bytes;
    if (scales.units > 0) scales.src += static_cast<size_t>(a.T) * scales.bytes;
  }
}

// scales: of no units where there are none.
void move_both(const Rows& r, const Rows& scales, const int32_t* idx, int64_t T, int64_t k, int64_t R, hipStream_t stream) {
  const MoveArgs a{idx, static_cast<uint32_t>(T), static_cast<uint32_t>(k), static_cast<uint32_t>(R)};
  // Aligned rows are written past the caches: 16384 rows of 14 KiB, 235 MB, take 53.6 us so
  // and 61 through them, 8192 rows of 2 KiB 11.0 and 12.6; of 940 MB both take the same
  // within 2%.
  if (whole_units(r.bytes, r.dst))
    move_all<true>(a, r, scales, stream);
  else
    move_all<false>(a, r, scales, stream);
}

constexpr uint32_t place_lds(uint32_t runs, uint32_t E) { return (runs + 2) * (E + 1) * 4; }
constexpr uint32_t kMostLds = 60 * 1024;
static_assert(place_lds(1, kPermuteMaxExperts) <= kMostLds, "experts' places in LDS");
static_assert(kPermuteBlockChoices % (16 * 64) == 0 && kPermuteSelfBlock % (16 * 64) == 0, "a wave's run of choices");

template <bool kSelf>
void place_all(const SortArgs& a, hipStream_t stream) {
  if (place_lds(16, a.E) <= kMostLds)
    permute_place_kernel<16, kSelf><<<a.blocks, kSortThreads, place_lds(16, a.E), stream>>>(a);
  else if (place_lds(4, a.E) <= kMostLds)
    permute_place_kernel<4, kSelf><<<a.blocks, kSortThreads, place_lds(4, a.E), stream>>>(a);
  else
    permute_place_kernel<1, kSelf><<<a.blocks, kSortThreads, place_lds(1, a.E), stream>>>(a);
}

}  // namespace

void move_rows(const void* src, void* dst, int64_t row_bytes, const int32_t* idx, int64_t T, int64_t k, int64_t R,
               hipStream_t stream) {
  move_both(rows_of(src, dst, row_bytes), Rows{}, idx, T, k, R, stream);
}

}  // namespace mrr

extern "C" mrr_status mrr_token_permute(const mrr_token_permute_args* args, void* workspace, size_t workspace_bytes,
                                        struct ihipStream_t* stream) {
  using namespace mrr;
  const mrr_status st = check_token_permute(args, workspace, workspace_bytes);
  if (st != MRR_SUCCESS) return st;
  const int64_t n = args->T * args->top_k, row = permute_row_bytes(args);
  const int64_t scale_row = args->per_token_scales == nullptr ? 0 : permute_scale_bytes(args);
  SortArgs a;
  a.ids = args->expert_ids;
  a.weight = args->expert_weight;
  a.idx = args->permute_token_idx;
  a.num = args->expert_token_num;
  a.out_weight = args->permute_topk_weight;
  a.counts = static_cast<int32_t*>(workspace);
  a.n = static_cast<uint32_t>(n);
  a.T = static_cast<uint32_t>(args->T);
  a.k = static_cast<uint32_t>(args->top_k);
  a.E = static_cast<uint32_t>(args->E);
  a.cumsum = args->expert_token_num_type == 0;
  a.block = static_cast<uint32_t>(permute_block(n, args->E));
  a.blocks = static_cast<uint32_t>(permute_blocks(n, args->E));
  const Rows tokens = rows_of(args->tokens, args->permute_tokens, row);
  Rows scales{};
  if (scale_row > 0) scales = rows_of(args->per_token_scales, args->permute_per_token_scales, scale_row);
  if (n <= kPermuteFewChoices) {
    const dim3 grid((tokens.units + kFewUnits - 1) / kFewUnits, a.T + 1);
    if (a.k <= 2)
      permute_few_kernel<2><<<grid, kFewThreads, 0, stream>>>(a, tokens, scales);
    else if (a.k <= 4)
      permute_few_kernel<4><<<grid, kFewThreads, 0, stream>>>(a, tokens, scales);
    else if (a.k <= 8)
      permute_few_kernel<8><<<grid, kFewThreads, 0, stream>>>(a, tokens, scales);
    else
      permute_few_kernel<16><<<grid, kFewThreads, 0, stream>>>(a, tokens, scales);
    return hipGetLastError() == hipSuccess ? MRR_SUCCESS : MRR_ERROR_HIP;
  }
  if (n <= kPermuteSelfChoices) {
    a.block = kPermuteSelfBlock;
    a.blocks = static_cast<uint32_t>((n + kPermuteSelfBlock - 1) / kPermuteSelfBlock);
    place_all<true>(a, stream);
  } else {
    permute_count_kernel<<<a.blocks, kSortThreads, 0, stream>>>(a);
    if (hipGetLastError() != hipSuccess) return MRR_ERROR_HIP;
    place_all<false>(a, stream);
  }
  if (hipGetLastError() != hipSuccess) return MRR_ERROR_HIP;
  move_both(tokens, scales, a.idx, args->T, args->top_k, n, stream);
  return hipGetLastError() == hipSuccess ? MRR_SUCCESS : MRR_ERROR_HIP;
}
