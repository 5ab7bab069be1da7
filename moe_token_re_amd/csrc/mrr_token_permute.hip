// mrr_token_permute.hip -- tokens sorted by expert: a stable counting sort of the
// choices (t, j) by expert, and the move of every token's row to the rows of its choices.
//
// Bound by memory: a row is read once and written top_k times. Few choices: one kernel,
// whose workgroups find their own token's rows, each the number of choices before it in
// the order of (expert, place), by comparing all choices with it (a ballot and a count
// for 64 of them). Many: blocks of choices are counted by expert, then placed (every
// block adds up the blocks before it), and the rows follow the index.
//
// Rows move in units of 16 bytes at any alignment; the last unit of a row that is no
// whole number of them begins earlier, so that two lanes write the same bytes twice.
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
      v = load16<false>(p + at);
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
  template <bool kStream>
  __device__ __forceinline__ void store(const Rows& r, size_t row, bool zero) const {
    uint8_t* p = r.dst + row * r.bytes + at;
    if (r.unit == 16) {
      store16<kStream>(p, zero ? rows_u32x4{0, 0, 0, 0} : v);
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
// A workgroup moves so much of a token's row.
constexpr uint32_t kFewUnits = kFewThreads;

__global__ __launch_bounds__(kFewThreads) void permute_few_kernel(SortArgs a, Rows tokens, Rows scales) {
  __shared__ uint32_t sh[kPermuteMaxExperts + 1];
  __shared__ uint32_t sh_wave[kFewThreads / 64][kLayerMaxTopK], sh_own[kLayerMaxTopK];
  const uint32_t tid = threadIdx.x, token = blockIdx.y;
  if (token == a.T) {  // the last workgroup counts
    if (blockIdx.x != 0) return;
    for (uint32_t e = tid; e < a.E; e += kFewThreads) sh[e] = 0;
    __syncthreads();
    for (uint32_t i = tid; i < a.n; i += kFewThreads) {
      const uint32_t e = expert_of(a.ids[i], a.E);
      if (e < a.E) atomicAdd(&sh[e], 1u);
    }
    __syncthreads();
    write_num<kFewThreads>(sh, a, sh_wave[0]);
    return;
  }
  const uint32_t unit = blockIdx.x * kFewUnits + tid;
  Unit u, s;
  if (unit < tokens.units) u.load(tokens, token, unit);
  const bool moves_scales = blockIdx.x == 0 && tid < scales.units;  // the first of them; more below
  if (moves_scales) s.load(scales, token, tid);
  // (expert, place) as one number
  const uint32_t first = token * a.k;
  uint32_t own[kLayerMaxTopK], before[kLayerMaxTopK] = {};
#pragma unroll
  for (uint32_t j = 0; j < kLayerMaxTopK; ++j)
    own[j] = j < a.k ? expert_of(a.ids[first + j], a.E) * a.n + first + j : 0;
  for (uint32_t i0 = tid / 64 * 64; i0 < a.n; i0 += kFewThreads) {
    const uint32_t i = i0 + tid % 64;
    const uint32_t c = i < a.n ? expert_of(a.ids[i], a.E) * a.n + i : 0xffffffffu;
#pragma unroll
    for (uint32_t j = 0; j < kLayerMaxTopK; ++j)
      if (j < a.k) before[j] += static_cast<uint32_t>(__popcll(__ballot(c < own[j])));
  }
#pragma unroll
  for (uint32_t j = 0; j < kLayerMaxTopK; ++j) {
    if (tid % 64 == 0) sh_wave[tid / 64][j] = before[j];
    if (tid == 0) sh_own[j] = own[j];
  }
  __syncthreads();
  const uint32_t away = a.E * a.n;
  for (uint32_t j = 0; j < a.k; ++j) {
    uint32_t row = 0;
#pragma unroll
    for (int w = 0; w < kFewThreads / 64; ++w) row += sh_wave[w][j];
    const bool zero = sh_own[j] >= away;
    if (unit < tokens.units) u.store<false>(tokens, row, zero);
    if (moves_scales) s.store<false>(scales, row, zero);
    if (blockIdx.x == 0) {
      for (uint32_t more = tid + kFewThreads; more < scales.units; more += kFewThreads) {
        Unit m;
        m.load(scales, token, more);
        m.store<false>(scales, row, zero);
      }
      if (tid == j) {
        a.idx[first + j] = static_cast<int32_t>(zero ? ~row : row);
        if (a.weight != nullptr) a.out_weight[row] = zero ? 0.0f : a.weight[first + j];
      }
    }
  }
}

// ------------------------------------------------------------ many choices

constexpr int kCountThreads = 1024;

__global__ __launch_bounds__(kCountThreads) void permute_count_kernel(SortArgs a) {
  __shared__ uint32_t count[kPermuteMaxExperts + 1];
  for (uint32_t e = threadIdx.x; e <= a.E; e += kCountThreads) count[e] = 0;
  __syncthreads();
  const uint32_t first = blockIdx.x * a.block, end = min(a.n, first + a.block);
  for (uint32_t i = first + threadIdx.x; i < end; i += kCountThreads) atomicAdd(&count[expert_of(a.ids[i], a.E)], 1u);
  __syncthreads();
  for (uint32_t e = threadIdx.x; e <= a.E; e += kCountThreads)
    a.counts[static_cast<size_t>(blockIdx.x) * (a.E + 1) + e] = static_cast<int32_t>(count[e]);
}

// A block's choices take their rows. Its waves have a run of neighbouring choices each,
// count them by expert, and place them in order, 64 at a time: the lanes of the same
// expert are found by its bits.
template <int kWaves>
__global__ __launch_bounds__(64 * kWaves) void permute_place_kernel(SortArgs a) {
  constexpr int kThreads = 64 * kWaves;
  extern __shared__ uint32_t at[];  // [kWaves, E + 1]
  __shared__ uint32_t sh[kWaves];
  const uint32_t tid = threadIdx.x, lane = tid % 64, wave = tid / 64, width = a.E + 1;
  for (uint32_t i = tid; i < width * kWaves; i += kThreads) at[i] = 0;
  __syncthreads();
  const uint32_t run = a.block / kWaves;  // a multiple of 64
  const uint32_t first = blockIdx.x * a.block + wave * run, end = min(a.n, first + run);
  uint32_t* mine = at + wave * width;
  for (uint32_t i = first + lane; i < end; i += 64) atomicAdd(&mine[expert_of(a.ids[i], a.E)], 1u);
  __syncthreads();
  // where an expert's rows begin, then where this block's of them do, then each wave's
  const uint32_t per = (width + kThreads - 1) / kThreads, e0 = tid * per;
  uint32_t sum = 0;
  for (uint32_t i = 0; i < per; ++i) {
    const uint32_t e = e0 + i;
    if (e >= width) break;
    for (uint32_t b = 0; b < a.blocks; ++b) sum += static_cast<uint32_t>(a.counts[static_cast<size_t>(b) * width + e]);
  }
  uint32_t begin = scan_threads<kThreads>(sum, sh) - sum;
  for (uint32_t i = 0; i < per; ++i) {
    const uint32_t e = e0 + i;
    if (e >= width) break;
    uint32_t all = 0, place = begin;
    for (uint32_t b = 0; b < a.blocks; ++b) {
      const uint32_t c = static_cast<uint32_t>(a.counts[static_cast<size_t>(b) * width + e]);
      if (b < blockIdx.x) place += c;
      all += c;
    }
    begin += all;
    if (blockIdx.x == 0 && e < a.E) a.num[e] = static_cast<int32_t>(a.cumsum ? begin : all);
    for (int w = 0; w < kWaves; ++w) {
      const uint32_t c = at[w * width + e];
      at[w * width + e] = place;
      place += c;
    }
  }
  __syncthreads();
  const int bits = 32 - __builtin_clz(a.E);
  for (uint32_t i0 = first; i0 < end; i0 += 64) {
    const uint32_t i = i0 + lane;
    const bool here = i < end;
    const uint32_t e = here ? expert_of(a.ids[i], a.E) : 0;
    uint64_t same = __ballot(here);
    for (int bit = 0; bit < bits; ++bit) {
      const bool set = e >> bit & 1;
      const uint64_t with = __ballot(set);
      same &= set ? with : ~with;
    }
    if (here) {
      const uint32_t rank = static_cast<uint32_t>(__popcll(same & ((uint64_t(1) << lane) - 1)));
      const uint32_t row = mine[e] + rank;
      // the last of them, after all have read
      if ((same >> lane) == 1) mine[e] = row + 1;
      a.idx[i] = static_cast<int32_t>(e < a.E ? row : ~row);
      if (a.weight != nullptr) a.out_weight[row] = e < a.E ? a.weight[i] : 0.0f;
    }
  }
}

struct MoveArgs {
  const int32_t* idx;
  uint32_t T, k;
  uint32_t R;  // rows of the output
};

// Rows of more than 64 units: a wave moves 1 KiB of a token's row.
template <bool kStream>
__global__ __launch_bounds__(64) void move_rows_kernel(MoveArgs a, Rows r) {
  const uint32_t token = blockIdx.y, unit = blockIdx.x * 64 + threadIdx.x;
  if (unit >= r.units) return;
  Unit u;
  u.load(r, token, unit);
  const int32_t* idx = a.idx + static_cast<size_t>(token) * a.k;
  for (uint32_t j = 0; j < a.k; ++j) {
    const int32_t i = idx[j];
    const uint32_t row = static_cast<uint32_t>(i < 0 ? ~i : i);
    if (row < a.R) u.store<kStream>(r, row, i < 0);
  }
}

// Shorter ones: as many tokens a wave as fit.
template <bool kStream>
__global__ __launch_bounds__(256) void move_short_rows_kernel(MoveArgs a, Rows r) {
  const uint32_t lane = threadIdx.x % 64, tokens = 64 / r.units, in_wave = lane / r.units;
  const size_t token = (static_cast<size_t>(blockIdx.x) * 4 + threadIdx.x / 64) * tokens + in_wave;
  if (in_wave >= tokens || token >= a.T) return;
  Unit u;
  u.load(r, token, lane - in_wave * r.units);
  const int32_t* idx = a.idx + token * a.k;
  for (uint32_t j = 0; j < a.k; ++j) {
    const int32_t i = idx[j];
    const uint32_t row = static_cast<uint32_t>(i < 0 ? ~i : i);
    if (row < a.R) u.store<kStream>(r, row, i < 0);
  }
}

constexpr uint32_t kMostGridY = 65535;
// Outputs of so many bytes are written past the caches, which would not hold them.
constexpr int64_t kStreamBytes = int64_t(64) << 20;

template <bool kStream>
void move_all(const MoveArgs& all, const Rows& rows, hipStream_t stream) {
  if (rows.units > 64) {
    for (uint32_t t = 0; t < all.T; t += kMostGridY) {
      MoveArgs a = all;
      Rows r = rows;
      a.idx += static_cast<size_t>(t) * a.k;
      r.src += static_cast<size_t>(t) * r.bytes;
      a.T = all.T - t < kMostGridY ? all.T - t : kMostGridY;
      move_rows_kernel<kStream><<<dim3((r.units + 63) / 64, a.T), 64, 0, stream>>>(a, r);
    }
    return;
  }
  constexpr uint32_t kMostTokens = 1u << 24;  // of a launch, which holds less than 2^32 threads
  for (uint32_t t = 0; t < all.T;) {
    MoveArgs a = all;
    Rows r = rows;
    a.idx += static_cast<size_t>(t) * a.k;
    r.src += static_cast<size_t>(t) * r.bytes;
    a.T = all.T - t < kMostTokens ? all.T - t : kMostTokens;
    const uint32_t each = 4 * (64 / r.units);
    move_short_rows_kernel<kStream><<<(a.T + each - 1) / each, 256, 0, stream>>>(a, r);
    t += a.T;
  }
}

void place_all(const SortArgs& a, hipStream_t stream) {
  const uint32_t width = a.E + 1;
  constexpr uint32_t kMostLds = 60 * 1024;
  if (16 * width * 4 <= kMostLds)
    permute_place_kernel<16><<<a.blocks, 1024, 16 * width * 4, stream>>>(a);
  else if (8 * width * 4 <= kMostLds)
    permute_place_kernel<8><<<a.blocks, 512, 8 * width * 4, stream>>>(a);
  else
    permute_place_kernel<2><<<a.blocks, 128, 2 * width * 4, stream>>>(a);
}
static_assert(2 * (kPermuteMaxExperts + 1) * 4 <= 60 * 1024, "experts' places in LDS");
static_assert(kPermuteBlockChoices % (16 * 64) == 0, "a wave's run of choices");

}  // namespace

void move_rows(const void* src, void* dst, int64_t row_bytes, const int32_t* idx, int64_t T, int64_t k, int64_t R,
               hipStream_t stream) {
  const MoveArgs a{idx, static_cast<uint32_t>(T), static_cast<uint32_t>(k), static_cast<uint32_t>(R)};
  const Rows r = rows_of(src, dst, row_bytes);
  if (R * row_bytes >= kStreamBytes)
    move_all<true>(a, r, stream);
  else
    move_all<false>(a, r, stream);
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
    permute_few_kernel<<<dim3((tokens.units + kFewUnits - 1) / kFewUnits, a.T + 1), kFewThreads, 0, stream>>>(a, tokens,
                                                                                                         scales);
    return hipGetLastError() == hipSuccess ? MRR_SUCCESS : MRR_ERROR_HIP;
  }
  permute_count_kernel<<<a.blocks, kCountThreads, 0, stream>>>(a);
  place_all(a, stream);
  move_rows(args->tokens, args->permute_tokens, row, a.idx, args->T, args->top_k, n, stream);
  if (scale_row > 0)
    move_rows(args->per_token_scales, args->permute_per_token_scales, scale_row, a.idx, args->T, args->top_k, n, stream);
  return hipGetLastError() == hipSuccess ? MRR_SUCCESS : MRR_ERROR_HIP;
}
