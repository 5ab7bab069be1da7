// mrr_few_tokens.hip -- a whole mixture-of-experts layer for a few tokens:
//     h[t, j] = p[t, j] silu(Wg[e] x[t]) * (Wu[e] x[t])   for e = ids[t, j],
//     y[t]    = sum over j of Wd[e] h[t, j].
// Bound by reading the chosen experts' weights, once each (a kernel that does nothing
// else reads 6.3 TB/s by way of the caches, 7.1 past them). Two kernels, one a product;
// for more than a few tokens a third before them finds the routing (softmax and top-k
// of the router's logits), which every workgroup of the first would otherwise find for
// itself. The second adds an output row's experts in a fixed order, so results do not
// depend on timing. What it measured: one token, 8 of 64 4-bit experts, H 7168, I 2048
// (187 MB): 49 us, 3.8 TB/s; 16 tokens, 6 of 64 fp16 experts by ids, a quarter of them
// elsewhere, H 2048, I 1408 (762 MB): 148 us, 5.1 TB/s; 64 tokens, 4 of 32 4-bit
// experts, H 4096, I 2048 (428 MB): 128 us, 3.3 TB/s, of which half is issuing
// instructions: in the first kernel a chunk of 4 KiB of weights takes 250 of them, 64 to
// widen the weights, 52 to sort lanes. Here and below weights come from memory, as
// several layers' take turns, and h and tokens from the caches.
//
// Both feed the matrix instructions with 16 weight rows and up to 16 of the tokens
// that chose the expert. A lane reads 32 bytes of a weight row at a time: 16 16-bit
// values, or two blocks of 32 4-bit values, widened to bf16 with their scale, which is
// exact but for the two largest scales (take_blocks). x has 16 bits as it comes. h has
// no such type, and 16 bits would round it or, fp16, end at 65504: it is held as two
// bf16 values, hi + lo, off by at most 2^-15. They take two columns of the instruction's
// 16, so that 8 tokens cost what 16 of one column would; fp16 weights are multiplied as
// the two bf16 values that they are the sum of. (fp32 products, 16x16x4, would need
// neither: 64 tokens, 8 of 16 bf16 experts, H 4096, took 289 us with them and 267 so, at
// one run of rows a wave.)
#include "mrr_device.h"
#include "mrr_experts.h"

#include <algorithm>

namespace mrr {
namespace {

using u32x4 = uint32_t __attribute__((ext_vector_type(4)));
using f32x4 = float __attribute__((ext_vector_type(4)));
using bf16x2 = __bf16 __attribute__((ext_vector_type(2)));
using bf16x8 = __bf16 __attribute__((ext_vector_type(8)));
using f16x2 = _Float16 __attribute__((ext_vector_type(2)));
using f16x8 = _Float16 __attribute__((ext_vector_type(8)));

constexpr int kMaxExperts = static_cast<int>(kFewMaxExperts);
constexpr int kExpertBits = 10;   // of an expert's number
static_assert(kMaxExperts == 1 << kExpertBits, "all of them");
constexpr int kUpWaves = 4;       // first kernel: they share a unit's rows, each a part of their length
constexpr int kRows = 16;         // weight rows of a fragment
constexpr int kDownTokens = 64;   // tokens of a workgroup of the second kernel
constexpr int kPlaces = 8;        // tokens of a tile there: a column for hi, one for lo
constexpr int kManyChoices = 10;  // of an expert, on average: more tiles of tokens at once
constexpr int kSelfRouted = 4;    // so many tokens, a wave each, the first kernel routes itself

struct FewArgs {
  const uint8_t* x;
  const float* logits;
  const int32_t* ids;
  const float* weight;
  const uint8_t* gate_up;
  const uint8_t* gate_up_scales;
  const uint8_t* down;
  const uint8_t* down_scales;
  uint8_t* y;
  int32_t* ws_ids;
  float* ws_weight;
  int32_t* ws_between;  // of a choice: where its h lies (Between)
  int32_t* ws_arrived;  // of a run of output rows: the workgroups that are done
  f32x4* ws_part;
  uint8_t* ws_h;
  int32_t T, H, E, I, k;
  int32_t renormalize;
};

inline __host__ __device__ constexpr size_t up_part_bytes(int tiles) {
  return 2 * sizeof(f32x4) * kUpWaves * 2 * tiles * 64;
}
inline __host__ __device__ constexpr size_t down_sum_bytes(int tokens, int waves, int parts) {
  return sizeof(f32x4) * waves * tokens * 4 * parts;
}

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  constexpr int kRowShr1 = 0x111, kRowShr2 = 0x112, kRowShr4 = 0x114, kRowShr8 = 0x118;
  constexpr int kRowBcast15 = 0x142, kRowBcast31 = 0x143;
  auto step = [&](auto ctrl, auto rows) {
    v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), decltype(ctrl)::value,
                                                                 decltype(rows)::value, 0xf, false)));
  };
  using std::integral_constant;
  step(integral_constant<int, kRowShr1>{}, integral_constant<int, 0xf>{});
  step(integral_constant<int, kRowShr2>{}, integral_constant<int, 0xf>{});
  step(integral_constant<int, kRowShr4>{}, integral_constant<int, 0xf>{});
  step(integral_constant<int, kRowShr8>{}, integral_constant<int, 0xf>{});
  step(integral_constant<int, kRowBcast15>{}, integral_constant<int, 0xa>{});
  step(integral_constant<int, kRowBcast31>{}, integral_constant<int, 0xc>{});
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
}

__device__ __forceinline__ float wave_sum_f32(float v) {
#pragma unroll
  for (int d = 32; d > 0; d /= 2) v += __shfl_xor(v, d);
  return v;
}

// A logit as an unsigned key of the same order; 0 for -inf (never chosen),
// NaN above all, both zeros alike.
__device__ __forceinline__ uint32_t logit_key(float l) {
  const uint32_t b = __float_as_uint(l + 0.0f);
  if (l != l) return 0xffffffffu;
  if (b == 0xff800000u) return 0;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// One wave chooses the k experts of a token: k rounds of the largest key left,
// ties to the lowest expert. Lane r < k ends with the r-th expert (-1: none)
// and its weight.
template <int kPerLane>
__device__ __forceinline__ void choose(const FewArgs& a, int token, int lane, int* id, float* weight) {
  const float* row = a.logits + static_cast<int64_t>(token) * a.E;
  float l[kPerLane];
  uint32_t key[kPerLane];
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int e = i * 64 + lane;
    l[i] = e < a.E ? row[e] : -INFINITY;
    key[i] = logit_key(l[i]);
  }
  float top = 0.0f, mine = -INFINITY;
  *id = -1;
  for (int r = 0; r < a.k; ++r) {
    uint32_t best = 0;
    int at = 0;
    float value = 0.0f;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
        value = l[i];
      }
    const uint32_t m = wave_max_u32(best);
    if (m == 0) break;
    const bool has = best == m;
    const uint32_t index = has ? static_cast<uint32_t>(at * 64 + lane) : 0xffffffffu;
    const uint64_t holders = __ballot(has);
    const int first = __ffsll(static_cast<unsigned long long>(holders)) - 1;
    uint32_t e = __builtin_amdgcn_readlane(index, first);
    if (holders & (holders - 1)) e = ~wave_max_u32(~index);  // a tie: the lowest expert
    const float chosen = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(value), e % 64));
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
      if (e == static_cast<uint32_t>(i * 64 + lane)) key[i] = 0;
    if (r == 0) top = chosen;
    if (lane == r) {
      *id = static_cast<int>(e);
      mine = chosen;
    }
  }
  const float p = *id >= 0 ? __expf(mine - top) : 0.0f;
  float sum = p;
  if (!a.renormalize) {
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
      if (i * 64 + lane < a.E) sum += __expf(l[i] - top);
  }
  *weight = p / wave_sum_f32(sum);
}

// The routing of token t by one wave: its experts (-1: none) and their weights.
__device__ __forceinline__ void route_token(const FewArgs& a, int t, int lane, int* id, float* weight) {
  if (a.E <= 64)
    choose<1>(a, t, lane, id, weight);
  else if (a.E <= 256)
    choose<4>(a, t, lane, id, weight);
  else
    choose<kMaxExperts / 64>(a, t, lane, id, weight);
}

// For more than kSelfRouted tokens: a wave a token, once for the other kernels.
__global__ __launch_bounds__(64) void few_route_kernel(FewArgs a) {
  int id;
  float weight;
  route_token(a, blockIdx.x, threadIdx.x, &id, &weight);
  if (static_cast<int>(threadIdx.x) < a.k) {
    a.ws_ids[blockIdx.x * a.k + threadIdx.x] = id;
    a.ws_weight[blockIdx.x * a.k + threadIdx.x] = weight;
  }
}

// Which tokens an expert has, in LDS sized by the call.
struct Plan {
  int32_t* count;     // [E]: tokens of an expert, then the place of its next one
  int32_t* wave_sum;  // [16]
  float* weight;      // [slots] (first kernel)
  int16_t* id;        // [slots]: the expert of token t's choice j, at t k + j; -1: none
  int16_t* slot;      // [slots]: the slots by expert, and in their order among an expert's
  int32_t* between;   // [slots]: where a slot's h lies (second kernel)
  int16_t* active;    // [E]: the experts that have tokens
  int16_t* first;     // [E + 1]: of an active expert: its first place in `slot`
  int experts;        // that have tokens
};

inline __host__ __device__ constexpr size_t plan_bytes(int slots, int E) {
  return (4 * (E + 16 + 2 * slots) + 2 * (2 * slots + 2 * E + 1) + 15) / 16 * 16;
}

// What a workgroup may have without asking for more; the first kernel takes two tiles
// of tokens with more than kManyChoices an expert alone.
constexpr size_t kMostLds = 64 * 1024;
constexpr int kMostSlots = MRR_FEW_TOKENS_MAX * static_cast<int>(kFewMaxTopK);
static_assert(up_part_bytes(1) + plan_bytes(kMostSlots, kMaxExperts) <= kMostLds, "first kernel");
static_assert(up_part_bytes(2) + plan_bytes(kMostSlots, kMostSlots / kManyChoices) <= kMostLds,
              "first kernel, two tiles");
static_assert(down_sum_bytes(kDownTokens, 8, 1) + plan_bytes(kDownTokens * kFewMaxTopK, kMaxExperts) <= kMostLds &&
                  down_sum_bytes(kDownTokens, 4, 2) <= down_sum_bytes(kDownTokens, 8, 1),
              "second kernel");

__device__ __forceinline__ Plan carve(uint8_t* lds, int slots, int E) {
  Plan p;
  p.count = reinterpret_cast<int32_t*>(lds);
  p.wave_sum = p.count + E;
  p.weight = reinterpret_cast<float*>(p.wave_sum + 16);
  p.between = reinterpret_cast<int32_t*>(p.weight + slots);
  p.id = reinterpret_cast<int16_t*>(p.between + slots);
  p.slot = p.id + slots;
  p.active = p.slot + slots;
  p.first = p.active + E;
  p.experts = 0;
  return p;
}

// The plan of a few slots, of which a lane has one's expert (-1: none): by every
// wave alone, without a barrier, as all of them write the same (one token, 2 of 16
// experts, H 1024: the layer takes 11.1 us so and 12.6 by the counting below; 4 tokens,
// 8 of 16, 32 slots: 23.1 and 21.1; 64 slots: 30.4 and 24.4).
constexpr int kSmallPlan = 16;
static_assert(kSmallPlan >= kFewMaxTopK, "one token's slots");
__device__ __forceinline__ void make_small_plan(Plan& p, int expert, int slots) {
  const int lane = threadIdx.x % 64;
  int rank = 0, lead = lane, count = 0;  // among the expert's slots; its first slot; how many it has
  for (int i = slots - 1; i >= 0; --i) {
    const int other = __builtin_amdgcn_readlane(expert, i);
    const bool same = other >= 0 && other == expert;
    rank += same && i < lane;
    count += same;
    if (same) lead = i;
  }
  const bool leads = expert >= 0 && lead == lane;
  const uint64_t leaders = __ballot(leads);
  const int which = __popcll(leaders & ((uint64_t(1) << lane) - 1));
  const int first = static_cast<int>(wave_scan_u32(leads ? count : 0)) - (leads ? count : 0);
  p.experts = __popcll(leaders);
  const int place = __shfl(first, lead) + rank;
  if (leads) {
    p.active[which] = static_cast<int16_t>(expert);
    p.first[which] = static_cast<int16_t>(first);
    if (which == p.experts - 1) p.first[p.experts] = static_cast<int16_t>(first + count);
  }
  if (expert >= 0) p.slot[place] = static_cast<int16_t>(lane);
}

// From p.id (written, not yet waited for) the rest of the plan, by all kWaves
// waves of the workgroup.
template <int kWaves>
__device__ __forceinline__ void make_plan(Plan& p, int slots, int E) {
  constexpr int kThreads = kWaves * 64;
  const int tid = threadIdx.x;
  for (int e = tid; e < E; e += kThreads) p.count[e] = 0;
  __syncthreads();
  if (slots <= kSmallPlan) {
    make_small_plan(p, tid % 64 < slots ? p.id[tid % 64] : -1, slots);
    return;
  }
  for (int i = tid; i < slots; i += kThreads)
    if (p.id[i] >= 0) atomicAdd(&p.count[p.id[i]], 1);
  __syncthreads();
  const int per = (E + kThreads - 1) / kThreads;
  uint32_t used = 0, tokens = 0;
  for (int i = 0; i < per; ++i) {
    const int e = tid * per + i;
    const int c = e < E ? p.count[e] : 0;
    used += c > 0;
    tokens += c;
  }
  // both sums in one word: at most 1024 experts and 2048 slots
  const uint32_t in = wave_scan_u32(used << 16 | tokens);
  if (tid % 64 == 63) p.wave_sum[tid / 64] = static_cast<int>(in);
  __syncthreads();
  uint32_t before = in - (used << 16 | tokens), all = 0;
  for (int w = 0; w < kWaves; ++w) {
    if (w < tid / 64) before += p.wave_sum[w];
    all += p.wave_sum[w];
  }
  int next = before >> 16, place = before & 0xffff;
  for (int i = 0; i < per; ++i) {
    const int e = tid * per + i;
    const int c = e < E ? p.count[e] : 0;
    if (c > 0) {
      p.active[next] = static_cast<int16_t>(e);
      p.first[next++] = static_cast<int16_t>(place);
      p.count[e] = place;
      place += c;
    }
  }
  p.experts = __builtin_amdgcn_readfirstlane(all >> 16);
  if (tid == 0) p.first[p.experts] = static_cast<int16_t>(all & 0xffff);
  __syncthreads();
  // An expert's slots in their order, so that all workgroups agree on their places:
  // one wave, 64 slots at a time. The lanes of the same expert are found by its ten
  // bits.
  if (tid < 64) {
    for (int i0 = 0; i0 < slots; i0 += 64) {
      const int i = i0 + tid, e = i < slots ? p.id[i] : -1;
      uint64_t same = __ballot(e >= 0);
#pragma unroll
      for (int bit = 0; bit < kExpertBits; ++bit) {
        const bool set = e >> bit & 1;
        const uint64_t with = __ballot(set);
        same &= set ? with : ~with;
      }
      if (e >= 0) {
        const int rank = __popcll(same & ((uint64_t(1) << tid) - 1)), first = p.count[e];
        p.slot[first + rank] = static_cast<int16_t>(i);
        if (rank == 0) p.count[e] = first + __popcll(same);
      }
    }
  }
  __syncthreads();
}

// A chunk is 128 bytes of a weight row, a whole line of the caches: eight pieces
// of 16 bytes, 32 4-bit values each, which share a scale, or 8 values of 16 bits.
// The matrix instruction wants lane 16 g + r to have row r. Read like that, no
// two neighbouring lanes would read neighbouring bytes, and each lane's 16 bytes
// would take a cycle of the address unit of their own. So lane 4 r + g reads piece
// g or 4 + g of row r, and sort_lanes() moves it to lane 16 g + r afterwards
// (64 tokens, 4 of 32 4-bit experts, H 4096: the layer took 172 us before, 129 so).
template <bool kMx>
struct Weights {
  u32x4 v[2];
  uint32_t scale[2];  // of the row's eight pieces
};

// The tokens' side of a product: rows of x as they are, the same read by neighbouring
// lanes (kSorted, below), or h as the first kernel left it.
enum class From { kRows, kSorted, kBetween };

// The tokens' values that go with a chunk, by products of 8 values a lane.
template <bool kMx, int kTiles, From kFrom>
struct Tokens {
  u32x4 v[kTiles][kMx ? 8 : 2];
};

// Where the h of a token's choice of an expert lies in the workspace: the `count`
// choices of an expert, from the `first` place on, are [I / 8][hi, lo][count][8] in
// bf16, so that the lanes of its tokens read bytes that follow each other, in the
// order in which the instruction wants them, and an expert's lines hold nothing else.
// (With [I / 8][places][8] for all experts together two tokens have 32 bytes of a
// line: 16 tokens, 6 of 64 fp16 experts, took 155 us then, 148 so.)
struct Between {
  uint32_t first, count, rank;

  __device__ __forceinline__ int32_t packed() const { return static_cast<int32_t>(first | count << 12 | rank << 20); }
  static __device__ __forceinline__ Between of(int32_t v) {
    const uint32_t u = static_cast<uint32_t>(v);
    return {u & 0xfff, u >> 12 & 0xff, u >> 20};
  }
  __device__ __forceinline__ uint32_t pitch() const { return count * 32; }  // of 8 columns
  // The offset of columns 8 group .. 8 group + 7, of hi or lo.
  __device__ __forceinline__ uint32_t at(int I, int group, int lo) const {
    return first * I * 4 + group * pitch() + (lo * count + rank) * 16;
  }
};
static_assert(MRR_FEW_TOKENS_MAX < 256 && MRR_FEW_TOKENS_MAX * kFewMaxTopK < 4096, "Between::packed");

template <bool kMx>
__device__ __forceinline__ int row_bytes(int n) { return kMx ? n / 2 : n * 2; }

using Buffer = __amdgpu_buffer_rsrc_t;

// Memory as a buffer: what lies outside reads as zeros, without traffic. The
// address is the same for all lanes.
__device__ __forceinline__ Buffer buffer_at(const uint8_t* p, uint32_t bytes) {
  constexpr int kRaw = 0x00027000;  // 32-bit data, no swizzle, no stride
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t low = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t high = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(static_cast<uint64_t>(high) << 32 | low), 0, bytes,
                                           kRaw);
}
constexpr uint32_t kOutside = 0x80000000u;  // an offset outside of any buffer here, and so is a little more

__device__ __forceinline__ u32x4 load16(Buffer from, uint32_t lane_offset, uint32_t offset) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(from, lane_offset, offset, 0));
}

// Where a wave reads: chunk `c` on of kParts runs of 16 weight rows and of
// kTiles * 16 tokens' rows, `left` chunks of them, every `step`-th.
template <int kTiles, int kParts>
struct Place {
  Buffer rows[kParts];            // the 16 rows
  const uint8_t* scales[kParts];  // of the 16 rows; the same for all lanes
  uint32_t x[kTiles];             // what the lane reads of a chunk 0 in the tokens' buffer; kOutside: nothing
  uint32_t pitch;                 // h: bytes of 8 columns
  int c, left, step;
};

// What is the same for all chunks of a kernel.
struct Rows {
  Buffer x;
  int pieces, bytes, scale_bytes;  // of a weight row
  uint32_t at, scales_at;          // what the lane reads of a chunk 0 of 16 rows, and their scales
  int scales_shift;                // bits that it read too early (rows of fewer than 8 scales alone)
};

template <bool kMx>
__device__ __forceinline__ Rows make_rows(const uint8_t* x, uint32_t x_bytes, int n) {
  const int r = threadIdx.x % 64 / 4, g = threadIdx.x % 4;
  Rows a;
  a.x = buffer_at(x, x_bytes);
  a.bytes = row_bytes<kMx>(n);
  a.pieces = a.bytes / 16;
  a.scale_bytes = 2 * ((n + 63) / 64);
  a.at = r * a.bytes + g * 16;
  const int scales_at = min(r * a.scale_bytes, 16 * a.scale_bytes - 8);
  a.scales_at = scales_at;
  a.scales_shift = 8 * (r * a.scale_bytes - scales_at);
  return a;
}

// Eight pieces of 16 weight rows from piece `q` on, by lane 4 r + g. Where rows
// are shorter, other rows' bytes follow, or zeros behind the last one.
template <bool kMx>
__device__ __forceinline__ void load_weights(Weights<kMx>& w, Buffer rows, const uint8_t* scales, const Rows& all, int q) {
#pragma unroll
  for (int p = 0; p < 2; ++p) w.v[p] = load16(rows, all.at + p * 64, q * 16);
  if constexpr (kMx) __builtin_memcpy(w.scale, scales + q + all.scales_at, 8);
}

// The same of the tokens' rows. Of 16-bit values a piece of 4-bit weights takes
// 64 bytes: four lanes' worth.
template <bool kMx, int kTiles, From kFrom>
__device__ __forceinline__ void load_tokens(Tokens<kMx, kTiles, kFrom>& x, const uint32_t (&at)[kTiles], const Rows& all,
                                            int q, uint32_t pitch) {
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int i = 0; i < (kMx ? 8 : 2); ++i) {
      if constexpr (kFrom == From::kBetween)
        x.v[t][i] = load16(all.x, at[t], (kMx ? (q + i) * 4 : q + i * 4) * pitch);
      else
        x.v[t][i] = load16(all.x, at[t] + i * 64, q * (kMx ? 64 : 16));
    }
}

// Zeros for what is not in pieces lo .. hi - 1 of the eight; a scale of zero
// (2^-127) goes with zeros.
template <bool kMx>
__device__ __forceinline__ void cut_weights(Weights<kMx>& w, int lo, int hi, int scales_shift) {
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int piece = p * 4 + threadIdx.x % 4;
    if (piece < lo || piece >= hi) w.v[p] = u32x4{0, 0, 0, 0};
  }
  if constexpr (kMx) {
    uint64_t v = (static_cast<uint64_t>(w.scale[1]) << 32 | w.scale[0]) >> scales_shift;
    if (hi < 8) v &= (uint64_t(1) << 8 * hi) - 1;
    v = v >> 8 * lo << 8 * lo;
    w.scale[0] = static_cast<uint32_t>(v);
    w.scale[1] = static_cast<uint32_t>(v >> 32);
  }
}
// Widened to bf16, values under a scale of 2^126 or 2^127 may be infinities where their
// products with the tokens' values are none. So where a workgroup of the first kernel,
// or a wave of the second, has had a sum that is not finite, it makes its sums again,
// carefully: of the other blocks, and then of an eighth of these. (To make each sum
// again by itself kept enough scalar registers busy to cost 2 to 4% of every call; this
// costs 0.3 to 2%.)
__device__ __forceinline__ bool is_large(uint32_t scale) { return scale == 253 || scale == 254; }
__device__ __forceinline__ void take_blocks(Weights<true>& w, bool large) {
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const uint32_t mine = w.scale[p] >> threadIdx.x % 4 * 8 & 0xff;
    if (mine != 255 && is_large(mine) != large) w.v[p] = u32x4{0, 0, 0, 0};
    if (!large) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (is_large(w.scale[p] >> 8 * i & 0xff)) w.scale[p] -= 3u << 8 * i;
  }
}

// Whether a lane's sums are finite.
__device__ __forceinline__ bool is_finite(f32x4 v) {
  const f32x4 nothing = v * 0.0f;  // or a NaN
  return (nothing[0] + nothing[1]) + (nothing[2] + nothing[3]) == 0.0f;
}

template <bool kMx, int kTiles, From kFrom>
__device__ __forceinline__ void cut_tokens(Tokens<kMx, kTiles, kFrom>& x, int lo, int hi) {
  const int g = kFrom == From::kSorted ? threadIdx.x % 4 : threadIdx.x % 64 / 16;
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int i = 0; i < (kMx ? 8 : 2); ++i) {
      const int piece = kMx ? i : i * 4 + g;
      if (piece < lo || piece >= hi) x.v[t][i] = u32x4{0, 0, 0, 0};
    }
}

// From lane 4 r + g to lane 16 g + r.
__device__ __forceinline__ uint32_t sort_lanes(uint32_t v) {
  const int lane = threadIdx.x % 64;
  return static_cast<uint32_t>(
      __builtin_amdgcn_ds_bpermute((lane % 16 * 4 + lane / 16) * 4, static_cast<int>(v)));
}
__device__ __forceinline__ u32x4 sort_lanes(u32x4 v) {
  return u32x4{sort_lanes(v[0]), sort_lanes(v[1]), sort_lanes(v[2]), sort_lanes(v[3])};
}

// Dword i of lane group g and dword g of lane group i change places: a
// transposition of 4 x 4 by two rounds of swaps between groups.
__device__ __forceinline__ u32x4 transpose_groups(u32x4 v) {
  const auto a = __builtin_amdgcn_permlane16_swap(v[0], v[1], false, false);
  const auto b = __builtin_amdgcn_permlane16_swap(v[2], v[3], false, false);
  const auto e = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false);
  const auto f = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
  return u32x4{e[0], f[0], e[1], f[1]};
}

template <bool kBf16>
__device__ __forceinline__ f32x4 product(u32x4 w, u32x4 x, f32x4 c) {
  if constexpr (kBf16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), c, 0,
                                                   0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, w), __builtin_bit_cast(f16x8, x), c, 0, 0,
                                                  0);
}

// fp16 values as the sums of two bf16 values of the same sign: `a` has the eight bits
// on top of the next value towards zero, `b` the rest, which is never nothing. So what
// meets an infinity meets it twice with the same sign, and an infinity is a finite
// value and an infinity.
__device__ __forceinline__ void split_f16(u32x4 v, u32x4& a, u32x4& b) {
  using u16x2 = uint16_t __attribute__((ext_vector_type(2)));
  // their eight bits, or fewer, are the upper half of fp32
  auto bf16_pair = [](f16x2 h) {
    return __builtin_amdgcn_perm(__float_as_uint(static_cast<float>(h[1])), __float_as_uint(static_cast<float>(h[0])),
                                 0x07060302u);
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = v[i];  // a bit cast of an element itself takes the first one's bits
    const u16x2 size = __builtin_bit_cast(u16x2, w & 0x7fff7fffu), one = {1, 1};
    const uint32_t below = __builtin_bit_cast(uint32_t, __builtin_elementwise_sub_sat(size, one));
    const f16x2 top = __builtin_bit_cast(f16x2, (below & 0x7ff87ff8u) | (w & 0x80008000u));
    a[i] = bf16_pair(top);
    b[i] = bf16_pair(__builtin_bit_cast(f16x2, w) - top);
  }
}

// acc[n] += the products of a chunk with kTiles tiles of tokens, whose lanes are
// sorted already. Of 16-bit values lane group g of a tokens' register has those of
// dword g of a piece of 4-bit weights, so the weights' dwords are brought there.
template <bool kMx, bool kBf16, int kTiles, From kFrom>
__device__ __forceinline__ void multiply(const Weights<kMx>& w, const Tokens<kMx, kTiles, kFrom>& x,
                                         f32x4 (&acc)[kTiles]) {
  uint32_t scale[2];
  if constexpr (kMx) {
    scale[0] = sort_lanes(w.scale[0]);
    scale[1] = sort_lanes(w.scale[1]);
  }
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    u32x4 v = sort_lanes(w.v[p]);
    if constexpr (kMx) {
      v = transpose_groups(v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // the conversion reads the scale's exponent alone
        const float s = __uint_as_float((scale[p] >> 8 * i & 0xff) << 23);
        u32x4 wide;
        wide[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[i], s, 0));
        wide[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[i], s, 1));
        wide[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[i], s, 2));
        wide[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[i], s, 3));
#pragma unroll
        for (int n = 0; n < kTiles; ++n) acc[n] = product<kBf16>(wide, x.v[n][p * 4 + i], acc[n]);
      }
    } else if constexpr (kFrom == From::kBetween && !kBf16) {
      u32x4 a, b;
      split_f16(v, a, b);
#pragma unroll
      for (int n = 0; n < kTiles; ++n) acc[n] = product<true>(b, x.v[n][p], product<true>(a, x.v[n][p], acc[n]));
    } else {
#pragma unroll
      for (int n = 0; n < kTiles; ++n) acc[n] = product<kBf16>(v, x.v[n][p], acc[n]);
    }
  }
}

template <bool kBf16>
__device__ __forceinline__ void store_row4(uint8_t* p, f32x4 v) {
  if constexpr (kBf16) {
    __bf16 q[4] = {(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
    __builtin_memcpy(p, q, 8);
  } else {
    _Float16 q[4] = {(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
    __builtin_memcpy(p, q, 8);
  }
}

// Four columns of h, from `col` on: hi is the next bf16 towards zero, lo what is left,
// rounded. An infinity is a finite value and an infinity.
__device__ __forceinline__ void store_between(uint8_t* h, const Between& to, int I, int col, f32x4 v) {
  f32x4 hi;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t bits = __float_as_uint(v[i]), size = bits & 0x7fffffffu;
    hi[i] = __uint_as_float(((size - (size > 0)) & 0xffff0000u) | (bits & 0x80000000u));
  }
  store_row4<true>(h + to.at(I, col / 8, 0) + col % 8 * 2, hi);
  store_row4<true>(h + to.at(I, col / 8, 1) + col % 8 * 2, v - hi);
}

// A wave's stream of chunks. The next chunk is on its way while one is
// multiplied, also the first one of the next sum; there is no branch over loads, so
// that the wait for one chunk does not wait for the next. The chunk that a row ends
// in is read as its last eight pieces, and those that were counted before are cut
// (rows of fewer than eight pieces: those that follow). kSorted: the tokens are read
// by neighbouring lanes too; up to four cost less as they are (one token, 8 of 64
// 4-bit experts, H 7168: 49.0 us so, 50.3 sorted; four tokens, H 4096: 87 and 90). `next` moves a place to the next
// sum's first chunk, `again` brings the present one's back.
template <bool kMx, bool kBf16, int kTiles, From kFrom, int kParts, bool kCareful>
struct Stream {
  Weights<kMx> w[2][kParts];
  Tokens<kMx, kTiles, kFrom> x[2];
  int low[2];  // the chunk's first piece that counts

  template <typename Next>
  __device__ __forceinline__ void load(int b, Place<kTiles, kParts>& at, const Rows& all, Next&& next) {
    const int q = max(min(at.c * 8, all.pieces - 8), 0);
    low[b] = at.c * 8 - q;
#pragma unroll
    for (int i = 0; i < kParts; ++i) load_weights<kMx>(w[b][i], at.rows[i], at.scales[i], all, q);
    load_tokens(x[b], at.x, all, q, at.pitch);
    __builtin_amdgcn_sched_barrier(0);  // or they sink to their use
    at.c += at.step;
    if (--at.left == 0) next(at);
  }

  __device__ __forceinline__ void use(int b, f32x4 (&acc)[kParts][kTiles], const Rows& all, bool large) {
    if (low[b] > 0 || all.pieces < 8) {
#pragma unroll
      for (int i = 0; i < kParts; ++i) cut_weights<kMx>(w[b][i], low[b], all.pieces, all.scales_shift);
      cut_tokens(x[b], low[b], all.pieces);
    }
    if constexpr (kCareful) {
#pragma unroll
      for (int i = 0; i < kParts; ++i) take_blocks(w[b][i], large);
    }
    if constexpr (kFrom == From::kSorted) {
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int i = 0; i < (kMx ? 8 : 2); ++i) x[b].v[t][i] = sort_lanes(x[b].v[t][i]);
    }
#pragma unroll
    for (int i = 0; i < kParts; ++i) multiply<kMx, kBf16>(w[b][i], x[b], acc[i]);
    __builtin_amdgcn_sched_barrier(0);
  }

  // The sums of the next n > 0 chunks, whose first is in the first buffer.
  template <typename Next, typename Again>
  __device__ __forceinline__ void sum(f32x4 (&acc)[kParts][kTiles], int n, Place<kTiles, kParts>& at, const Rows& all,
                                      Next&& next, Again&& again) {
    each(acc, [](f32x4) { return f32x4{0, 0, 0, 0}; });
    add(acc, n, at, all, next, false);
    if constexpr (kCareful) {
      each(acc, [](f32x4 v) { return v * 0.125f; });
      again();
      add(acc, n, at, all, next, true);
      each(acc, [](f32x4 v) { return v * 8.0f; });
    }
  }

  template <typename F>
  static __device__ __forceinline__ void each(f32x4 (&acc)[kParts][kTiles], F&& f) {
#pragma unroll
    for (int i = 0; i < kParts; ++i)
#pragma unroll
      for (int t = 0; t < kTiles; ++t) acc[i][t] = f(acc[i][t]);
  }

  template <typename Next>
  __device__ __forceinline__ void add(f32x4 (&acc)[kParts][kTiles], int n, Place<kTiles, kParts>& at, const Rows& all,
                                      Next&& next, bool large) {
    for (;;) {
      load(1, at, all, next);
      use(0, acc, all, large);
      if (--n == 0) {
#pragma unroll
        for (int i = 0; i < kParts; ++i) w[0][i] = w[1][i];
        x[0] = x[1];
        low[0] = low[1];
        return;
      }
      load(0, at, all, next);
      use(1, acc, all, large);
      if (--n == 0) return;
    }
  }
};

// A barrier of LDS alone: loads from memory stay on their way.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// The first kernel. A unit is 16 gate rows and the same 16 up rows of an expert,
// for kTiles * 16 of its tokens; the waves share the rows' length, chunk by chunk.
template <bool kMx, bool kBf16, int kTiles, bool kSort>
__global__ __launch_bounds__(kUpWaves * 64, 2) void few_up_kernel(FewArgs a) {
  extern __shared__ __align__(16) uint8_t lds[];
  constexpr int kThreads = kUpWaves * 64;
  const int slots = a.T * a.k, tid = threadIdx.x, lane = tid % 64;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  Plan s = carve(lds + up_part_bytes(kTiles), slots, a.E);
  if (a.logits != nullptr && a.T == 1) {  // by every wave, so that none waits
    int id;
    float weight;
    route_token(a, 0, lane, &id, &weight);
    if (lane < a.k) {
      s.id[lane] = static_cast<int16_t>(id);
      s.weight[lane] = weight;
    }
    make_small_plan(s, lane < a.k ? id : -1, slots);
  } else if (a.logits != nullptr && a.T <= kSelfRouted) {
    for (int t = wave; t < a.T; t += kUpWaves) {
      int id;
      float weight;
      route_token(a, t, lane, &id, &weight);
      if (lane < a.k) {
        s.id[t * a.k + lane] = static_cast<int16_t>(id);
        s.weight[t * a.k + lane] = weight;
      }
    }
  } else if (a.logits != nullptr) {  // by few_route_kernel
    for (int i = tid; i < slots; i += kThreads) {
      s.id[i] = static_cast<int16_t>(a.ws_ids[i]);
      s.weight[i] = a.ws_weight[i];
    }
  } else {
    // An expert that a token names again counts at its first place, with the
    // sum of the weights.
    for (int i = tid; i < slots; i += kThreads) {
      const int t = i / a.k, j = i - t * a.k;
      const int id = a.ids[i];
      float weight = a.weight[i];
      bool keep = id >= 0 && id < a.E;
      for (int n = 0; n < a.k; ++n) {
        if (n == j || a.ids[t * a.k + n] != id) continue;
        if (n < j)
          keep = false;
        else
          weight += a.weight[t * a.k + n];
      }
      s.id[i] = static_cast<int16_t>(keep ? id : -1);
      s.weight[i] = weight;
    }
  }
  if (a.logits == nullptr || a.T > 1) make_plan<kUpWaves>(s, slots, a.E);
  if (blockIdx.x == 0 && (a.logits == nullptr || a.T <= kSelfRouted))  // for the second kernel
    for (int i = tid; i < slots; i += kThreads) a.ws_ids[i] = s.id[i];
  if (blockIdx.x == 0) {
    for (int i = tid; i < kFewMostRuns; i += kThreads) a.ws_arrived[i] = 0;
    for (int n = tid; n < s.experts; n += kThreads) {
      const int first = s.first[n], count = s.first[n + 1] - first;
      for (int i = 0; i < count; ++i)
        a.ws_between[s.slot[first + i]] = Between{uint32_t(first), uint32_t(count), uint32_t(i)}.packed();
    }
  }

  // This workgroup's units: row tile `tile` of active expert `n`, its tokens from
  // place `at` on.
  struct Unit {
    int unit, n, tile, at, end;
  };
  const int tiles = a.I / kRows, units = s.experts * tiles;
  auto begin = [&](Unit& u) {
    if (u.unit >= units) return;
    u.n = u.unit / tiles;
    u.tile = u.unit - u.n * tiles;
    u.at = __builtin_amdgcn_readfirstlane(s.first[u.n]);
    u.end = __builtin_amdgcn_readfirstlane(s.first[u.n + 1]);
  };
  auto advance = [&](Unit& u) {
    u.at += 16 * kTiles;
    if (u.at < u.end) return;
    u.unit += gridDim.x;
    begin(u);
  };
  if (static_cast<int>(blockIdx.x) >= units) return;

  const Rows all = make_rows<kMx>(a.x, a.T * a.H * 2, a.H);
  const int chunks = (all.pieces + 7) / 8;
  const int n = wave < chunks ? (chunks - wave + kUpWaves - 1) / kUpWaves : 0;  // of this wave
  using Where = Place<kTiles, 2>;
  auto set = [&](Where& p, const Unit& u) {
    const int expert = __builtin_amdgcn_readfirstlane(s.active[u.n]);
    const int64_t row = static_cast<int64_t>(expert) * 2 * a.I + u.tile * kRows;
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // the gate's rows and the up projection's
      p.rows[i] = buffer_at(a.gate_up + (row + i * a.I) * all.bytes, kRows * all.bytes);
      p.scales[i] = a.gate_up_scales + (row + i * a.I) * all.scale_bytes;
    }
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      const int place = u.at + t * 16 + (kSort ? lane / 4 : lane % 16), g = kSort ? lane % 4 : lane / 16;
      p.x[t] = place < u.end ? static_cast<uint32_t>(s.slot[place] / a.k) * a.H * 2 + g * 16 : kOutside;
    }
    p.c = wave;
    p.left = n;
    p.step = kUpWaves;
  };
  f32x4* part = reinterpret_cast<f32x4*>(lds);  // two of [waves][2][tiles][64]: partial sums of a unit
  constexpr int kPart = kUpWaves * 2 * kTiles * 64;
  int finisher = 0;
  // All units; whether the sums that the lane saw were finite.
  auto compute = [&](auto careful) {
    bool finite = true;
    Unit u{static_cast<int>(blockIdx.x), 0, 0, 0, 0};
    begin(u);
    Unit ahead = u;
    Where where;
    auto next = [&](Where& p) {  // behind the last unit: its first chunk again
      if (ahead.unit < units) advance(ahead);
      if (ahead.unit < units) {
        set(p, ahead);
      } else {
        p.c = wave;
        p.left = 1 << 30;
        p.step = 0;
      }
    };
    Stream<kMx, kBf16, kTiles, kSort ? From::kSorted : From::kRows, 2, decltype(careful)::value> stream;
    auto again = [&]() {
      ahead = u;
      set(where, u);
      stream.load(0, where, all, next);
    };
    set(where, u);
    if (n > 0) stream.load(0, where, all, next);
    for (; u.unit < units; advance(u)) {
      f32x4 acc[2][kTiles];
      if (n > 0) {
        stream.sum(acc, n, where, all, next, again);
      } else {
#pragma unroll
        for (int t = 0; t < kTiles; ++t) acc[0][t] = acc[1][t] = f32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int t = 0; t < kTiles; ++t) part[((wave * 2 + i) * kTiles + t) * 64 + lane] = acc[i][t];
      lds_barrier();
      // a wave finishes a tile of tokens, each its turn: a lane has four rows of one
      // token. Meanwhile the others go on, in the other half of `part`.
      for (int t = 0; t < kTiles; ++t, finisher = (finisher + 1) % kUpWaves) {
        if (wave != finisher) continue;
        f32x4 gs = part[t * 64 + lane], us = part[(kTiles + t) * 64 + lane];
#pragma unroll
        for (int w = 1; w < kUpWaves; ++w) {
          gs += part[(w * 2 * kTiles + t) * 64 + lane];
          us += part[((w * 2 + 1) * kTiles + t) * 64 + lane];
        }
        const int place = u.at + t * 16 + lane % 16, first = s.first[u.n];
        if (place < u.end) {
          if constexpr (kMx) finite &= is_finite(gs), finite &= is_finite(us);
          const float p = s.weight[s.slot[place]];
          f32x4 h;
#pragma unroll
          for (int i = 0; i < 4; ++i) h[i] = p * (gs[i] / (1.0f + __expf(-gs[i]))) * us[i];
          const int col = u.tile * kRows + lane / 16 * 4;
          const Between to{uint32_t(first), uint32_t(u.end - first), uint32_t(place - first)};
          store_between(a.ws_h, to, a.I, col, h);
        }
      }
      part = part == reinterpret_cast<f32x4*>(lds) ? part + kPart : reinterpret_cast<f32x4*>(lds);
    }
    return finite;
  };
  const bool finite = compute(std::false_type{});
  if constexpr (kMx) {
    s.wave_sum[wave] = !__all(finite);
    __syncthreads();
    int bad = 0;
    for (int w = 0; w < kUpWaves; ++w) bad |= s.wave_sum[w];
    if (__builtin_expect(__builtin_amdgcn_readfirstlane(bad), 0)) compute(std::true_type{});
  }
}

// What the lane eight away, of sixteen, has.
__device__ __forceinline__ f32x4 eighth_lane(f32x4 v) {
  constexpr int kRotate8 = 0x128;  // row_ror:8
  f32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
        0, static_cast<int>(__float_as_uint(v[i])), kRotate8, 0xf, 0xf, false)));
  return r;
}

// Values that workgroups on different XCDs share: past the XCD's own L2 both ways.
// (A fence of the whole L2 in their place made the kernel take 100 us more.)
__device__ __forceinline__ void store_shared(f32x4* p, f32x4 v) {
  uint64_t w[2];
  __builtin_memcpy(w, &v, 16);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    __hip_atomic_store(reinterpret_cast<uint64_t*>(p) + i, w[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ f32x4 load_shared(f32x4* p) {
  uint64_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = __hip_atomic_load(reinterpret_cast<uint64_t*>(p) + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  f32x4 v;
  __builtin_memcpy(&v, w, 16);
  return v;
}

// The second kernel: 16 kParts rows of y, a run, for up to 64 tokens. Its waves take the
// experts in turn, or parts of their rows when the experts are few, for 8 kTiles
// of the expert's tokens at a time, and add the results to sums of their own in
// LDS: each in its fixed order. Where there are fewer runs than the chip holds
// workgroups, a run has several (blockIdx.z), which share the experts; each leaves
// its sums in the workspace, and the last one to arrive adds them, in their order.
// So nothing depends on timing.
template <bool kMx, bool kBf16, int kTiles, int kParts, int kWaves>
__global__ __launch_bounds__(kWaves * 64, 2) void few_down_kernel(FewArgs a) {
  extern __shared__ __align__(16) uint8_t lds[];
  constexpr int kThreads = kWaves * 64;
  const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int r = lane % 16, group = lane / 16;
  const int t0 = blockIdx.y * kDownTokens, tokens = min(a.T - t0, kDownTokens), slots = tokens * a.k;
  constexpr int kGroups = 4 * kParts;  // of four rows
  f32x4* sums = reinterpret_cast<f32x4*>(lds);  // [waves][tokens][groups]
  f32x4* mine = sums + wave * tokens * kGroups;
  Plan s = carve(lds + down_sum_bytes(tokens, kWaves, kParts), slots, a.E);
  for (int i = lane; i < tokens * kGroups; i += 64) mine[i] = f32x4{0, 0, 0, 0};
  if (slots <= kSmallPlan) {
    if (lane < slots) s.between[lane] = a.ws_between[t0 * a.k + lane];
    make_small_plan(s, lane < slots ? a.ws_ids[t0 * a.k + lane] : -1, slots);
  } else {
    for (int i = tid; i < slots; i += kThreads) {
      s.id[i] = static_cast<int16_t>(a.ws_ids[t0 * a.k + i]);
      s.between[i] = a.ws_between[t0 * a.k + i];
    }
    make_plan<kWaves>(s, slots, a.E);
  }

  const Rows all = make_rows<kMx>(a.ws_h, a.T * a.k * a.I * 4, a.I);
  const int chunks = (all.pieces + 7) / 8;
  // parts of an expert's rows: enough for two a wave, of two chunks at least
  const int waves = kWaves * static_cast<int>(gridDim.z), first_unit = blockIdx.z * kWaves + wave;
  const int wanted = (2 * waves + s.experts - 1) / max(s.experts, 1);
  const int part_chunks = max(2, (chunks + wanted - 1) / wanted);
  const int parts = (chunks + part_chunks - 1) / part_chunks;
  // This wave's units: part `part` of active expert `n`, its tokens from place
  // `at` on.
  struct Unit {
    int unit, n, part, at, end;
  };
  const int units = s.experts * parts;
  auto begin = [&](Unit& u) {
    if (u.unit >= units) return;
    u.n = u.unit / parts;
    u.part = u.unit - u.n * parts;
    u.at = __builtin_amdgcn_readfirstlane(s.first[u.n]);
    u.end = __builtin_amdgcn_readfirstlane(s.first[u.n + 1]);
  };
  auto advance = [&](Unit& u) {
    u.at += kPlaces * kTiles;
    if (u.at < u.end) return;
    u.unit += waves;
    begin(u);
  };
  auto length = [&](const Unit& u) { return min(part_chunks, chunks - u.part * part_chunks); };
  using Where = Place<kTiles, kParts>;
  auto set = [&](Where& p, const Unit& u) {
    const int expert = __builtin_amdgcn_readfirstlane(s.active[u.n]);
    const int64_t row = static_cast<int64_t>(expert) * a.H + blockIdx.x * (kRows * kParts);
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      p.rows[i] = buffer_at(a.down + (row + i * kRows) * all.bytes, kRows * all.bytes);
      p.scales[i] = a.down_scales + (row + i * kRows) * all.scale_bytes;
    }
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      const int place = u.at + t * kPlaces + r % kPlaces;
      p.x[t] = place < u.end ? Between::of(s.between[s.slot[place]]).at(a.I, group, r / kPlaces) : kOutside;
    }
    p.pitch = __builtin_amdgcn_readfirstlane(Between::of(s.between[s.slot[u.at]]).pitch());
    p.c = u.part * part_chunks;
    p.left = length(u);
    p.step = 1;
  };
  // All units; whether the sums that the lane saw were finite.
  auto compute = [&](auto careful) {
    bool finite = true;
    Unit u{first_unit, 0, 0, 0, 0};
    begin(u);
    Unit ahead = u;
    Where where;
    auto next = [&](Where& p) {  // behind the last unit: its last chunk again
      if (ahead.unit < units) advance(ahead);
      if (ahead.unit < units) {
        set(p, ahead);
      } else {
        p.c -= p.step;
        p.left = 1 << 30;
        p.step = 0;
      }
    };
    Stream<kMx, kBf16, kTiles, From::kBetween, kParts, decltype(careful)::value> stream;
    auto again = [&]() {
      ahead = u;
      set(where, u);
      stream.load(0, where, all, next);
    };
    again();
    for (; u.unit < units; advance(u)) {
      f32x4 acc[kParts][kTiles];
      stream.sum(acc, length(u), where, all, next, again);
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        const int place = u.at + t * kPlaces + r;
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
          const f32x4 sum = acc[i][t] + eighth_lane(acc[i][t]);
          if (r < kPlaces && place < u.end) {
            if constexpr (kMx) finite &= is_finite(sum);
            mine[s.slot[place] / a.k * kGroups + i * 4 + group] += sum;
          }
        }
      }
    }
    return finite;
  };
  if (first_unit < units) {
    const bool finite = compute(std::false_type{});
    if constexpr (kMx) {
      if (__builtin_expect(!__all(finite), 0)) {
        for (int i = lane; i < tokens * kGroups; i += 64) mine[i] = f32x4{0, 0, 0, 0};
        compute(std::true_type{});
      }
    }
  }
  __syncthreads();
  auto store = [&](int i, f32x4 sum) {
    store_row4<kBf16>(
        a.y + (static_cast<int64_t>(t0 + i / kGroups) * a.H + (blockIdx.x * kGroups + i % kGroups) * 4) * 2, sum);
  };
  // [workgroups of a run][runs][tokens][groups]; the last run of tokens may have fewer
  const int run = blockIdx.y * gridDim.x + blockIdx.x, pitch = min(a.T, kDownTokens) * kGroups;
  f32x4* part = a.ws_part + static_cast<int64_t>(run) * pitch;
  const int64_t apart = static_cast<int64_t>(gridDim.y * gridDim.x) * pitch;
  for (int i = tid; i < tokens * kGroups; i += kThreads) {
    f32x4 sum = sums[i];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) sum += sums[w * tokens * kGroups + i];
    if (gridDim.z == 1)
      store(i, sum);
    else
      store_shared(part + blockIdx.z * apart + i, sum);
  }
  if (gridDim.z == 1) return;
  // the sums are where every XCD sees them before this workgroup is counted
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (tid == 0) *s.wave_sum = atomicAdd(a.ws_arrived + run, 1);
  __syncthreads();
  if (*s.wave_sum != static_cast<int>(gridDim.z) - 1) return;
  constexpr unsigned kAtOnce = 4;
  for (int i = tid; i < tokens * kGroups; i += kThreads) {
    f32x4 sum = load_shared(part + i);
    for (unsigned z = 1; z < gridDim.z; z += kAtOnce) {  // several on their way, added in their order
      f32x4 v[kAtOnce];
#pragma unroll
      for (unsigned n = 0; n < kAtOnce; ++n) v[n] = load_shared(part + min(z + n, gridDim.z - 1) * apart + i);
#pragma unroll
      for (unsigned n = 0; n < kAtOnce; ++n)
        if (z + n < gridDim.z) sum += v[n];
    }
    store(i, sum);
  }
}

template <bool kMx, bool kBf16, int kTiles, bool kSort>
mrr_status launch_up(const FewArgs& a, hipStream_t stream) {
  const int slots = a.T * a.k;
  // the workgroups that the chip holds at once (by their registers: two a CU with 4-bit
  // weights, three with two tiles, else four), each taking its units in turn
  const int64_t units = static_cast<int64_t>(slots < a.E ? slots : a.E) * (a.I / kRows);
  const int64_t most = 256 * (kMx ? 2 : kTiles == 2 ? 3 : 4), grid = units < most ? units : most;
  hipLaunchKernelGGL((few_up_kernel<kMx, kBf16, kTiles, kSort>), dim3(static_cast<unsigned>(grid)), dim3(kUpWaves * 64),
                     up_part_bytes(kTiles) + plan_bytes(slots, a.E), stream, a);
  return hipGetLastError() == hipSuccess ? MRR_SUCCESS : MRR_ERROR_HIP;
}

template <bool kMx, bool kBf16, int kTiles, int kParts>
mrr_status launch_down(const FewArgs& a, hipStream_t stream) {
  const int slots = a.T * a.k, tokens = a.T < kDownTokens ? a.T : kDownTokens;
  dim3 grid(a.H / (kRows * kParts), (a.T + kDownTokens - 1) / kDownTokens);
  const int runs = static_cast<int>(grid.x * grid.y);
  // Workgroups of a run: with few runs as many as the chip holds (two a CU, by their
  // registers), with four chunks a wave at least, more tokens counting as more chunks
  // (16 tokens, 6 of 64 fp16 experts, H 2048: 173 us with one, 147 with four; 16 tokens,
  // 8 of 64 4-bit experts, H 1024: 57 and 34). Few: of eight waves half the CUs, of four,
  // with two parts, two thirds of them (64 tokens, 4 of 8 4-bit experts, 160 runs: 100 us
  // with one, 93 with three; 4 of 32, 224 runs: 216 and 221 with two).
  const int used = slots < a.E ? slots : a.E, chunks = ((kMx ? a.I / 32 : a.I / 8) + 7) / 8;
  const int steps = used * chunks + slots * chunks / 8;
  if (runs <= (kParts == 1 ? 128 : 170))
    grid.z = std::max(1, std::min(static_cast<int>(kFewMostRuns) / runs, steps / 32));
  // Eight waves of one part, four of two: their sums take the same LDS.
  constexpr int kWaves = kParts == 1 ? 8 : 4;
  hipLaunchKernelGGL((few_down_kernel<kMx, kBf16, kTiles, kParts, kWaves>), grid, dim3(kWaves * 64),
                     down_sum_bytes(tokens, kWaves, kParts) + plan_bytes(tokens * a.k, a.E), stream, a);
  return hipGetLastError() == hipSuccess ? MRR_SUCCESS : MRR_ERROR_HIP;
}

template <bool kMx, bool kBf16>
mrr_status launch_few(const FewArgs& a, hipStream_t stream) {
  if (a.logits != nullptr && a.T > kSelfRouted) {
    hipLaunchKernelGGL(few_route_kernel, dim3(a.T), dim3(64), 0, stream, a);
    if (hipGetLastError() != hipSuccess) return MRR_ERROR_HIP;
  }
  // The second kernel's tiles are of eight tokens: one where an expert has fewer than
  // half of it, on average (48 tokens, 4 of 64 4-bit experts: 194 us, 207 with two;
  // 64 tokens, 4 of 32: 139 and 130). What takes its time beside the weights are the
  // loads of h, which two runs of rows share: always with 4-bit weights (one token, 8 of
  // 64 experts, H 7168: 49.1 us, 52.8 with one run; 64 tokens, 4 of 32: 134 and 146), with
  // 16-bit ones, which are four times as many bytes, where there are two tiles (64
  // tokens, 8 of 16 bf16 experts: 233 us and 264; with one tile, 32 tokens, 4 of 64: 245
  // us and 241 with one run).
  // From ten choices an expert on 16-bit weights have two tiles of sixteen tokens in the
  // first kernel and four of eight in the second (64 tokens, 4 of 15 bf16 experts, H
  // 4096: 165 us, 199 with one tile in the first, 181 with two in the second; 48 tokens,
  // 4 of 16: 158 and 162; 32 tokens: 155 and 154). 4-bit ones would not leave the
  // registers for them: 64 tokens, 8 of 16 experts, H 4096: 238 us so, 156 with one tile
  // in the first kernel, and weights read again for each 16 tokens.
  const int slots = a.T * a.k;
  const bool few = a.T <= kPlaces || slots <= 4 * a.E, many = slots > kManyChoices * a.E;
  const mrr_status st = a.T <= kSelfRouted ? launch_up<kMx, kBf16, 1, false>(a, stream)
                        : kMx || !many     ? launch_up<kMx, kBf16, 1, true>(a, stream)
                                           : launch_up<kMx, kBf16, kMx ? 1 : 2, true>(a, stream);
  if (st != MRR_SUCCESS) return st;
  if (few) return launch_down<kMx, kBf16, 1, kMx ? 2 : 1>(a, stream);
  return kMx || !many ? launch_down<kMx, kBf16, 2, 2>(a, stream) : launch_down<kMx, kBf16, kMx ? 2 : 4, 2>(a, stream);
}

}  // namespace
}  // namespace mrr

extern "C" mrr_status mrr_few_tokens(const mrr_few_tokens_args* args, void* workspace, size_t workspace_bytes,
                                     struct ihipStream_t* stream) {
  const mrr_status st = mrr::check_few_tokens(args, workspace, workspace_bytes);
  if (st != MRR_SUCCESS || args->T == 0) return st;
  const mrr::FewLayout l = mrr::few_layout(args->T, args->top_k, args->I);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  mrr::FewArgs a{};
  a.x = static_cast<const uint8_t*>(args->x);
  a.logits = args->router_logits;
  a.ids = args->expert_ids;
  a.weight = args->expert_weight;
  a.gate_up = static_cast<const uint8_t*>(args->gate_up);
  a.gate_up_scales = static_cast<const uint8_t*>(args->gate_up_scales);
  a.down = static_cast<const uint8_t*>(args->down);
  a.down_scales = static_cast<const uint8_t*>(args->down_scales);
  a.y = static_cast<uint8_t*>(args->y);
  a.ws_ids = reinterpret_cast<int32_t*>(ws + l.ids);
  a.ws_weight = reinterpret_cast<float*>(ws + l.weight);
  a.ws_between = reinterpret_cast<int32_t*>(ws + l.between);
  a.ws_arrived = reinterpret_cast<int32_t*>(ws + l.arrived);
  a.ws_part = reinterpret_cast<mrr::f32x4*>(ws + l.part);
  a.ws_h = ws + l.h;
  a.T = static_cast<int32_t>(args->T);
  a.H = static_cast<int32_t>(args->H);
  a.E = static_cast<int32_t>(args->E);
  a.I = static_cast<int32_t>(args->I);
  a.k = static_cast<int32_t>(args->top_k);
  a.renormalize = args->renormalize == 1;
  if (args->weights_dtype == MRR_F4_E2M1) return mrr::launch_few<true, true>(a, stream);
  return args->dtype == MRR_BF16 ? mrr::launch_few<false, true>(a, stream) : mrr::launch_few<false, false>(a, stream);
}
