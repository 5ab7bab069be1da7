// mrr_few_tokens.hip -- a whole mixture-of-experts layer for a few tokens in
// two kernels:
//     h[t, j] = p[t, j] silu(Wg[e] x[t]) * (Wu[e] x[t])   for e = ids[t, j],
//     y[t]    = sum over j of Wd[e] h[t, j].
// Bound by reading the chosen experts' weights, once each. The first kernel
// also finds the routing (softmax and top-k of the router's logits, or given
// ids): every workgroup does it for itself, as it needs it to know its work.
// The second adds an output row's experts in one workgroup, in a fixed order,
// so no sum crosses workgroups and results do not depend on timing.
//
// Both feed the 16x16x32 matrix instruction with 16 weight rows and up to 16
// tokens. A lane reads 16 bytes of a weight row at a time: eight 16-bit values
// (one product), or a block of 32 4-bit values (four products), widened to
// bf16 with their scale, which is exact.
#include "mrr_device.h"
#include "mrr_experts.h"

namespace mrr {
namespace {

using u32x4 = uint32_t __attribute__((ext_vector_type(4)));
using f32x4 = float __attribute__((ext_vector_type(4)));
using bf16x2 = __bf16 __attribute__((ext_vector_type(2)));
using bf16x8 = __bf16 __attribute__((ext_vector_type(8)));
using f16x8 = _Float16 __attribute__((ext_vector_type(8)));

constexpr int kMaxExperts = static_cast<int>(kFewMaxExperts);
constexpr int kUpWaves = 4;       // first kernel: they share a unit's rows, each a part of their length
constexpr int kDownWaves = 8;     // second kernel: each takes experts, or parts of them
constexpr int kRows = 16;         // weight rows of a fragment
constexpr int kDownTokens = 64;   // tokens of a workgroup of the second kernel

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
  uint8_t* ws_h;
  int32_t T, H, E, I, k;
  int32_t renormalize;
};

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

struct Routing {
  float* weight;  // [T][k]
  int16_t* id;    // [T][k], -1: none
};

// The routing of all tokens into LDS, by all waves of the workgroup.
template <int kWaves>
__device__ void find_routing(const FewArgs& a, const Routing& r) {
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  if (a.logits != nullptr) {
    for (int t = wave; t < a.T; t += kWaves) {
      int id;
      float weight;
      if (a.E <= 64)
        choose<1>(a, t, lane, &id, &weight);
      else if (a.E <= 256)
        choose<4>(a, t, lane, &id, &weight);
      else
        choose<kMaxExperts / 64>(a, t, lane, &id, &weight);
      if (lane < a.k) {
        r.id[t * a.k + lane] = static_cast<int16_t>(id);
        r.weight[t * a.k + lane] = weight;
      }
    }
  } else {
    // An expert that a token names again counts at its first place, with the
    // sum of the weights.
    for (int s = threadIdx.x; s < a.T * a.k; s += kWaves * 64) {
      const int t = s / a.k, j = s - t * a.k;
      const int id = a.ids[s];
      float weight = a.weight[s];
      bool keep = id >= 0 && id < a.E;
      for (int i = 0; i < a.k; ++i) {
        if (i == j || a.ids[t * a.k + i] != id) continue;
        if (i < j)
          keep = false;
        else
          weight += a.weight[t * a.k + i];
      }
      r.id[s] = static_cast<int16_t>(keep ? id : -1);
      r.weight[s] = weight;
    }
  }
}

template <bool kMx>
__device__ __forceinline__ int row_bytes(int n) { return kMx ? n / 2 : n * 2; }

// What a lane reads of a weight row for one chunk (64 bytes of the row over
// the four lane groups).
template <bool kMx>
struct WeightPiece {
  u32x4 v;
  uint32_t scale;
};

template <bool kMx>
__device__ __forceinline__ WeightPiece<kMx> load_weight(const uint8_t* row, const uint8_t* scales, int piece,
                                                        bool valid) {
  WeightPiece<kMx> w;
  w.v = u32x4{0, 0, 0, 0};
  w.scale = 127;
  if (valid) {
    w.v = *reinterpret_cast<const u32x4*>(row + static_cast<int64_t>(piece) * 16);
    if constexpr (kMx) w.scale = scales[piece];
  }
  return w;
}

// The token's values that go with a weight piece: 32 (4-bit weights) or 8.
template <bool kMx>
struct TokenPiece {
  u32x4 v[kMx ? 4 : 1];
};

template <bool kMx>
__device__ __forceinline__ TokenPiece<kMx> load_token(const uint8_t* row, int piece, bool valid) {
  constexpr int n = kMx ? 4 : 1;
  TokenPiece<kMx> t;
#pragma unroll
  for (int i = 0; i < n; ++i) t.v[i] = u32x4{0, 0, 0, 0};
  if (valid) {
    const u32x4* p = reinterpret_cast<const u32x4*>(row) + static_cast<int64_t>(piece) * n;
#pragma unroll
    for (int i = 0; i < n; ++i) t.v[i] = p[i];
  }
  return t;
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

// acc[n] += the products of a weight piece with kTiles tiles of tokens.
template <bool kMx, bool kBf16, int kTiles>
__device__ __forceinline__ void multiply(const WeightPiece<kMx>& w, const TokenPiece<kMx> (&x)[kTiles],
                                         f32x4 (&acc)[kTiles]) {
  if constexpr (kMx) {
    const float s = __uint_as_float(w.scale << 23);  // the conversion reads the exponent alone
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u32x4 wide;
      wide[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w.v[i], s, 0));
      wide[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w.v[i], s, 1));
      wide[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w.v[i], s, 2));
      wide[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w.v[i], s, 3));
#pragma unroll
      for (int n = 0; n < kTiles; ++n) acc[n] = product<kBf16>(wide, x[n].v[i], acc[n]);
    }
  } else {
#pragma unroll
    for (int n = 0; n < kTiles; ++n) acc[n] = product<kBf16>(w.v, x[n].v[0], acc[n]);
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

// The first kernel's LDS, sized by the call (a few KiB for one token, so that
// several workgroups share a CU).
struct UpShared {
  f32x4* part;        // [waves][2][tiles][64]: partial sums of a unit
  int32_t* count;     // [E]: tokens of an expert, then the place of its next one
  int32_t* wave_sum;  // [waves]
  Routing routing;
  int16_t* slot;      // [T k]: token * 16 + choice, by expert
  int16_t* active;    // [E]: the experts that have tokens
  int16_t* first;     // [E + 1]: of an active expert: its first place in `slot`
};

inline __host__ __device__ size_t up_shared_bytes(int slots, int E, int tiles) {
  return sizeof(f32x4) * kUpWaves * 2 * tiles * 64 + 4 * (E + kUpWaves + slots) + 2 * (2 * slots + 2 * E + 1);
}

__device__ __forceinline__ UpShared carve(uint8_t* lds, int slots, int E, int tiles) {
  UpShared s;
  s.part = reinterpret_cast<f32x4*>(lds);
  s.count = reinterpret_cast<int32_t*>(s.part + kUpWaves * 2 * tiles * 64);
  s.wave_sum = s.count + E;
  s.routing.weight = reinterpret_cast<float*>(s.wave_sum + kUpWaves);
  s.routing.id = reinterpret_cast<int16_t*>(s.routing.weight + slots);
  s.slot = s.routing.id + slots;
  s.active = s.slot + slots;
  s.first = s.active + E;
  return s;
}

// One unit of the first kernel: 16 gate rows and the same 16 up rows of an
// expert, for kTiles * 16 of its tokens from place `at` on. The waves share
// the rows' length, chunk by chunk.
template <bool kMx, bool kBf16, int kTiles>
__device__ __forceinline__ void up_unit(const FewArgs& a, const UpShared& s, int expert, int tile, int at, int end) {
  constexpr int kUnroll = kMx ? 2 : 4;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int r = lane % 16, group = lane / 16;
  const int bytes = row_bytes<kMx>(a.H);
  const int pieces = bytes / 16;
  const int chunks = (pieces + 3) / 4;
  const int64_t row = static_cast<int64_t>(expert) * 2 * a.I + tile * kRows + r;
  const uint8_t* g_row = a.gate_up + row * bytes;
  const uint8_t* u_row = g_row + static_cast<int64_t>(a.I) * bytes;
  const int scale_bytes = 2 * ((a.H + 63) / 64);
  const uint8_t* g_scale = a.gate_up_scales + (kMx ? row * scale_bytes : 0);
  const uint8_t* u_scale = g_scale + (kMx ? static_cast<int64_t>(a.I) * scale_bytes : 0);
  const uint8_t* x_row[kTiles];
  bool has[kTiles];
#pragma unroll
  for (int n = 0; n < kTiles; ++n) {
    const int place = at + n * 16 + r;
    has[n] = place < end;
    x_row[n] = a.x + (has[n] ? static_cast<int64_t>(s.slot[place] / 16) * a.H * 2 : 0);
  }
  f32x4 g[kTiles], u[kTiles];
#pragma unroll
  for (int n = 0; n < kTiles; ++n) g[n] = u[n] = f32x4{0, 0, 0, 0};
  for (int c0 = wave; c0 < chunks; c0 += kUpWaves * kUnroll) {
    WeightPiece<kMx> wg[kUnroll], wu[kUnroll];
    TokenPiece<kMx> x[kUnroll][kTiles];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int piece = (c0 + i * kUpWaves) * 4 + group;
      wg[i] = load_weight<kMx>(g_row, g_scale, piece, piece < pieces);
      wu[i] = load_weight<kMx>(u_row, u_scale, piece, piece < pieces);
#pragma unroll
      for (int n = 0; n < kTiles; ++n) x[i][n] = load_token<kMx>(x_row[n], piece, has[n] && piece < pieces);
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      multiply<kMx, kBf16, kTiles>(wg[i], x[i], g);
      multiply<kMx, kBf16, kTiles>(wu[i], x[i], u);
    }
  }
#pragma unroll
  for (int n = 0; n < kTiles; ++n) {
    s.part[((wave * 2 + 0) * kTiles + n) * 64 + lane] = g[n];
    s.part[((wave * 2 + 1) * kTiles + n) * 64 + lane] = u[n];
  }
  __syncthreads();
  // a wave finishes a tile of tokens: a lane has four rows of one token
  for (int n = wave; n < kTiles; n += kUpWaves) {
    f32x4 gs = s.part[n * 64 + lane], us = s.part[(kTiles + n) * 64 + lane];
#pragma unroll
    for (int w = 1; w < kUpWaves; ++w) {
      gs += s.part[(w * 2 * kTiles + n) * 64 + lane];
      us += s.part[((w * 2 + 1) * kTiles + n) * 64 + lane];
    }
    const int place = at + n * 16 + r;
    if (place < end) {
      const int slot = s.slot[place] / 16 * a.k + s.slot[place] % 16;
      const float p = s.routing.weight[slot];
      f32x4 h;
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = p * (gs[i] / (1.0f + __expf(-gs[i]))) * us[i];
      store_row4<kBf16>(a.ws_h + (static_cast<int64_t>(slot) * a.I + tile * kRows + group * 4) * 2, h);
    }
  }
  __syncthreads();
}

// kMaxTiles: tiles of 16 tokens that all tokens fill.
template <bool kMx, bool kBf16, int kMaxTiles>
__global__ __launch_bounds__(kUpWaves * 64) void few_up_kernel(FewArgs a) {
  extern __shared__ __align__(16) uint8_t lds[];
  const UpShared s = carve(lds, a.T * a.k, a.E, kMaxTiles);
  const int tid = threadIdx.x;
  constexpr int kThreads = kUpWaves * 64;
  for (int e = tid; e < a.E; e += kThreads) s.count[e] = 0;
  find_routing<kUpWaves>(a, s.routing);
  __syncthreads();
  const int slots = a.T * a.k;
  if (blockIdx.x == 0)
    for (int i = tid; i < slots; i += kThreads) a.ws_ids[i] = s.routing.id[i];
  for (int i = tid; i < slots; i += kThreads)
    if (s.routing.id[i] >= 0) atomicAdd(&s.count[s.routing.id[i]], 1);
  __syncthreads();
  // the experts that have tokens, and where their tokens start
  constexpr int kPer = kMaxExperts / kThreads;
  uint32_t used = 0, tokens = 0;
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    const int c = e < a.E ? s.count[e] : 0;
    used += c > 0;
    tokens += c;
  }
  // both sums in one word: at most 1024 experts and 2048 slots
  const uint32_t in = wave_scan_u32(used << 16 | tokens);
  if (tid % 64 == 63) s.wave_sum[tid / 64] = static_cast<int>(in);
  __syncthreads();
  uint32_t before = in - (used << 16 | tokens), all = 0;
  for (int w = 0; w < kUpWaves; ++w) {
    if (w < tid / 64) before += s.wave_sum[w];
    all += s.wave_sum[w];
  }
  int next = before >> 16, place = before & 0xffff;
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    const int c = e < a.E ? s.count[e] : 0;
    if (c > 0) {
      s.active[next] = static_cast<int16_t>(e);
      s.first[next++] = static_cast<int16_t>(place);
      s.count[e] = place;
      place += c;
    }
  }
  const int active = all >> 16;
  if (tid == 0) s.first[active] = static_cast<int16_t>(all & 0xffff);
  __syncthreads();
  // the order within an expert does not matter: a token's sums are its own
  for (int i = tid; i < slots; i += kThreads) {
    const int e = s.routing.id[i];
    if (e >= 0) s.slot[atomicAdd(&s.count[e], 1)] = static_cast<int16_t>(i / a.k * 16 + i % a.k);
  }
  __syncthreads();

  const int tiles = a.I / kRows;
  const int units = active * tiles;
  for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int n = unit / tiles, tile = unit - n * tiles;
    const int expert = s.active[n], end = s.first[n + 1];
    for (int at = s.first[n]; at < end;) {
      if (kMaxTiles == 1 || end - at <= 16) {
        up_unit<kMx, kBf16, 1>(a, s, expert, tile, at, end);
        at += 16;
      } else if (kMaxTiles == 2 || end - at <= 32) {
        up_unit<kMx, kBf16, kMaxTiles < 2 ? 1 : 2>(a, s, expert, tile, at, end);
        at += 32;
      } else {
        up_unit<kMx, kBf16, kMaxTiles>(a, s, expert, tile, at, end);
        at += 64;
      }
    }
  }
}

// The second kernel: a workgroup computes 16 rows of y for up to 64 tokens.
// Its waves take the tokens' experts in turn, or parts of their rows when the
// experts are few; a wave's sums cover all tokens, the ones that do not use an
// expert entering as zeros.
template <bool kMx, bool kBf16, int kTiles>
__global__ __launch_bounds__(kDownWaves * 64) void few_down_kernel(FewArgs a) {
  constexpr int kThreads = kDownWaves * 64;
  constexpr int kUnroll = kMx ? 2 : 4;
  __shared__ int16_t s_id[kDownTokens * static_cast<int>(kFewMaxTopK)];
  __shared__ int32_t s_used[kMaxExperts];
  __shared__ int16_t s_active[kMaxExperts];
  __shared__ int32_t s_sum[kDownWaves];
  __shared__ f32x4 s_part[kDownWaves][kTiles][64];
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int r = lane % 16, group = lane / 16;
  const int t0 = blockIdx.y * kDownTokens, tokens = min(a.T - t0, kDownTokens);
  for (int e = tid; e < a.E; e += kThreads) s_used[e] = 0;
  __syncthreads();
  for (int i = tid; i < tokens * a.k; i += kThreads) {
    const int id = a.ws_ids[t0 * a.k + i];
    s_id[i] = static_cast<int16_t>(id);
    if (id >= 0) s_used[id] = 1;
  }
  __syncthreads();
  constexpr int kPer = kMaxExperts / kThreads;
  uint32_t used = 0;
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    used += e < a.E ? s_used[e] : 0;
  }
  const uint32_t in = wave_scan_u32(used);
  if (lane == 63) s_sum[wave] = static_cast<int>(in);
  __syncthreads();
  int next = static_cast<int>(in - used), active = 0;
  for (int w = 0; w < kDownWaves; ++w) {
    if (w < wave) next += s_sum[w];
    active += s_sum[w];
  }
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    if (e < a.E && s_used[e]) s_active[next++] = static_cast<int16_t>(e);
  }
  __syncthreads();

  const int bytes = row_bytes<kMx>(a.I);
  const int pieces = bytes / 16, chunks = (pieces + 3) / 4;
  const int scale_bytes = 2 * ((a.I + 63) / 64);
  const int row = blockIdx.x * kRows + r;
  // parts of an expert's rows: enough for two a wave, of four chunks at least
  const int parts = max(1, min((chunks + 3) / 4, (2 * kDownWaves + active - 1) / max(active, 1)));
  const int part_chunks = (chunks + parts - 1) / parts;
  f32x4 acc[kTiles];
#pragma unroll
  for (int n = 0; n < kTiles; ++n) acc[n] = f32x4{0, 0, 0, 0};
  for (int unit = wave; unit < active * parts; unit += kDownWaves) {
    const int which = unit / parts, part = unit - which * parts;
    const int expert = s_active[which];
    const uint8_t* w_row = a.down + (static_cast<int64_t>(expert) * a.H + row) * bytes;
    const uint8_t* w_scale = a.down_scales + (kMx ? (static_cast<int64_t>(expert) * a.H + row) * scale_bytes : 0);
    const uint8_t* h_row[kTiles];
    bool has[kTiles];
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      const int t = n * 16 + r;
      int choice = -1;
      if (t < tokens)
        for (int j = 0; j < a.k; ++j)
          if (s_id[t * a.k + j] == expert) choice = j;
      has[n] = choice >= 0;
      h_row[n] = a.ws_h + (has[n] ? (static_cast<int64_t>(t0 + t) * a.k + choice) * a.I * 2 : 0);
    }
    const int end = min(chunks, (part + 1) * part_chunks);
    for (int c0 = part * part_chunks; c0 < end; c0 += kUnroll) {
      WeightPiece<kMx> w[kUnroll];
      TokenPiece<kMx> h[kUnroll][kTiles];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int piece = (c0 + i) * 4 + group;
        const bool valid = c0 + i < end && piece < pieces;
        w[i] = load_weight<kMx>(w_row, w_scale, piece, valid);
#pragma unroll
        for (int n = 0; n < kTiles; ++n) h[i][n] = load_token<kMx>(h_row[n], piece, has[n] && valid);
      }
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) multiply<kMx, kBf16, kTiles>(w[i], h[i], acc);
    }
  }
#pragma unroll
  for (int n = 0; n < kTiles; ++n) s_part[wave][n][lane] = acc[n];
  __syncthreads();
  for (int n = wave; n < kTiles; n += kDownWaves) {
    const int t = n * 16 + r;
    f32x4 sum = s_part[0][n][lane];
#pragma unroll
    for (int w = 1; w < kDownWaves; ++w) sum += s_part[w][n][lane];
    if (t < tokens)
      store_row4<kBf16>(a.y + (static_cast<int64_t>(t0 + t) * a.H + blockIdx.x * kRows + group * 4) * 2, sum);
  }
}

template <bool kMx, bool kBf16, int kTiles>
mrr_status launch_few_tiles(const FewArgs& a, hipStream_t stream) {
  const int64_t slots = static_cast<int64_t>(a.T) * a.k;
  const int64_t units = (slots < a.E ? slots : a.E) * (a.I / kRows);
  const int64_t most = 256 * 4;
  hipLaunchKernelGGL((few_up_kernel<kMx, kBf16, kTiles>), dim3(static_cast<unsigned>(units < most ? units : most)),
                     dim3(kUpWaves * 64), up_shared_bytes(static_cast<int>(slots), a.E, kTiles), stream, a);
  if (hipGetLastError() != hipSuccess) return MRR_ERROR_HIP;
  hipLaunchKernelGGL((few_down_kernel<kMx, kBf16, kTiles>), dim3(a.H / kRows, (a.T + kDownTokens - 1) / kDownTokens),
                     dim3(kDownWaves * 64), 0, stream, a);
  return hipGetLastError() == hipSuccess ? MRR_SUCCESS : MRR_ERROR_HIP;
}

template <bool kMx, bool kBf16>
mrr_status launch_few(const FewArgs& a, hipStream_t stream) {
  return a.T <= 16   ? launch_few_tiles<kMx, kBf16, 1>(a, stream)
         : a.T <= 32 ? launch_few_tiles<kMx, kBf16, 2>(a, stream)
                     : launch_few_tiles<kMx, kBf16, 4>(a, stream);
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
