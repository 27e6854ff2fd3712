// Products of one or a few tokens with experts' NVFP4 weights, the activations left in bf16:
//
//   y[t, j, n] = gB[e] sum_b sB[e, n, b] sum_{i < 16} x[r, 16 b + i] b[e, n, 16 b + i],  e = ids[t, j]
//
// and with them silu(gate) up, or the sum over a token's slots j of w[t, j] y[t, j].
//
// The weights are read once and their decoding has to keep up with HBM, so what counts is how few
// instructions a weight takes.  A lane loads 16 bytes, 32 codes of one weight row, which are two scale
// blocks, so sums over lanes may only be taken after the scales.  The 4x4x4 MFMA (16 independent
// blocks) fits that: a lane's four weights of one row meet four tokens' elements, summed within the lane,
// and 4 MFMAs sum a scale block.  Per 16 weights and lane that is 8 conversions (two codes to bf16
// each, exact), 4 MFMAs on the matrix pipe and one fma per token with the block's scale: one vector
// instruction per 1.3 to 1.8 weights, for up to 4 tokens.  Products are exact and sums binary32.
//
// A wave takes 16 weight rows (lane 16 g + r: row r, elements [64 g, 64 g + 64) of a 256-wide step, as
// the packed layout has them) of two tiles, which share the tokens' elements: gate and up rows, or
// neighbouring tiles.  The waves of a workgroup share a pair of tiles and deal the steps, or the steps
// of all experts, among themselves; their partial sums are added in order through LDS.
//
// Tokens that chose the same expert share the read of its weights: the pairs (t, j) of up to 16 tokens
// are collected into groups of one expert, at most one slot of each token (a token's second slot with
// the same expert goes to a second group).
#include "gemv_nvfp4.hpp"

#pragma clang fp contract(off)

namespace moe {
namespace gemv {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short short4v __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kStep = 256;         // elements of K in a step
constexpr int kPackBlock = 2304;   // bytes of one (16-row tile, step) block of packed weights
constexpr int kMaxWaves = 8;
constexpr int kMaxTokens = 16, kMaxSlots = 32;
constexpr int kMaxPairs = kMaxTokens * kMaxSlots;
constexpr int NT = 2;              // tiles of 16 weight rows that a wave takes together

// One step's weights of a tile in this lane: 64 codes of its row and their four scales.
struct Weights {
  u32x4 code[2];
  uint32_t scale;
};

struct Tile {
  const uint8_t *code;      // of this lane's row (packed: of the tile)
  const uint8_t *scale;
};

// `left`: elements of K from the lane's first one of the step (may be negative).
template <bool PACKED>
__device__ __forceinline__ Weights load_weights(const Tile &t, int step, int left, bool scales4) {
  Weights w;
  const int lane = threadIdx.x & 63;
  if (PACKED) {
    const uint8_t *at = t.code + static_cast<int64_t>(step) * kPackBlock;
    w.code[0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(at + lane * 16));
    w.code[1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(at + 1024 + lane * 16));
    w.scale = __builtin_nontemporal_load(reinterpret_cast<const uint32_t *>(at + 2048 + lane * 4));
  } else {
    const uint8_t *at = t.code + step * (kStep / 2) + lane / 16 * 32;
    const uint8_t *sf = t.scale + step * (kStep / 16) + lane / 16 * 4;
    w.code[0] = w.code[1] = u32x4{0, 0, 0, 0};
    w.scale = 0;
    if (left > 0) w.code[0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(at));
    if (left > 32) w.code[1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(at + 16));
    if (scales4) {
      if (left > 0) w.scale = __builtin_nontemporal_load(reinterpret_cast<const uint32_t *>(sf));
    } else {
      if (left > 0) w.scale = *reinterpret_cast<const uint16_t *>(sf);
      if (left > 32) w.scale |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(sf + 2)) << 16;
    }
  }
  return w;
}

// One step's elements of this lane's token: 64 of its lane group.
struct Elements {
  u32x4 v[8];
};
__device__ __forceinline__ Elements load_elements(const uint16_t *row, int step, int left) {
  Elements e;
  const u32x4 *at = reinterpret_cast<const u32x4 *>(row + step * kStep + (threadIdx.x & 63) / 16 * 64);
#pragma unroll
  for (int i = 0; i < 8; i++) {
    e.v[i] = u32x4{0, 0, 0, 0};
    if (left > 8 * i) e.v[i] = at[i];
  }
  return e;
}

__device__ __forceinline__ short4v pair_up(uint32_t a, uint32_t b) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(short4v, u32x2{a, b});
}

// acc[c] += the step's products with token c (of 4), scaled.
template <int TB>
__device__ __forceinline__ void multiply(const Weights &w, const Elements (&x)[TB], float4v (&acc)[TB]) {
#pragma unroll
  for (int b = 0; b < 4; b++) {       // the lane's scale blocks
    const float s = b == 0   ? __builtin_amdgcn_cvt_f32_fp8(w.scale, 0)
                    : b == 1 ? __builtin_amdgcn_cvt_f32_fp8(w.scale, 1)
                    : b == 2 ? __builtin_amdgcn_cvt_f32_fp8(w.scale, 2)
                             : __builtin_amdgcn_cvt_f32_fp8(w.scale, 3);
    short4v q[4];
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const uint32_t c = w.code[b / 2][b % 2 * 2 + h];
      const uint32_t p0 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 0));
      const uint32_t p1 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 1));
      const uint32_t p2 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 2));
      const uint32_t p3 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 3));
      q[2 * h] = pair_up(p0, p1);
      q[2 * h + 1] = pair_up(p2, p3);
    }
#pragma unroll
    for (int tb = 0; tb < TB; tb++) {
      float4v v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const u32x4 &e = x[tb].v[2 * b + i / 2];
        v = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(pair_up(e[i % 2 * 2], e[i % 2 * 2 + 1]), q[i], v, 0, 0, 0);
      }
#pragma unroll
      for (int c = 0; c < 4; c++) acc[tb][c] = fmaf(v[c], s, acc[tb][c]);
    }
  }
}

// acc += steps [from, to) by `by` of expert e's two tiles.
template <int TB, bool PACKED>
__device__ __forceinline__ void accumulate(const Params &P, const Tile (&tile)[NT], const uint16_t *const (&row)[TB], int from, int to, int by,
                                           float4v (&acc)[NT][TB]) {
  if (from >= to) return;
  const int off = (threadIdx.x & 63) / 16 * 64;
  const bool scales4 = P.K % 64 == 0;
  Weights w[NT];
  Elements x[TB];
#pragma unroll
  for (int t = 0; t < NT; t++) w[t] = load_weights<PACKED>(tile[t], from, P.K - from * kStep - off, scales4);
#pragma unroll
  for (int tb = 0; tb < TB; tb++) x[tb] = load_elements(row[tb], from, P.K - from * kStep - off);
  for (int s = from; s < to; s += by) {
    Weights wn[NT];
    Elements xn[TB];
    const int next = s + by < to ? s + by : s;   // (the last step is loaded again, into nothing)
#pragma unroll
    for (int t = 0; t < NT; t++) wn[t] = load_weights<PACKED>(tile[t], next, P.K - next * kStep - off, scales4);
#pragma unroll
    for (int tb = 0; tb < TB; tb++) xn[tb] = load_elements(row[tb], next, P.K - next * kStep - off);
#pragma unroll
    for (int t = 0; t < NT; t++) multiply<TB>(w[t], x, acc[t]);
#pragma unroll
    for (int t = 0; t < NT; t++) w[t] = wn[t];
#pragma unroll
    for (int tb = 0; tb < TB; tb++) x[tb] = xn[tb];
  }
}

// The groups of a workgroup's tokens, in LDS: ids of their pairs and the first pair of each group.
struct Groups {
  int id[kMaxPairs];
  uint64_t lead[kMaxPairs / kWave];
  uint16_t first[kMaxPairs];
  int count;
};

// Slots of token t before slot `end` that chose e.
__device__ __forceinline__ int chosen(const Groups &g, int k, int t, int e, int end) {
  int n = 0;
  for (int j = 0; j < end; j++) n += g.id[t * k + j] == e ? 1 : 0;
  return n;
}

__device__ __forceinline__ void build_groups(const Params &P, int t0, int tokens, Groups &g) {
  const int pairs = tokens * P.k;
  for (int p = threadIdx.x; p < pairs; p += blockDim.x) {
    const int id = P.ids ? P.ids[static_cast<int64_t>(t0) * P.k + p] : 0;
    g.id[p] = id >= 0 && id < P.E ? id : -1;
  }
  __syncthreads();
  const int rounds = (pairs + blockDim.x - 1) / blockDim.x;
  for (int i = 0; i < rounds; i++) {
    const int p = i * blockDim.x + threadIdx.x;
    bool lead = false;
    if (p < pairs && g.id[p] >= 0) {
      const int t = p / P.k, e = g.id[p], nth = chosen(g, P.k, t, e, p - t * P.k);
      lead = true;
      for (int u = 0; u < t && lead; u++) lead = chosen(g, P.k, u, e, P.k) <= nth;
    }
    const uint64_t mask = __ballot(lead);
    if ((threadIdx.x & 63) == 0 && p < pairs) g.lead[p / kWave] = mask;
  }
  __syncthreads();
  int total = 0;
  for (int w = 0; w * kWave < pairs; w++) {
    const uint64_t mask = g.lead[w];
    const int p = w * kWave + threadIdx.x;
    if (threadIdx.x < kWave && (mask >> threadIdx.x & 1)) g.first[total + __popcll(mask & ((uint64_t(1) << threadIdx.x) - 1))] = static_cast<uint16_t>(p);
    total += __popcll(mask);
  }
  if (threadIdx.x == 0) g.count = total;
  __syncthreads();
}

// The slot of token t in group number i, or -1.
__device__ __forceinline__ int slot_in(const Groups &g, int k, int i, int t, int tokens) {
  if (t >= tokens) return -1;
  const int p = g.first[i], u = p / k, e = g.id[p], nth = chosen(g, k, u, e, p - u * k);
  int n = 0;
  for (int j = 0; j < k; j++) {
    if (g.id[t * k + j] != e) continue;
    if (n == nth) return j;
    n++;
  }
  return -1;
}

// TB: blocks of four tokens.
template <int TB, Epilogue MODE, bool PACKED>
__global__ __launch_bounds__(kMaxWaves *kWave) void gemv_kernel(const Params P) {
  __shared__ Groups groups;
  __shared__ float part[kMaxWaves][NT][TB * 4][16];
  const int t0 = blockIdx.z * TB * 4, tokens = min(TB * 4, P.T - t0);
  build_groups(P, t0, tokens, groups);
  const int waves = blockDim.x / kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = threadIdx.x & 63, r = lane % 16;
  const int width = MODE == kGated ? P.N / 2 : P.N;
  // first columns of the two tiles; a second one past the end is the first again, and not stored
  const int n0 = blockIdx.x * (MODE == kGated ? 16 : 32);
  const int steps = (P.K + kStep - 1) / kStep;
  int base[NT] = {n0, MODE == kGated ? width + n0 : n0 + 16};
  if (MODE != kGated && base[1] >= P.N) base[1] = n0;

  auto tiles_of = [&](int e, Tile (&tile)[NT]) {
#pragma unroll
    for (int t = 0; t < NT; t++) {
      if (PACKED) {
        tile[t].code = P.B + (static_cast<int64_t>(e) * P.N + base[t]) / 16 * steps * kPackBlock;
        tile[t].scale = nullptr;
      } else {
        const int64_t n = static_cast<int64_t>(e) * P.N + base[t] + r;
        tile[t].code = P.B + n * (P.K / 2);
        tile[t].scale = P.B_sf + n * (P.K / 16);
      }
    }
  };
  // the rows of x of group i that this lane multiplies (a token outside it: any row, not stored)
  auto rows_of = [&](int i, const uint16_t *(&row)[TB]) {
#pragma unroll
    for (int tb = 0; tb < TB; tb++) {
      const int t = tb * 4 + lane % 4, j = slot_in(groups, P.k, i, t, tokens);
      const int64_t at = j < 0 ? 0 : P.per_pair ? static_cast<int64_t>(t0 + t) * P.k + j : t0 + t;
      row[tb] = P.x + at * P.K;
    }
  };
  // sums over lane groups and waves; afterwards sum(tile, token, column)
  auto join = [&](float4v (&acc)[NT][TB]) {
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
      for (int tb = 0; tb < TB; tb++)
#pragma unroll
        for (int c = 0; c < 4; c++) {
          float v = acc[t][tb][c];
          v += __shfl_xor(v, 16, kWave);
          v += __shfl_xor(v, 32, kWave);
          if (lane < 16) part[wave][t][tb * 4 + c][r] = v;
        }
    __syncthreads();
  };
  auto sum = [&](int t, int token, int col) {
    float v = part[0][t][token][col];
    for (int w = 1; w < waves; w++) v += part[w][t][token][col];
    return v;
  };

  float4v acc[NT][TB];
  auto clear = [&] {
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
      for (int tb = 0; tb < TB; tb++) acc[t][tb] = float4v{0.f, 0.f, 0.f, 0.f};
  };

  if (MODE == kWeighted) {
    float4v out[NT][TB];
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
      for (int tb = 0; tb < TB; tb++) out[t][tb] = float4v{0.f, 0.f, 0.f, 0.f};
    // the steps of all groups, in order, dealt to the waves in equal parts
    const int total = groups.count * steps, per = (total + waves - 1) / waves;
    const int end = min(total, (wave + 1) * per);
    for (int at = wave * per; at < end;) {
      const int i = at / steps, from = at - i * steps, to = min(steps, from + end - at);
      const int e = __builtin_amdgcn_readfirstlane(groups.id[groups.first[i]]);
      Tile tile[NT];
      const uint16_t *row[TB];
      tiles_of(e, tile);
      rows_of(i, row);
      clear();
      accumulate<TB, PACKED>(P, tile, row, from, to, 1, acc);
      const float gs = P.B_gs[e];
#pragma unroll
      for (int tb = 0; tb < TB; tb++)
#pragma unroll
        for (int c = 0; c < 4; c++) {
          const int t = tb * 4 + c, j = slot_in(groups, P.k, i, t, tokens);
          if (j < 0) continue;
          const float w = (P.topk_w ? P.topk_w[static_cast<int64_t>(t0 + t) * P.k + j] : 1.0f) * gs;
#pragma unroll
          for (int n = 0; n < NT; n++) out[n][tb][c] = fmaf(acc[n][tb][c], w, out[n][tb][c]);
        }
      at += to - from;
    }
    join(out);
    for (int i = threadIdx.x; i < NT * tokens * 16; i += blockDim.x) {
      const int col = i % 16, t = i / 16 % NT, token = i / 16 / NT;
      if (n0 + t * 16 < P.N) P.D[static_cast<int64_t>(t0 + token) * P.N + n0 + t * 16 + col] = f32_to_bf16(sum(t, token, col));
    }
    return;
  }

  if (blockIdx.y == 0) {   // dropped slots: zeros
    const int cols = MODE == kGated ? 16 : min(32, P.N - n0);
    for (int i = threadIdx.x; i < tokens * P.k * cols; i += blockDim.x) {
      const int p = i / cols;
      if (groups.id[p] < 0) P.D[(static_cast<int64_t>(t0) * P.k + p) * width + n0 + i % cols] = 0;
    }
  }
  for (int i = blockIdx.y; i < groups.count; i += gridDim.y) {
    const int e = __builtin_amdgcn_readfirstlane(groups.id[groups.first[i]]);
    Tile tile[NT];
    const uint16_t *row[TB];
    tiles_of(e, tile);
    rows_of(i, row);
    clear();
    accumulate<TB, PACKED>(P, tile, row, wave, steps, waves, acc);
    join(acc);
    const float gs = P.B_gs[e];
    constexpr int kOut = MODE == kGated ? 1 : NT;
    for (int o = threadIdx.x; o < kOut * tokens * 16; o += blockDim.x) {
      const int col = o % 16, t = o / 16 % kOut, token = o / 16 / kOut;
      const int j = slot_in(groups, P.k, i, token, tokens);
      if (j < 0 || n0 + t * 16 >= width) continue;
      float v = sum(t, token, col) * gs;
      if (MODE == kGated) {
        const float up = sum(1, token, col) * gs;
        v = v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.4426950408889634f)) * up;
      }
      P.D[(static_cast<int64_t>(t0 + token) * P.k + j) * width + n0 + t * 16 + col] = f32_to_bf16(v);
    }
    __syncthreads();   // the sums are read before the next group's are written
  }
}

template <Epilogue MODE, bool PACKED>
hipError_t run(const Params &p, hipStream_t stream) {
  const int steps = (p.K + kStep - 1) / kStep;
  const int tb = p.T <= 4 ? 1 : p.T <= 8 ? 2 : 4;
  const int chunk = p.T < tb * 4 ? p.T : tb * 4, pairs = chunk * p.k;
  const int groups = pairs < p.E ? pairs : p.E;
  const int tasks = MODE == kWeighted ? steps * groups : steps;
  const int waves = tasks < kMaxWaves ? tasks : kMaxWaves;
  const dim3 grid(MODE == kGated ? p.N / 32 : (p.N + 31) / 32, MODE == kWeighted ? 1 : groups, (p.T + tb * 4 - 1) / (tb * 4));
  const dim3 block(waves * kWave);
  if (tb == 1) hipLaunchKernelGGL((gemv_kernel<1, MODE, PACKED>), grid, block, 0, stream, p);
  else if (tb == 2) hipLaunchKernelGGL((gemv_kernel<2, MODE, PACKED>), grid, block, 0, stream, p);
  else hipLaunchKernelGGL((gemv_kernel<4, MODE, PACKED>), grid, block, 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch(const Params &p, Epilogue epilogue, bool packed, hipStream_t stream) {
  if (p.T == 0) return hipSuccess;
  if (epilogue == kPlain) return packed ? run<kPlain, true>(p, stream) : run<kPlain, false>(p, stream);
  if (epilogue == kGated) return packed ? run<kGated, true>(p, stream) : run<kGated, false>(p, stream);
  return packed ? run<kWeighted, true>(p, stream) : run<kWeighted, false>(p, stream);
}

}  // namespace gemv
}  // namespace moe
