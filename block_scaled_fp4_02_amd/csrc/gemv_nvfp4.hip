// Products of one or a few tokens with experts' NVFP4 weights, the activations left in bf16:
//
//   y[t, j, n] = gB[e] sum_b sB[e, n, b] sum_{i < 16} x[r, 16 b + i] b[e, n, 16 b + i],  e = ids[t, j]
//
// and with them silu(gate) up, or the sum over a token's slots j of w[t, j] y[t, j].
//
// The weights are read once and their decoding has to keep up with HBM, so what counts is how few
// instructions a weight takes.  A lane takes 16 bytes, 32 codes of one weight row, which are two scale
// blocks, so sums over lanes may only be taken after the scales.  The 4x4x4 MFMA (16 independent
// blocks) fits that: a lane's four weights of one row meet four tokens' elements, summed within the lane,
// and 4 MFMAs sum a scale block.  Per 16 weights and lane that is 8 conversions (two codes to bf16
// each, exact), 4 MFMAs on the matrix pipe and one fma per token with the block's scale: one vector
// instruction per 1.3 to 1.8 weights, for up to 4 tokens.  Products are exact and sums binary32.
//
// A wave takes two tiles of 16 weight rows, which share the tokens' elements: gate and up rows, or
// neighbouring tiles.  It copies them in steps of 256 elements (4.6 KB), and the tokens' elements beside
// them, into a ring of its own in LDS (no registers, whole 128-byte lines: lanes that load what they
// multiply straight from a row-major matrix touch 64 lines with each load, and 50 us for 113 MB was what
// that took), and waits for nothing but its own copies.  Lane 16 g + r multiplies elements
// [64 g, 64 g + 64) of row r, the order that the packed layout has; rows in LDS keep their 8 pieces of 16
// bytes swizzled as in the other products, so 16 lanes fall on all banks once.
//
// Tokens that chose the same expert share the read of its weights: the pairs (t, j) of up to 16 tokens
// are collected into groups of one expert, at most one slot of each token (a token's second slot with
// the same expert goes to a second group).
#include "gemv_nvfp4.hpp"
#include "lds_tiles.hpp"

#include <limits.h>

#include <type_traits>

#pragma clang fp contract(off)

namespace moe {
namespace gemv {
namespace {

using namespace lds;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short short4v __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kStep = 256;         // elements of K in a step
constexpr int kPackBlock = 2304;   // bytes of one (16-row tile, step) block of packed weights
constexpr int kMaxSlots = 32;
constexpr int NT = 2;              // tiles of 16 weight rows that a wave takes together
constexpr int kCodes = kStep / 2;  // bytes of a row's codes in a step

// Row-major weights, K a multiple of 64, or of 32 (rows of scales then start at even bytes); packed.
enum Layout { kRows64, kRows32, kPacked };

// TB: blocks of four tokens.  SINGLE: one token, whose slots are the groups.
template <int TB_, Layout L_, bool SINGLE_, int WAVES_, int STAGES_>
struct Shape {
  static constexpr int TB = TB_, WAVES = WAVES_, STAGES = STAGES_;
  static constexpr Layout L = L_;
  static constexpr bool SINGLE = SINGLE_;
  static constexpr int kTokens = TB * 4, kPairs = SINGLE ? 1 : kTokens * kMaxSlots;
  static constexpr int kScaleCopies = L == kRows32 ? 2 * NT : NT;   // of 256 bytes
  static constexpr int kXCopies = SINGLE ? 1 : kTokens / 2;         // of 1 KB: two tokens
  static constexpr int kCopies = NT * 2 + kScaleCopies + kXCopies;
  static constexpr int kScales = NT * 2048, kX = kScales + kScaleCopies * 256, kStage = kX + kXCopies * 1024;
  static constexpr int kRing = WAVES * STAGES * kStage;
  static_assert(WAVES * NT * kTokens * 16 * 4 <= kRing, "partial sums");
};

// One step's weights of a tile in this lane: 64 codes of its row and their four scales.
struct Weights {
  u32x4 code[2];
  uint32_t scale;
};
// One step's elements of this lane's token: 64 of its lane group.
struct Elements {
  u32x4 v[8];
};

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

// The tiles and tokens that a wave's copies come from.
template <class S>
struct Source {
  Buf code[NT], scale[NT], x;
  uint32_t row[S::kXCopies];   // byte in x of the token that this lane's copies move (kOob: none)
};

// The copies of step `step` into the stage at LDS byte `at` (`none`: they move nothing).
template <class S>
__device__ __forceinline__ void issue(const Source<S> &src, int K, uint32_t at, int step, bool none) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int c = 0; c < NT * 2; c++) {
    uint32_t from;
    if (S::L == kPacked) {
      from = none ? kOob : step * kPackBlock + c % 2 * 1024 + lane * 16;
    } else {
      const int row = c % 2 * 8 + lane / 8, piece = (lane & 7) ^ ((row >> 1) & 7);
      from = none || step * kStep + piece * 32 >= K ? kOob : row * (K / 2) + step * kCodes + piece * 16;
    }
    copy16<true>(uniform(src.code[c / 2]), at + c * 1024, from);
  }
#pragma unroll
  for (int c = 0; c < S::kScaleCopies; c++) {
    uint32_t from;
    if (S::L == kPacked) {
      from = none ? kOob : step * kPackBlock + 2048 + lane * 4;
    } else if (S::L == kRows64) {
      from = none || step * kStep + lane % 4 * 64 >= K ? kOob : lane / 4 * (K / 16) + step * 16 + lane % 4 * 4;
    } else {   // the two words around four scales that may start between them (a tile's scales are whole words)
      from = (lane / 4 * (K / 16) + step * 16 + lane % 4 * 4) / 4 * 4 + c % 2 * 4;
      if (none || step * kStep + lane % 4 * 64 >= K || from >= static_cast<uint32_t>(K)) from = kOob;
    }
    copy4(uniform(src.scale[S::L == kRows32 ? c / 2 : c]), at + S::kScales + c * 256, from);
  }
#pragma unroll
  for (int c = 0; c < S::kXCopies; c++) {
    const int t = 2 * c + lane / 32, piece = lane % 32 ^ (t & 3);
    const bool in = !none && src.row[c] != kOob && step * kStep + piece * 8 < K;
    copy16(src.x, at + S::kX + c * 1024, in ? src.row[c] + step * (kStep * 2) + piece * 16 : kOob);
  }
}

// acc += the products of the step in the stage at `stage`.
template <class S>
__device__ __forceinline__ void consume(const uint8_t *stage, int K, int step, float4v (&acc)[NT][S::TB], Weights (&w)[NT], Elements (&x)[S::TB]) {
  const int lane = threadIdx.x & 63, g = lane / 16, r = lane % 16;
#pragma unroll
  for (int t = 0; t < NT; t++) {
#pragma unroll
    for (int q = 0; q < 2; q++) {
      const int at = S::L == kPacked ? q * 1024 + lane * 16 : r * kCodes + ((2 * g + q) ^ ((r >> 1) & 7)) * 16;
      w[t].code[q] = *reinterpret_cast<const u32x4 *>(stage + t * 2048 + at);
    }
    if (S::L == kPacked) {
      w[t].scale = *reinterpret_cast<const uint32_t *>(stage + S::kScales + t * 256 + lane * 4);
    } else if (S::L == kRows64) {
      w[t].scale = *reinterpret_cast<const uint32_t *>(stage + S::kScales + t * 256 + r * 16 + g * 4);
    } else {
      const uint32_t lo = *reinterpret_cast<const uint32_t *>(stage + S::kScales + t * 512 + r * 16 + g * 4);
      const uint32_t hi = *reinterpret_cast<const uint32_t *>(stage + S::kScales + t * 512 + 256 + r * 16 + g * 4);
      w[t].scale = r * (K / 16) % 4 ? lo >> 16 | hi << 16 : lo;
    }
  }
#pragma unroll
  for (int tb = 0; tb < S::TB; tb++) {
    const int t = S::SINGLE ? 0 : tb * 4 + lane % 4;
#pragma unroll
    for (int i = 0; i < 8; i++) x[tb].v[i] = *reinterpret_cast<const u32x4 *>(stage + S::kX + t * 512 + ((g * 8 + i) ^ (t & 3)) * 16);
  }
  asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");   // the stage is read before it is filled again
}

// The groups of a workgroup's tokens, in LDS: ids of their pairs and the first pair of each group.
template <int PAIRS>
struct Groups {
  int id[PAIRS];
  uint64_t lead[(PAIRS + kWave - 1) / kWave];
  uint16_t first[PAIRS];
  int count;
};

// Slots of token t before slot `end` that chose e.
template <int PAIRS>
__device__ __forceinline__ int chosen(const Groups<PAIRS> &g, int k, int t, int e, int end) {
  int n = 0;
  for (int j = 0; j < end; j++) n += g.id[t * k + j] == e ? 1 : 0;
  return n;
}

template <int PAIRS>
__device__ __forceinline__ void build_groups(const Params &P, int t0, int tokens, Groups<PAIRS> &g) {
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
template <int PAIRS>
__device__ __forceinline__ int slot_in(const Groups<PAIRS> &g, int k, int i, int t, int tokens) {
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

// KS (PLAIN, GATED): waves that share a pair of tiles and deal its steps among themselves.
template <class S, Epilogue MODE>
__global__ __launch_bounds__(S::WAVES *kWave) void gemv_kernel(const Params P, int KS) {
  __shared__ __align__(1024) uint8_t ring[S::kRing];
  __shared__ Groups<S::kPairs> groups;
  constexpr int TB = S::TB;
  constexpr bool SINGLE = S::SINGLE;
  const int t0 = SINGLE ? 0 : blockIdx.z * S::kTokens, tokens = SINGLE ? 1 : min(S::kTokens, P.T - t0);
  if (!SINGLE) build_groups(P, t0, tokens, groups);
  const int count = SINGLE ? P.k : __builtin_amdgcn_readfirstlane(groups.count);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x & 63, r = lane % 16;
  const int width = MODE == kGated ? P.N / 2 : P.N;
  constexpr int kCols = MODE == kGated ? 16 : 32;   // columns of the result in a pair of tiles
  const int pairs = (width + kCols - 1) / kCols, steps = (P.K + kStep - 1) / kStep;
  // this wave's pair of tiles, and which of its steps (MODE == kWeighted: all waves have one pair)
  const int pair = MODE == kWeighted ? blockIdx.x : blockIdx.x * (S::WAVES / KS) + wave / KS;
  const int n0 = pair * kCols;
  const bool idle = pair >= pairs;

  // expert of group i; -1: a dropped slot of the only token
  auto expert = [&](int i) {
    if (!SINGLE) return __builtin_amdgcn_readfirstlane(groups.id[groups.first[i]]);
    const int id = P.ids ? P.ids[i] : 0;
    return __builtin_amdgcn_readfirstlane(id >= 0 && id < P.E ? id : -1);
  };
  auto slot = [&](int i, int t) { return SINGLE ? (t == 0 ? i : -1) : slot_in(groups, P.k, i, t, tokens); };

  Source<S> src = {};   // (no bytes: what has no source copies zeros)
  // the workgroup's rows of x (at most 16 * 32 * 2^20 * 2 bytes)
  const int per = P.per_pair ? P.k : 1;
  src.x = uniform(Buf{reinterpret_cast<uint64_t>(P.x + static_cast<int64_t>(t0) * per * P.K), static_cast<uint32_t>(tokens * per) * P.K * 2});
  auto set_source = [&](int i) {
    const int e = expert(i);
#pragma unroll
    for (int t = 0; t < NT; t++) {
      // a second tile past the end is the first again, and not stored
      int base = n0 + (MODE == kGated ? t * width : t * 16);
      if (MODE != kGated && base >= P.N) base = n0;
      const int64_t n = static_cast<int64_t>(e) * P.N + base;
      const bool none = e < 0 || idle;
      if (S::L == kPacked) {
        src.code[t] = src.scale[t] = uniform(Buf{reinterpret_cast<uint64_t>(P.B + n / 16 * steps * kPackBlock), none ? 0u : steps * kPackBlock});
      } else {
        src.code[t] = uniform(Buf{reinterpret_cast<uint64_t>(P.B + n * (P.K / 2)), none ? 0u : 8u * P.K});
        src.scale[t] = uniform(Buf{reinterpret_cast<uint64_t>(P.B_sf + n * (P.K / 16)), none ? 0u : static_cast<uint32_t>(P.K)});
      }
    }
#pragma unroll
    for (int c = 0; c < S::kXCopies; c++) {
      const int t = 2 * c + lane / 32, j = slot(i, t);
      src.row[c] = j < 0 ? kOob : static_cast<uint32_t>(P.per_pair ? t * P.k + j : t) * P.K * 2;
    }
  };

  uint8_t *const mine = ring + wave * S::STAGES * S::kStage;
  const uint32_t mine0 = lds_address(mine);
  float4v acc[NT][TB];
  auto clear = [&] {
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
      for (int tb = 0; tb < TB; tb++) acc[t][tb] = float4v{0.f, 0.f, 0.f, 0.f};
  };
  // Steps `first`, first + by, ... of group i, `todo` of them (across the groups' ends where by == 1).
  // The copies run STAGES - 1 steps ahead; done(i) is called behind a group's last step, or this wave's.
  auto stream = [&](int i, int first, int by, int todo, auto done) {
    int ci = i, cs = first, left = todo;   // the copies' place
    if (todo > 0) set_source(ci);
    auto next_copies = [&](int slot) {
      if (left > 0 && cs >= steps) {
        cs -= steps;
        set_source(++ci);
      }
      issue<S>(src, P.K, mine0 + slot * S::kStage, cs, left <= 0);
      cs += by;
      left--;
    };
#pragma unroll
    for (int u = 0; u < S::STAGES; u++) next_copies(u);
    int s = first, at = 0;
    for (int n = 0; n < todo; n++) {
      asm volatile("s_waitcnt vmcnt(%0)" : : "n"(S::kCopies * (S::STAGES - 1)) : "memory");
      Weights w[NT];
      Elements x[TB];
      consume<S>(mine + at * S::kStage, P.K, s, acc, w, x);
      next_copies(at);
#pragma unroll
      for (int t = 0; t < NT; t++) multiply<TB>(w[t], x, acc[t]);
      at = at == S::STAGES - 1 ? 0 : at + 1;
      s += by;
      if (n == todo - 1 || s >= steps) {
        done(i);
        s -= steps;
        i++;
      }
    }
  };
  // sums over lane groups, put beside the other waves'
  float(*part)[NT][S::kTokens][16] = reinterpret_cast<float(*)[NT][S::kTokens][16]>(ring);
  auto join = [&](const float4v (&v)[NT][TB]) {
    arrive<0>();   // no copy is under way into the ring, which the partial sums reuse
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
      for (int tb = 0; tb < TB; tb++)
#pragma unroll
        for (int c = 0; c < 4; c++) {
          float u = v[t][tb][c];
          u += __shfl_xor(u, 16, kWave);
          u += __shfl_xor(u, 32, kWave);
          if (lane < 16) part[wave][t][tb * 4 + c][r] = u;
        }
    __syncthreads();
  };
  auto sum = [&](int from, int waves, int t, int token, int col) {
    float v = part[from][t][token][col];
    for (int w = 1; w < waves; w++) v += part[from + w][t][token][col];
    return v;
  };

  if (MODE == kWeighted) {
    float4v out[NT][TB];
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
      for (int tb = 0; tb < TB; tb++) out[t][tb] = float4v{0.f, 0.f, 0.f, 0.f};
    // the steps of all groups, in order, dealt to the waves in equal parts
    const int total = count * steps, share = (total + S::WAVES - 1) / S::WAVES;
    const int begin = min(total, wave * share), end = min(total, begin + share);
    clear();
    stream(begin / steps, begin % steps, 1, end - begin, [&](int i) {
      const int e = expert(i);
      if (e >= 0) {
        const float gs = P.B_gs[e];
#pragma unroll
        for (int tb = 0; tb < TB; tb++)
#pragma unroll
          for (int c = 0; c < 4; c++) {
            const int t = tb * 4 + c, j = slot(i, t);
            if (j < 0) continue;
            const float w = (P.topk_w ? P.topk_w[static_cast<int64_t>(t0 + t) * P.k + j] : 1.0f) * gs;
#pragma unroll
            for (int n = 0; n < NT; n++) out[n][tb][c] = fmaf(acc[n][tb][c], w, out[n][tb][c]);
          }
      }
      clear();
    });
    join(out);
    for (int i = threadIdx.x; i < NT * tokens * 16; i += S::WAVES * kWave) {
      const int col = i % 16, t = i / 16 % NT, token = i / 16 / NT;
      if (n0 + t * 16 < P.N) P.D[static_cast<int64_t>(t0 + token) * P.N + n0 + t * 16 + col] = f32_to_bf16(sum(0, S::WAVES, t, token, col));
    }
    return;
  }

  constexpr int kOut = MODE == kGated ? 1 : NT;   // tiles of results
  const int lead = wave / KS * KS, rank = (wave - lead) * kWave + lane;   // the waves of this pair, the thread among theirs
  if (!SINGLE && blockIdx.y == 0 && !idle) {      // dropped slots: zeros
    const int cols = min(kCols, width - n0);
    for (int i = rank; i < tokens * P.k * cols; i += KS * kWave) {
      const int p = i / cols;
      if (groups.id[p] < 0) P.D[(static_cast<int64_t>(t0) * P.k + p) * width + n0 + i % cols] = 0;
    }
  }
  for (int i = blockIdx.y; i < count; i += gridDim.y) {
    const int e = expert(i), from = wave - lead;
    clear();
    stream(i, from, KS, idle || e < 0 || from >= steps ? 0 : (steps - from + KS - 1) / KS, [](int) {});
    join(acc);
    const float gs = e < 0 ? 0.f : P.B_gs[e];
    for (int o = idle ? INT_MAX : rank; o < kOut * tokens * 16; o += KS * kWave) {
      const int col = o % 16, t = o / 16 % kOut, token = o / 16 / kOut;
      const int j = slot(i, token);
      if (j < 0 || n0 + t * 16 >= width) continue;
      float v = sum(lead, KS, t, token, col) * gs;
      if (MODE == kGated) {
        const float up = sum(lead, KS, 1, token, col) * gs;
        v = v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.4426950408889634f)) * up;
      }
      P.D[(static_cast<int64_t>(t0 + token) * P.k + j) * width + n0 + t * 16 + col] = e < 0 ? 0 : f32_to_bf16(v);
    }
    __syncthreads();   // the sums are read before the ring is filled again
  }
}

template <class S, Epilogue MODE>
hipError_t run(const Params &p, hipStream_t stream) {
  const int steps = (p.K + kStep - 1) / kStep, width = MODE == kGated ? p.N / 2 : p.N, cols = MODE == kGated ? 16 : 32;
  const int pairs = (width + cols - 1) / cols, chunk = p.T < S::kTokens ? p.T : S::kTokens;
  const int groups = chunk * p.k < p.E ? chunk * p.k : p.E;   // (more of them, of one expert each, take turns)
  // waves that share a pair of tiles: as many as leave each of the card's waves work
  int ks = 1;
  while (ks < S::WAVES && ks < steps && static_cast<int64_t>(pairs) * groups * ks < 256 * 8) ks *= 2;
  const int per = S::WAVES / ks;
  const dim3 grid(MODE == kWeighted ? pairs : (pairs + per - 1) / per, MODE == kWeighted ? 1 : groups, (p.T + S::kTokens - 1) / S::kTokens);
  hipLaunchKernelGGL((gemv_kernel<S, MODE>), grid, dim3(S::WAVES * kWave), 0, stream, p, ks);
  return hipGetLastError();
}

template <Epilogue MODE, Layout L>
hipError_t run_layout(const Params &p, hipStream_t stream) {
  if (p.T == 1) return run<Shape<1, L, true, 8, 3>, MODE>(p, stream);
  if (p.T <= 4) return run<Shape<1, L, false, 4, 3>, MODE>(p, stream);
  if (p.T <= 8) return run<Shape<2, L, false, 4, 2>, MODE>(p, stream);
  return run<Shape<4, L, false, 4, 2>, MODE>(p, stream);
}

}  // namespace

hipError_t launch(const Params &p, Epilogue epilogue, bool packed, hipStream_t stream) {
  if (p.T == 0) return hipSuccess;
  auto run_for = [&](auto layout) {
    constexpr Layout L = decltype(layout)::value;
    if (epilogue == kPlain) return run_layout<kPlain, L>(p, stream);
    if (epilogue == kGated) return run_layout<kGated, L>(p, stream);
    return run_layout<kWeighted, L>(p, stream);
  };
  if (packed) return run_for(std::integral_constant<Layout, kPacked>());
  if (p.K % 64 == 0) return run_for(std::integral_constant<Layout, kRows64>());
  return run_for(std::integral_constant<Layout, kRows32>());
}

}  // namespace gemv
}  // namespace moe
