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
//
// HBM and the latency of a step's copies bound it: one token through 8 experts of 2048 x 6144, gate/up (113
// MB) 28 us row-major and 25 packed (4.0 and 4.5 TB/s), down (57 MB) 17.5 and 15.5; through 8 of width 256
// 8.8 and 5.7; a dense 8192 x 8192 for one token 11.6, for seven 16.5, of which 5.6 is its bytes.
#include "gemv_nvfp4.hpp"
#include "lds_tiles.hpp"

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
constexpr int kCodes = kStep / 2;  // bytes of a row's codes in a step
constexpr int kCus = 256;

// Row-major weights, K a multiple of 64, or of 32 (rows of scales then start at even bytes); packed.
enum Layout { kRows64, kRows32, kPacked };

// NT: tiles of 16 weight rows that a wave takes together.  TB: blocks of four tokens.  SINGLE: one token,
// whose slots are the groups.
template <int NT_, int TB_, Layout L_, bool SINGLE_, int WAVES_, int STAGES_>
struct Shape {
  static constexpr int NT = NT_, TB = TB_, WAVES = WAVES_, STAGES = STAGES_;
  static constexpr Layout L = L_;
  static constexpr bool SINGLE = SINGLE_;
  static constexpr int kTokens = TB * 4, kPairs = SINGLE ? kMaxSlots : kTokens * kMaxSlots;
  static constexpr int kScaleCopies = L == kRows32 ? 2 * NT : NT;   // of 256 bytes
  static constexpr int kXCopies = SINGLE ? 1 : kTokens / 2;         // of 1 KB: two tokens
  static constexpr int kCopies = NT * 2 + kScaleCopies + kXCopies;
  static constexpr int kScales = NT * 2048, kX = kScales + kScaleCopies * 256, kStage = kX + kXCopies * 1024;
  static constexpr int kRing = WAVES * STAGES * kStage;
  static_assert(kMaxSlots <= 127, "slots in 8 bits");
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
  Buf code[S::NT], scale[S::NT], x;
  uint32_t row[S::kXCopies];   // byte in x of the token that this lane's copies move (kOob: none)
};

// The copies of step `step` into the stage at LDS byte `at` (`none`: they move nothing).
template <class S>
__device__ __forceinline__ void issue(const Source<S> &src, int K, uint32_t at, int step, bool none) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int c = 0; c < S::NT * 2; c++) {
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
__device__ __forceinline__ void consume(const uint8_t *stage, int K, int step, float4v (&acc)[S::NT][S::TB], Weights (&w)[S::NT], Elements (&x)[S::TB]) {
  const int lane = threadIdx.x & 63, g = lane / 16, r = lane % 16;
#pragma unroll
  for (int t = 0; t < S::NT; t++) {
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
      if (step * kStep + g * 64 + 32 >= K) w[t].scale &= 0xffff;   // the next row's scales, which may be NaN
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

// The groups of a workgroup's tokens, in LDS: ids of their pairs, what a pair's product is multiplied by,
// and for each group its expert and every token's slot in it.
template <int PAIRS, int TOKENS>
struct Groups {
  int id[PAIRS];
  float coef[PAIRS];
  uint64_t lead[(PAIRS + kWave - 1) / kWave];
  int expert[PAIRS];
  int8_t slot[PAIRS][TOKENS];   // -1: none
  int count;
};

// Slots of token t before slot `end` that chose e.
template <class G>
__device__ __forceinline__ int chosen(const G &g, int k, int t, int e, int end) {
  int n = 0;
  for (int j = 0; j < end; j++) n += g.id[t * k + j] == e ? 1 : 0;
  return n;
}

// A pair's group is led by the first token that chose its expert as often (`nth` times before).
template <int PAIRS, int TOKENS>
__device__ __forceinline__ void build_groups(const Params &P, int t0, int tokens, bool weighted, Groups<PAIRS, TOKENS> &g) {
  const int pairs = tokens * P.k, threads = blockDim.x;
  for (int p = threadIdx.x; p < pairs; p += threads) {
    const int64_t at = static_cast<int64_t>(t0) * P.k + p;
    const int id = P.ids ? P.ids[at] : 0;
    const bool in = id >= 0 && id < P.E;
    g.id[p] = in ? id : -1;
    if (in) g.coef[p] = P.B_gs[id] * (weighted && P.topk_w ? P.topk_w[at] : 1.0f);
    for (int t = 0; t < TOKENS; t++) g.slot[p][t] = -1;
  }
  __syncthreads();
  const int rounds = (pairs + threads - 1) / threads;
  // the pair that leads pair p's group; -1 for a dropped slot
  auto leader = [&](int p) {
    const int e = g.id[p], t = p / P.k;
    if (e < 0) return -1;
    const int nth = chosen(g, P.k, t, e, p - t * P.k);
    for (int u = 0; u < t; u++) {
      int n = 0;
      for (int j = 0; j < P.k; j++)
        if (g.id[u * P.k + j] == e && n++ == nth) return u * P.k + j;
    }
    return p;
  };
  for (int i = 0; i < rounds; i++) {
    const int p = i * threads + threadIdx.x;
    const uint64_t mask = __ballot(p < pairs && leader(p) == p);
    if ((threadIdx.x & 63) == 0 && p < pairs) g.lead[p / kWave] = mask;
  }
  __syncthreads();
  for (int p = threadIdx.x; p < pairs; p += threads) {
    const int q = leader(p);
    if (q < 0) continue;
    int group = __popcll(g.lead[q / kWave] & ((uint64_t(1) << (q % kWave)) - 1));
    for (int w = 0; w < q / kWave; w++) group += __popcll(g.lead[w]);
    g.expert[group] = g.id[p];
    g.slot[group][p / P.k] = static_cast<int8_t>(p % P.k);
  }
  if (threadIdx.x == 0) {
    int total = 0;
    for (int w = 0; w * kWave < pairs; w++) total += __popcll(g.lead[w]);
    g.count = total;
  }
  __syncthreads();
}

// An item is a pair of tiles of one group (MODE kWeighted: a group; the workgroup has one pair).  A
// workgroup takes a run of items, whose steps are dealt to its waves in equal runs, so the copies of one
// item follow those of another without a pause; an item that several waves had parts of is summed by
// all of them at the end, in the order of its steps.
template <class S, Epilogue MODE>
__global__ __launch_bounds__(S::WAVES *kWave) void gemv_kernel(const Params P) {
  constexpr int NT = S::NT, TB = S::TB, kHeld = S::SINGLE ? 1 : S::kTokens;
  constexpr bool SINGLE = S::SINGLE;
  static_assert(MODE == kWeighted || NT == 2, "pairs of tiles");
  __shared__ __align__(1024) uint8_t ring[S::kRing];
  __shared__ float part[S::WAVES][2][NT][kHeld][16];   // of a wave's first item, of its last one
  __shared__ Groups<S::kPairs, kHeld> groups;
  const int t0 = SINGLE ? 0 : blockIdx.z * S::kTokens, tokens = SINGLE ? 1 : min(S::kTokens, P.T - t0);
  if (!SINGLE) build_groups(P, t0, tokens, MODE == kWeighted, groups);
  const int count = SINGLE ? P.k : __builtin_amdgcn_readfirstlane(groups.count);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x & 63, r = lane % 16;
  const int width = MODE == kGated ? P.N / 2 : P.N;
  constexpr int kCols = MODE == kGated ? 16 : NT * 16;   // columns of the result in the tiles
  const int pairs = (width + kCols - 1) / kCols, steps = (P.K + kStep - 1) / kStep;

  // SINGLE: slot j's expert is in lane j (-1: dropped); every wave writes the same ids and factors
  int my_id = -1;
  if (SINGLE && lane < P.k) {
    const int id = P.ids ? P.ids[lane] : 0;
    const bool in = id >= 0 && id < P.E;
    if (in) my_id = id;
    groups.id[lane] = my_id;
    groups.coef[lane] = in ? P.B_gs[id] * (MODE == kWeighted && P.topk_w ? P.topk_w[lane] : 1.0f) : 0.f;
  }
  if (SINGLE) wave_order();
  auto expert = [&](int i) { return SINGLE ? __builtin_amdgcn_readlane(my_id, i) : __builtin_amdgcn_readfirstlane(groups.expert[i]); };
  auto slot = [&](int i, int t) { return SINGLE ? (t == 0 ? i : -1) : static_cast<int>(groups.slot[i][t]); };
  // of token t, whose slot in group i is j
  auto coef = [&](int i, int t, int j) { return groups.coef[SINGLE ? i : t * P.k + j]; };

  Source<S> src = {};
  // the workgroup's rows of x (at most 16 * 32 * 2^20 * 2 bytes)
  const int per = P.per_pair ? P.k : 1;
  src.x = uniform(Buf{reinterpret_cast<uint64_t>(P.x + static_cast<int64_t>(t0) * per * P.K), static_cast<uint32_t>(tokens * per) * P.K * 2});
  auto set_source = [&](int i, int pair) {
    const int e = expert(i), n0 = pair * kCols;
#pragma unroll
    for (int t = 0; t < NT; t++) {
      // a second tile past the end is the first again, and not stored
      int base = n0 + (MODE == kGated ? t * width : t * 16);
      if (MODE != kGated && base >= P.N) base = n0;
      const int64_t n = static_cast<int64_t>(e) * P.N + base;
      if (S::L == kPacked) {
        src.code[t] = src.scale[t] = uniform(Buf{reinterpret_cast<uint64_t>(P.B + n / 16 * steps * kPackBlock), e < 0 ? 0u : steps * kPackBlock});
      } else {
        src.code[t] = uniform(Buf{reinterpret_cast<uint64_t>(P.B + n * (P.K / 2)), e < 0 ? 0u : 8u * P.K});
        src.scale[t] = uniform(Buf{reinterpret_cast<uint64_t>(P.B_sf + n * (P.K / 16)), e < 0 ? 0u : static_cast<uint32_t>(P.K)});
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
  // Steps [begin, end) of all items' steps; the copies run STAGES - 1 steps ahead.  done(q, from, to) is
  // called with the sums of item q's steps [from, to) in acc, and clears them.
  auto stream = [&](int begin, int end, auto source_of, auto done) {
    int cq = begin / steps, cs = begin - cq * steps, left = end - begin;   // the copies' place
    if (left > 0) source_of(cq);
    auto next_copies = [&](int at) {
      if (left > 0 && cs == steps) {
        cs = 0;
        source_of(++cq);
      }
      issue<S>(src, P.K, mine0 + at * S::kStage, cs, left <= 0);
      cs++;
      left--;
    };
#pragma unroll
    for (int u = 0; u < S::STAGES; u++) next_copies(u);
    int q = begin / steps, s = begin - q * steps, from = s, at = 0;
    clear();
    for (int n = end - begin; n > 0; n--) {
      asm volatile("s_waitcnt vmcnt(%0)" : : "n"(S::kCopies * (S::STAGES - 1)) : "memory");
      Weights w[NT];
      Elements x[TB];
      consume<S>(mine + at * S::kStage, P.K, s, acc, w, x);
      next_copies(at);
#pragma unroll
      for (int t = 0; t < NT; t++) multiply<TB>(w[t], x, acc[t]);
      at = at == S::STAGES - 1 ? 0 : at + 1;
      s++;
      if (n == 1 || s == steps) {
        done(q, from, s);
        clear();
        q++;
        s = from = 0;
      }
    }
  };
  // v summed over the lane groups
  auto over_groups = [&](float v) {
    v += __shfl_xor(v, 16, kWave);
    return v + __shfl_xor(v, 32, kWave);
  };

  if (MODE == kWeighted) {
    const int n0 = blockIdx.x * kCols;
    float4v out[NT][TB];
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
      for (int tb = 0; tb < TB; tb++) out[t][tb] = float4v{0.f, 0.f, 0.f, 0.f};
    const int total = count * steps, share = (total + S::WAVES - 1) / S::WAVES;
    const int begin = min(total, wave * share), end = min(total, begin + share);
    stream(begin, end, [&](int i) { set_source(i, blockIdx.x); },
           [&](int i, int, int) {
#pragma unroll
             for (int tb = 0; tb < TB; tb++)
#pragma unroll
               for (int c = 0; c < 4; c++) {
                 const int t = tb * 4 + c, j = t < kHeld ? slot(i, t) : -1;
                 if (j < 0 || expert(i) < 0) continue;
                 const float f = coef(i, t, j);
#pragma unroll
                 for (int n = 0; n < NT; n++) out[n][tb][c] = fmaf(acc[n][tb][c], f, out[n][tb][c]);
               }
           });
#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
      for (int t = 0; t < kHeld; t++) {
        const float v = over_groups(out[n][t / 4][t % 4]);
        if (lane < 16) part[wave][0][n][t][r] = v;
      }
    arrive<0>();
    for (int i = threadIdx.x; i < NT * tokens * 16; i += S::WAVES * kWave) {
      const int col = i % 16, t = i / 16 % NT, token = i / 16 / NT;
      float v = part[0][0][t][token][col];
#pragma unroll
      for (int w = 1; w < S::WAVES; w++) v += part[w][0][t][token][col];
      if (n0 + t * 16 < P.N) P.D[static_cast<int64_t>(t0 + token) * P.N + n0 + t * 16 + col] = f32_to_bf16(v);
    }
    return;
  }

  if (!SINGLE) {   // dropped slots: zeros
    for (int p = 0; p < tokens * P.k; p++)
      if (groups.id[p] < 0)
        for (int c = blockIdx.x * blockDim.x + threadIdx.x; c < width; c += gridDim.x * blockDim.x)
          P.D[(static_cast<int64_t>(t0) * P.k + p) * width + c] = 0;
  }
  const int items = count * pairs, run = (items + gridDim.x - 1) / gridDim.x;
  const int first = min(items, static_cast<int>(blockIdx.x) * run), total = min(items - first, run) * steps;
  const int share = (total + S::WAVES - 1) / S::WAVES;
  const int begin = first * steps + min(total, wave * share), end = first * steps + min(total, (wave + 1) * share);
  // column `col` of token t's row of item q, from the sums of the two tiles
  auto store = [&](int q, int t, int col, float a, float b) {
    const int i = q / pairs, n = (q - i * pairs) * kCols + col, j = slot(i, t);
    if (j < 0) return;
    if (SINGLE && groups.id[i] < 0) a = b = 0.f;   // (no weights times an infinity is a NaN)
    const float f = coef(i, t, j);
    uint16_t *at = P.D + (static_cast<int64_t>(t0 + t) * P.k + j) * width + n;
    if (MODE == kGated) {
      const float gate = a * f;
      *at = f32_to_bf16(gate * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(gate * -1.4426950408889634f)) * (b * f));
    } else {
      *at = f32_to_bf16(a * f);
      if (n + 16 < width) at[16] = f32_to_bf16(b * f);
    }
  };
  stream(begin, end,
         [&](int q) {
           const int i = q / pairs;
           set_source(i, q - i * pairs);
         },
         [&](int q, int from, int to) {
           const bool whole = from == 0 && to == steps;
           const int nth = q == begin / steps ? 0 : 1;
#pragma unroll
           for (int t = 0; t < kHeld; t++) {
             const float a = over_groups(acc[0][t / 4][t % 4]), b = over_groups(acc[NT - 1][t / 4][t % 4]);
             if (!whole) {
               if (lane < 16) part[wave][nth][0][t][r] = a;
               else if (lane < 32) part[wave][nth][NT - 1][t][r] = b;
             } else if (lane / 16 == t % 4 && t < tokens) {
               store(q, t, r, a, b);
             }
           }
         });
  arrive<0>();
  // items in parts: wave w's part is its first one where the item is its first
  for (int o = threadIdx.x; o < total / steps * tokens * 16; o += S::WAVES * kWave) {
    const int col = o % 16, t = o / 16 % tokens, local = o / 16 / tokens;
    const int from = local * steps / share, to = (local * steps + steps - 1) / share;
    if (from == to) continue;
    float a = 0.f, b = 0.f;
    for (int w = from; w <= to; w++) {
      const int nth = w * share / steps == local ? 0 : 1;
      a += part[w][nth][0][t][col];
      b += part[w][nth][NT - 1][t][col];
    }
    store(first + local, t, col, a, b);
  }
}

template <class S, Epilogue MODE>
hipError_t run(const Params &p, hipStream_t stream) {
  const int width = MODE == kGated ? p.N / 2 : p.N, cols = MODE == kGated ? 16 : S::NT * 16;
  const int pairs = (width + cols - 1) / cols, chunk = p.T < S::kTokens ? p.T : S::kTokens;
  const int64_t items = static_cast<int64_t>(pairs) * (chunk * p.k < p.E ? chunk * p.k : p.E);
  const dim3 grid(static_cast<uint32_t>(MODE == kWeighted ? pairs : items < kCus ? items : kCus), 1, (p.T + S::kTokens - 1) / S::kTokens);
  hipLaunchKernelGGL((gemv_kernel<S, MODE>), grid, dim3(S::WAVES * kWave), 0, stream, p);
  return hipGetLastError();
}

// The fewest blocks of four tokens that hold them, up to 16 tokens: 1 token through 8 of 64 experts, 4096 x
// 6144, 24 us without groups, 28 with, 31 with two blocks, 64 with four; 4 tokens 85, 90, 190 with one, two,
// four; 8 tokens 148, 295 with two, four.  Eight waves with two stages each (three: 25 us) where LDS has
// room for them, else four.
template <Epilogue MODE, Layout L, int NT>
hipError_t run_tokens(const Params &p, hipStream_t stream) {
  if (p.T == 1) return run<Shape<NT, 1, L, true, 8, 2>, MODE>(p, stream);
  if (p.T <= 4) return run<Shape<NT, 1, L, false, 8, 2>, MODE>(p, stream);
  if (p.T <= 8) return run<Shape<NT, 2, L, false, L == kRows32 ? 4 : 8, 2>, MODE>(p, stream);
  return run<Shape<NT, 4, L, false, 4, 2>, MODE>(p, stream);
}

// A weighted sum's workgroup has its columns for all groups: one tile of them where pairs of tiles are at most
// half of the CUs.  8 of 64 experts, us with one tile | two: 4096 x 2048, one token 11.1 | 15.2, sixteen 162 |
// 261; 6144 x 2048 18.0 | 18.2, eight tokens 118 | 96.
template <Epilogue MODE, Layout L>
hipError_t run_layout(const Params &p, hipStream_t stream) {
  if (MODE == kWeighted && p.N <= kCus / 2 * 32) return run_tokens<MODE, L, MODE == kWeighted ? 1 : 2>(p, stream);
  return run_tokens<MODE, L, 2>(p, stream);
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
