// Grouped FP8 (E4M3FN) matrix products with one binary32 scale per 128 elements of the
// contraction: the experts' forward product and its input gradient (gemm_kernel), and the
// weight gradient (wgrad_kernel).
//
//   y[p, n]     = sum_b sA[r, b] sB[e, n / 128, b] sum_{i < 128} a[r, 128 b + i] b[e, n, 128 b + i]
//   dW[e, n, k] = sum_b sY[b, n] sX[b, k] sum_{t < 128} y[b, n, t] x[b, k, t]   (b: token blocks of e)
//
// gemm_kernel: one 16x16x128 FP8 MFMA holds exactly one scale block of its contraction, so every
// MFMA starts from zero and its 4 results per lane join the binary32 accumulators by one fma
// with the product of the two scales.  (The scaled form of the MFMA takes power-of-two scales
// per 32 only.)  The FP8 matrix core adds 8 products at a time after aligning them to the
// largest exponent and cutting them off 13 bits below it; those sums and all later ones are
// binary32 (measured on gfx950: the same for the 16x16x32 form).  That is 5e-5 of the result in
// the 2-norm, a thirtieth of the rounding of D to bf16, for twice the rate of the fp16 matrix core.
//
// Where that would show, the codes become fp16 (exactly) and the fp16 matrix core, whose products
// and sums are whole, takes them: in wgrad_kernel, whose D may be binary32, and in the SwiGLU
// epilogue's smaller tiles, whose act is rounded again to E4M3 (a code next to a border falls the
// other way for the least difference: 1.3 to 1.6 times the error of the down projection's result,
// against 4 % of a decode batch's time; the large tile keeps FP8, a prompt's gate/up product taking 467 us
// with it and 1027 with fp16).  MOE_SUMS_WHOLE takes the fp16 matrix core for every call.
//
// Both products have the same inner form.  The "row" operand P (weight rows; columns k of x)
// gives the MFMA's rows, of which a lane holds 4 consecutive ones, so results are contiguous
// along P; the "column" operand Q (tokens; rows n of dW) gives its columns, one per lane.
// Tiles of both are copied from memory straight into LDS (16 bytes per lane, no registers) in
// a ring of STAGES buffers, one scale block per stage.  A tile row is 128 bytes in 8 pieces;
// row r keeps piece c at place c ^ ((r >> 1) & 7), so the 16 rows that 16 lanes read together
// fall on all 64 banks once.  The copies are range-checked: rows and pieces outside the
// operand arrive as zeros.
#include "common.hpp"
#include "fp8_gemm.hpp"
#include "fp8_round.hpp"
#include "groups.hpp"
#include "lds_tiles.hpp"

#include <type_traits>

#pragma clang fp contract(off)

namespace moe {
namespace fp8 {
namespace {

using namespace lds;

typedef int int8v __attribute__((ext_vector_type(8)));
enum Mode { kNone, kSwigluFp8, kWgradF32, kWgradBf16 };

// ---- one tile -----------------------------------------------------------------------------

template <int BQ_, int BP_, int WQ_, int WP_, int STAGES_>
struct Tile {
  static constexpr int BQ = BQ_, BP = BP_, WQ = WQ_, WP = WP_, STAGES = STAGES_;
  static constexpr int kWaves = WQ * WP, kThreadsT = kWaves * kWave;
  static constexpr int kHalves = BP / kFp8Block;             // 128-row halves of P
  static constexpr int kPerHalf = kFp8Block / WP / 16;       // a wave's 16-row tiles in each half
  static constexpr int TP = kHalves * kPerHalf, TQ = BQ / WQ / 16;
  static constexpr int kCopiesP = BP / 8 / kWaves;           // copies per wave and stage: 8 rows each
  static constexpr int kCopiesQ = (BQ / 8 + kWaves - 1) / kWaves;
  static constexpr int kCopies = kCopiesP + kCopiesQ + 1;    // and one of scales
  static constexpr int kRowsQ = kCopiesQ * kWaves * 8;       // Q rows in LDS (at least BQ)
  static constexpr int kBytesP = BP * kFp8Block, kBytesQ = kRowsQ * kFp8Block, kBytesS = kWaves * kWave * 4;
  static constexpr int kScaleP = BQ < kWave ? kWave : BQ;    // P's scales stand behind Q's, in another wave's copy
  static constexpr int kStage = kBytesP + kBytesQ + kBytesS;
  static constexpr bool kLarge = BQ == 256 && BP == 256;     // contract_large
  // contract_large keeps its scales apart: two groups of four steps, a float4 per row
  static constexpr int kScaleRows = kScaleP + kWave, kScaleGroup = kScaleRows * 16;
  static constexpr int kLds = kLarge ? 2 * (kBytesP + kBytesQ) + 2 * kScaleGroup : STAGES * kStage;
  static_assert(BP % 128 == 0 && BP / 8 % kWaves == 0 && BQ % (16 * WQ) == 0 && kPerHalf >= 1, "tile split");
  static_assert(kScaleP + kHalves <= kWaves * kWave, "a stage's scales fit one copy per wave");
  static_assert(STAGES >= 2 && kCopies * (STAGES - 2) < 64, "copies under way fit the counter");
};

// Where one lane's copies of a stage come from: byte offsets of its pieces in the two buffers
// (kOob: nothing), the offset of its scale, and the steps between stages.
template <class T>
struct Source {
  Buf p, q, s;                 // operands and scales; `s` serves this wave's scale copy
  uint32_t vp[T::kCopiesP], vq[T::kCopiesQ], vs;
  uint32_t step_p, step_q, step_s;   // bytes that the buffers advance per stage
  int last_pieces;             // 16-byte pieces that the last stage holds of a row (8: all)
};

// First LDS row of copy j of P: in the large tile a wave copies as many rows of either half.
template <class T>
__device__ __forceinline__ int copy_row_p(int wave, int j) {
  constexpr int kHalf = T::kCopiesP / 2;
  return T::kLarge ? j / kHalf * kFp8Block + (wave * kHalf + j % kHalf) * 8 : (wave * T::kCopiesP + j) * 8;
}

// Row and logical piece that a copy of the rows from `first_row` moves in this lane.
__device__ __forceinline__ void copy_place(int first_row, int &row, int &piece) {
  const int lane = threadIdx.x & 63;
  row = first_row + lane / 8;
  piece = (lane & 7) ^ ((row >> 1) & 7);
}

// This lane's offset in a copy of the rows from `first_row`: nothing if the last stage ends before
// the lane's piece.
__device__ __forceinline__ uint32_t piece_or_none(uint32_t voff, int first_row, bool last, int last_pieces) {
  int row, piece;
  copy_place(first_row, row, piece);
  return last && piece >= last_pieces ? kOob : voff;
}

template <class T, bool ONCE, int FROM, int TO>
__device__ __forceinline__ void issue_p(const Source<T> &src, uint32_t lds, int wave, bool last) {
#pragma unroll
  for (int j = FROM; j < TO; j++) {
    const int row = copy_row_p<T>(wave, j);
    copy16<ONCE>(src.p, lds + row * kFp8Block, piece_or_none(src.vp[j], row, last, src.last_pieces));
  }
}
template <class T>
__device__ __forceinline__ void issue_q(const Source<T> &src, uint32_t lds, int wave, bool last) {
#pragma unroll
  for (int j = 0; j < T::kCopiesQ; j++) {
    const int row = (wave * T::kCopiesQ + j) * 8;
    copy16(src.q, lds + T::kBytesP + row * kFp8Block, piece_or_none(src.vq[j], row, last, src.last_pieces));
  }
}

// The copies of stage `kb` into the buffer at `lds`; beyond the last stage they move nothing.
template <class T, bool ONCE>
__device__ __forceinline__ void issue(Source<T> &src, uint32_t lds, int wave, int kb, int steps) {
  const bool last = kb == steps - 1 && src.last_pieces < 8;
  if (kb >= steps) src.p.bytes = src.q.bytes = src.s.bytes = 0;
  issue_p<T, ONCE, 0, T::kCopiesP>(src, lds, wave, last);
  issue_q<T>(src, lds, wave, last);
  copy4(src.s, lds + T::kBytesP + T::kBytesQ + wave * kWave * 4, src.vs);
  src.p.base += src.step_p;
  src.q.base += src.step_q;
  src.s.base += src.step_s;
}

// 32 bytes of a tile row: pieces g and g + 4 for lane group g (both operands take this order;
// within a scale block the contraction's order is free).
__device__ __forceinline__ int8v fragment(const uint8_t *rows, int row, int g) {
  const int sw = (row >> 1) & 7;
  const uint8_t *p = rows + row * kFp8Block;
  const int4x a = *reinterpret_cast<const int4x *>(p + (g ^ sw) * 16);
  const int4x b = *reinterpret_cast<const int4x *>(p + ((g + 4) ^ sw) * 16);
  return int8v{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// The same 32 values as fp16, in four pieces of 8 (every E4M3 value is an fp16 value).
struct Half32 {
  half8 h[4];
};
__device__ __forceinline__ Half32 to_f16(const int8v &v) {
  Half32 r;
#pragma unroll
  for (int i = 0; i < 4; i++) {
#pragma unroll
    for (int w = 0; w < 2; w++) {
      const half2v a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v[2 * i + w], 1.0f, false);
      const half2v b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v[2 * i + w], 1.0f, true);
      r.h[i][4 * w] = a[0];
      r.h[i][4 * w + 1] = a[1];
      r.h[i][4 * w + 2] = b[0];
      r.h[i][4 * w + 3] = b[1];
    }
  }
  return r;
}

// The whole contraction of one tile.  Scales of a stage: [0, BQ) of the Q rows, from kScaleP one
// per half of P.
template <class T, bool ONCE, bool WHOLE, int ACTIVE>
__device__ __forceinline__ void contract(Source<T> &src, uint8_t *lds, int steps, float4v (&acc)[T::TP][T::TQ]) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = threadIdx.x & 63, g = lane / 16, r = lane % 16;
  const int wp = wave % T::WP, wq = wave / T::WP;
  const uint32_t lds0 = lds_address(lds);
#pragma unroll
  for (int i = 0; i < T::TP; i++)
#pragma unroll
    for (int j = 0; j < T::TQ; j++) acc[i][j] = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < T::STAGES - 1; s++) issue<T, ONCE>(src, lds0 + s * T::kStage, wave, s, steps);
  int slot = 0;
  for (int kb = 0; kb < steps; kb++) {
    arrive<T::kCopies *(T::STAGES - 2)>();
    const int next = slot == 0 ? T::STAGES - 1 : slot - 1;
    issue<T, ONCE>(src, lds0 + next * T::kStage, wave, kb + T::STAGES - 1, steps);
    const uint8_t *P = lds + slot * T::kStage, *Q = P + T::kBytesP;
    const float *S = reinterpret_cast<const float *>(Q + T::kBytesQ);
    std::conditional_t<WHOLE, Half32, int8v> q[ACTIVE];
    float sq[ACTIVE];
#pragma unroll
    for (int j = 0; j < ACTIVE; j++) {
      const int row = (wq * T::TQ + j) * 16 + r;
      if constexpr (WHOLE) q[j] = to_f16(fragment(Q, row, g));
      else q[j] = fragment(Q, row, g);
      sq[j] = S[row];
    }
#pragma unroll
    for (int i = 0; i < T::TP; i++) {
      const int row0 = (i / T::kPerHalf) * kFp8Block + wp * (kFp8Block / T::WP) + (i % T::kPerHalf) * 16;
      const int8v p = fragment(P, row0 + r, g);
      const float sp = S[T::kScaleP + i / T::kPerHalf];
      float4v v[ACTIVE];
      if constexpr (WHOLE) {
        const Half32 ph = to_f16(p);
#pragma unroll
        for (int j = 0; j < ACTIVE; j++) v[j] = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 4; h++)
#pragma unroll
          for (int j = 0; j < ACTIVE; j++) v[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ph.h[h], q[j].h[h], v[j], 0, 0, 0);
      } else {
#pragma unroll
        for (int j = 0; j < ACTIVE; j++)
          v[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(p, q[j], float4v{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < ACTIVE; j++) {
        const float s = sp * sq[j];
#pragma unroll
        for (int c = 0; c < 4; c++) acc[i][j][c] = fmaf(v[j][c], s, acc[i][j][c]);
      }
    }
    slot = slot == T::STAGES - 1 ? 0 : slot + 1;
  }
  arrive<0>();   // the copies past the end (zeros) are in before the buffers serve anything else
}

// ---- the large tile -------------------------------------------------------------------------
//
// 256 x 256 results in eight waves, two on each SIMD, each 128 P rows (64 of either half) by 64 Q
// rows.  A step (one scale block) has four phases per wave: read half 0 of P and all of Q from LDS
// into registers, 16 MFMAs, read half 1 of P, 16 MFMAs.  Two workgroup barriers a step, after an
// MFMA phase of waves 0-3 and a reading phase of waves 4-7, keep the two halves of the workgroup
// one phase apart, so on every SIMD one wave's matrix instructions run while the other reads.  A
// stage has two parts, X (Q, half 0 of P) and Y (half 1 of P), whose buffers are free again at
// the next barrier after they were read: part X of step b + 2 is copied in the reading phase of
// half 1 of step b, part Y of step b + 1 in that of half 0, about six phases before they are read.
//
// A step's scales are one float in each of 256 rows, as many requests to L2 as half the codes;
// four steps' scales of a row are one 16-byte copy instead, issued with part X of every fourth
// step.  The last group of a row that has no whole number of groups starts at its fourth scale
// from the end (a large tile has at least four steps).
//
// Measured, one group of 8192 rows, N = K = 8192 (1.1 TFLOP): 472 us, 2.3 PFLOP/s (128 x 128 tiles
// 680 us).  What bounds it: the matrix cores are busy for 56 % of the cycles at a clock that this
// load holds at 1.9 GHz (the same launch on zeros takes 420 us; a loop of these MFMAs and fmas
// alone runs at 3.5 PFLOP/s on random data, 4.5 on constants); writing D costs 25 us, the copies
// from L2 some 30.
constexpr int kLag = 4;   // an MFMA's result is read that many MFMAs later (3: the same within 1 %; 2: 3 % slower)

template <class T, bool ONCE>
__device__ __forceinline__ void issue_x(Source<T> &src, uint32_t lds0, int wave, int kb, int steps) {
  const uint32_t lds = lds0 + (kb & 1) * (T::kBytesP + T::kBytesQ), scales = lds0 + 2 * (T::kBytesP + T::kBytesQ);
  const bool last = kb == steps - 1 && src.last_pieces < 8;
  if (kb >= steps) src.p.bytes = src.q.bytes = 0;
  issue_q<T>(src, lds, wave, last);
  issue_p<T, ONCE, 0, T::kCopiesP / 2>(src, lds, wave, last);
  // (kOob plus an offset inside a row of scales is out of range too)
  copy16_if((kb & 3) == 0 && kb < steps && wave * kWave < T::kScaleRows, src.s,
            scales + (kb >> 2 & 1) * T::kScaleGroup + wave * kWave * 16, src.vs + 4 * min(kb, steps - 4));
  src.q.base += src.step_q;
}
template <class T, bool ONCE>
__device__ __forceinline__ void issue_y(Source<T> &src, uint32_t lds0, int wave, int kb, int steps) {
  if (kb >= steps) src.p.bytes = 0;
  issue_p<T, ONCE, T::kCopiesP / 2, T::kCopiesP>(src, lds0 + (kb & 1) * (T::kBytesP + T::kBytesQ), wave,
                                          kb == steps - 1 && src.last_pieces < 8);
  src.p.base += src.step_p;
}

template <class T>
__device__ __forceinline__ void mfma_half(const int8v (&p)[T::kPerHalf], const int8v (&q)[T::TQ], const float (&s)[T::TQ],
                                          float4v (*acc)[T::TQ]) {
  constexpr int kAll = T::kPerHalf * T::TQ;
  float4v t[kLag + 1];
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int n = 0; n < kAll + kLag; n++) {
    if (n < kAll)
      t[n % (kLag + 1)] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(p[n / T::TQ], q[n % T::TQ],
                                                                           float4v{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
    if (n >= kLag) {
      const int m = n - kLag;
#pragma unroll
      for (int c = 0; c < 4; c++)
        acc[m / T::TQ][m % T::TQ][c] = fmaf(t[m % (kLag + 1)][c], s[m % T::TQ], acc[m / T::TQ][m % T::TQ][c]);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

// Copies that may be under way at a barrier: the two parts issued after the one it waits for.  A
// group's scales, the last copy of its part X, are not counted, so a barrier with one of them
// under way waits for one copy more than it has to.
template <class T>
constexpr int kLaterCopies = T::kCopiesQ + T::kCopiesP;

// BEHIND: waves 4-7, whose barriers follow their reading phases.
template <class T, bool ONCE, bool BEHIND>
__device__ __forceinline__ void large_loop(Source<T> &src, uint8_t *lds, int steps, int wave, float4v (&acc)[T::TP][T::TQ]) {
  constexpr int kLater = kLaterCopies<T>;
  const int lane = threadIdx.x & 63, g = lane / 16, r = lane % 16;
  const int wp = wave % T::WP, wq = wave / T::WP;
  const uint32_t lds0 = lds_address(lds);
  for (int kb = 0; kb < steps; kb++) {
    const uint8_t *P = lds + (kb & 1) * (T::kBytesP + T::kBytesQ), *Q = P + T::kBytesP;
    const float *S = reinterpret_cast<const float *>(lds + 2 * (T::kBytesP + T::kBytesQ) + (kb >> 2 & 1) * T::kScaleGroup) +
                     (kb - min(kb & ~3, steps - 4));
    int8v p[T::kPerHalf], q[T::TQ];
    float s[2][T::TQ];
    issue_y<T, ONCE>(src, lds0, wave, kb + 1, steps);
#pragma unroll
    for (int j = 0; j < T::TQ; j++) q[j] = fragment(Q, (wq * T::TQ + j) * 16 + r, g);
#pragma unroll
    for (int i = 0; i < T::kPerHalf; i++) p[i] = fragment(P, wp * (kFp8Block / T::WP) + i * 16 + r, g);
#pragma unroll
    for (int j = 0; j < T::TQ; j++) {
      const float sq = S[4 * ((wq * T::TQ + j) * 16 + r)];
      s[0][j] = sq * S[4 * T::kScaleP];
      s[1][j] = sq * S[4 * (T::kScaleP + 1)];
    }
    if (BEHIND) arrive<kLater>();    // part Y of this step is there
    mfma_half<T>(p, q, s[0], acc);
    if (!BEHIND) arrive<kLater>();
    issue_x<T, ONCE>(src, lds0, wave, kb + 2, steps);
#pragma unroll
    for (int i = 0; i < T::kPerHalf; i++) p[i] = fragment(P, kFp8Block + wp * (kFp8Block / T::WP) + i * 16 + r, g);
    if (BEHIND) arrive<kLater>();    // part X of the next step is there
    mfma_half<T>(p, q, s[1], acc + T::kPerHalf);
    if (!BEHIND) arrive<kLater>();
  }
}

// `rows`: rows of Q in use; a wave whose 64 rows are all behind them only copies.
template <class T, bool ONCE>
__device__ __forceinline__ void contract_large(Source<T> &src, uint8_t *lds, int steps, int rows, float4v (&acc)[T::TP][T::TQ]) {
  static_assert(T::kWaves == 8 && T::WP == 2 && T::kHalves == 2, "the schedule above");
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t lds0 = lds_address(lds);
#pragma unroll
  for (int i = 0; i < T::TP; i++)
#pragma unroll
    for (int j = 0; j < T::TQ; j++) acc[i][j] = float4v{0.f, 0.f, 0.f, 0.f};
  issue_x<T, ONCE>(src, lds0, wave, 0, steps);
  issue_y<T, ONCE>(src, lds0, wave, 0, steps);
  issue_x<T, ONCE>(src, lds0, wave, 1, steps);
  constexpr int kLater = kLaterCopies<T>;
  arrive<kLater>();                  // part X of step 0 is there
  if (wave / T::WP * T::TQ * 16 >= rows) {
    for (int kb = 0; kb < steps; kb++) {
      issue_y<T, ONCE>(src, lds0, wave, kb + 1, steps);
      arrive<kLater>();
      issue_x<T, ONCE>(src, lds0, wave, kb + 2, steps);
      arrive<kLater>();
    }
  } else if (wave >= T::kWaves / 2) {
    large_loop<T, ONCE, true>(src, lds, steps, wave, acc);
  } else {
    large_loop<T, ONCE, false>(src, lds, steps, wave, acc);
  }
  arrive<0>();
}

// The item of this workgroup: group g, its chunk of `size` rows and n tile.
__device__ __forceinline__ bool find_item(const GemmParams &P, int size, groups::Chunk &g, int &chunk, int &nt) {
  int64_t w = 0;
  int i;
  auto index = [&](int total) {
    return item_of(blockIdx.x, static_cast<int64_t>(total) * P.n_tiles, w) ? static_cast<int>(w / P.n_tiles) : -1;
  };
  if (!groups::find_chunk_of_all(P.offsets, P.E, P.R, size, index, i, g)) return false;
  place_in_band(static_cast<int>(w - static_cast<int64_t>(i - g.index) * P.n_tiles), g.total, P.n_tiles, chunk, nt);
  return true;
}

// Row of A that permuted row p reads.
__device__ __forceinline__ int64_t row_of_a(const GemmParams &P, int p) {
  const int64_t a = P.A_rows[p];
  return a < 0 ? 0 : (a >= P.rows_A ? P.rows_A - 1 : a);
}

// One tile: up to BQ rows from `first` of group g, n tile `nt`.  WHOLE: fp16 matrix core.
template <class T, Mode MODE, bool WHOLE>
__device__ __forceinline__ void gemm_tile(const GemmParams &P, uint8_t *lds, const groups::Chunk &g, int first, int count, int nt) {
  const int half_n = P.N / 2;                       // SWIGLU: gate rows, then up rows
  const int n0 = nt * (MODE == kSwigluFp8 ? kFp8Block : T::BP);

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = threadIdx.x & 63, lg = lane / 16, r = lane % 16;
  Source<T> src;
  src.last_pieces = P.K % kFp8Block ? P.K % kFp8Block / 16 : 8;
  src.step_p = src.step_q = kFp8Block;
  src.step_s = 4;
  src.p.base = reinterpret_cast<uint64_t>(P.B) + static_cast<uint64_t>(g.group) * P.N * P.K;
  src.p.bytes = static_cast<uint32_t>(P.N) * P.K;
#pragma unroll
  for (int j = 0; j < T::kCopiesP; j++) {
    int row, piece;
    copy_place(copy_row_p<T>(wave, j), row, piece);
    int n = n0 + row;
    if (MODE == kSwigluFp8) n = n0 + row % kFp8Block + row / kFp8Block * half_n;   // half_n % 128 == 0
    src.vp[j] = n < P.N ? static_cast<uint32_t>(n) * P.K + piece * 16 : kOob;
  }
  // token rows: gathered from all of A, or the group's own
  const bool gather = P.A_rows != nullptr;
  src.q.base = reinterpret_cast<uint64_t>(P.A) + (gather ? 0 : static_cast<uint64_t>(first) * P.K);
  src.q.bytes = static_cast<uint32_t>((gather ? P.rows_A : count) * P.K);
  auto row_of = [&](int row) -> int64_t { return gather ? row_of_a(P, first + row) : row; };
#pragma unroll
  for (int j = 0; j < T::kCopiesQ; j++) {
    int row, piece;
    copy_place((wave * T::kCopiesQ + j) * 8, row, piece);
    src.vq[j] = row < count ? static_cast<uint32_t>(row_of(row)) * P.K + piece * 16 : kOob;
  }
  // this wave's scales of a stage: 64 of [Q rows, then the halves of P]; a wave has one kind
  static_assert(T::BQ % kWave == 0 || T::BQ < kWave, "a wave copies scales of one operand");
  const int kb_n = (P.K + kFp8Block - 1) / kFp8Block, nb_n = (P.N + kFp8Block - 1) / kFp8Block;
  const int slot0 = wave * kWave;
  src.vs = kOob;
  if (slot0 < T::BQ) {
    src.s.base = reinterpret_cast<uint64_t>(P.A_sf) + (gather ? 0 : static_cast<uint64_t>(first) * kb_n * 4);
    src.s.bytes = static_cast<uint32_t>((gather ? P.rows_A : count) * kb_n * 4);
    if (slot0 + lane < count) src.vs = static_cast<uint32_t>(row_of(slot0 + lane)) * kb_n * 4;
  } else {
    src.s.base = reinterpret_cast<uint64_t>(P.B_sf) + static_cast<uint64_t>(g.group) * nb_n * kb_n * 4;
    src.s.bytes = static_cast<uint32_t>(nb_n) * kb_n * 4;
    const int h = slot0 + lane - T::kScaleP;
    if (h >= 0 && h < T::kHalves) {
      const int nb = MODE == kSwigluFp8 ? (n0 + h * half_n) / kFp8Block : n0 / kFp8Block + h;
      if (nb < nb_n) src.vs = static_cast<uint32_t>(nb) * kb_n * 4;
    }
  }

  src.s = uniform(src.s);

  float4v acc[T::TP][T::TQ];
  // the weights of a group of one chunk are read by this workgroup alone (measured at 32 rows per
  // expert, 805 MB of weights: 130 us past the caches, 138 us through them; with two chunks, whose
  // second one finds them in L2, 35 us against 24 us for 77 MB)
  const bool once = g.total == 1 && P.stream_weights;
  if constexpr (T::kLarge) {
    static_assert(!WHOLE, "the large tile has the FP8 form alone");
    if (once) contract_large<T, true>(src, lds, kb_n, count, acc);
    else contract_large<T, false>(src, lds, kb_n, count, acc);
  } else {
    // Q tiles behind the last row are left out
    auto run = [&](auto active) {
      constexpr int kActive = decltype(active)::value;
      if (once) contract<T, true, WHOLE, kActive>(src, lds, kb_n, acc);
      else contract<T, false, WHOLE, kActive>(src, lds, kb_n, acc);
    };
    const int active = T::WQ == 1 ? (count + 15) / 16 : T::TQ;
    if (T::TQ >= 4 && active == 3) run(std::integral_constant<int, T::TQ >= 4 ? 3 : T::TQ>());
    else if (T::TQ >= 4 && active == 2) run(std::integral_constant<int, T::TQ >= 4 ? 2 : T::TQ>());
    else if (T::TQ >= 2 && active == 1) run(std::integral_constant<int, T::TQ >= 2 ? 1 : T::TQ>());
    else run(std::integral_constant<int, T::TQ>());
  }

  const int wp = wave % T::WP, wq = wave / T::WP;
  if (MODE == kNone) {
    // each wave turns its tile around in LDS, 16 rows (or a few times 16, to have a piece for every
    // lane) at a time, and stores whole pieces of rows (straight from the MFMA layout they would be
    // 32 bytes long: 490 us against 480 us for the large tile's 1.1 TFLOP)
    constexpr int kCols = kFp8Block / T::WP, kRow = T::kHalves * kCols * 2, kStride = kRow + 16;   // bytes
    constexpr int kTurn = kRow < kWave ? kWave / kRow : 1;   // 16-row tiles turned together
    constexpr int kPieces = kTurn * 16 * kRow / 16 / kWave;
    static_assert(T::TQ % kTurn == 0 && kPieces * kWave == kTurn * kRow && T::kWaves * kTurn * 16 * kStride <= T::kLds, "staging");
    uint8_t *mine = lds + wave * kTurn * 16 * kStride;
    uint16_t *D = static_cast<uint16_t *>(P.D);
#pragma unroll
    for (int j0 = 0; j0 < T::TQ; j0 += kTurn) {
#pragma unroll
      for (int j = 0; j < kTurn; j++)
#pragma unroll
        for (int ti = 0; ti < T::TP; ti++)
          *reinterpret_cast<uint2 *>(mine + (j * 16 + r) * kStride + ti * 32 + lg * 8) = bf16x4(acc[ti][j0 + j]);
      wave_order();
#pragma unroll
      for (int c = 0; c < kPieces; c++) {
        const int at = c * kWave + lane, row = at / (kRow / 16), col = at % (kRow / 16) * 8;   // col: of the wave's columns
        const int t = (wq * T::TQ + j0) * 16 + row;
        const int n = n0 + col / kCols * kFp8Block + wp * kCols + col % kCols;
        const uint4 v = *reinterpret_cast<const uint4 *>(mine + row * kStride + col * 2);
        if (t >= count || n >= P.N) continue;
        store16<T::kLarge>(D + static_cast<int64_t>(first + t) * P.N + n, v);
      }
      wave_order();
    }
  } else {
    // act = silu(gate) up in binary32 (hardware exp2 and reciprocal); its maximum over the 128
    // columns: a lane's own, the 4 lane groups', then the WP waves' through LDS
    uint32_t *red = reinterpret_cast<uint32_t *>(lds);   // [WP][BQ]
    uint32_t m[T::TQ];
#pragma unroll
    for (int j = 0; j < T::TQ; j++) {
      m[j] = 0;
#pragma unroll
      for (int ti = 0; ti < T::kPerHalf; ti++) {
#pragma unroll
        for (int c = 0; c < 4; c++) {
          const float gate = acc[ti][j][c], up = acc[(T::kHalves - 1) * T::kPerHalf + ti][j][c];
          const float act = gate * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(gate * -1.4426950408889634f)) * up;
          acc[ti][j][c] = act;
          m[j] = max(m[j], abs_bits(act));
        }
      }
      m[j] = max(m[j], static_cast<uint32_t>(__shfl_xor(static_cast<int>(m[j]), 16, kWave)));
      m[j] = max(m[j], static_cast<uint32_t>(__shfl_xor(static_cast<int>(m[j]), 32, kWave)));
      if (lg == 0) red[wp * T::BQ + (wq * T::TQ + j) * 16 + r] = m[j];
    }
    __syncthreads();
    uint8_t *D = static_cast<uint8_t *>(P.D);
#pragma unroll
    for (int j = 0; j < T::TQ; j++) {
      const int t = (wq * T::TQ + j) * 16 + r;
      if (t >= count) continue;
      uint32_t mm = 0;
#pragma unroll
      for (int k = 0; k < T::WP; k++) mm = max(mm, red[k * T::BQ + t]);
      const Fp8Block s = fp8_block(mm);
      const int64_t p = first + t;
      if (wp == 0 && lg == 0) P.D_sf[p * (half_n / kFp8Block) + nt] = s.scale;
#pragma unroll
      for (int ti = 0; ti < T::kPerHalf; ti++) {
        const int n = n0 + wp * (kFp8Block / T::WP) + ti * 16 + 4 * lg;
        *reinterpret_cast<uint32_t *>(D + p * half_n + n) =
            fp8_quantize4(acc[ti][j][0], acc[ti][j][1], acc[ti][j][2], acc[ti][j][3], s);
      }
    }
  }
}

template <class T, Mode MODE, bool WHOLE, int TILES>
__global__ __launch_bounds__(T::kThreadsT) void gemm_kernel(const GemmParams P) {
  __shared__ __align__(1024) uint8_t lds[T::kLds];
  groups::Chunk g;
  int chunk, nt;
  if (!find_item(P, T::BQ, g, chunk, nt)) return;
  const int first = g.lo + chunk * T::BQ, count = min(T::BQ, g.hi - first);
  gemm_tile<T, MODE, WHOLE>(P, lds, g, first, count, TILES * nt);
#pragma unroll 1
  for (int i = 1; i < TILES; i++) {
    if ((TILES * nt + i) * T::BP >= P.N) return;
    __syncthreads();   // the tile before is out of LDS
    gemm_tile<T, MODE, WHOLE>(P, lds, g, first, count, TILES * nt + i);
  }
}

// ---- few items ------------------------------------------------------------------------------
//
// Where there are few rows and columns (a single token: k experts' weights, each a few hundred
// rows), the contraction is dealt to the eight waves of a workgroup: wave w takes the
// scale blocks w, w + 8, ... of a tile of 32 columns (16 where even those are one round: 7.9 us against
// 8.4 for the token below) and 16 rows, with a ring of its own and no barrier before the end, and the
// eight partial tiles are added in order through LDS.  Bound by latency: the item lookup, about two
// round trips to HBM and the sum.  One token, eight experts of 512 x 6144: 7.9 us (28 us in 64 x 128
// tiles).
template <int Q_, int P_, int WAVES_, int STAGES_>
struct Split {
  static constexpr int Q = Q_, P = P_, WAVES = WAVES_, STAGES = STAGES_;
  static constexpr int TQ = Q / 16, TP = P / 16;
  static constexpr int kCopies = (P + Q) / 8 + 2;
  static constexpr int kStage = (P + Q) * kFp8Block + 2 * kWave * 4;
  static constexpr int kLds = WAVES * STAGES * kStage;
  static_assert(Q <= kWave && TP * TQ * kWave * 16 <= STAGES * kStage, "a wave's scales and partial tiles fit");
};

template <class T>
__global__ __launch_bounds__(T::WAVES *kWave) void split_kernel(const GemmParams P) {
  __shared__ __align__(1024) uint8_t lds[T::kLds];
  groups::Chunk g;
  int chunk, nt;
  if (!find_item(P, T::Q, g, chunk, nt)) return;
  const int first = g.lo + chunk * T::Q, count = min(T::Q, g.hi - first), n0 = nt * T::P;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = threadIdx.x & 63, lg = lane / 16, r = lane % 16;
  const int kb_n = (P.K + kFp8Block - 1) / kFp8Block, nb_n = (P.N + kFp8Block - 1) / kFp8Block;
  const bool gather = P.A_rows != nullptr;
  auto row_of = [&](int row) -> int64_t { return gather ? row_of_a(P, first + row) : row; };
  const Buf bp = {reinterpret_cast<uint64_t>(P.B) + static_cast<uint64_t>(g.group) * P.N * P.K, static_cast<uint32_t>(P.N) * P.K};
  const Buf bq = {reinterpret_cast<uint64_t>(P.A) + (gather ? 0 : static_cast<uint64_t>(first) * P.K),
                  static_cast<uint32_t>((gather ? P.rows_A : count) * P.K)};
  const Buf bsq = {reinterpret_cast<uint64_t>(P.A_sf) + (gather ? 0 : static_cast<uint64_t>(first) * kb_n * 4),
                   static_cast<uint32_t>((gather ? P.rows_A : count) * kb_n * 4)};
  const Buf bsp = {reinterpret_cast<uint64_t>(P.B_sf) + (static_cast<uint64_t>(g.group) * nb_n + n0 / kFp8Block) * kb_n * 4,
                   static_cast<uint32_t>(kb_n) * 4};
  uint32_t vp[T::P / 8], vq[T::Q / 8];
#pragma unroll
  for (int j = 0; j < T::P / 8; j++) {
    int row, piece;
    copy_place(8 * j, row, piece);
    vp[j] = n0 + row < P.N ? static_cast<uint32_t>(n0 + row) * P.K + piece * 16 : kOob;
  }
#pragma unroll
  for (int j = 0; j < T::Q / 8; j++) {
    int row, piece;
    copy_place(8 * j, row, piece);
    vq[j] = row < count ? static_cast<uint32_t>(row_of(row)) * P.K + piece * 16 : kOob;
  }
  const uint32_t vsq = lane < count ? static_cast<uint32_t>(row_of(lane)) * kb_n * 4 : kOob;
  const int last_pieces = P.K % kFp8Block ? P.K % kFp8Block / 16 : 8;
  uint8_t *ring = lds + wave * T::STAGES * T::kStage;
  const uint32_t ring0 = lds_address(ring);
  // the wave's i-th scale block into buffer `slot`
  auto issue_block = [&](int i, int slot) {
    const int kb = wave + T::WAVES * i;
    const uint32_t at = ring0 + slot * T::kStage;
    const bool past = kb >= kb_n, last = kb == kb_n - 1;
#pragma unroll
    for (int j = 0; j < T::P / 8; j++) {
      int row, piece;
      copy_place(8 * j, row, piece);
      copy16(bp, at + j * 1024, past || (last && piece >= last_pieces) ? kOob : vp[j] + kb * kFp8Block);
    }
#pragma unroll
    for (int j = 0; j < T::Q / 8; j++) {
      int row, piece;
      copy_place(8 * j, row, piece);
      copy16(bq, at + T::P * kFp8Block + j * 1024, past || (last && piece >= last_pieces) ? kOob : vq[j] + kb * kFp8Block);
    }
    copy4(bsq, at + (T::P + T::Q) * kFp8Block, past ? kOob : vsq + kb * 4);
    copy4(bsp, at + (T::P + T::Q) * kFp8Block + kWave * 4, past || lane != 0 ? kOob : kb * 4);
  };
  float4v acc[T::TP][T::TQ] = {};
#pragma unroll
  for (int i = 0; i < T::STAGES; i++) issue_block(i, i);
  int slot = 0;
  for (int i = 0; wave + T::WAVES * i < kb_n; i++) {
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(T::kCopies * (T::STAGES - 1)) : "memory");
    const uint8_t *S = ring + slot * T::kStage;
    const float *sc = reinterpret_cast<const float *>(S + (T::P + T::Q) * kFp8Block);
    int8v q[T::TQ], p[T::TP];
    float s[T::TQ];
#pragma unroll
    for (int j = 0; j < T::TQ; j++) {
      q[j] = fragment(S + T::P * kFp8Block, j * 16 + r, lg);
      s[j] = sc[j * 16 + r] * sc[kWave];
    }
#pragma unroll
    for (int t = 0; t < T::TP; t++) p[t] = fragment(S, t * 16 + r, lg);
    asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");   // the buffer is read before it is filled again
    issue_block(i + T::STAGES, slot);
#pragma unroll
    for (int t = 0; t < T::TP; t++)
#pragma unroll
      for (int j = 0; j < T::TQ; j++) {
        const float4v v =
            __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(p[t], q[j], float4v{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
#pragma unroll
        for (int c = 0; c < 4; c++) acc[t][j][c] = fmaf(v[c], s[j], acc[t][j][c]);
      }
    slot = slot == T::STAGES - 1 ? 0 : slot + 1;
  }
  arrive<0>();
  float4v *part = reinterpret_cast<float4v *>(lds);   // [wave][tile][lane]
  constexpr int kTiles = T::TP * T::TQ;
#pragma unroll
  for (int t = 0; t < kTiles; t++) part[(wave * kTiles + t) * kWave + lane] = acc[t / T::TQ][t % T::TQ];
  __syncthreads();
  for (int t = wave; t < kTiles; t += T::WAVES) {
    float4v sum = part[t * kWave + lane];
#pragma unroll
    for (int w = 1; w < T::WAVES; w++) sum += part[(w * kTiles + t) * kWave + lane];
    const int n = n0 + t / T::TQ * 16 + 4 * lg, row = t % T::TQ * 16 + r;
    if (row < count && n < P.N)
      *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(P.D) + static_cast<int64_t>(first + row) * P.N + n) = bf16x4(sum);
  }
}

// ---- the weight gradient -----------------------------------------------------------------------
//
// A tile of D has a few steps (one per 128 tokens of its expert).  Measured, 16 experts of 512 rows, N
// 4096, K 6144, binary32 D (412 GFLOP, 1.6 GB written): 565 us (rows dealt at random, a
// fifth, nearly empty block for some experts: 587), matrix cores busy for 34 % of the cycles; 64 rows
// each: 300 us, 5.4 TB/s written.  Per step and wave 64 MFMAs (1024 cycles) stand against 128 conversions and 128
// scalings (1024), which the MFMAs hide in part only.  One pipeline through several tiles, the
// next one's first stage copied during the last step: 620 to 710 us.
struct GradTile {
  Buf p, q, s;     // this wave's stages: X codes, Y codes, scales of one of them
  int steps, last; // token blocks, tokens of the last one
  int e, n0, k0;
};

template <class T>
__device__ __forceinline__ bool grad_tile(const WgradParams &P, int wave, GradTile &t) {
  const int n_tiles = (P.N + T::BQ - 1) / T::BQ, k_tiles = (P.K + T::BP - 1) / T::BP, per = n_tiles * k_tiles;
  int64_t w;
  if (!item_of(blockIdx.x, static_cast<int64_t>(P.E) * per, w)) return false;
  t.e = static_cast<int>(w / per);
  int nt, kt;
  place_in_band(static_cast<int>(w - static_cast<int64_t>(t.e) * per), n_tiles, k_tiles, nt, kt);
  t.n0 = nt * T::BQ;
  t.k0 = kt * T::BP;
  const int b0 = groups::chunks_before(P.offsets, t.e, P.E, P.R, kFp8Block);
  int lo = __builtin_amdgcn_readfirstlane(P.offsets[t.e]), hi = __builtin_amdgcn_readfirstlane(P.offsets[t.e + 1]);
  groups::clamp_pair(lo, hi, P.R);
  t.steps = (hi - lo + kFp8Block - 1) / kFp8Block;
  t.last = hi - lo - (t.steps - 1) * kFp8Block;
  t.steps = max(0, min(t.steps, P.blocks - b0));   // offsets that are not monotone stay inside the buffers
  const bool of_q = wave * kWave < T::BQ;
  const uint32_t rows_p = min(T::BP, P.K - t.k0), rows_q = min(T::BQ, P.N - t.n0);
  t.p.base = reinterpret_cast<uint64_t>(P.X) + (static_cast<uint64_t>(b0) * P.K + t.k0) * kFp8Block;
  t.q.base = reinterpret_cast<uint64_t>(P.Y) + (static_cast<uint64_t>(b0) * P.N + t.n0) * kFp8Block;
  t.s.base = of_q ? reinterpret_cast<uint64_t>(P.Y_sf) + (static_cast<uint64_t>(b0) * P.N + t.n0) * 4
                  : reinterpret_cast<uint64_t>(P.X_sf) + (static_cast<uint64_t>(b0) * P.K + t.k0) * 4;
  t.p.bytes = rows_p * kFp8Block;
  t.q.bytes = rows_q * kFp8Block;
  t.s.bytes = 4 * (of_q ? rows_q : rows_p);
  t.p = uniform(t.p);
  t.q = uniform(t.q);
  t.s = uniform(t.s);
  return true;
}

template <class T, Mode MODE>
__global__ __launch_bounds__(T::kThreadsT) void wgrad_kernel(const WgradParams P) {
  static_assert(T::BQ % kWave == 0 && T::BQ + T::BP <= T::kThreadsT && T::STAGES == 2 && !T::kLarge, "the schedule below");
  __shared__ __align__(1024) uint8_t lds[T::kLds];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = threadIdx.x & 63, g = lane / 16, r = lane % 16;
  const int wp = wave % T::WP, wq = wave / T::WP;
  const uint32_t lds0 = lds_address(lds);
  uint32_t vp[T::kCopiesP], vq[T::kCopiesQ];
#pragma unroll
  for (int j = 0; j < T::kCopiesP; j++) {
    int row, piece;
    copy_place((wave * T::kCopiesP + j) * 8, row, piece);
    vp[j] = row * kFp8Block + piece * 16;
  }
#pragma unroll
  for (int j = 0; j < T::kCopiesQ; j++) {
    int row, piece;
    copy_place((wave * T::kCopiesQ + j) * 8, row, piece);
    vq[j] = row * kFp8Block + piece * 16;
  }
  const bool of_q = wave * kWave < T::BQ;
  const uint32_t vs = 4 * static_cast<uint32_t>(wave * kWave + lane - (of_q ? 0 : T::BQ));
  const uint32_t step_p = static_cast<uint32_t>(P.K) * kFp8Block, step_q = static_cast<uint32_t>(P.N) * kFp8Block;
  const uint32_t step_s = uniform(4u * static_cast<uint32_t>(of_q ? P.N : P.K));
  GradTile t;
  if (!grad_tile<T>(P, wave, t)) return;
  auto issue_stage = [&](int kb) {   // past the last one: nothing
    const uint32_t at = lds0 + (kb & 1) * T::kStage;
    if (kb >= t.steps) t.p.bytes = t.q.bytes = t.s.bytes = 0;
#pragma unroll
    for (int j = 0; j < T::kCopiesP; j++) copy16(t.p, at + (wave * T::kCopiesP + j) * 8 * kFp8Block, vp[j]);
#pragma unroll
    for (int j = 0; j < T::kCopiesQ; j++) copy16(t.q, at + T::kBytesP + (wave * T::kCopiesQ + j) * 8 * kFp8Block, vq[j]);
    copy4(t.s, at + T::kBytesP + T::kBytesQ + wave * kWave * 4, vs);
    t.p.base += step_p;
    t.q.base += step_q;
    t.s.base += step_s;
  };
  float4v acc[T::TP][T::TQ];
#pragma unroll
  for (int i = 0; i < T::TP; i++)
#pragma unroll
    for (int j = 0; j < T::TQ; j++) acc[i][j] = float4v{0.f, 0.f, 0.f, 0.f};
  issue_stage(0);
  // One token block.  kPieces 2: the block has up to 64 tokens (pieces 0 and 1 of a lane's 32 bytes are
  // the block's first 64), so half its MFMAs and conversions would work on padding.  Measured, 16
  // experts of about 512 rows, N 4096, K 6144: 616 -> 600 us, 175 rows: 385 -> 369, 2048 rows (bf16 D):
  // 1694 -> 1659; 64 experts of 128 rows, N 1024, K 4096: 238 -> 226; 16 of 64 rows, where writing D
  // is the bound: 294 -> 300.
  auto step = [&](int kb, auto pieces) {
    constexpr int kPieces = decltype(pieces)::value;
    arrive<0>();
    issue_stage(kb + 1);
    const uint8_t *Ps = lds + (kb & 1) * T::kStage, *Qs = Ps + T::kBytesP;
    const float *S = reinterpret_cast<const float *>(Qs + T::kBytesQ);
    Half32 q[T::TQ];
    float sq[T::TQ];
#pragma unroll
    for (int j = 0; j < T::TQ; j++) {
      const int row = (wq * T::TQ + j) * 16 + r;
      q[j] = to_f16(fragment(Qs, row, g));
      sq[j] = S[row];
    }
#pragma unroll
    for (int i = 0; i < T::TP; i++) {
      const int row0 = (i / T::kPerHalf) * kFp8Block + wp * (kFp8Block / T::WP) + (i % T::kPerHalf) * 16;
      const Half32 p = to_f16(fragment(Ps, row0 + r, g));
      const float4v sp = *reinterpret_cast<const float4v *>(S + T::kScaleP + row0 + 4 * g);
      float4v v[T::TQ];
#pragma unroll
      for (int j = 0; j < T::TQ; j++) v[j] = float4v{0.f, 0.f, 0.f, 0.f};
      // piece by piece over all columns: neighbouring MFMAs do not wait for each other
#pragma unroll
      for (int h = 0; h < kPieces; h++)
#pragma unroll
        for (int j = 0; j < T::TQ; j++) v[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(p.h[h], q[j].h[h], v[j], 0, 0, 0);
#pragma unroll
      for (int j = 0; j < T::TQ; j++)
#pragma unroll
        for (int c = 0; c < 4; c++) acc[i][j][c] = fmaf(v[j][c], sp[c] * sq[j], acc[i][j][c]);
    }
  };
  for (int kb = 0; kb + 1 < t.steps; kb++) step(kb, std::integral_constant<int, 4>());
  if (t.steps > 0) {
    if (t.last <= kFp8Block / 2) step(t.steps - 1, std::integral_constant<int, 2>());
    else step(t.steps - 1, std::integral_constant<int, 4>());
  }
  arrive<0>();   // the copies past the end (zeros) are in before the buffers serve anything else
  // each wave turns 16 rows of its tile at a time in LDS and stores whole pieces of them (16 rows
  // of 64 bytes straight from the MFMA layout: 444 us against 306 us where every expert has one step)
  constexpr int kElem = MODE == kWgradF32 ? 4 : 2, kRow = T::TP * 16 * kElem, kStride = kRow + 16;   // bytes
  constexpr int kCols = kFp8Block / T::WP, kPieces = kRow / kWave, kPer = 16 / kElem;
  static_assert(kPieces >= 1 && T::kWaves * 16 * kStride <= T::kBytesP + T::kBytesQ, "staging");
  uint8_t *mine = lds + wave * 16 * kStride;
#pragma unroll
  for (int j = 0; j < T::TQ; j++) {
#pragma unroll
    for (int ti = 0; ti < T::TP; ti++) {
      uint8_t *at = mine + r * kStride + (ti * 16 + 4 * g) * kElem;
      if (MODE == kWgradF32) *reinterpret_cast<float4v *>(at) = acc[ti][j];
      else *reinterpret_cast<uint2 *>(at) = bf16x4(acc[ti][j]);
    }
    wave_order();
#pragma unroll
    for (int c = 0; c < kPieces; c++) {
      const int at = c * kWave + lane, row = at / (kRow / 16), col = at % (kRow / 16) * kPer;   // col: of the wave's columns
      const int n = t.n0 + (wq * T::TQ + j) * 16 + row;
      const int k = t.k0 + col / kCols * kFp8Block + wp * kCols + col % kCols;
      const uint4 v = *reinterpret_cast<const uint4 *>(mine + row * kStride + col * kElem);
      if (n >= P.N || k >= P.K) continue;
      store16<true>(static_cast<uint8_t *>(P.D) + ((static_cast<int64_t>(t.e) * P.N + n) * P.K + k) * kElem, v);
    }
    wave_order();
  }
}

// TILES: n tiles that a workgroup does one after the other.
template <class T, Mode MODE, bool WHOLE, int TILES = 1>
hipError_t run_gemm(GemmParams p, hipStream_t stream) {
  static_assert(MODE != kSwigluFp8 || TILES == 1, "an n tile is 128 columns of act");
  p.n_tiles = MODE == kSwigluFp8 ? p.N / 2 / kFp8Block : (p.N + TILES * T::BP - 1) / (TILES * T::BP);
  const int64_t items = groups::max_chunks(p.R, p.E, T::BQ) * p.n_tiles;
  const int64_t grid = (items + kXcds - 1) / kXcds * kXcds;
  if (grid > 0)
    hipLaunchKernelGGL((gemm_kernel<T, MODE, WHOLE, TILES>), dim3(static_cast<uint32_t>(grid)), dim3(T::kThreadsT), 0, stream, p);
  return hipGetLastError();
}

template <class T>
hipError_t run_split(GemmParams p, hipStream_t stream) {
  p.n_tiles = (p.N + T::P - 1) / T::P;
  const int64_t items = groups::max_chunks(p.R, p.E, T::Q) * p.n_tiles;
  const int64_t grid = (items + kXcds - 1) / kXcds * kXcds;
  hipLaunchKernelGGL(split_kernel<T>, dim3(static_cast<uint32_t>(grid)), dim3(T::WAVES * kWave), 0, stream, p);
  return hipGetLastError();
}

using Large = Tile<256, 256, 4, 2, 2>;
constexpr int64_t kCacheBytes = 256 << 20;   // MI355X's memory-side cache
// Fewer tiles leave CUs without one.  One group, N = K = 4096: of 1024 rows, 64 large tiles 55 us, 512
// 64-row tiles 31; of 2048, 128 large tiles 59 us, 256 128-row tiles 46.  N = K = 2048: of 4096 rows, 128
// large tiles 34 us, 512 128-row tiles 27; of 6144, 192 and 768, 36 and 39.  N 8192, K 2048: of 1024
// rows (128, 512) 34 and 27, of 2048 (256, 1024) 40 and 49.
constexpr int kManyTiles = 192;
// Rows per expert above which 64-row tiles read weights twice too often, in us of 64-row tiles and of
// large ones, rows dealt to the experts at random.  32 experts, N 4096, K 6144: mean of 32 rows 136 and
// 136; 44: 147 and 136; 64: 203 and 138.  64 experts, N = K = 2048: 44: 51 and 58; 64: 59 and 57; 80: 71
// and 60.  32 experts, N 6144, K 2048: 50: 79 and 84; 56: 86 and 84; 64: 92 and 85.  128 experts, N 1024, K
// 4096: 50: 124 and 133; 64: 124 and 134; 80: 155 and 136.  So the two meet between 32 and 70
// rows: with 44 up to 18 % are lost (the last case just above it), with 64 up to 47 % would be (the first).
constexpr int kLargeRows = 44;
// The split tiles' rings take a CU's LDS, so a second round of workgroups costs as much as the first.
// Groups of 8 rows, in us of 64-row tiles and of the split: N = K = 2048: 4 groups (256 split tiles) 9.4
// and 7.0, 6 (384) 9.4 and 9.6, 8 (512) 9.6 and 10.8.  N 2048, K 6144: 4 groups 19.0 and 11.6, 6: 19.2 and
// 17.4, 8: 19.6 and 21.0.  N 6144, K 1024: 1 group (192) 7.2 and 5.6, 4 (768) 7.3 and 14.1.  One group, N 2048, K
// 2048: of 64 rows 12.5 and 7.2, of 256 (256 tiles) 12.5 and 8.1, of 384 (384) 12.6 and 13.1.  The 16-column
// form against 32 columns, K 6144, N 512: 8 groups (256 tiles of 16 columns) 6.9 and 7.1, 10 (320) 10.8 and 7.4.
constexpr int kCus = 256;

template <class T, Mode MODE>
hipError_t run_wgrad(const WgradParams &p, hipStream_t stream) {
  const int64_t items = static_cast<int64_t>(p.E) * ((p.N + T::BQ - 1) / T::BQ) * ((p.K + T::BP - 1) / T::BP);
  const int64_t grid = (items + kXcds - 1) / kXcds * kXcds;
  hipLaunchKernelGGL((wgrad_kernel<T, MODE>), dim3(static_cast<uint32_t>(grid)), dim3(T::kThreadsT), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm(GemmParams p, bool swiglu, bool whole, hipStream_t stream) {
  const int64_t hit = p.R < p.E ? p.R : p.E;   // at most so many experts have rows
  if (hit == 0) return hipSuccess;
  const int64_t mean = p.R / hit;
  p.stream_weights = static_cast<int64_t>(p.E) * p.N * p.K > kCacheBytes / 2;
  // tiles of q rows by c columns that there can be
  auto tiles = [&](int q, int c) { return groups::max_chunks(p.R, p.E, q) * ((p.N + c - 1) / c); };
  // q rows by c columns of groups of the mean size: at most one tile for each CU
  auto one_round = [&](int q, int c) { return hit * ((mean + q - 1) / q) * ((p.N + c - 1) / c) <= kCus; };
  const bool large = mean > kLargeRows && p.K > 3 * kFp8Block && tiles(256, 256) >= kManyTiles;
  if (swiglu) {
    if (large && !whole) return run_gemm<Large, kSwigluFp8, false>(p, stream);
    // fewer rows a tile while that makes no second round, in us of 32-row and of 64-row tiles: 8 experts, N
    // 4096, K 6144, of 64 rows (256 tiles) 49 and 69, of 100 (512) 87 and 66; 32, N 1024, K 2048, of 64 rows (256)
    // 20 and 25, of 100 (512) 35 and 26; 48, of 48 rows (384) 35 and 23; up to 32 rows no difference
    if (one_round(32, 256)) return run_gemm<Tile<32, 256, 1, 4, 3>, kSwigluFp8, true>(p, stream);
    return run_gemm<Tile<64, 256, 1, 8, 3>, kSwigluFp8, true>(p, stream);
  }
  const bool middle = mean > 2 * kLargeRows && tiles(128, 128) >= kManyTiles;
  if (whole) {
    // (32 experts, N 4096, K 2048, us in 128-row and in 64-row tiles: of 64 rows 80 and 72, of 96 83 and 99, of 512 320
    // and 380; 16, N 2048, K 4096: of 96 rows 43 and 44, of 512 156 and 173)
    if (middle) return run_gemm<Tile<128, 128, 2, 2, 2>, kNone, true>(p, stream);
    return run_gemm<Tile<64, 128, 1, 4, 3>, kNone, true>(p, stream);
  }
  if (large) return run_gemm<Large, kNone, false>(p, stream);
  if (p.K >= 4 * kFp8Block) {
    if (mean > 32) {
      if (one_round(64, 32)) return run_split<Split<64, 32, 4, 3>>(p, stream);
    } else if (mean > 16) {
      if (one_round(32, 32)) return run_split<Split<32, 32, 8, 2>>(p, stream);
    } else if (one_round(16, 16)) {
      return run_split<Split<16, 16, 8, 3>>(p, stream);
    } else if (one_round(16, 32)) {
      return run_split<Split<16, 32, 8, 3>>(p, stream);
    }
  }
  if (middle) return run_gemm<Tile<128, 128, 2, 2, 2>, kNone, false>(p, stream);
  // two steps a tile: looking the item up takes as long (256 experts of 32 rows, N 6144, K 256: 119 us, one
  // tile a workgroup 136; with K 512 no difference; 32 of 64 rows, N 8192: K 128 18.0 and 19.6, K 256 22.5 and
  // 25.7; 256 of 32, N 2048, K 256: 37.1 and 37.7, K 384: 58.3 and 55.9)
  if (p.K <= 2 * kFp8Block && tiles(64, 512) >= 4 * kManyTiles) return run_gemm<Tile<64, 128, 1, 4, 2>, kNone, false, 4>(p, stream);
  if (p.K <= 4 * kFp8Block) return run_gemm<Tile<64, 128, 1, 4, 2>, kNone, false>(p, stream);
  return run_gemm<Tile<64, 128, 1, 4, 3>, kNone, false>(p, stream);
}

hipError_t launch_wgrad(const WgradParams &p, bool bf16, hipStream_t stream) {
  if (bf16) return run_wgrad<Tile<128, 128, 2, 2, 2>, kWgradBf16>(p, stream);
  return run_wgrad<Tile<128, 128, 2, 2, 2>, kWgradF32>(p, stream);
}

}  // namespace fp8
}  // namespace moe
