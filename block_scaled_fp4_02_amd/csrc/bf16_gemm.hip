// Grouped bf16 matrix products of an expert layer's training: the forward product and the input
// gradient with their epilogues (gemm_kernel, split_kernel), and the weight gradient (wgrad_kernel).
//
//   y[p, n]     = sum_k a[r, k] b[e, n, k]      or, b transposed, sum_k a[r, k] b[e, k, n]
//   gated:        g = y[p, i], u = y[p, I + i]; act = silu(g) u, with g and u kept on request
//   backward:     y = d act; dg = y u s (1 + g (1 - s)), du = y g s, s = sigmoid(g), of the kept g, u
//   dW[e, n, k] = sum_p dy[p, n] x[r, k]        over the rows p of group e
//
// The bf16 matrix core's products are whole and its sums binary32; one 16x16x32 MFMA takes 8
// consecutive elements of the contraction from each of four lane groups.  The "row" operand P
// (weight rows n; columns k of dW) gives the MFMA's rows, of which a lane holds 4 consecutive ones, so
// results are contiguous along P; the "column" operand Q (tokens; rows n of dW) gives its columns.
//
// A stage holds 64 elements of the contraction of both operands (32 in the large tile), in panels of 128
// rows or columns, copied from memory straight into LDS (16 bytes per lane, no registers).  An operand
// whose rows run along the contraction keeps 128 bytes of a row together in 8 pieces (64 in 4); row r has
// piece c at place c ^ ((r >> 1) & 7) (c ^ (-(r >> 2) & 3)), so the 16 lanes that read together, which are
// rows 0-3 and 12-15 of one lane group and 4-11 of the next, or the other way round, fall on all 64 banks
// once.  (With c ^ ((r >> 2) & 3) half of the LDS cycles of the large tile were conflicts; now 3 %.)  An
// operand whose rows run across it (b transposed, both operands of dW) keeps 256 bytes of each row of the
// stage, in 8 pairs of pieces of 16 columns, and is read through the transposing LDS load: 16 lanes read
// four rows of a pair and each gets one column's four elements.  Row k has pair c at place c ^ (k & 3 |
// (k >> 3 & 1) << 2): the eight rows that 32 lanes read together fall on all banks once.
// The copies are range-checked and what lies outside an operand arrives as zeros, in both
// operands, so nothing outside (a NaN, an infinity) meets a zero.
#include "bf16_gemm.hpp"
#include "groups.hpp"
#include "lds_tiles.hpp"

#include <type_traits>

#pragma clang fp contract(off)

namespace moe {
namespace bf16 {
namespace {

using namespace lds;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short short4v __attribute__((ext_vector_type(4)));
typedef short short8v __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) short4v lds_short4;

#define INLINED __attribute__((always_inline))

constexpr int kPanelCols = 128;      // rows or columns of an operand in a panel
constexpr int kAcross = kPanelCols * 2;          // bytes of a row across the contraction

// ---- one tile -----------------------------------------------------------------------------

// Elements of the contraction in a stage, and how an operand lies in LDS.
template <int STEP_>
struct Stage {
  static constexpr int STEP = STEP_;
  static constexpr int kRowBytes = STEP * 2;            // of a row along the contraction
  static constexpr int kPieces = kRowBytes / 16;        // in such a row
  static constexpr int kPanel = kPanelCols * kRowBytes; // bytes
  static constexpr int kCopyRows = 64 / kPieces;        // rows along, and
  static constexpr int kPanelCopies = STEP / 4;         // copies of a panel: 1 KB each, four rows across
};

// PT, QT: the operand's rows run across the contraction.
template <int BQ_, int BP_, int WQ_, int WP_, int STAGES_, bool PT_, bool QT_ = false, int STEP_ = 64>
struct Tile : Stage<STEP_> {
  using St = Stage<STEP_>;
  static constexpr int BQ = BQ_, BP = BP_, WQ = WQ_, WP = WP_, STAGES = STAGES_;
  static constexpr bool PT = PT_, QT = QT_;
  static constexpr int kWaves = WQ * WP, kThreadsT = kWaves * kWave;
  static constexpr int kHalves = BP / kPanelCols;            // panels of P
  static constexpr int kPerHalf = kPanelCols / WP / 16;      // a wave's 16-row tiles in each panel
  static constexpr int TP = kHalves * kPerHalf, TQ = BQ / WQ / 16;
  static constexpr int kCopiesP = BP / St::kCopyRows / kWaves;   // per wave and stage
  static constexpr int kCopiesQ = (BQ / St::kCopyRows + kWaves - 1) / kWaves;
  static constexpr int kCopies = kCopiesP + kCopiesQ;
  static constexpr int kBytesP = BP * St::kRowBytes, kBytesQ = kCopiesQ * kWaves * 1024;
  static constexpr int kStage = kBytesP + kBytesQ;
  static constexpr bool kLarge = BQ == 256 && BP == 256;     // contract_large
  static constexpr int kLds = STAGES * kStage;
  static_assert(BP % kPanelCols == 0 && BP / St::kCopyRows % kWaves == 0 && BQ % (16 * WQ) == 0 && kPerHalf >= 1, "tile split");
  static_assert(!QT || BQ % kPanelCols == 0, "whole panels");
  static_assert(STAGES >= 2 && kCopies * (STAGES - 1) < 64, "copies under way fit the counter");
};

// f(integral_constant 0), ..., f(integral_constant N - 1).
template <int N, class F, int I = 0>
__device__ __forceinline__ void for_constants(F f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>());
    for_constants<N, F, I + 1>(f);
  }
}

// The place of piece c of row r along the contraction among the row's pieces, or back.
template <class S>
__device__ __forceinline__ int swizzle_along(int r, int c) {
  return S::kPieces == 8 ? c ^ ((r >> 1) & 7) : c ^ (-(r >> 2) & 3);
}
// What copy number c moves in this lane.  Along: 16-byte piece `piece` of row `row` of the operand.
// Across: row `k` of the stage, columns from `col`.
template <class S>
__device__ __forceinline__ void place_along(int c, int &row, int &piece) {
  const int lane = threadIdx.x & 63;
  row = c * S::kCopyRows + lane / S::kPieces;
  piece = swizzle_along<S>(row, lane % S::kPieces);
}
__device__ __forceinline__ int swizzle_across(int k) { return (k & 3) | ((k >> 3) & 1) << 2; }
template <class S>
__device__ __forceinline__ void place_across(int c, int &k, int &col) {
  const int lane = threadIdx.x & 63;
  k = c % S::kPanelCopies * 4 + lane / 16;
  const int pair = ((lane & 15) >> 1) ^ swizzle_across(k);
  col = c / S::kPanelCopies * kPanelCols + pair * 16 + (lane & 1) * 8;
}

// Where one lane's copies of a stage come from: byte offsets of its pieces in the two buffers (kOob:
// nothing) and what the buffers advance per stage.  An operand across the contraction ends with its
// buffer (`left`: bytes of it from the stage on), so the range check drops the rows past the contraction's
// end; one along it has more rows there, and `last`, the elements of the contraction in the last stage.
template <class T>
struct Source {
  Buf p, q;
  int64_t left_p, left_q;
  uint32_t vp[T::kCopiesP], vq[T::kCopiesQ];
  uint32_t step_p, step_q;
  int last;
};

__device__ __forceinline__ uint32_t range_of(int64_t left) {
  return left <= 0 ? 0u : static_cast<uint32_t>(left < kOob ? left : static_cast<int64_t>(kOob));
}

// On to stage `kb`.
template <bool ACROSS>
__device__ __forceinline__ void advance_one(Buf &b, int64_t &left, uint32_t step, bool past) {
  b.base += step;
  if (ACROSS) {
    left -= step;
    b.bytes = range_of(left);
  } else if (past) {
    b.bytes = 0;
  }
}
template <class T>
__device__ __forceinline__ void advance_to(Source<T> &src, int kb, int steps) {
  advance_one<T::PT>(src.p, src.left_p, src.step_p, kb >= steps);
  advance_one<T::QT>(src.q, src.left_q, src.step_q, kb >= steps);
}

// This lane's offset in copy c of an operand along the contraction: nothing if that ends before its piece.
template <class S>
__device__ __forceinline__ uint32_t in_range(uint32_t voff, int c, bool is_last, int last) {
  int row, piece;
  place_along<S>(c, row, piece);
  return is_last && piece * 8 >= last ? kOob : voff;
}

// Copy number j of a wave's stage: first those of P, then those of Q.
template <class T, bool ONCE>
__device__ __forceinline__ void issue_one(const Source<T> &src, uint32_t lds, int wave, int j, bool is_last) {
  if (j < T::kCopiesP) {
    const int c = wave * T::kCopiesP + j;
    copy16<ONCE>(src.p, lds + c * 1024, T::PT ? src.vp[j] : in_range<T>(src.vp[j], c, is_last, src.last));
  } else {
    const int i = j - T::kCopiesP, c = wave * T::kCopiesQ + i;
    copy16(src.q, lds + T::kBytesP + c * 1024, T::QT ? src.vq[i] : in_range<T>(src.vq[i], c, is_last, src.last));
  }
}

// The copies of stage `kb` into the buffer at `lds`; beyond the last stage they move nothing.
template <class T, bool ONCE>
__device__ __forceinline__ void issue(Source<T> &src, uint32_t lds, int wave, int kb, int steps) {
#pragma unroll
  for (int j = 0; j < T::kCopies; j++) issue_one<T, ONCE>(src, lds, wave, j, kb == steps - 1 && src.last < T::STEP);
  advance_to<T>(src, kb + 1, steps);
}

// Elements [32 h + 8 g, + 8) of the stage, for lane group g, of row `row` of an operand along it ...
template <class S>
__device__ __forceinline__ bf16x8 along(const uint8_t *rows, int row, int h, int g) {
  return *reinterpret_cast<const bf16x8 *>(rows + row * S::kRowBytes + swizzle_along<S>(row, 4 * h + g) * 16);
}
// ... or of column r of the 16 from `tile` * 16 of an operand across it.
template <class S>
__device__ __forceinline__ bf16x8 across(const uint8_t *operand, int tile, int h, int g, int r) {
  const int k = 32 * h + 8 * g + (r >> 2);   // and k + 4, whose swizzle is the same
  const uint8_t *at = operand + tile / 8 * S::kPanel + k * kAcross + ((tile % 8) ^ ((r >> 2) | (g & 1) << 2)) * 32 + (r & 3) * 8;
  const short4v a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4 *)at);
  const short4v b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4 *)(at + 4 * kAcross));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// The wave's 16-row tile i of panel `half` of P, and its column tile j of Q.
template <class T>
__device__ __forceinline__ bf16x8 fragment_p(const uint8_t *P, int wp, int half, int i, int h, int g, int r) {
  const int tile = half * (kPanelCols / 16) + wp * T::kPerHalf + i;
  if constexpr (T::PT) return across<T>(P, tile, h, g, r);
  else return along<T>(P, tile * 16 + r, h, g);
}
// (The large tile deals its 16-row tiles to the waves in turn, so that few rows are few for every wave.)
template <class T>
__device__ __forceinline__ int tile_q(int wq, int j) { return T::kLarge ? j * T::WQ + wq : wq * T::TQ + j; }
// Row number `row` of a wave's TQ * 16 as a row of the tile.
template <class T>
__device__ __forceinline__ int row_of_tile(int wq, int row) { return tile_q<T>(wq, row / 16) * 16 + row % 16; }
template <class T>
__device__ __forceinline__ bf16x8 fragment_q(const uint8_t *Q, int wq, int j, int h, int g, int r) {
  const int tile = tile_q<T>(wq, j);
  if constexpr (T::QT) return across<T>(Q, tile, h, g, r);
  else return along<T>(Q, tile * 16 + r, h, g);
}

template <class T>
__device__ __forceinline__ void clear(float4v (&acc)[T::TP][T::TQ]) {
#pragma unroll
  for (int i = 0; i < T::TP; i++)
#pragma unroll
    for (int j = 0; j < T::TQ; j++) acc[i][j] = float4v{0.f, 0.f, 0.f, 0.f};
}

template <class T>
__device__ __forceinline__ void mfma_row(const bf16x8 &p, const bf16x8 (&q)[T::TQ], float4v (&acc)[T::TQ]) {
#pragma unroll
  for (int j = 0; j < T::TQ; j++) acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(p, q[j], acc[j], 0, 0, 0);
}

// The whole contraction of one tile of the smaller kinds; ACTIVE of the wave's TQ column tiles are in use.
template <class T, bool ONCE, int ACTIVE>
__device__ __forceinline__ void contract(Source<T> &src, uint8_t *lds, int steps, float4v (&acc)[T::TP][T::TQ]) {
  constexpr int kHalvesK = T::STEP / 32;   // MFMAs along the contraction
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = threadIdx.x & 63, g = lane / 16, r = lane % 16;
  const int wp = wave % T::WP, wq = wave / T::WP;
  const uint32_t lds0 = lds_address(lds);
  clear<T>(acc);
#pragma unroll
  for (int s = 0; s < T::STAGES - 1; s++) issue<T, ONCE>(src, lds0 + s * T::kStage, wave, s, steps);
  int slot = 0;
  for (int kb = 0; kb < steps; kb++) {
    arrive<T::kCopies *(T::STAGES - 2)>();
    const int next = slot == 0 ? T::STAGES - 1 : slot - 1;
    issue<T, ONCE>(src, lds0 + next * T::kStage, wave, kb + T::STAGES - 1, steps);
    const uint8_t *P = lds + slot * T::kStage, *Q = P + T::kBytesP;
    bf16x8 q[kHalvesK][ACTIVE];
#pragma unroll
    for (int h = 0; h < kHalvesK; h++)
#pragma unroll
      for (int j = 0; j < ACTIVE; j++) q[h][j] = fragment_q<T>(Q, wq, j, h, g, r);
#pragma unroll
    for (int i = 0; i < T::TP; i++)
#pragma unroll
      for (int h = 0; h < kHalvesK; h++) {
        const bf16x8 p = fragment_p<T>(P, wp, i / T::kPerHalf, i % T::kPerHalf, h, g, r);
#pragma unroll
        for (int j = 0; j < ACTIVE; j++) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(p, q[h][j], acc[i][j], 0, 0, 0);
      }
    slot = slot == T::STAGES - 1 ? 0 : slot + 1;
  }
  arrive<0>();   // the copies past the end (zeros) are in before the buffers serve anything else
}

// ---- the large tile -------------------------------------------------------------------------
//
// 256 x 256 results in four waves, one on each SIMD, each 128 x 128: every element that a wave reads from
// LDS then meets 128 others, and LDS has 768 cycles of work (512 of reads, 256 of copies) for the 1024
// that the matrix cores take for a stage.  A stage holds 32 elements of the contraction, 32 KB, and there
// are five of them, all of LDS: one that is read and four, 128 KB, under way, which the latency of HBM
// needs (with two stages of 64 elements, 64 KB under way, the same loop took 2.2 us for 64 elements,
// twice what the matrix cores take).  A wave's 256 accumulators are AGPRs, and it keeps the matrix core
// busy by itself: while the 64 MFMAs of one stage run, the next stage's operands are read.  One barrier a
// stage tells that the next one is there and that this one is read, so that its buffer takes the copies
// of the fifth one after it, issued between the MFMAs.
//
// Dense 8192^3 on random data 815 to 960 us (1.14 to 1.35 PFLOP/s; torch.matmul beside it 844 to 884), where
// the board's power sets the clock: on zeros 629 to 683.  A tile's start and end take about 10 us in which its
// matrix cores idle (the first copies, 128 KB of results by every CU at once), so a contraction of
// 512 leaves 36 % of the cycles to them, one of 6144 60 %.  Tiles of 128 x 256, 256 x 128 and 128 x 128, two
// to a CU, were slower for every product of that size.

// acc += p q^T, in accumulation registers.  (Of the builtin the compiler gives a wave's 256 accumulators to
// both kinds of registers and moves 580 of them in every step.)  The compiler does not know these statements as
// MFMAs and waits for no result of theirs.  Nothing in the loop reads one but the MFMA of the next stage, and SETTLE, with
// the last MFMA before a place where the loop may end, waits in the same statement: an MFMA's result is there
// after 8 wait states, and the results before it are older.  (A wait after the loop, in a statement of its own, came behind
// moves of accumulators.  This one takes 32 cycles of every two stages' 2048: dense 8192^3 785 us, 782
// without; 16 groups of 512 rows, transposed, 345 and 342.  A branch around it took longer, 790 and 354, and
// accumulators as operands of a statement after the loop are moved first.)
template <bool SETTLE>
__device__ __forceinline__ void mfma_agpr(const bf16x8 &p, const bf16x8 &q, float4v &acc) {
  if constexpr (SETTLE) asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0\n\ts_nop 7" : "+a"(acc) : "v"(p), "v"(q));
  else asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(p), "v"(q));
}

// issue(j, kb, at): copy number j (a constant) of stage kb into the buffer at LDS address `at`; locate(j, kb,
// phase): before it the address, in kPhases steps that stand between different MFMAs; prepare(kb): the
// loads that stage kb's copies need, while the stage before is issued; advance(kb): on to stage kb.  ACTIVE of a wave's
// 8 column tiles are in use.
constexpr int kPhases = 4;
template <class T, int ACTIVE, class I, class L, class R, class A>
__device__ __forceinline__ void contract_large(I issue, L locate, R prepare, A advance, const uint8_t *lds, int steps, float4v (&acc)[T::TP][T::TQ]) {
  static_assert(T::kWaves == 4 && T::TP == 8 && T::TQ == 8 && T::STEP == 32 && T::kCopies == T::TP, "the schedule above");
  constexpr int kLater = T::kCopies * (T::STAGES - 2);   // copies of the stages after the next one
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = threadIdx.x & 63, g = lane / 16, r = lane % 16;
  const int wp = wave % T::WP, wq = wave / T::WP;
  const uint32_t lds0 = lds_address(lds);
  clear<T>(acc);
#pragma unroll
  for (int i = 0; i < T::STAGES; i++) {
    prepare(i + 1);
    for_constants<T::kCopies>([&](auto j) INLINED {
      for_constants<kPhases>([&](auto phase) INLINED { locate(j, i, phase); });
      issue(j, i, lds0 + i * T::kStage);
    });
    advance(i + 1);
  }
  int slot = 0;
  bf16x8 p[2][T::TP], q[2][ACTIVE];
  // number n of the next stage's operands: P's and Q's tiles in turn
  auto read = [&](auto half, const uint8_t *stage, int n) INLINED {
    constexpr int h = decltype(half)::value;
    const int u = n / 2;
    if (n % 2 == 0) p[h][u] = fragment_p<T>(stage, wp, u / T::kPerHalf, u % T::kPerHalf, 0, g, r);
    else if (u < ACTIVE) q[h][u] = fragment_q<T>(stage + T::kBytesP, wq, u, 0, g, r);
  };
  // Stage kb, whose operands are in p[h] and q[h].  A wave issues an instruction in four cycles and an MFMA
  // takes sixteen, so what stands between two of them is at most a read or a copy.
  auto stage_of = [&](auto half, int kb) INLINED {
    constexpr int h = decltype(half)::value;
    arrive<kLater>();                // the next stage is there, and no wave reads this one any more
    prepare(kb + T::STAGES + 1);
    const int next = slot == T::STAGES - 1 ? 0 : slot + 1;
    for_constants<T::TP>([&](auto row) INLINED {
      constexpr int i = decltype(row)::value;
      constexpr bool kSettle = h == 1 && i == T::TP - 1;   // the loop ends behind its second stage
#pragma unroll
      for (int j = 0; j < ACTIVE; j++) {
        if (kSettle && j == ACTIVE - 1) mfma_agpr<kSettle>(p[h][i], q[h][j], acc[i][j]);
        else mfma_agpr<false>(p[h][i], q[h][j], acc[i][j]);
        // (past the end: zeros)
        constexpr int kReads = 4, kPer = ACTIVE >= 8 ? 1 : ACTIVE >= 4 ? 2 : 4;   // reads of a row of MFMAs, after one of them
        if (i < 4 && j >= 1 && (j - 1) * kPer < kReads) {
#pragma unroll
          for (int n = 0; n < kPer; n++) read(std::integral_constant<int, 1 - h>(), lds + next * T::kStage, i * kReads + (j - 1) * kPer + n);
        }
        // P's copies, whose addresses may take work, beside the rows of MFMAs that have no reads
        constexpr std::integral_constant<int, (i + T::kCopiesQ) % T::kCopies> copy;
        for_constants<kPhases>([&](auto phase) INLINED {
          if (j == (ACTIVE > 4 ? 2 + decltype(phase)::value : ACTIVE - 1)) locate(copy, kb + T::STAGES, phase);
        });
        if (j == (ACTIVE > 4 ? 6 : ACTIVE - 1)) issue(copy, kb + T::STAGES, lds0 + slot * T::kStage);
        __builtin_amdgcn_sched_barrier(0);
      }
    });
    advance(kb + T::STAGES + 1);
    slot = next;
  };
  arrive<kLater + T::kCopies>();     // stage 0 is there
#pragma unroll
  for (int i = 0; i < 2 * T::TP; i++) read(std::integral_constant<int, 0>(), lds, i);
  for (int kb = 0; kb < steps; kb += 2) {
    stage_of(std::integral_constant<int, 0>(), kb);
    stage_of(std::integral_constant<int, 1>(), kb + 1);   // (an odd number of stages: one of zeros)
  }
  arrive<0>();
}

// run(ACTIVE) for `rows` rows of Q in use.  The last chunk of a group of, say, 540 rows has 28: 2 of a
// wave's 8 tiles.
template <class T, class F>
__device__ __forceinline__ void with_active(int rows, F run) {
  const int tiles = (rows + 16 * T::WQ - 1) / (16 * T::WQ);
  if (tiles > 4) run(std::integral_constant<int, 8>());
  else if (tiles > 2) run(std::integral_constant<int, 4>());
  else run(std::integral_constant<int, 2>());
}

// ---- results --------------------------------------------------------------------------------

// Rounded to nearest even by the hardware's conversion, two at a time (by integer operations a large
// tile's results took 5 us).
__device__ __forceinline__ uint2 rounded4(const float4v &v) {
  typedef __bf16 bf16x4v __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(uint2, __builtin_convertvector(v, bf16x4v));
}

__device__ __forceinline__ float sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.4426950408889634f));
}

// Each wave turns 16 rows of its results at a time around in LDS (or a few times 16, to have a piece
// for every lane), NT tiles of P wide, and hands whole 16-byte pieces of them to store(row of the
// wave's Q rows, column of its NT * 16, piece).
template <class T, int NT, class V, class S>
__device__ __forceinline__ void turn(uint8_t *lds, V value, S store) {
  constexpr int kRow = NT * 32, kStride = kRow + 16;   // bytes
  constexpr int kTurn = kRow < kWave ? kWave / kRow : 1;
  constexpr int kPieces = kTurn * kRow / kWave;
  static_assert(T::TQ % kTurn == 0 && kPieces * kWave == kTurn * kRow && T::kWaves * kTurn * 16 * kStride <= T::kLds, "staging");
  const int lane = threadIdx.x & 63, lg = lane / 16, r = lane % 16;
  uint8_t *mine = lds + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave) * kTurn * 16 * kStride;
#pragma unroll
  for (int j0 = 0; j0 < T::TQ; j0 += kTurn) {
#pragma unroll
    for (int j = 0; j < kTurn; j++)
#pragma unroll
      for (int ti = 0; ti < NT; ti++) *reinterpret_cast<uint2 *>(mine + (j * 16 + r) * kStride + ti * 32 + lg * 8) = rounded4(value(ti, j0 + j));
    wave_order();
#pragma unroll
    for (int c = 0; c < kPieces; c++) {
      const int at = c * kWave + lane, row = at / (kRow / 16), col = at % (kRow / 16) * 8;
      store(j0 * 16 + row, col, *reinterpret_cast<const uint4 *>(mine + row * kStride + col * 2));
    }
    wave_order();
  }
}

// The same with binary32 values, handed over COUNT = 4 or 8 at a time, the address of the first.
template <class T, int NT, int COUNT, class S>
__device__ __forceinline__ void turn_f32(uint8_t *lds, const float4v (&acc)[NT][T::TQ], S store) {
  constexpr int kRow = NT * 64, kStride = kRow + 16, kPieces = kRow / (COUNT * 16);   // bytes
  static_assert(kPieces >= 1 && kPieces * COUNT * 16 == kRow && T::kWaves * 16 * kStride <= T::kLds, "staging");
  const int lane = threadIdx.x & 63, lg = lane / 16, r = lane % 16;
  uint8_t *mine = lds + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave) * 16 * kStride;
#pragma unroll
  for (int j = 0; j < T::TQ; j++) {
#pragma unroll
    for (int ti = 0; ti < NT; ti++) *reinterpret_cast<float4v *>(mine + r * kStride + ti * 64 + lg * 16) = acc[ti][j];
    wave_order();
#pragma unroll
    for (int c = 0; c < kPieces; c++) {
      const int at = c * kWave + lane, row = at / (kRow / 4 / COUNT), col = at % (kRow / 4 / COUNT) * COUNT;
      store(j * 16 + row, col, reinterpret_cast<const float4v *>(mine + row * kStride + col * 4));
    }
    wave_order();
  }
}

__device__ __forceinline__ float element(const uint4 &v, int i) {
  const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
  return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
}

// ---- the product ----------------------------------------------------------------------------

// Items of the large tile, of which a CU holds one at a time: where the items that an XCD has beyond whole
// rounds of its CUs are at most half a round (a quarter), each is cut into two (four) along Q, for a
// last round of about half (a quarter of) the time: 384 tiles of 8192 rows 501 us whole, 453 cut.  Part `part` of the tile has rows from part * Q / parts on.
constexpr int kXcdCus = 32, kMostParts = 24;   // more workgroups for an XCD's cut items
__device__ __forceinline__ bool part_of(int b, int64_t count, int64_t &w, int &part, int &parts) {
  const int64_t per = (count + kXcds - 1) / kXcds, first = b % kXcds * per;
  const int64_t mine = min(per, count - first), whole = mine <= 0 ? 0 : mine / kXcdCus * kXcdCus, rest = mine - whole, i = b / kXcds;
  parts = rest <= kXcdCus / 4 ? 4 : rest <= kXcdCus / 2 ? 2 : 1;
  part = 0;
  if (i < whole) {
    parts = 1;
    w = first + i;
    return true;
  }
  const int64_t at = (i - whole) / parts;
  part = static_cast<int>((i - whole) % parts);
  w = first + whole + at;
  return at < rest;
}

// The item of this workgroup: group g, `count` rows of it from row `first` on, and n tile.
template <int SIZE, bool LARGE>
__device__ __forceinline__ bool find_item(const GemmParams &P, groups::Chunk &g, int &first, int &count, int &nt) {
  int64_t w = 0;
  int i, chunk, part = 0, parts = 1;
  auto index = [&](int total) {
    const int64_t items = static_cast<int64_t>(total) * P.n_tiles;
    return (LARGE ? part_of(blockIdx.x, items, w, part, parts) : item_of(blockIdx.x, items, w)) ? static_cast<int>(w / P.n_tiles) : -1;
  };
  if (!groups::find_chunk_of_all(P.offsets, P.E, P.R, SIZE, index, i, g)) return false;
  place_in_band(static_cast<int>(w - static_cast<int64_t>(i - g.index) * P.n_tiles), g.total, P.n_tiles, chunk, nt);
  const int size = SIZE / parts;
  first = g.lo + chunk * SIZE + part * size;
  count = min(size, g.hi - first);
  return count > 0;
}

// Row number v of an operand of `rows` rows, kept inside it.
__device__ __forceinline__ int64_t clamped(int64_t v, int64_t rows) { return v < 0 ? 0 : (v >= rows ? rows - 1 : v); }

template <class T, Epilogue MODE>
__global__ __launch_bounds__(T::kThreadsT) void gemm_kernel(const GemmParams P) {
  static_assert(MODE != kGated || (T::kHalves == 2 && !T::PT), "gate and up panels");
  __shared__ __align__(1024) uint8_t lds[T::kLds];
  groups::Chunk g;
  int first, count, nt;
  if (!find_item<T::BQ, T::kLarge>(P, g, first, count, nt)) return;
  const int width = MODE == kGated ? P.N / 2 : P.N;   // columns of act, or of y
  const int n0 = nt * (MODE == kGated ? kPanelCols : T::BP);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);

  Source<T> src;
  const int steps = (P.K + T::STEP - 1) / T::STEP;
  src.last = P.K - (steps - 1) * T::STEP;
  src.p.base = reinterpret_cast<uint64_t>(P.B) + static_cast<uint64_t>(g.group) * P.N * P.K * 2;
  src.left_p = static_cast<int64_t>(P.N) * P.K * 2;
  src.p.bytes = range_of(src.left_p);
  src.step_p = T::PT ? static_cast<uint32_t>(P.N) * T::STEP * 2 : T::kRowBytes;
#pragma unroll
  for (int j = 0; j < T::kCopiesP; j++) {
    const int c = wave * T::kCopiesP + j;
    if (T::PT) {
      int k, col;
      place_across<T>(c, k, col);
      src.vp[j] = n0 + col < P.N ? (static_cast<uint32_t>(k) * P.N + n0 + col) * 2 : kOob;
    } else {
      int row, piece;
      place_along<T>(c, row, piece);
      const int i = n0 + (MODE == kGated ? row % kPanelCols : row);
      const int n = MODE == kGated ? i + row / kPanelCols * width : i;
      src.vp[j] = i < width ? static_cast<uint32_t>(n) * P.K * 2 + piece * 16 : kOob;
    }
  }
  // token rows: gathered from all of A, or the group's own
  const bool gather = P.A_rows != nullptr;
  src.q.base = reinterpret_cast<uint64_t>(P.A) + (gather ? 0 : static_cast<uint64_t>(first) * P.K * 2);
  src.q.bytes = static_cast<uint32_t>((gather ? P.rows_A : count) * P.K * 2);
  src.step_q = T::kRowBytes;
#pragma unroll
  for (int j = 0; j < T::kCopiesQ; j++) {
    int row, piece;
    place_along<T>(wave * T::kCopiesQ + j, row, piece);
    src.vq[j] = kOob;
    if (row < count) {
      const int64_t a = gather ? clamped(P.A_rows[first + row], P.rows_A) : row;
      src.vq[j] = static_cast<uint32_t>(a) * P.K * 2 + piece * 16;
    }
  }

  float4v acc[T::TP][T::TQ];
  if constexpr (T::kLarge) {
    with_active<T>(count, [&](auto active) INLINED {
      contract_large<T, decltype(active)::value>(
          [&](auto j, int kb, uint32_t at) INLINED { issue_one<T, false>(src, at, wave, j, kb == steps - 1 && src.last < T::STEP); },
          [](auto, int, auto) INLINED {}, [](int) INLINED {}, [&](int kb) INLINED { advance_to<T>(src, kb, steps); }, lds, steps, acc);
    });
  } else {
    // the weights of a group of one chunk are read by this workgroup alone: where they do not stay in the
    // memory-side cache between calls, past the caches (32 groups of 32 rows, 1.6 GB, 280 us, 293 through them; 16 of 20,
    // 53 MB, the other way 25 and 16)
    const bool once = g.total == 1 && P.stream_weights;
    // Q tiles behind the last row are left out
    auto run = [&](auto active) {
      constexpr int kActive = decltype(active)::value;
      if (once) contract<T, true, kActive>(src, lds, steps, acc);
      else contract<T, false, kActive>(src, lds, steps, acc);
    };
    const int active = T::WQ == 1 ? (count + 15) / 16 : T::TQ;
    if (T::TQ >= 4 && active == 3) run(std::integral_constant<int, T::TQ >= 4 ? 3 : T::TQ>());
    else if (T::TQ >= 4 && active == 2) run(std::integral_constant<int, T::TQ >= 4 ? 2 : T::TQ>());
    else if (T::TQ >= 2 && active == 1) run(std::integral_constant<int, T::TQ >= 2 ? 1 : T::TQ>());
    else run(std::integral_constant<int, T::TQ>());
  }

  const int wp = wave % T::WP, wq = wave / T::WP;
  constexpr int kCols = kPanelCols / T::WP;           // a wave's columns of a panel
  if (MODE == kPlain) {
    turn<T, T::TP>(lds, [&](int ti, int j) { return acc[ti][j]; },
                   [&](int row, int col, const uint4 &v) {
                     const int t = row_of_tile<T>(wq, row);
                     const int n = n0 + col / kCols * kPanelCols + wp * kCols + col % kCols;
                     if (t < count && n < P.N) store16<T::kLarge>(P.D + static_cast<int64_t>(first + t) * P.N + n, v);
                   });
  } else if (MODE == kGated) {
    const int i0 = n0 + wp * kCols;
    if (P.Z != nullptr) {
#pragma unroll
      for (int half = 0; half < T::kHalves; half++)
        turn<T, T::kPerHalf>(lds, [&](int ti, int j) { return acc[half * T::kPerHalf + ti][j]; },
                             [&](int row, int col, const uint4 &v) {
                               const int t = row_of_tile<T>(wq, row);
                               if (t < count && i0 + col < width)
                                 store16<T::kLarge>(P.Z + static_cast<int64_t>(first + t) * P.N + half * width + i0 + col, v);
                             });
    }
    turn<T, T::kPerHalf>(lds,
                         [&](int ti, int j) {
                           float4v act;
#pragma unroll
                           for (int c = 0; c < 4; c++) {
                             const float gate = acc[ti][j][c], up = acc[(T::kHalves - 1) * T::kPerHalf + ti][j][c];
                             act[c] = gate * sigmoid(gate) * up;
                           }
                           return act;
                         },
                         [&](int row, int col, const uint4 &v) {
                           const int t = row_of_tile<T>(wq, row);
                           if (t < count && i0 + col < width)
                             store16<T::kLarge>(P.D + static_cast<int64_t>(first + t) * width + i0 + col, v);
                         });
  } else {
    turn_f32<T, T::TP, 8>(lds, acc, [&](int row, int col, const float4v *v) {
      const float4v lo = v[0], hi = v[1];
      const int n = n0 + col / kCols * kPanelCols + wp * kCols + col % kCols;
      const int t = row_of_tile<T>(wq, row);
      if (t >= count || n >= P.N) return;
      const int64_t at = static_cast<int64_t>(first + t) * 2 * P.N + n;
      const uint4 gate = *reinterpret_cast<const uint4 *>(P.Z + at), up = *reinterpret_cast<const uint4 *>(P.Z + at + P.N);
      float4v dg[2], du[2];
#pragma unroll
      for (int c = 0; c < 8; c++) {
        const float y = c < 4 ? lo[c & 3] : hi[c & 3], gv = element(gate, c), uv = element(up, c), s = sigmoid(gv);
        dg[c / 4][c & 3] = y * uv * (s * (1.0f + gv * (1.0f - s)));
        du[c / 4][c & 3] = y * (gv * s);
      }
      const uint2 a = rounded4(dg[0]), b = rounded4(dg[1]), c = rounded4(du[0]), d = rounded4(du[1]);
      store16<T::kLarge>(P.D + at, make_uint4(a.x, a.y, b.x, b.y));
      store16<T::kLarge>(P.D + at + P.N, make_uint4(c.x, c.y, d.x, d.y));
    });
  }
}

// ---- few items ------------------------------------------------------------------------------
//
// Where there are few rows and columns (a single token: k experts' weights, each a few hundred rows),
// the contraction is dealt to the eight waves of a workgroup: wave w takes the steps w, w + 8, ... of a
// tile of P rows of the weights and 16 rows of A, with a ring of its own and no barrier before the end,
// and the eight partial tiles are added in order through LDS.  Gated: a 16-row tile of the weights
// holds 8 gate rows and the 8 up rows that belong to them, which end in lane groups two apart.
template <int P_, int WAVES_, int STAGES_>
struct Split : Stage<64> {
  static constexpr int Q = 16, P = P_, WAVES = WAVES_, STAGES = STAGES_;
  static constexpr int TP = P / 16;
  static constexpr int kCopiesP = P / 8, kCopies = kCopiesP + Q / 8;
  static constexpr int kStage = (P + Q) * kRowBytes;
  static constexpr int kLds = WAVES * STAGES * kStage;
  static_assert(TP * kWave * 16 <= STAGES * kStage, "a wave's partial tiles fit");
};

template <class T, Epilogue MODE>
__global__ __launch_bounds__(T::WAVES *kWave) void split_kernel(const GemmParams P) {
  static_assert(MODE != kGatedBackward, "weights along the contraction");
  __shared__ __align__(1024) uint8_t lds[T::kLds];
  groups::Chunk g;
  int first, count, nt;
  if (!find_item<T::Q, false>(P, g, first, count, nt)) return;
  constexpr int kTile = MODE == kGated ? 8 : 16;      // columns of the result in a 16-row tile
  const int width = MODE == kGated ? P.N / 2 : P.N, n0 = nt * T::TP * kTile;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = threadIdx.x & 63, lg = lane / 16, r = lane % 16;
  const int steps = (P.K + T::STEP - 1) / T::STEP, last = P.K - (steps - 1) * T::STEP;
  const bool gather = P.A_rows != nullptr;
  const Buf bp = {reinterpret_cast<uint64_t>(P.B) + static_cast<uint64_t>(g.group) * P.N * P.K * 2, static_cast<uint32_t>(P.N) * P.K * 2};
  const Buf bq = {reinterpret_cast<uint64_t>(P.A) + (gather ? 0 : static_cast<uint64_t>(first) * P.K * 2),
                  static_cast<uint32_t>((gather ? P.rows_A : count) * P.K * 2)};
  uint32_t vp[T::kCopiesP], vq[T::Q / 8];
#pragma unroll
  for (int j = 0; j < T::kCopiesP; j++) {
    int row, piece;
    place_along<T>(j, row, piece);
    const int i = n0 + row / 16 * kTile + row % kTile;
    const int n = MODE == kGated ? i + row % 16 / 8 * width : i;
    vp[j] = i < width ? static_cast<uint32_t>(n) * P.K * 2 + piece * 16 : kOob;
  }
#pragma unroll
  for (int j = 0; j < T::Q / 8; j++) {
    int row, piece;
    place_along<T>(j, row, piece);
    vq[j] = kOob;
    if (row < count) {
      const int64_t a = gather ? clamped(P.A_rows[first + row], P.rows_A) : row;
      vq[j] = static_cast<uint32_t>(a) * P.K * 2 + piece * 16;
    }
  }
  uint8_t *ring = lds + wave * T::STAGES * T::kStage;
  const uint32_t ring0 = lds_address(ring);
  // the wave's i-th step into buffer `slot`
  auto issue_step = [&](int i, int slot) {
    const int kb = wave + T::WAVES * i;
    const uint32_t at = ring0 + slot * T::kStage;
    const bool past = kb >= steps, is_last = kb == steps - 1;
#pragma unroll
    for (int j = 0; j < T::kCopiesP; j++) {
      const uint32_t v = in_range<T>(vp[j], j, is_last, last);
      copy16<true>(bp, at + j * 1024, past || v == kOob ? kOob : v + kb * T::kRowBytes);
    }
#pragma unroll
    for (int j = 0; j < T::Q / 8; j++) {
      const uint32_t v = in_range<T>(vq[j], j, is_last, last);
      copy16(bq, at + T::P * T::kRowBytes + j * 1024, past || v == kOob ? kOob : v + kb * T::kRowBytes);
    }
  };
  float4v acc[T::TP] = {};
#pragma unroll
  for (int i = 0; i < T::STAGES; i++) issue_step(i, i);
  int slot = 0;
  for (int i = 0; wave + T::WAVES * i < steps; i++) {
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(T::kCopies * (T::STAGES - 1)) : "memory");
    const uint8_t *S = ring + slot * T::kStage;
    bf16x8 q[2], p[2][T::TP];
#pragma unroll
    for (int h = 0; h < 2; h++) {
      q[h] = along<T>(S + T::P * T::kRowBytes, r, h, lg);
#pragma unroll
      for (int t = 0; t < T::TP; t++) p[h][t] = along<T>(S, t * 16 + r, h, lg);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");   // the buffer is read before it is filled again
    issue_step(i + T::STAGES, slot);
#pragma unroll
    for (int h = 0; h < 2; h++)
#pragma unroll
      for (int t = 0; t < T::TP; t++) acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(p[h][t], q[h], acc[t], 0, 0, 0);
    slot = slot == T::STAGES - 1 ? 0 : slot + 1;
  }
  arrive<0>();
  float4v *part = reinterpret_cast<float4v *>(lds);   // [wave][tile][lane]
#pragma unroll
  for (int t = 0; t < T::TP; t++) part[(wave * T::TP + t) * kWave + lane] = acc[t];
  __syncthreads();
  for (int t = wave; t < T::TP; t += T::WAVES) {
    float4v sum = part[t * kWave + lane];
#pragma unroll
    for (int w = 1; w < T::WAVES; w++) sum += part[(w * T::TP + t) * kWave + lane];
    const int64_t p = first + r;
    if (MODE == kPlain) {
      const int n = n0 + t * 16 + 4 * lg;
      if (r < count && n < P.N) *reinterpret_cast<uint2 *>(P.D + p * P.N + n) = rounded4(sum);
    } else {
      float4v other, act;
#pragma unroll
      for (int c = 0; c < 4; c++) other[c] = __shfl_xor(sum[c], 32, kWave);
      const int i = n0 + t * 8 + 4 * (lg & 1);
#pragma unroll
      for (int c = 0; c < 4; c++) act[c] = sum[c] * sigmoid(sum[c]) * other[c];   // of gate lanes
      if (r >= count || i >= width) continue;
      if (P.Z != nullptr) *reinterpret_cast<uint2 *>(P.Z + p * P.N + lg / 2 * width + i) = rounded4(sum);
      if (lg < 2) *reinterpret_cast<uint2 *>(P.D + p * width + i) = rounded4(act);
    }
  }
}

// ---- the weight gradient -----------------------------------------------------------------------

// Read through scalar loads.
typedef const __attribute__((address_space(4))) int32_t *const_rows;
typedef int int16x __attribute__((ext_vector_type(16)));
typedef int int16x_unaligned __attribute__((ext_vector_type(16), aligned(4)));
typedef const __attribute__((address_space(4))) int16x_unaligned *const_rows16;

// One tile of D: Q is Y's columns n, P is X's columns k, the contraction the tokens of group e.
template <class T, bool BF16, bool GATHER>
__global__ __launch_bounds__(T::kThreadsT) void wgrad_kernel(const WgradParams P) {
  static_assert(T::PT && T::QT, "columns of X and Y");
  __shared__ __align__(1024) uint8_t lds[T::kLds];
  const int n_tiles = (P.N + T::BQ - 1) / T::BQ, k_tiles = (P.K + T::BP - 1) / T::BP, per = n_tiles * k_tiles;
  int64_t w;
  int part = 0, parts = 1;
  if (!(T::kLarge ? part_of(blockIdx.x, static_cast<int64_t>(P.E) * per, w, part, parts) : item_of(blockIdx.x, static_cast<int64_t>(P.E) * per, w))) return;
  const int e = static_cast<int>(w / per);
  int nt, kt;
  place_in_band(static_cast<int>(w - static_cast<int64_t>(e) * per), n_tiles, k_tiles, nt, kt);
  const int n0 = nt * T::BQ + part * (T::BQ / parts), k0 = kt * T::BP, n1 = min(n0 + T::BQ / parts, P.N);
  if (n0 >= n1) return;
  int lo = __builtin_amdgcn_readfirstlane(P.offsets[e]), hi = __builtin_amdgcn_readfirstlane(P.offsets[e + 1]);
  groups::clamp_pair(lo, hi, P.R);
  const int rows = hi - lo, steps = (rows + T::STEP - 1) / T::STEP;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x & 63;
  const_rows index = (const_rows)(uintptr_t)P.X_rows;

  Source<T> src;
  src.last = 0;   // (both operands lie across the contraction)
  src.q.base = reinterpret_cast<uint64_t>(P.Y) + static_cast<uint64_t>(lo) * P.N * 2;
  src.p.base = reinterpret_cast<uint64_t>(P.X) + (GATHER ? 0 : static_cast<uint64_t>(lo) * P.K * 2);
  src.left_q = static_cast<int64_t>(rows) * P.N * 2;
  src.left_p = (GATHER ? P.rows_X : rows) * P.K * 2;
  src.q.bytes = range_of(src.left_q);
  src.p.bytes = range_of(src.left_p);
  src.step_q = static_cast<uint32_t>(P.N) * T::STEP * 2;
  src.step_p = GATHER ? 0 : static_cast<uint32_t>(P.K) * T::STEP * 2;
#pragma unroll
  for (int j = 0; j < T::kCopiesQ; j++) {
    int k, col;
    place_across<T>(wave * T::kCopiesQ + j, k, col);
    src.vq[j] = n0 + col < n1 ? (static_cast<uint32_t>(k) * P.N + n0 + col) * 2 : kOob;
  }
#pragma unroll
  for (int j = 0; j < T::kCopiesP; j++) {
    int k, col;
    place_across<T>(wave * T::kCopiesP + j, k, col);
    src.vp[j] = k0 + col < P.K ? (static_cast<uint32_t>(GATHER ? 0 : k) * P.K + k0 + col) * 2 : kOob;
  }
  const uint32_t lds0 = lds_address(lds);
  // The numbers of the gathered rows of a stage's copies, four each, come through the scalar cache, so
  // that no vector load stands between the copies, and a stage ahead, so that none waits for them.  A lane
  // takes the one of its row; past the group's end it takes none.  (A number outside X is outside the
  // buffer's range, or wraps to another place in it.)
  constexpr int kRows = 4 * T::kCopiesP;
  static_assert(kRows == 16 && T::kPanelCopies % T::kCopiesP == 0, "a wave's rows are 16 neighbours");
  int16x row_of = {}, next_row_of = {};
  auto load_rows = [&](int kb) INLINED {
    if (!GATHER) return;
    const int row0 = lo + kb * T::STEP + wave * T::kCopiesP % T::kPanelCopies * 4;
    if (row0 + kRows <= P.R) {
      next_row_of = *reinterpret_cast<const_rows16>(index + row0);
    } else {   // (near the end of the list only: the wait for this load is one for the copies under way too)
      const int mine = P.X_rows[min(row0 + lane % kRows, P.R - 1)];
#pragma unroll
      for (int q = 0; q < kRows; q++) next_row_of[q] = __builtin_amdgcn_readlane(mine, q);
    }
  };
  auto take_rows = [&]() INLINED { row_of = next_row_of; };
  load_rows(0);
  take_rows();
  const uint32_t row_bytes = static_cast<uint32_t>(P.K) * 2;
  // The gathered copy's offset, in steps: all at once between two MFMAs they kept the next one waiting (16
  // groups of 512 rows, 4096 x 6144, 572 us; now 538, and 510 where the rows need no gathering).
  uint32_t from = 0, other = 0;
  auto locate = [&](auto number, int kb, auto phase) INLINED {
    constexpr int j = decltype(number)::value, step = decltype(phase)::value;
    if constexpr (GATHER && j < T::kCopiesP) {
      const int k = kb * T::STEP + (wave * T::kCopiesP + j) % T::kPanelCopies * 4 + lane / 16;
      if (step == 0) {
        int row[4] = {row_of[4 * j], row_of[4 * j + 1], row_of[4 * j + 2], row_of[4 * j + 3]};
#pragma unroll
        for (int q = 0; q < 4; q++) asm("" : "+s"(row[q]));   // (or they become one element with a variable index)
        from = lane / 16 & 1 ? row[1] : row[0];
        other = lane / 16 & 1 ? row[3] : row[2];
      } else if (step == 1) {
        from = lane / 32 ? other : from;
      } else if (step == 2) {
        from = src.vp[j] + from * row_bytes;
      } else {
        from = k < rows ? from : kOob;
      }
      asm volatile("" : "+v"(from));   // (or the compiler branches around the product, four times a stage)
    }
  };
  auto issue_copy = [&](auto number, int kb, uint32_t at) INLINED {
    constexpr int j = decltype(number)::value;
    if constexpr (GATHER && j < T::kCopiesP) copy16(src.p, at + (wave * T::kCopiesP + j) * 1024, from);
    else issue_one<T, false>(src, at, wave, j, false);
  };
  auto advance = [&](int kb) INLINED {
    if (GATHER) {
      advance_one<false>(src.p, src.left_p, 0, false);
      advance_one<true>(src.q, src.left_q, src.step_q, false);
      take_rows();
    } else {
      advance_to<T>(src, kb, steps);
    }
  };
  float4v acc[T::TP][T::TQ];
  if constexpr (T::kLarge) {
    with_active<T>(n1 - n0, [&](auto active) INLINED { contract_large<T, decltype(active)::value>(issue_copy, locate, load_rows, advance, lds, steps, acc); });
  } else {
    const int g = lane / 16, r = lane % 16, wp = wave % T::WP, wq = wave / T::WP;
    constexpr int kHalvesK = T::STEP / 32;
    auto issue_stage = [&](int kb, int slot) INLINED {
      load_rows(kb + 1);
      for_constants<T::kCopies>([&](auto j) INLINED {
        for_constants<kPhases>([&](auto phase) INLINED { locate(j, kb, phase); });
        issue_copy(j, kb, lds0 + slot * T::kStage);
      });
      advance(kb + 1);
    };
    clear<T>(acc);
#pragma unroll
    for (int i = 0; i < T::STAGES - 1; i++) issue_stage(i, i);
    int slot = 0;
    for (int kb = 0; kb < steps; kb++) {
      arrive<T::kCopies *(T::STAGES - 2)>();
      issue_stage(kb + T::STAGES - 1, slot == 0 ? T::STAGES - 1 : slot - 1);
      const uint8_t *Ps = lds + slot * T::kStage, *Qs = Ps + T::kBytesP;
      bf16x8 q[kHalvesK][T::TQ];
#pragma unroll
      for (int h = 0; h < kHalvesK; h++)
#pragma unroll
        for (int j = 0; j < T::TQ; j++) q[h][j] = fragment_q<T>(Qs, wq, j, h, g, r);
#pragma unroll
      for (int i = 0; i < T::TP; i++)
#pragma unroll
        for (int h = 0; h < kHalvesK; h++) mfma_row<T>(fragment_p<T>(Ps, wp, i / T::kPerHalf, i % T::kPerHalf, h, g, r), q[h], acc[i]);
      slot = slot == T::STAGES - 1 ? 0 : slot + 1;
    }
    arrive<0>();
  }
  const int wp = wave % T::WP, wq = wave / T::WP;
  constexpr int kCols = kPanelCols / T::WP;
  auto column = [&](int col) { return k0 + col / kCols * kPanelCols + wp * kCols + col % kCols; };
  if (BF16) {
    uint16_t *D = static_cast<uint16_t *>(P.D);
    turn<T, T::TP>(lds, [&](int ti, int j) { return acc[ti][j]; },
                   [&](int row, int col, const uint4 &v) {
                     const int n = n0 + row_of_tile<T>(wq, row), k = column(col);
                     if (n < n1 && k < P.K) store16<true>(D + (static_cast<int64_t>(e) * P.N + n) * P.K + k, v);
                   });
  } else {
    float *D = static_cast<float *>(P.D);
    turn_f32<T, T::TP, 4>(lds, acc, [&](int row, int col, const float4v *v) {
      const int n = n0 + row_of_tile<T>(wq, row), k = column(col);
      if (n < n1 && k < P.K) store16<true>(D + (static_cast<int64_t>(e) * P.N + n) * P.K + k, __builtin_bit_cast(uint4, *v));
    });
  }
}

// ---- launches -----------------------------------------------------------------------------------

template <class T, Epilogue MODE>
hipError_t run_gemm(GemmParams p, hipStream_t stream) {
  p.n_tiles = MODE == kGated ? (p.N / 2 + kPanelCols - 1) / kPanelCols : (p.N + T::BP - 1) / T::BP;
  const int64_t items = groups::max_chunks(p.R, p.E, T::BQ) * p.n_tiles;
  const int64_t grid = ((items + kXcds - 1) / kXcds + (T::kLarge ? kMostParts : 0)) * kXcds;
  if (items > 0) hipLaunchKernelGGL((gemm_kernel<T, MODE>), dim3(static_cast<uint32_t>(grid)), dim3(T::kThreadsT), 0, stream, p);
  return hipGetLastError();
}

template <class T, Epilogue MODE>
hipError_t run_split(GemmParams p, hipStream_t stream) {
  constexpr int kCols = MODE == kGated ? T::P / 2 : T::P;
  const int width = MODE == kGated ? p.N / 2 : p.N;
  p.n_tiles = (width + kCols - 1) / kCols;
  const int64_t items = groups::max_chunks(p.R, p.E, T::Q) * p.n_tiles;
  const int64_t grid = (items + kXcds - 1) / kXcds * kXcds;
  hipLaunchKernelGGL((split_kernel<T, MODE>), dim3(static_cast<uint32_t>(grid)), dim3(T::WAVES * kWave), 0, stream, p);
  return hipGetLastError();
}

template <class T, bool BF16>
hipError_t run_wgrad(const WgradParams &p, hipStream_t stream) {
  const int64_t items = static_cast<int64_t>(p.E) * ((p.N + T::BQ - 1) / T::BQ) * ((p.K + T::BP - 1) / T::BP);
  const int64_t grid = ((items + kXcds - 1) / kXcds + (T::kLarge ? kMostParts : 0)) * kXcds;
  if (p.X_rows != nullptr)
    hipLaunchKernelGGL((wgrad_kernel<T, BF16, true>), dim3(static_cast<uint32_t>(grid)), dim3(T::kThreadsT), 0, stream, p);
  else
    hipLaunchKernelGGL((wgrad_kernel<T, BF16, false>), dim3(static_cast<uint32_t>(grid)), dim3(T::kThreadsT), 0, stream, p);
  return hipGetLastError();
}

constexpr int64_t kCacheBytes = 256 << 20;   // MI355X's memory-side cache

template <bool PT>
using Large = Tile<256, 256, 2, 2, 5, PT, false, 32>;

template <Epilogue MODE, bool PT>
hipError_t run_tile(GemmTile tile, const GemmParams &p, hipStream_t stream) {
  if (tile == kSquare256) return run_gemm<Large<PT>, MODE>(p, stream);
  if constexpr (!PT) {
    if (tile == kSplit16) return run_split<Split<16, 8, 3>, MODE>(p, stream);
    if (tile == kSplit32) return run_split<Split<32, 8, 3>, MODE>(p, stream);
  }
  if constexpr (MODE == kGated) {
    return run_gemm<Tile<64, 256, 1, 8, 3, PT>, MODE>(p, stream);
  } else {
    if (tile == kSquare128) return run_gemm<Tile<128, 128, 2, 2, 2, PT>, MODE>(p, stream);
    if (tile == kRows32) return run_gemm<Tile<32, 128, 1, 4, 3, PT>, MODE>(p, stream);
    return run_gemm<Tile<64, 128, 1, 4, 3, PT>, MODE>(p, stream);
  }
}

}  // namespace

hipError_t launch_gemm(GemmParams p, Epilogue epilogue, bool transposed, hipStream_t stream) {
  if (p.R == 0) return hipSuccess;
  p.stream_weights = static_cast<int64_t>(p.E) * p.N * p.K * 2 > kCacheBytes / 2;
  const GemmTile tile = gemm_tile(p.E, p.N, p.R, epilogue, transposed);
  if (epilogue == kGated) return run_tile<kGated, false>(tile, p, stream);
  if (epilogue == kGatedBackward) return run_tile<kGatedBackward, true>(tile, p, stream);
  return transposed ? run_tile<kPlain, true>(tile, p, stream) : run_tile<kPlain, false>(tile, p, stream);
}

hipError_t launch_wgrad(const WgradParams &p, bool bf16, hipStream_t stream) {
  if (wgrad_large(p.E, p.N, p.K, p.R)) {
    using T = Tile<256, 256, 2, 2, 5, true, true, 32>;
    return bf16 ? run_wgrad<T, true>(p, stream) : run_wgrad<T, false>(p, stream);
  }
  using T = Tile<128, 128, 2, 2, 2, true, true>;
  return bf16 ? run_wgrad<T, true>(p, stream) : run_wgrad<T, false>(p, stream);
}

}  // namespace bf16
}  // namespace moe
