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
// wgrad_kernel: D may be binary32, where that would show, so the codes become fp16 (exactly) and
// the fp16 matrix core, whose products and sums are whole, takes them.  A launch of a few hundred
// tokens per expert is bound by writing D all the same.
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

#include <type_traits>

#pragma clang fp contract(off)

namespace moe {
namespace fp8 {
namespace {

typedef int int8v __attribute__((ext_vector_type(8)));
typedef int int4x __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;

constexpr uint32_t kOob = 0x80000000u;   // an offset that no operand's range reaches

enum Mode { kNone, kSwigluFp8, kWgradF32, kWgradBf16 };

// ---- copies into LDS ----------------------------------------------------------------------

struct Buf {
  uint64_t base;
  uint32_t bytes;
};

__device__ __forceinline__ int4x descriptor(const Buf &b) {
  return int4x{static_cast<int>(b.base), static_cast<int>((b.base >> 32) & 0xffffu), static_cast<int>(b.bytes), 0x00020000};
}

// The same value, known to the compiler to be uniform over the wave.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ Buf uniform(const Buf &b) {
  return {(static_cast<uint64_t>(uniform(static_cast<uint32_t>(b.base >> 32))) << 32) | uniform(static_cast<uint32_t>(b.base)),
          uniform(b.bytes)};
}

__device__ __forceinline__ uint32_t lds_address(const void *p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const lds_u8 *)p));
}

// Copies 16 (4) bytes per lane from `voff` of the buffer to LDS bytes lds + 16 (4) * lane.  The
// copy is counted by vmcnt like a load; it has no destination registers, so nothing waits for
// it but the explicit wait in `arrive`.
__device__ __forceinline__ void copy16(const Buf &b, uint32_t lds, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(descriptor(b))
               : "memory");
}
__device__ __forceinline__ void copy4(const Buf &b, uint32_t lds, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(descriptor(b))
               : "memory");
}

// Waits until at most `LATER` copies of this wave are under way and its LDS reads are done,
// then for the workgroup: after it every wave's older copies are in LDS, and no wave still
// reads the buffer that the stage before used.
template <int LATER>
__device__ __forceinline__ void arrive() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(LATER) : "memory");
}

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
  static constexpr int kLds = STAGES * kStage;
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

// Row and logical piece that copy j of this wave and lane moves.
__device__ __forceinline__ void copy_place(int first_row, int &row, int &piece) {
  const int lane = threadIdx.x & 63;
  row = first_row + lane / 8;
  piece = (lane & 7) ^ ((row >> 1) & 7);
}

// The copies of stage `kb` into buffer `slot`; beyond the last stage they move nothing.
template <class T>
__device__ __forceinline__ void issue(Source<T> &src, uint32_t lds, int wave, int kb, int steps) {
  const bool tail = kb == steps - 1 && src.last_pieces < 8;
  const int lane = threadIdx.x & 63;
  if (kb >= steps) src.p.bytes = src.q.bytes = src.s.bytes = 0;
#pragma unroll
  for (int j = 0; j < T::kCopiesP; j++) {
    const int row8 = (wave * T::kCopiesP + j) * 8;
    uint32_t v = src.vp[j];
    if (tail && ((lane & 7) ^ (((row8 + lane / 8) >> 1) & 7)) >= src.last_pieces) v = kOob;
    copy16(src.p, lds + row8 * kFp8Block, v);
  }
#pragma unroll
  for (int j = 0; j < T::kCopiesQ; j++) {
    const int row8 = (wave * T::kCopiesQ + j) * 8;
    uint32_t v = src.vq[j];
    if (tail && ((lane & 7) ^ (((row8 + lane / 8) >> 1) & 7)) >= src.last_pieces) v = kOob;
    copy16(src.q, lds + T::kBytesP + row8 * kFp8Block, v);
  }
  copy4(src.s, lds + T::kBytesP + T::kBytesQ + wave * kWave * 4, src.vs);
  src.p.base += src.step_p;
  src.q.base += src.step_q;
  src.s.base += src.step_s;
}

// 32 bytes of a tile row: pieces 2g and 2g + 1 for lane group g (both operands take this order;
// within a scale block the contraction's order is free).
__device__ __forceinline__ int8v fragment(const uint8_t *rows, int row, int g) {
  const int sw = (row >> 1) & 7;
  const uint8_t *p = rows + row * kFp8Block;
  const int4x a = *reinterpret_cast<const int4x *>(p + ((2 * g) ^ sw) * 16);
  const int4x b = *reinterpret_cast<const int4x *>(p + ((2 * g + 1) ^ sw) * 16);
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
// per half of P (WGRAD false) or one per P row.
template <class T, bool WGRAD>
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
  for (int s = 0; s < T::STAGES - 1; s++) issue<T>(src, lds0 + s * T::kStage, wave, s, steps);
  int slot = 0;
  for (int kb = 0; kb < steps; kb++) {
    arrive<T::kCopies *(T::STAGES - 2)>();
    const int next = slot == 0 ? T::STAGES - 1 : slot - 1;
    issue<T>(src, lds0 + next * T::kStage, wave, kb + T::STAGES - 1, steps);
    const uint8_t *P = lds + slot * T::kStage, *Q = P + T::kBytesP;
    const float *S = reinterpret_cast<const float *>(Q + T::kBytesQ);
    using Frag = std::conditional_t<WGRAD, Half32, int8v>;
    Frag q[T::TQ];
    float sq[T::TQ];
#pragma unroll
    for (int j = 0; j < T::TQ; j++) {
      const int row = (wq * T::TQ + j) * 16 + r;
      if constexpr (WGRAD) q[j] = to_f16(fragment(Q, row, g));
      else q[j] = fragment(Q, row, g);
      sq[j] = S[row];
    }
#pragma unroll
    for (int i = 0; i < T::TP; i++) {
      const int row0 = (i / T::kPerHalf) * kFp8Block + wp * (kFp8Block / T::WP) + (i % T::kPerHalf) * 16;
      const int8v p = fragment(P, row0 + r, g);
      if constexpr (WGRAD) {
        const Half32 ph = to_f16(p);
        const float4v sp = *reinterpret_cast<const float4v *>(S + T::kScaleP + row0 + 4 * g);
#pragma unroll
        for (int j = 0; j < T::TQ; j++) {
          float4v t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int h = 0; h < 4; h++) t = __builtin_amdgcn_mfma_f32_16x16x32_f16(ph.h[h], q[j].h[h], t, 0, 0, 0);
#pragma unroll
          for (int c = 0; c < 4; c++) acc[i][j][c] = fmaf(t[c], sp[c] * sq[j], acc[i][j][c]);
        }
      } else {
        const float sp = S[T::kScaleP + i / T::kPerHalf];
#pragma unroll
        for (int j = 0; j < T::TQ; j++) {
          const float4v t =
              __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(p, q[j], float4v{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
          const float s = sp * sq[j];
#pragma unroll
          for (int c = 0; c < 4; c++) acc[i][j][c] = fmaf(t[c], s, acc[i][j][c]);
        }
      }
    }
    slot = slot == T::STAGES - 1 ? 0 : slot + 1;
  }
  arrive<0>();   // the copies past the end (zeros) are in before the buffers serve anything else
}

__device__ __forceinline__ uint2 bf16x4(const float4v &v) {
  return make_uint2(f32_to_bf16(v[0]) | (static_cast<uint32_t>(f32_to_bf16(v[1])) << 16),
                    f32_to_bf16(v[2]) | (static_cast<uint32_t>(f32_to_bf16(v[3])) << 16));
}

// Item number of workgroup b out of `count`: workgroups are dealt to the 8 XCDs in turn, so
// each XCD gets a contiguous range of items and neighbours (tiles that share operands) its L2.
__device__ __forceinline__ bool item_of(int b, int64_t count, int64_t &w) {
  const int64_t per = (count + kXcds - 1) / kXcds;
  w = (b % kXcds) * per + b / kXcds;
  return b / kXcds < per && w < count;
}

// Tile (row chunk, column tile) number `l` out of chunks x tiles: bands of kBand row chunks, in
// a band the row chunk runs fastest, so the ~32 tiles that one XCD works on at a time share a
// few P and Q tiles.
constexpr int kBand = 8;
__device__ __forceinline__ void place_in_band(int l, int chunks, int tiles, int &chunk, int &tile) {
  const int band = l / (kBand * tiles);
  const int rem = l - band * kBand * tiles;
  const int width = min(kBand, chunks - band * kBand);
  tile = rem / width;
  chunk = band * kBand + rem - tile * width;
}

template <class T, Mode MODE>
__global__ __launch_bounds__(T::kThreadsT) void gemm_kernel(const GemmParams P) {
  __shared__ __align__(1024) uint8_t lds[T::kLds];
  // the item: an expert's row chunk and n tile
  int64_t w;
  const int total = groups::chunk_count(P.offsets, P.E, P.R, T::BQ);
  if (!item_of(blockIdx.x, static_cast<int64_t>(total) * P.n_tiles, w)) return;
  const int i = static_cast<int>(w / P.n_tiles);
  groups::Chunk g;
  if (!groups::find_chunk(P.offsets, P.E, P.R, T::BQ, i, g)) return;
  int chunk, nt;
  place_in_band(static_cast<int>(w - static_cast<int64_t>(i - g.index) * P.n_tiles), g.total, P.n_tiles, chunk, nt);
  const int first = g.lo + chunk * T::BQ, count = min(T::BQ, g.hi - first);
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
    copy_place((wave * T::kCopiesP + j) * 8, row, piece);
    int n = n0 + row;
    if (MODE == kSwigluFp8) n = n0 + row % kFp8Block + row / kFp8Block * half_n;   // half_n % 128 == 0
    src.vp[j] = n < P.N ? static_cast<uint32_t>(n) * P.K + piece * 16 : kOob;
  }
  // token rows: gathered from all of A, or the group's own
  const bool gather = P.A_rows != nullptr;
  src.q.base = reinterpret_cast<uint64_t>(P.A) + (gather ? 0 : static_cast<uint64_t>(first) * P.K);
  src.q.bytes = static_cast<uint32_t>((gather ? P.rows_A : count) * P.K);
  auto row_of = [&](int row) -> int64_t {
    if (!gather) return row;
    const int64_t a = P.A_rows[first + row];
    return a < 0 ? 0 : (a >= P.rows_A ? P.rows_A - 1 : a);
  };
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
  contract<T, false>(src, lds, kb_n, acc);

  const int wp = wave % T::WP, wq = wave / T::WP;
  if (MODE == kNone) {
    uint16_t *D = static_cast<uint16_t *>(P.D);
#pragma unroll
    for (int j = 0; j < T::TQ; j++) {
      const int t = (wq * T::TQ + j) * 16 + r;
      if (t >= count) continue;
      uint16_t *row = D + static_cast<int64_t>(first + t) * P.N;
#pragma unroll
      for (int ti = 0; ti < T::TP; ti++) {
        const int n = n0 + (ti / T::kPerHalf) * kFp8Block + wp * (kFp8Block / T::WP) + (ti % T::kPerHalf) * 16 + 4 * lg;
        if (n < P.N) *reinterpret_cast<uint2 *>(row + n) = bf16x4(acc[ti][j]);
      }
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

template <class T, Mode MODE>
__global__ __launch_bounds__(T::kThreadsT) void wgrad_kernel(const WgradParams P) {
  __shared__ __align__(1024) uint8_t lds[T::kLds];
  const int n_tiles = (P.N + T::BQ - 1) / T::BQ, k_tiles = (P.K + T::BP - 1) / T::BP;
  int64_t w;
  if (!item_of(blockIdx.x, static_cast<int64_t>(P.E) * n_tiles * k_tiles, w)) return;
  const int per = n_tiles * k_tiles;
  const int e = static_cast<int>(w / per);
  int nt, kt;
  place_in_band(static_cast<int>(w - static_cast<int64_t>(e) * per), n_tiles, k_tiles, nt, kt);
  const int n0 = nt * T::BQ, k0 = kt * T::BP;
  // the expert's token blocks
  const int b0 = groups::chunks_before(P.offsets, e, P.E, P.R, kFp8Block);
  int lo = __builtin_amdgcn_readfirstlane(P.offsets[e]), hi = __builtin_amdgcn_readfirstlane(P.offsets[e + 1]);
  groups::clamp_pair(lo, hi, P.R);
  int steps = (hi - lo + kFp8Block - 1) / kFp8Block;
  steps = max(0, min(steps, P.blocks - b0));   // offsets that are not monotone stay inside the buffers

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = threadIdx.x & 63, lg = lane / 16, r = lane % 16;
  Source<T> src;
  src.last_pieces = 8;
  src.step_p = static_cast<uint32_t>(P.K) * kFp8Block;
  src.step_q = static_cast<uint32_t>(P.N) * kFp8Block;
  src.p.base = reinterpret_cast<uint64_t>(P.X) + (static_cast<uint64_t>(b0) * P.K + k0) * kFp8Block;
  src.p.bytes = static_cast<uint32_t>(min(T::BP, P.K - k0)) * kFp8Block;
  src.q.base = reinterpret_cast<uint64_t>(P.Y) + (static_cast<uint64_t>(b0) * P.N + n0) * kFp8Block;
  src.q.bytes = static_cast<uint32_t>(min(T::BQ, P.N - n0)) * kFp8Block;
#pragma unroll
  for (int j = 0; j < T::kCopiesP; j++) {
    int row, piece;
    copy_place((wave * T::kCopiesP + j) * 8, row, piece);
    src.vp[j] = row * kFp8Block + piece * 16;
  }
#pragma unroll
  for (int j = 0; j < T::kCopiesQ; j++) {
    int row, piece;
    copy_place((wave * T::kCopiesQ + j) * 8, row, piece);
    src.vq[j] = row * kFp8Block + piece * 16;
  }
  static_assert(T::BQ % kWave == 0 && T::BQ + T::BP <= T::kThreadsT, "one scale copy per wave serves both operands");
  const int slot0 = wave * kWave;
  const bool of_q = slot0 < T::BQ;
  src.s.base = of_q ? reinterpret_cast<uint64_t>(P.Y_sf) + (static_cast<uint64_t>(b0) * P.N + n0) * 4
                    : reinterpret_cast<uint64_t>(P.X_sf) + (static_cast<uint64_t>(b0) * P.K + k0) * 4;
  src.s.bytes = 4 * static_cast<uint32_t>(of_q ? min(T::BQ, P.N - n0) : min(T::BP, P.K - k0));
  src.step_s = 4 * static_cast<uint32_t>(of_q ? P.N : P.K);
  src.vs = 4 * static_cast<uint32_t>(slot0 + lane - (of_q ? 0 : T::BQ));

  src.s = uniform(src.s);
  src.step_s = uniform(src.step_s);

  float4v acc[T::TP][T::TQ];
  contract<T, true>(src, lds, steps, acc);

  const int wp = wave % T::WP, wq = wave / T::WP;
#pragma unroll
  for (int j = 0; j < T::TQ; j++) {
    const int n = n0 + (wq * T::TQ + j) * 16 + r;
    if (n >= P.N) continue;
    const int64_t row = (static_cast<int64_t>(e) * P.N + n) * P.K;
#pragma unroll
    for (int ti = 0; ti < T::TP; ti++) {
      const int k = k0 + (ti / T::kPerHalf) * kFp8Block + wp * (kFp8Block / T::WP) + (ti % T::kPerHalf) * 16 + 4 * lg;
      if (k >= P.K) continue;
      if (MODE == kWgradF32)
        *reinterpret_cast<float4v *>(static_cast<float *>(P.D) + row + k) = acc[ti][j];
      else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(P.D) + row + k) = bf16x4(acc[ti][j]);
    }
  }
}

template <class T, Mode MODE>
hipError_t run_gemm(GemmParams p, hipStream_t stream) {
  p.n_tiles = MODE == kSwigluFp8 ? p.N / 2 / kFp8Block : (p.N + T::BP - 1) / T::BP;
  const int64_t items = groups::max_chunks(p.R, p.E, T::BQ) * p.n_tiles;
  const int64_t grid = (items + kXcds - 1) / kXcds * kXcds;
  if (grid > 0)
    hipLaunchKernelGGL((gemm_kernel<T, MODE>), dim3(static_cast<uint32_t>(grid)), dim3(T::kThreadsT), 0, stream, p);
  return hipGetLastError();
}

template <class T, Mode MODE>
hipError_t run_wgrad(const WgradParams &p, hipStream_t stream) {
  const int64_t items = static_cast<int64_t>(p.E) * ((p.N + T::BQ - 1) / T::BQ) * ((p.K + T::BP - 1) / T::BP);
  const int64_t grid = (items + kXcds - 1) / kXcds * kXcds;
  hipLaunchKernelGGL((wgrad_kernel<T, MODE>), dim3(static_cast<uint32_t>(grid)), dim3(T::kThreadsT), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm(const GemmParams &p, bool swiglu, hipStream_t stream) {
  if (swiglu) return run_gemm<Tile<64, 256, 1, 4, 2>, kSwigluFp8>(p, stream);
  return run_gemm<Tile<128, 128, 2, 2, 2>, kNone>(p, stream);
}

hipError_t launch_wgrad(const WgradParams &p, bool bf16, hipStream_t stream) {
  if (bf16) return run_wgrad<Tile<128, 128, 2, 2, 2>, kWgradBf16>(p, stream);
  return run_wgrad<Tile<128, 128, 2, 2, 2>, kWgradF32>(p, stream);
}

}  // namespace fp8
}  // namespace moe
