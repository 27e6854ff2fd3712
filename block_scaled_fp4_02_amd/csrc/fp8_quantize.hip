// FP8 (E4M3FN) quantisation with one binary32 scale per 128 elements, in the three forms that
// the FP8 grouped GEMM and its gradients read: rows (1 x 128 along a row: activations, output
// gradients), weights (128 x 128 tiles, optionally with the transposed copy that the input
// gradient contracts over), and tokens (128 x 1 down each column of a group of rows, stored
// with the tokens of a block contiguous: the operands of the weight gradient).
//
// The pages hold their FP8 data as one-byte scales of the FP4 operands only ("Cracking the
// SM120 Shared Memory Ceiling", section "The Shared Memory Calculation"); the steps are this
// library's (fp8_round.hpp) and bit-exact.  All three kernels are bound by HBM: a bf16
// element is 2 bytes read and 1 byte written.
#include "common.hpp"
#include "fp8_round.hpp"
#include "groups.hpp"

#pragma clang fp contract(off)

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kLanes = 16;            // lanes that share a block's row: 8 elements each
constexpr int kRows = kThreads / kLanes;

struct Vec8 {
  float v[8];
};

// Eight consecutive elements from element offset `at` (a multiple of 8) as they stand in memory.
template <bool BF16>
struct Raw8 {
  uint4 w[BF16 ? 1 : 2];
};
template <bool BF16>
__device__ __forceinline__ Raw8<BF16> load_raw8(const void *x, int64_t at) {
  Raw8<BF16> r;
  const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(x) + at * (BF16 ? 2 : 4));
#pragma unroll
  for (int i = 0; i < (BF16 ? 1 : 2); i++) r.w[i] = p[i];
  return r;
}
template <bool BF16>
__device__ __forceinline__ Vec8 values(const Raw8<BF16> &r) {
  if constexpr (BF16) {
    const uint32_t p[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
    Vec8 v;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v.v[2 * i] = __uint_as_float(p[i] << 16);
      v.v[2 * i + 1] = __uint_as_float(p[i] & 0xffff0000u);
    }
    return v;
  } else {
    const uint4 a = r.w[0], b = r.w[1];
    return {{__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z), __uint_as_float(a.w), __uint_as_float(b.x),
             __uint_as_float(b.y), __uint_as_float(b.z), __uint_as_float(b.w)}};
  }
}

__device__ __forceinline__ uint32_t amax8(const Vec8 &r) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) m = max(m, abs_bits(r.v[i]));
  return m;
}

__device__ __forceinline__ uint2 codes8(const Vec8 &r, const Fp8Block &b) {
  return make_uint2(fp8_quantize4(r.v[0], r.v[1], r.v[2], r.v[3], b), fp8_quantize4(r.v[4], r.v[5], r.v[6], r.v[7], b));
}

__device__ __forceinline__ uint32_t max_over16(uint32_t m) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), o, kWave)));
  return m;
}

// 16 lanes per block of 128: 256 contiguous bytes of bf16, one scale.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void quant_rows_kernel(const void *__restrict__ x, uint32_t nblk, uint32_t per_row,
                                                              int C, uint8_t *__restrict__ q, float *__restrict__ sf) {
  const uint32_t b = blockIdx.x * kRows + threadIdx.x / kLanes;
  const uint32_t bc = b < nblk ? b : nblk - 1;
  const uint32_t row = bc / per_row;
  const int c = static_cast<int>(bc - row * per_row) * kFp8Block + 8 * static_cast<int>(threadIdx.x % kLanes);
  const int64_t at = static_cast<int64_t>(row) * C + c;
  Raw8<BF16> raw = {};
  if (c < C) raw = load_raw8<BF16>(x, at);
  const Vec8 r = values(raw);
  const Fp8Block s = fp8_block(max_over16(amax8(r)));
  if (b >= nblk) return;
  if (c < C) *reinterpret_cast<uint2 *>(q + at) = codes8(r, s);
  if (threadIdx.x % kLanes == 0) sf[b] = s.scale;
}

// Byte b of four words, for b = 0..3.
__device__ __forceinline__ void turn4(const uint32_t (&w)[4], uint32_t (&t)[4]) {
  const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400), b = __builtin_amdgcn_perm(w[1], w[0], 0x07030602);
  const uint32_t c = __builtin_amdgcn_perm(w[3], w[2], 0x05010400), d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602);
  t[0] = __builtin_amdgcn_perm(c, a, 0x05040100);
  t[1] = __builtin_amdgcn_perm(c, a, 0x07060302);
  t[2] = __builtin_amdgcn_perm(d, b, 0x05040100);
  t[3] = __builtin_amdgcn_perm(d, b, 0x07060302);
}

// Columns of a 128 x 128 tile of codes in LDS as rows of `out`: column c of the tile is row c0 + c
// (< rows_end), its elements stand from column n0 (< cols_end) on.  A thread turns 16 x 4 codes, and
// 8 neighbouring lanes write one row's 128 bytes (with 8 bytes a lane and neighbouring lanes on
// other rows the weight quantiser takes 400 us instead of 330 us for 403 M weights).
typedef uint32_t TileRow[kFp8Block / 4 + 1];   // one word of padding
__device__ __forceinline__ void store_turned(const TileRow *tile, uint8_t *out, int c0, int rows_end, int n0, int cols_end,
                                             int64_t stride) {
  const int part = threadIdx.x % 8, word = threadIdx.x / 8;
  uint32_t t[4][4];   // [group of 4 elements][column]
#pragma unroll
  for (int i = 0; i < 4; i++) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; j++) w[j] = tile[16 * part + 4 * i + j][word];
    turn4(w, t[i]);
  }
#pragma unroll
  for (int b = 0; b < 4; b++) {
    const int row = c0 + 4 * word + b, col = n0 + 16 * part;
    if (row < rows_end && col < cols_end)
      *reinterpret_cast<uint4 *>(out + row * stride + col) = make_uint4(t[0][b], t[1][b], t[2][b], t[3][b]);
  }
}

// One 128 x 128 tile of one expert per workgroup; a thread holds 8 columns of 8 rows.
template <bool BF16>
__global__ __launch_bounds__(kThreads, 6) void quant_weights_kernel(const void *__restrict__ w, int N, int K, int nb, int kb,
                                                                 uint8_t *__restrict__ q, float *__restrict__ sf,
                                                                 uint8_t *__restrict__ qt, float *__restrict__ sft) {
  __shared__ uint32_t wave_amax[kThreads / kWave];
  __shared__ TileRow tile[kFp8Block];   // codes
  const int tk = blockIdx.x % kb, tn = blockIdx.x / kb % nb;
  const int64_t e = blockIdx.x / kb / nb;
  const int n0 = tn * kFp8Block, k0 = tk * kFp8Block;
  const int lr = threadIdx.x / kLanes, lc = threadIdx.x % kLanes;
  const int64_t base = e * N * K;
  Raw8<BF16> r[8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const int n = n0 + lr + kRows * i, k = k0 + 8 * lc;
    r[i] = {};
    if (n < N && k < K) r[i] = load_raw8<BF16>(w, base + static_cast<int64_t>(n) * K + k);
  }
#pragma unroll
  for (int i = 0; i < 8; i++) m = max(m, amax8(values(r[i])));
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), o, kWave)));
  if (threadIdx.x % kWave == 0) wave_amax[threadIdx.x / kWave] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / kWave; i++) m = max(m, wave_amax[i]);
  const Fp8Block s = fp8_block(m);
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const int row = lr + kRows * i, n = n0 + row, k = k0 + 8 * lc;
    const uint2 c = codes8(values(r[i]), s);
    if (n < N && k < K) *reinterpret_cast<uint2 *>(q + base + static_cast<int64_t>(n) * K + k) = c;
    tile[row][2 * lc] = c.x;
    tile[row][2 * lc + 1] = c.y;
  }
  if (threadIdx.x == 0) {
    sf[(e * nb + tn) * kb + tk] = s.scale;
    if (qt) sft[(e * kb + tk) * nb + tn] = s.scale;
  }
  if (!qt) return;
  __syncthreads();
  store_turned(tile, qt + base, k0, K, n0, N, N);
}

// One block of up to 128 rows of a group, 128 columns, per workgroup: a scale per column, and
// the codes of a column contiguous: q [block][C][128], zeros behind the group's last row.
template <bool BF16>
__global__ __launch_bounds__(kThreads, 6) void quant_tokens_kernel(const void *__restrict__ x, int64_t rows_x,
                                                                const int32_t *__restrict__ rows,
                                                                const int32_t *__restrict__ offsets, int E, int R, int C,
                                                                int col_tiles, uint8_t *__restrict__ q,
                                                                float *__restrict__ sf) {
  __shared__ uint32_t col_amax[kThreads / kWave][kFp8Block];
  __shared__ TileRow tile[kFp8Block];
  const int blk = blockIdx.x / col_tiles, c0 = blockIdx.x % col_tiles * kFp8Block;
  groups::Chunk g;
  if (!groups::find_chunk(offsets, E, R, kFp8Block, blk, g)) return;
  const int first = g.lo + g.index * kFp8Block, count = min(kFp8Block, g.hi - first);
  const int lr = threadIdx.x / kLanes, lc = threadIdx.x % kLanes;
  const int c = c0 + 8 * lc;
  Raw8<BF16> r[8];
  int64_t src[8];
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const int t = lr + kRows * i;
    int64_t p = first + min(t, count - 1);
    if (rows) p = rows[p];
    src[i] = p < 0 ? 0 : (p >= rows_x ? rows_x - 1 : p);
  }
#pragma unroll
  for (int i = 0; i < 8; i++) {
    r[i] = {};
    if (lr + kRows * i < count && c < C) r[i] = load_raw8<BF16>(x, src[i] * C + c);
  }
  // column maxima: over the thread's 8 rows, the wave's 4 row groups, then the 4 waves
  uint32_t m[8] = {};
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const Vec8 v = values(r[i]);
#pragma unroll
    for (int j = 0; j < 8; j++) m[j] = max(m[j], abs_bits(v.v[j]));
  }
#pragma unroll
  for (int j = 0; j < 8; j++) {
    m[j] = max(m[j], static_cast<uint32_t>(__shfl_xor(static_cast<int>(m[j]), 16, kWave)));
    m[j] = max(m[j], static_cast<uint32_t>(__shfl_xor(static_cast<int>(m[j]), 32, kWave)));
  }
  if (threadIdx.x % kWave < kLanes) {
#pragma unroll
    for (int j = 0; j < 8; j++) col_amax[threadIdx.x / kWave][8 * lc + j] = m[j];
  }
  __syncthreads();
  Fp8Block s[8];
#pragma unroll
  for (int j = 0; j < 8; j++) {
#pragma unroll
    for (int w = 0; w < kThreads / kWave; w++) m[j] = max(m[j], col_amax[w][8 * lc + j]);
    s[j] = fp8_block(m[j]);
    if (lr == 0 && c + j < C) sf[static_cast<int64_t>(blk) * C + c + j] = s[j].scale;
  }
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const Vec8 v = values(r[i]);
#pragma unroll
    for (int h = 0; h < 2; h++)
      tile[lr + kRows * i][2 * lc + h] =
          fp8_pack4(fp8_quotient(v.v[4 * h], s[4 * h]), fp8_quotient(v.v[4 * h + 1], s[4 * h + 1]),
                    fp8_quotient(v.v[4 * h + 2], s[4 * h + 2]), fp8_quotient(v.v[4 * h + 3], s[4 * h + 3]));
  }
  __syncthreads();
  store_turned(tile, q + static_cast<int64_t>(blk) * C * kFp8Block, c0, C, 0, kFp8Block, kFp8Block);
}

}  // namespace

hipError_t launch_quantize_fp8(const void *x, int x_dtype, int64_t rows, int C, uint8_t *q, float *sf, hipStream_t stream) {
  const int per_row = (C + kFp8Block - 1) / kFp8Block;
  const uint32_t nblk = static_cast<uint32_t>(rows * per_row);
  if (nblk > 0) {
    const auto k = x_dtype == MOE_DTYPE_BF16 ? quant_rows_kernel<true> : quant_rows_kernel<false>;
    hipLaunchKernelGGL(k, dim3((nblk + kRows - 1) / kRows), dim3(kThreads), 0, stream, x, nblk,
                       static_cast<uint32_t>(per_row), C, q, sf);
  }
  return hipGetLastError();
}

hipError_t launch_quantize_fp8_weights(const void *w, int w_dtype, int E, int N, int K, uint8_t *q, float *sf, uint8_t *qt,
                                       float *sft, hipStream_t stream) {
  const int nb = (N + kFp8Block - 1) / kFp8Block, kb = (K + kFp8Block - 1) / kFp8Block;
  const auto k = w_dtype == MOE_DTYPE_BF16 ? quant_weights_kernel<true> : quant_weights_kernel<false>;
  hipLaunchKernelGGL(k, dim3(static_cast<uint32_t>(E) * nb * kb), dim3(kThreads), 0, stream, w, N, K, nb, kb, q, sf, qt, sft);
  return hipGetLastError();
}

hipError_t launch_quantize_fp8_tokens(const void *x, int x_dtype, int64_t rows_x, const int32_t *rows,
                                      const int32_t *offsets, int E, int64_t R, int C, uint8_t *q, float *sf,
                                      hipStream_t stream) {
  const int col_tiles = (C + kFp8Block - 1) / kFp8Block;
  const int64_t grid = groups::max_chunks(R, E, kFp8Block) * col_tiles;
  if (grid > 0) {
    const auto k = x_dtype == MOE_DTYPE_BF16 ? quant_tokens_kernel<true> : quant_tokens_kernel<false>;
    hipLaunchKernelGGL(k, dim3(static_cast<uint32_t>(grid)), dim3(kThreads), 0, stream, x, rows_x, rows, offsets, E,
                       static_cast<int>(R), C, col_tiles, q, sf);
  }
  return hipGetLastError();
}

}  // namespace moe
