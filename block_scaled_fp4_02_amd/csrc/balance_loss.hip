// The router's load-balancing term and its gradient.  For every sequence s of n tokens (those
// that the mask keeps), with p the softmax of a token's E logits and c[s, e] the number of its
// tokens' slots that chose expert e:
//
//   loss = 1/S sum_s sum_e f[s, e] P[s, e],   f = E c / (k n),   P[s, e] = 1/n sum_t p[t, e]
//        = sum_s sum_e coef[s, e] sum_t p[t, e],   coef = E c / (k n^2 S)
//
// The counts are constants of the gradient, so coef is all that the backward pass needs:
// dlogit[t, e] = p (a - sum_e' p a),  a = dloss coef[s].  The same pass adds the gradient that
// reaches the logits through the routing weights w = softmax of the chosen logits:
// dlogit[t, id_j] += w_j (dw_j - sum_i w_i dw_i).
//
// Forward: loss_chunk_kernel reads the logits once (a wave per token, E / 64 logits per lane in
// registers) and leaves one partial row of probability sums and counts per chunk of at most
// 32 tokens of one sequence; loss_sum_kernel adds a sequence's partials (binary64, in a
// fixed order), writes counts and coef, and its last workgroup adds up the loss.  Backward: one
// pass that recomputes p.  Both are bound by HBM: 4 E bytes read per token, and 4 E written
// backward.  No floating-point atomics: results repeat bit for bit.  16384 tokens of 256 experts: loss 14.7 us,
// gradient 10.0 us (the floors are 3.3 and 6.6); 13.3 and 8.0 on inputs that stayed in the caches, as in the
// comparisons below.
#include "common.hpp"
#include "balance_loss.hpp"
#include "groups.hpp"

#include <algorithm>
#include <type_traits>

#pragma clang fp contract(off)

namespace moe {
namespace balance {
namespace {

constexpr int kThreads = 256;
constexpr int kWavesB = kThreads / kWave;
// Most tokens of a wave, all loaded before the first is used.  A chunk is a workgroup's tokens.
constexpr int kMaxPer = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_huge_valf();

// Wave-wide sum and maximum: rotations within rows of 16 lanes, then one lane of each of the four rows.
template <int N>
__device__ __forceinline__ float rotated(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(v), __float_as_int(v), 0x120 + N, 0xf, 0xf, false));
}
__device__ __forceinline__ float lane_of(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
__device__ __forceinline__ float wave_sum(float v) {
  v += rotated<1>(v);
  v += rotated<2>(v);
  v += rotated<4>(v);
  v += rotated<8>(v);
  return (lane_of(v, 0) + lane_of(v, 16)) + (lane_of(v, 32) + lane_of(v, 48));
}
__device__ __forceinline__ float wave_max_all(float v) {
  v = fmaxf(v, rotated<1>(v));
  v = fmaxf(v, rotated<2>(v));
  v = fmaxf(v, rotated<4>(v));
  v = fmaxf(v, rotated<8>(v));
  return fmaxf(fmaxf(lane_of(v, 0), lane_of(v, 16)), fmaxf(lane_of(v, 32), lane_of(v, 48)));
}

// The chunk of `size` tokens of workgroup `b`: rows [first, first + count) of sequence `seq`.
struct Rows {
  int seq, first, count;
};
__device__ __forceinline__ bool rows_of(const int32_t *off, int S, int T, int size, int b, Rows &r) {
  if (off == nullptr) {   // one sequence over all tokens
    r.seq = 0;
    r.first = b * size;
    r.count = min(size, T - r.first);
    return r.count > 0;
  }
  groups::Chunk c;
  if (!groups::find_chunk(off, S, T, size, b, c)) return false;
  r.seq = c.group;
  r.first = c.lo + c.index * size;
  r.count = min(size, c.hi - r.first);
  return true;
}

// The logits of this wave's tokens (wave, wave + 4, ... of the chunk, the last one again past its end),
// expert lane + 64 i in x[u][i] with -inf past E, and which of the tokens count.
template <int NV, int PER>
__device__ __forceinline__ void load_tokens(const float *logits, const uint8_t *mask, const Rows &rows, int wave, int E,
                                            float (&x)[PER][NV], bool (&keep)[PER]) {
  const int lane = threadIdx.x & 63;
  uint8_t m[PER];
#pragma unroll
  for (int u = 0; u < PER; u++) {
    const int64_t t = rows.first + min(wave + kWavesB * u, rows.count - 1);
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const int e = lane + kWave * i;
      x[u][i] = e < E ? logits[t * E + e] : kNegInf;
    }
    m[u] = mask ? mask[t] : 1;
  }
#pragma unroll
  for (int u = 0; u < PER; u++) keep[u] = wave + kWavesB * u < rows.count && m[u] != 0;
}

// x becomes its softmax over the wave (a row of -inf alone has no probability anywhere).
template <int NV>
__device__ __forceinline__ void softmax(float (&x)[NV]) {
  float m = x[0];
#pragma unroll
  for (int i = 1; i < NV; i++) m = fmaxf(m, x[i]);
  m = wave_max_all(m);
  const bool none = m == kNegInf;   // (a NaN among -inf also lands here and stays NaN below)
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; i++) {
    x[i] = __builtin_amdgcn_exp2f((x[i] - (none ? 0.f : m)) * kLog2e);
    s += x[i];
  }
  s = wave_sum(s);
  const float inv = s == 0.f ? 0.f : __builtin_amdgcn_rcpf(s);
#pragma unroll
  for (int i = 0; i < NV; i++) x[i] *= inv;
}

template <int NV, int PER>
__global__ __launch_bounds__(kThreads) void loss_chunk_kernel(const LossParams P) {
  __shared__ int hist[NV * kWave];
  __shared__ float sums[kWavesB][NV * kWave];
  __shared__ int kept;
  if (blockIdx.x == 0 && threadIdx.x == 0) *P.ticket = 0u;   // for the next kernel's last workgroup
  Rows rows;
  if (!rows_of(P.seq_offsets, P.S, P.T, kWavesB * PER, blockIdx.x, rows)) return;
  const int wave = threadIdx.x / kWave, lane = threadIdx.x & 63;
  float x[PER][NV];
  bool keep[PER];
  load_tokens<NV, PER>(P.logits, P.mask, rows, wave, P.E, x, keep);
  for (int e = threadIdx.x; e < NV * kWave; e += kThreads) hist[e] = 0;
  if (threadIdx.x == 0) kept = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < rows.count * P.k; i += kThreads) {
    const int64_t at = static_cast<int64_t>(rows.first) * P.k + i;
    const int id = P.ids[at];
    if ((!P.mask || P.mask[rows.first + i / P.k]) && id >= 0 && id < P.E) atomicAdd(&hist[id], 1);
  }
  if (static_cast<int>(threadIdx.x) < rows.count && (!P.mask || P.mask[rows.first + threadIdx.x])) atomicAdd(&kept, 1);
  float sum[NV];
#pragma unroll
  for (int i = 0; i < NV; i++) sum[i] = 0.f;
#pragma unroll
  for (int u = 0; u < PER; u++) {
    softmax<NV>(x[u]);
#pragma unroll
    for (int i = 0; i < NV; i++) sum[i] += keep[u] ? x[u][i] : 0.f;   // (a dropped row may hold anything)
  }
#pragma unroll
  for (int i = 0; i < NV; i++) sums[wave][lane + kWave * i] = sum[i];
  __syncthreads();
  for (int e = threadIdx.x; e < P.E; e += kThreads) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWavesB; w++) s += sums[w][e];
    P.part_sum[static_cast<int64_t>(blockIdx.x) * P.E + e] = s;
    P.part_count[static_cast<int64_t>(blockIdx.x) * P.E + e] = hist[e];
  }
  if (threadIdx.x == 0) P.part_kept[blockIdx.x] = kept;
}

// Workgroup (s, b): a block of EXPERTS experts of sequence s, THREADS / EXPERTS threads for each that
// stride over the sequence's chunks: 64 x 4 where that makes 64 workgroups, else 16 x 64 (one sequence
// of 16384 tokens and 256 experts: 13.4 us with the chunks' kernel, 17.0 in 64 x 4; four of 1024 tokens
// and 1024 experts: 19.2 and 17.0).
template <int EXPERTS, int THREADS>
__global__ __launch_bounds__(THREADS) void loss_sum_kernel(const LossParams P) {
  constexpr int kParts = THREADS / EXPERTS;
  __shared__ double mass[kParts][EXPERTS];
  __shared__ int count[kParts][EXPERTS];
  __shared__ int kept[THREADS / kWave];
  __shared__ int last;
  const int lane = threadIdx.x & 63, wave = threadIdx.x / kWave;
  const int ex = threadIdx.x % EXPERTS, part = threadIdx.x / EXPERTS;
  const int blocks = (P.E + EXPERTS - 1) / EXPERTS;
  const int s = blockIdx.x / blocks, e = blockIdx.x % blocks * EXPERTS + ex;
  int c0 = 0, n_chunks = (P.T + P.chunk - 1) / P.chunk;
  if (P.seq_offsets) {
    c0 = groups::chunks_before(P.seq_offsets, s, P.S, P.T, P.chunk);
    int lo = __builtin_amdgcn_readfirstlane(P.seq_offsets[s]), hi = __builtin_amdgcn_readfirstlane(P.seq_offsets[s + 1]);
    groups::clamp_pair(lo, hi, P.T);
    n_chunks = (hi - lo + P.chunk - 1) / P.chunk;
    n_chunks = max(0, min(n_chunks, P.chunks - c0));   // offsets that are not monotone stay inside the workspace
  }
  double m = 0.0;
  int c = 0, n = 0;
  const int64_t at = static_cast<int64_t>(c0) * P.E + min(e, P.E - 1);
#pragma unroll 8
  for (int i = part; i < n_chunks; i += kParts) {
    m += P.part_sum[at + static_cast<int64_t>(i) * P.E];
    c += P.part_count[at + static_cast<int64_t>(i) * P.E];
  }
  for (int i = threadIdx.x; i < n_chunks; i += THREADS) n += P.part_kept[c0 + i];
  n = __builtin_amdgcn_readlane(groups::wave_inclusive_sum(n), kWave - 1);
  mass[part][ex] = m;
  count[part][ex] = c;
  if (lane == 0) kept[wave] = n;
  __syncthreads();
  if (wave == 0) {
    // the lanes of an expert share its parts and then add up
    constexpr int kShare = kWave / EXPERTS;
    m = 0.0;
    c = 0;
    n = 0;
#pragma unroll
    for (int p = 0; p < kParts / kShare; p++) {
      m += mass[kShare * p + lane / EXPERTS][ex];
      c += count[kShare * p + lane / EXPERTS][ex];
    }
#pragma unroll
    for (int o = EXPERTS; o < kWave; o *= 2) {
      m += __shfl_xor(m, o, kWave);
      c += __shfl_xor(c, o, kWave);
    }
#pragma unroll
    for (int w = 0; w < THREADS / kWave; w++) n += kept[w];
    const double dn = n;
    const double coef = n > 0 ? static_cast<double>(P.E) * c / (dn * dn * P.k * P.S) : 0.0;
    double loss = 0.0;
    if (e < P.E && lane < EXPERTS) {
      P.counts[static_cast<int64_t>(s) * P.E + e] = c;
      P.coef[static_cast<int64_t>(s) * P.E + e] = static_cast<float>(coef);
      loss = coef * m;
    }
#pragma unroll
    for (int o = EXPERTS / 2; o > 0; o >>= 1) loss += __shfl_xor(loss, o, kWave);
    if (lane == 0) {
      __hip_atomic_store(&P.part_loss[blockIdx.x], loss, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      last = __hip_atomic_fetch_add(P.ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
    }
  }
  __syncthreads();
  if (!last || wave != 0) return;
  // the last workgroup to arrive: every other one's part is visible; fixed order
  double loss = 0.0;
  for (unsigned i = lane; i < gridDim.x; i += kWave)
    loss += __hip_atomic_load(&P.part_loss[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) loss += __shfl_xor(loss, o, kWave);
  if (lane == 0) *P.loss = static_cast<float>(loss);
}

template <int NV, int PER>
__global__ __launch_bounds__(kThreads) void backward_kernel(const GradParams P) {
  Rows rows;
  if (!rows_of(P.seq_offsets, P.S, P.T, kWavesB * PER, blockIdx.x, rows)) return;
  const int wave = threadIdx.x / kWave, lane = threadIdx.x & 63;
  float x[PER][NV];
  bool keep[PER];
  load_tokens<NV, PER>(P.logits, P.mask, rows, wave, P.E, x, keep);
  int id[PER];
  float w[PER], dw[PER];
  if (P.d_topk_w) {
#pragma unroll
    for (int u = 0; u < PER; u++) {
      const int64_t at = static_cast<int64_t>(rows.first + min(wave + kWavesB * u, rows.count - 1)) * P.k + min(lane, P.k - 1);
      id[u] = P.ids[at];
      w[u] = lane < P.k ? P.topk_w[at] : 0.f;
      dw[u] = lane < P.k ? P.d_topk_w[at] : 0.f;
    }
  }
  const float grad = *P.grad_loss;
  float a[NV];
#pragma unroll
  for (int i = 0; i < NV; i++) {
    const int e = lane + kWave * i;
    a[i] = e < P.E ? grad * P.coef[static_cast<int64_t>(rows.seq) * P.E + e] : 0.f;
  }
#pragma unroll
  for (int u = 0; u < PER; u++) {
    softmax<NV>(x[u]);
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < NV; i++) dot = fmaf(x[u][i], a[i], dot);
    dot = wave_sum(dot);
#pragma unroll
    for (int i = 0; i < NV; i++) x[u][i] *= a[i] - dot;
    if (P.d_topk_w) {
      const float v = w[u] * (dw[u] - wave_sum(w[u] * dw[u]));
      for (int j = 0; j < P.k; j++) {   // in slot order: an expert chosen twice gets both
        const int ej = __builtin_amdgcn_readlane(id[u], j);
        const float vj = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), j));
#pragma unroll
        for (int i = 0; i < NV; i++)
          if (ej == lane + kWave * i) x[u][i] += vj;
      }
    }
    const int r = wave + kWavesB * u;
    if (r >= rows.count) continue;
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const int e = lane + kWave * i;
      if (e < P.E) P.dlogits[static_cast<int64_t>(rows.first + r) * P.E + e] = keep[u] ? x[u][i] : 0.f;
    }
  }
}

// Calls f with the logits per lane, the smallest of 1, 2, 4, 8, 16 that holds E, and the tokens per
// wave.  Forward: up to 64 logits per lane, halved while that leaves CUs without work, since every
// chunk writes a row of partials (16384 tokens of 256 experts: 8 tokens 13.5 us, 4: 16.5, 2: 24).
// Backward, which writes none: two tokens or one (the same batch: 8.5 us, with 8 tokens 9.9).
template <int NV, class F>
int by_tokens(int wanted, F f) {
  constexpr int kPer = std::min(kMaxPer, 64 / NV);
  if constexpr (kPer >= 8)
    if (wanted >= 8) return f(std::integral_constant<int, NV>(), std::integral_constant<int, 8>());
  if (wanted >= 4) return f(std::integral_constant<int, NV>(), std::integral_constant<int, 4>());
  if (wanted >= 2) return f(std::integral_constant<int, NV>(), std::integral_constant<int, 2>());
  return f(std::integral_constant<int, NV>(), std::integral_constant<int, 1>());
}
template <class F>
int by_size(int wanted, int E, F f) {
  if (E <= 64) return by_tokens<1>(wanted, f);
  if (E <= 128) return by_tokens<2>(wanted, f);
  if (E <= 256) return by_tokens<4>(wanted, f);
  if (E <= 512) return by_tokens<8>(wanted, f);
  return by_tokens<16>(wanted, f);
}
int wanted_forward(int T) { return T / (256 * kWavesB); }
int wanted_backward(int T) { return std::min(2, T / (2 * 256 * kWavesB)); }

int chunk_size(int wanted, int E) {
  return by_size(wanted, E, [](auto, auto per) { return kWavesB * decltype(per)::value; });
}

int64_t chunks_of(bool one_sequence, int T, int S, int size) {
  return one_sequence ? (static_cast<int64_t>(T) + size - 1) / size : groups::max_chunks(T, S, size);
}

size_t align16(size_t n) { return (n + 15) & ~static_cast<size_t>(15); }

bool many_sums(int E, int S) { return static_cast<int64_t>(S) * ((E + 63) / 64) >= 64; }
size_t sum_blocks(int E, int S) {
  const int experts = many_sums(E, S) ? 64 : 16;
  return static_cast<size_t>(S) * ((E + experts - 1) / experts);
}

}  // namespace

size_t loss_ws_bytes(int T, int E, int S) {
  const int size = chunk_size(wanted_forward(T), E);
  const size_t chunks = static_cast<size_t>(std::max(chunks_of(true, T, 1, size), chunks_of(false, T, S, size)));
  return 16 + align16(sum_blocks(E, S) * sizeof(double)) + align16(chunks * 4) + 2 * align16(chunks * E * 4);
}

hipError_t launch_loss(LossParams p, void *ws, hipStream_t stream) {
  const int wanted = wanted_forward(p.T);
  p.chunk = chunk_size(wanted, p.E);
  const size_t chunks = static_cast<size_t>(chunks_of(p.seq_offsets == nullptr, p.T, p.S, p.chunk));
  p.chunks = static_cast<int>(chunks);
  uint8_t *at = static_cast<uint8_t *>(ws);
  p.ticket = reinterpret_cast<uint32_t *>(at);
  at += 16;
  p.part_loss = reinterpret_cast<double *>(at);
  at += align16(sum_blocks(p.E, p.S) * sizeof(double));
  p.part_kept = reinterpret_cast<int32_t *>(at);
  at += align16(chunks * 4);
  p.part_count = reinterpret_cast<int32_t *>(at);
  at += align16(chunks * p.E * 4);
  p.part_sum = reinterpret_cast<float *>(at);
  by_size(wanted, p.E, [&](auto nv, auto per) {
    hipLaunchKernelGGL((loss_chunk_kernel<decltype(nv)::value, decltype(per)::value>),
                       dim3(static_cast<uint32_t>(std::max<size_t>(chunks, 1))), dim3(kThreads), 0, stream, p);
    return 0;
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 grid(static_cast<uint32_t>(sum_blocks(p.E, p.S)));
  if (many_sums(p.E, p.S)) hipLaunchKernelGGL((loss_sum_kernel<64, 256>), grid, dim3(256), 0, stream, p);
  else hipLaunchKernelGGL((loss_sum_kernel<16, 1024>), grid, dim3(1024), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_backward(const GradParams &p, hipStream_t stream) {
  const int wanted = wanted_backward(p.T);
  const int64_t chunks = chunks_of(p.seq_offsets == nullptr, p.T, p.S, chunk_size(wanted, p.E));
  if (chunks > 0)
    by_size(wanted, p.E, [&](auto nv, auto per) {
      hipLaunchKernelGGL((backward_kernel<decltype(nv)::value, decltype(per)::value>), dim3(static_cast<uint32_t>(chunks)),
                         dim3(kThreads), 0, stream, p);
      return 0;
    });
  return hipGetLastError();
}

}  // namespace balance
}  // namespace moe
