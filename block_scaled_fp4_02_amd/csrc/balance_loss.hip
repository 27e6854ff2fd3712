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
// kTokens tokens of one sequence; loss_sum_kernel adds a sequence's partials (binary64, in a
// fixed order), writes counts and coef, and its last workgroup adds up the loss.  Backward: one
// pass that recomputes p.  Both are bound by HBM: 4 E bytes read per token, and 4 E written
// backward.  No floating-point atomics: results repeat bit for bit.
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
constexpr int kTokens = 32;     // tokens of a chunk (one workgroup), 8 per wave
constexpr int kBatch = 4;       // tokens whose logits a wave loads together
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_huge_valf();

// Wave-wide sum and maximum by lane moves within rows of 16, then across rows; the result of
// the last lane is read as a scalar.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ float dpp(float v, float identity) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(identity), __float_as_int(v), CTRL, ROW_MASK, 0xf, false));
}
__device__ __forceinline__ float last_lane(float v) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), kWave - 1)); }

__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<0x111, 0xf>(v, 0.f);
  v += dpp<0x112, 0xf>(v, 0.f);
  v += dpp<0x114, 0xf>(v, 0.f);
  v += dpp<0x118, 0xf>(v, 0.f);
  v += dpp<0x142, 0xa>(v, 0.f);
  v += dpp<0x143, 0xc>(v, 0.f);
  return last_lane(v);
}
__device__ __forceinline__ float wave_max_all(float v) {
  v = fmaxf(v, dpp<0x111, 0xf>(v, kNegInf));
  v = fmaxf(v, dpp<0x112, 0xf>(v, kNegInf));
  v = fmaxf(v, dpp<0x114, 0xf>(v, kNegInf));
  v = fmaxf(v, dpp<0x118, 0xf>(v, kNegInf));
  v = fmaxf(v, dpp<0x142, 0xa>(v, kNegInf));
  v = fmaxf(v, dpp<0x143, 0xc>(v, kNegInf));
  return last_lane(v);
}

// The chunk of workgroup `b`: rows [first, first + count) of sequence `seq`.
struct Rows {
  int seq, first, count;
};
__device__ __forceinline__ bool rows_of(const int32_t *off, int S, int T, int b, Rows &r) {
  if (off == nullptr) {   // one sequence over all tokens
    r.seq = 0;
    r.first = b * kTokens;
    r.count = min(kTokens, T - r.first);
    return r.count > 0;
  }
  groups::Chunk c;
  if (!groups::find_chunk(off, S, T, kTokens, b, c)) return false;
  r.seq = c.group;
  r.first = c.lo + c.index * kTokens;
  r.count = min(kTokens, c.hi - r.first);
  return true;
}

// A token's logits, expert lane + 64 i in x[i]; lanes past E hold -inf.
template <int NV>
__device__ __forceinline__ void load_logits(const float *logits, int64_t t, int E, float (&x)[NV]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < NV; i++) {
    const int e = lane + kWave * i;
    x[i] = e < E ? logits[t * E + e] : kNegInf;
  }
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
  const float inv = s == 0.f ? 0.f : 1.0f / s;
#pragma unroll
  for (int i = 0; i < NV; i++) x[i] *= inv;
}

template <int NV>
__global__ __launch_bounds__(kThreads) void loss_chunk_kernel(const LossParams P) {
  __shared__ int hist[NV * kWave];
  __shared__ float sums[kWavesB][NV * kWave];
  __shared__ int kept;
  if (blockIdx.x == 0 && threadIdx.x == 0) *P.ticket = 0u;   // for the next kernel's last workgroup
  Rows rows;
  if (!rows_of(P.seq_offsets, P.S, P.T, blockIdx.x, rows)) return;
  const int wave = threadIdx.x / kWave, lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < NV * kWave / kThreads + 1; i++)
    if (static_cast<int>(threadIdx.x) + kThreads * i < NV * kWave) hist[threadIdx.x + kThreads * i] = 0;
  if (threadIdx.x == 0) kept = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < rows.count * P.k; i += kThreads) {
    const int64_t t = rows.first + i / P.k;
    if (P.mask && !P.mask[t]) continue;
    const int id = P.ids[t * P.k + i % P.k];
    if (id >= 0 && id < P.E) atomicAdd(&hist[id], 1);
  }
  if (static_cast<int>(threadIdx.x) < rows.count && (!P.mask || P.mask[rows.first + threadIdx.x])) atomicAdd(&kept, 1);
  float sum[NV];
#pragma unroll
  for (int i = 0; i < NV; i++) sum[i] = 0.f;
#pragma unroll
  for (int b = 0; b < kTokens / kWavesB; b += kBatch) {
    float x[kBatch][NV];
#pragma unroll
    for (int u = 0; u < kBatch; u++) load_logits<NV>(P.logits, rows.first + min(wave + kWavesB * (b + u), rows.count - 1), P.E, x[u]);
#pragma unroll
    for (int u = 0; u < kBatch; u++) {
      const int t = wave + kWavesB * (b + u);
      if (t >= rows.count || (P.mask && !P.mask[rows.first + t])) continue;
      softmax<NV>(x[u]);
#pragma unroll
      for (int i = 0; i < NV; i++) sum[i] += x[u][i];
    }
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

// Workgroup (s, b): experts [64 b, 64 b + 64) of sequence s, 16 waves that stride over its chunks.
constexpr int kSumThreads = 1024;
constexpr int kSumWaves = kSumThreads / kWave;

__global__ __launch_bounds__(kSumThreads) void loss_sum_kernel(const LossParams P) {
  __shared__ double mass[kSumWaves][kWave];
  __shared__ int count[kSumWaves][kWave];
  __shared__ int kept[kSumWaves];
  __shared__ int last;
  const int lane = threadIdx.x & 63, wave = threadIdx.x / kWave;
  const int blocks = (P.E + kWave - 1) / kWave;
  const int s = blockIdx.x / blocks, e = blockIdx.x % blocks * kWave + lane;
  int c0 = 0, n_chunks = (P.T + kTokens - 1) / kTokens;
  if (P.seq_offsets) {
    c0 = groups::chunks_before(P.seq_offsets, s, P.S, P.T, kTokens);
    int lo = __builtin_amdgcn_readfirstlane(P.seq_offsets[s]), hi = __builtin_amdgcn_readfirstlane(P.seq_offsets[s + 1]);
    groups::clamp_pair(lo, hi, P.T);
    n_chunks = (hi - lo + kTokens - 1) / kTokens;
    n_chunks = max(0, min(n_chunks, P.chunks - c0));   // offsets that are not monotone stay inside the workspace
  }
  double m = 0.0;
  int c = 0, n = 0;
  const int64_t at = static_cast<int64_t>(c0) * P.E + min(e, P.E - 1);
#pragma unroll 8
  for (int i = wave; i < n_chunks; i += kSumWaves) {
    m += P.part_sum[at + static_cast<int64_t>(i) * P.E];
    c += P.part_count[at + static_cast<int64_t>(i) * P.E];
  }
  for (int i = threadIdx.x; i < n_chunks; i += kSumThreads) n += P.part_kept[c0 + i];
  n = __builtin_amdgcn_readlane(groups::wave_inclusive_sum(n), kWave - 1);
  mass[wave][lane] = m;
  count[wave][lane] = c;
  if (lane == 0) kept[wave] = n;
  __syncthreads();
  if (wave == 0) {
    m = 0.0;
    c = 0;
    n = 0;
#pragma unroll
    for (int w = 0; w < kSumWaves; w++) {
      m += mass[w][lane];
      c += count[w][lane];
      n += kept[w];
    }
    const double dn = n;
    const double coef = n > 0 ? static_cast<double>(P.E) * c / (dn * dn * P.k * P.S) : 0.0;
    double part = 0.0;
    if (e < P.E) {
      P.counts[static_cast<int64_t>(s) * P.E + e] = c;
      P.coef[static_cast<int64_t>(s) * P.E + e] = static_cast<float>(coef);
      part = coef * m;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) part += __shfl_xor(part, o, kWave);
    if (lane == 0) {
      __hip_atomic_store(&P.part_loss[blockIdx.x], part, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
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

template <int NV>
__global__ __launch_bounds__(kThreads) void backward_kernel(const GradParams P) {
  Rows rows;
  if (!rows_of(P.seq_offsets, P.S, P.T, blockIdx.x, rows)) return;
  const int wave = threadIdx.x / kWave, lane = threadIdx.x & 63;
  const float grad = *P.grad_loss;
  float a[NV];
#pragma unroll
  for (int i = 0; i < NV; i++) {
    const int e = lane + kWave * i;
    a[i] = e < P.E ? grad * P.coef[static_cast<int64_t>(rows.seq) * P.E + e] : 0.f;
  }
#pragma unroll
  for (int b = 0; b < kTokens / kWavesB; b += kBatch) {
    float x[kBatch][NV];
#pragma unroll
    for (int u = 0; u < kBatch; u++) load_logits<NV>(P.logits, rows.first + min(wave + kWavesB * (b + u), rows.count - 1), P.E, x[u]);
#pragma unroll
    for (int u = 0; u < kBatch; u++) {
      const int r = wave + kWavesB * (b + u);
      if (r >= rows.count) continue;
      const int64_t t = rows.first + r;
      float d[NV];
      if (P.mask && !P.mask[t]) {
#pragma unroll
        for (int i = 0; i < NV; i++) d[i] = 0.f;
      } else {
        softmax<NV>(x[u]);
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < NV; i++) dot = fmaf(x[u][i], a[i], dot);
        dot = wave_sum(dot);
#pragma unroll
        for (int i = 0; i < NV; i++) d[i] = x[u][i] * (a[i] - dot);
        if (P.d_topk_w) {
          int id = -1;
          float w = 0.f, dw = 0.f;
          if (lane < P.k) {
            id = P.ids[t * P.k + lane];
            w = P.topk_w[t * P.k + lane];
            dw = P.d_topk_w[t * P.k + lane];
          }
          const float v = w * (dw - wave_sum(w * dw));
          for (int j = 0; j < P.k; j++) {   // in slot order: an expert chosen twice gets both
            const int ej = __builtin_amdgcn_readlane(id, j);
            const float vj = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), j));
#pragma unroll
            for (int i = 0; i < NV; i++)
              if (ej == lane + kWave * i) d[i] += vj;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < NV; i++) {
        const int e = lane + kWave * i;
        if (e < P.E) P.dlogits[t * P.E + e] = d[i];
      }
    }
  }
}

// Logits per lane: the smallest of 1, 2, 4, 8, 16 that holds E.
template <class F>
void by_width(int E, F f) {
  if (E <= 64) f(std::integral_constant<int, 1>());
  else if (E <= 128) f(std::integral_constant<int, 2>());
  else if (E <= 256) f(std::integral_constant<int, 4>());
  else if (E <= 512) f(std::integral_constant<int, 8>());
  else f(std::integral_constant<int, 16>());
}

int64_t chunks_of(bool one_sequence, int T, int S) {
  return one_sequence ? (static_cast<int64_t>(T) + kTokens - 1) / kTokens : groups::max_chunks(T, S, kTokens);
}

size_t align16(size_t n) { return (n + 15) & ~static_cast<size_t>(15); }

}  // namespace

size_t loss_ws_bytes(int T, int E, int S) {
  const size_t chunks = static_cast<size_t>(std::max(chunks_of(true, T, 1), chunks_of(false, T, S)));
  const size_t parts = static_cast<size_t>(S) * ((E + kWave - 1) / kWave);
  return 16 + align16(parts * sizeof(double)) + align16(chunks * 4) + 2 * align16(chunks * E * 4);
}

hipError_t launch_loss(LossParams p, void *ws, hipStream_t stream) {
  const int64_t chunks = chunks_of(p.seq_offsets == nullptr, p.T, p.S);
  p.chunks = static_cast<int>(chunks);
  const size_t parts = static_cast<size_t>(p.S) * ((p.E + kWave - 1) / kWave);
  uint8_t *at = static_cast<uint8_t *>(ws);
  p.ticket = reinterpret_cast<uint32_t *>(at);
  at += 16;
  p.part_loss = reinterpret_cast<double *>(at);
  at += align16(parts * sizeof(double));
  p.part_kept = reinterpret_cast<int32_t *>(at);
  at += align16(static_cast<size_t>(chunks) * 4);
  p.part_count = reinterpret_cast<int32_t *>(at);
  at += align16(static_cast<size_t>(chunks) * p.E * 4);
  p.part_sum = reinterpret_cast<float *>(at);
  by_width(p.E, [&](auto nv) {
    hipLaunchKernelGGL(loss_chunk_kernel<decltype(nv)::value>, dim3(static_cast<uint32_t>(std::max<int64_t>(chunks, 1))),
                       dim3(kThreads), 0, stream, p);
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(loss_sum_kernel, dim3(static_cast<uint32_t>(parts)), dim3(kSumThreads), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_backward(const GradParams &p, hipStream_t stream) {
  const int64_t chunks = chunks_of(p.seq_offsets == nullptr, p.T, p.S);
  if (chunks > 0)
    by_width(p.E, [&](auto nv) {
      hipLaunchKernelGGL(backward_kernel<decltype(nv)::value>, dim3(static_cast<uint32_t>(chunks)), dim3(kThreads), 0, stream, p);
    });
  return hipGetLastError();
}

}  // namespace balance
}  // namespace moe
