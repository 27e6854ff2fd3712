// The global norm of many gradient tensors and their clipping:
//
//   norm = sqrt(sum over all elements of x^2),   out = x min(1, max_norm / (norm + 1e-6))
//
// Both are one read of the tensors (the second also a write), so HBM bounds them, and launches where
// the tensors are small.  The tensors' addresses travel in the kernel's arguments, up to kTable of them
// in a launch, so nothing is copied to the device and a captured launch holds what it needs.  A
// workgroup takes one chunk of kChunk elements of one tensor.  Squares are taken and summed in 64 bits:
// gfx950's vector units do that as fast as in 32, and no gradient is too large or too small for it.
// 1.2 GB of binary32: norm 194 us (6.2 TB/s), clipping 454 us (5.3 TB/s read and written; a copy 4.95).
#include "grad_clip.hpp"

#pragma clang fp contract(off)

namespace moe {
namespace grad {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kTable = 320;      // (10 KB of arguments: 301 tensors of 4 million elements 46 us with 96 a launch, 22 with all in one)
constexpr int kChunkBits = 14;   // (600 million binary32 elements, norm and clipping, 1341 us, with 15 1315; 1.2 billion bf16 1287 and 1320)
constexpr int64_t kChunk = int64_t(1) << kChunkBits;

enum { kBf16 = 1, kWide = 2 };   // kWide: 16 bytes at a time

// (Whole words only: the table lies in the kernel's arguments and is read with scalar loads, which
// drop the low bits of an address's base and of its offset, so neither may be built from byte indexes.)
struct Entry {
  const void *src;
  void *dst;
  int64_t n;
  int32_t first;               // chunks of the tensors before it
  int32_t flags;
};
struct Table {
  Entry e[kTable];
  int32_t count, chunks;
};

int64_t chunks_of(int64_t n) { return (n + kChunk - 1) / kChunk; }

// The tensor of chunk b, and its elements [lo, hi): a lane looks at an entry, all of them at once (a
// binary search would wait for the table eight times over).
__device__ __forceinline__ Entry find(const Table &t, int b, int64_t &lo, int64_t &hi) {
  const int lane = threadIdx.x & 63;
  int before = 0;
#pragma unroll
  for (int base = 0; base < kTable; base += kWave) {
    const int i = min(base + lane, kTable - 1);
    before += __popcll(__ballot(base + lane < t.count && t.e[i].first <= b));
  }
  const Entry e = t.e[__builtin_amdgcn_readfirstlane(before - 1)];
  lo = static_cast<int64_t>(b - e.first) << kChunkBits;
  hi = lo + kChunk < e.n ? lo + kChunk : e.n;
  return e;
}

// sum + the square of a binary32 value.
__device__ __forceinline__ double add_square(double sum, uint32_t bits) {
  const double v = __uint_as_float(bits);
  return fma(v, v, sum);
}
template <bool BF16>
__device__ __forceinline__ float element(const void *p, int64_t i) {
  return BF16 ? bf16_to_f32(static_cast<const uint16_t *>(p)[i]) : static_cast<const float *>(p)[i];
}

// The sum of v over the workgroup, in thread 0.
template <int THREADS>
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double part[THREADS / kWave];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x / kWave] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < THREADS / kWave; w++) s += part[w];
  return s;
}

// A whole chunk is 8 (bf16) or 16 pieces of 16 bytes for each thread, kAhead of which are loaded at once.
constexpr int kAhead = 8;

template <bool BF16>
__device__ __forceinline__ double sum_of_squares(const Entry &e, int64_t lo, int64_t hi) {
  constexpr int kPer = BF16 ? 3 : 2, kPieces = static_cast<int>(kChunk >> kPer) / kThreads;   // kPer: log2 of the elements in 16 bytes
  double sum[4] = {0.0, 0.0, 0.0, 0.0};
  auto add = [&](const u32x4 &v) {
#pragma unroll
    for (int c = 0; c < 4; c++) {
      if (BF16) sum[c] = add_square(sum[c], v[c] << 16);
      sum[c] = add_square(sum[c], BF16 ? v[c] & 0xffff0000u : v[c]);
    }
  };
  if (e.flags & kWide) {
    const u32x4 *p = static_cast<const u32x4 *>(e.src) + (lo >> kPer) + threadIdx.x;
    if (hi - lo == kChunk) {
#pragma unroll
      for (int a = 0; a < kPieces; a += kAhead) {
        u32x4 v[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; u++) v[u] = p[(a + u) * kThreads];
#pragma unroll
        for (int u = 0; u < kAhead; u++) add(v[u]);
      }
      lo = hi;
    } else {
      const int n = static_cast<int>((hi - lo) >> kPer);
#pragma unroll 4
      for (int a = threadIdx.x; a < n; a += kThreads) add(p[a - static_cast<int>(threadIdx.x)]);
      lo += static_cast<int64_t>(n) << kPer;
    }
  }
  for (int64_t a = lo + threadIdx.x; a < hi; a += kThreads) sum[0] = add_square(sum[0], __float_as_uint(element<BF16>(e.src, a)));
  return (sum[0] + sum[1]) + (sum[2] + sum[3]);
}

__global__ __launch_bounds__(kThreads) void norm_kernel(const Table t, double *partial) {
  int64_t lo, hi;
  const Entry e = find(t, blockIdx.x, lo, hi);
  const double sum = block_sum<kThreads>(e.flags & kBf16 ? sum_of_squares<true>(e, lo, hi) : sum_of_squares<false>(e, lo, hi));
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

constexpr int kSumThreads = 1024;
__global__ __launch_bounds__(kSumThreads) void sum_kernel(const double *partial, int64_t n, float *norm) {
  double sum = 0.0;
  for (int64_t a = threadIdx.x; a < n; a += 8 * kSumThreads) {   // (eight loads at once)
    double v[8];
#pragma unroll
    for (int u = 0; u < 8; u++) v[u] = a + u * kSumThreads < n ? partial[a + u * kSumThreads] : 0.0;
#pragma unroll
    for (int u = 0; u < 8; u++) sum += v[u];
  }
  sum = block_sum<kSumThreads>(sum);
  if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(sum));
}

__device__ __forceinline__ uint32_t scaled_pair(uint32_t v, float s) {
  return f32_to_bf16(__uint_as_float(v << 16) * s) | (static_cast<uint32_t>(f32_to_bf16(__uint_as_float(v & 0xffff0000u) * s)) << 16);
}

template <bool BF16>
__device__ __forceinline__ void scale(const Entry &e, int64_t lo, int64_t hi, float s) {
  constexpr int kPer = BF16 ? 3 : 2, kPieces = static_cast<int>(kChunk >> kPer) / kThreads;
  auto scaled = [&](u32x4 v) {
#pragma unroll
    for (int c = 0; c < 4; c++) v[c] = BF16 ? scaled_pair(v[c], s) : __float_as_uint(__uint_as_float(v[c]) * s);
    return v;
  };
  if (e.flags & kWide) {
    const u32x4 *p = static_cast<const u32x4 *>(e.src) + (lo >> kPer) + threadIdx.x;
    u32x4 *q = static_cast<u32x4 *>(e.dst) + (lo >> kPer) + threadIdx.x;
    if (hi - lo == kChunk) {
#pragma unroll
      for (int a = 0; a < kPieces; a += kAhead) {
        u32x4 v[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; u++) v[u] = p[(a + u) * kThreads];
#pragma unroll
        for (int u = 0; u < kAhead; u++) __builtin_nontemporal_store(scaled(v[u]), &q[(a + u) * kThreads]);
      }
      return;
    }
    const int n = static_cast<int>((hi - lo) >> kPer);
#pragma unroll 4
    for (int a = threadIdx.x; a < n; a += kThreads) q[a - static_cast<int>(threadIdx.x)] = scaled(p[a - static_cast<int>(threadIdx.x)]);
    lo += static_cast<int64_t>(n) << kPer;
  }
  for (int64_t a = lo + threadIdx.x; a < hi; a += kThreads) {
    const float v = element<BF16>(e.src, a) * s;
    if (BF16) static_cast<uint16_t *>(e.dst)[a] = f32_to_bf16(v);
    else static_cast<float *>(e.dst)[a] = v;
  }
}

__global__ __launch_bounds__(kThreads) void clip_kernel(const Table t, const float *norm, float max_norm) {
  int64_t lo, hi;
  // from the last chunk back: what the norm read last is still in the memory-side cache (600 million binary32
  // elements in place 1382 -> 1352 us, with stores past the caches 1341)
  const Entry e = find(t, t.chunks - 1 - blockIdx.x, lo, hi);
  float s = max_norm / (*norm + 1e-6f);
  if (s >= 1.0f || max_norm == INFINITY) s = 1.0f;   // (otherwise a NaN norm stays one)
  if (s == 1.0f && e.src == e.dst) return;           // x * 1 = x
  if (e.flags & kBf16) scale<true>(e, lo, hi, s);
  else scale<false>(e, lo, hi, s);
}

// Calls launch(table) for the non-empty tensors, kTable at a time.
template <class F>
hipError_t for_tables(const moe_tensor *tensors, int count, bool write, F launch) {
  Table t = {};
  for (int i = 0; i <= count; i++) {
    if (i < count && tensors[i].n > 0) {
      const moe_tensor &x = tensors[i];
      Entry &e = t.e[t.count++];
      e.src = x.src;
      e.dst = x.dst ? x.dst : x.src;
      e.n = x.n;
      e.first = t.chunks;
      const uintptr_t at = reinterpret_cast<uintptr_t>(e.src) | (write ? reinterpret_cast<uintptr_t>(e.dst) : 0);
      e.flags = (x.dtype == MOE_DTYPE_BF16 ? kBf16 : 0) | (at % 16 == 0 ? kWide : 0);
      t.chunks += static_cast<int32_t>(chunks_of(x.n));
    }
    if (t.count > 0 && (t.count == kTable || i == count)) {
      const hipError_t e = launch(t);
      if (e != hipSuccess) return e;
      t.count = t.chunks = 0;
    }
  }
  return hipSuccess;
}

}  // namespace

size_t norm_ws_bytes(const moe_tensor *tensors, int count) {
  int64_t chunks = 0;
  for (int i = 0; i < count; i++) chunks += chunks_of(tensors[i].n);
  return static_cast<size_t>(chunks < 2 ? 2 : chunks) * sizeof(double);
}

hipError_t launch_norm(const moe_tensor *tensors, int count, float *norm, void *ws, hipStream_t stream) {
  double *partial = static_cast<double *>(ws);
  int64_t done = 0;
  const hipError_t e = for_tables(tensors, count, false, [&](const Table &t) {
    hipLaunchKernelGGL(norm_kernel, dim3(t.chunks), dim3(kThreads), 0, stream, t, partial + done);
    done += t.chunks;
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(sum_kernel, dim3(1), dim3(kSumThreads), 0, stream, partial, done, norm);
  return hipGetLastError();
}

hipError_t launch_clip(const moe_tensor *tensors, int count, const float *norm, float max_norm, hipStream_t stream) {
  return for_tables(tensors, count, true, [&](const Table &t) {
    hipLaunchKernelGGL(clip_kernel, dim3(t.chunks), dim3(kThreads), 0, stream, t, norm, max_norm);
    return hipGetLastError();
  });
}

}  // namespace grad
}  // namespace moe
