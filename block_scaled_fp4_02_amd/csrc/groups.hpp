// Groups of consecutive rows given by offsets on the device (expert groups, sequences), cut
// into chunks: which group and rows does chunk number `i` hold?  Every wave works it out for
// itself, 256 groups per round (four per lane, their offsets loaded together), and the result
// is uniform over the wave.  Offsets are clamped to [0, limit] and made monotone pairwise, and
// numbers of chunks stop at 2^30, more than monotone offsets can give, so bad values give wrong
// groups but never a row outside [0, limit).
#pragma once

#include "common.hpp"

namespace moe {
namespace groups {

struct Chunk {
  int group;   // group of the chunk
  int lo, hi;  // rows [lo, hi) of the group
  int index;   // chunk number within the group: rows from lo + index * size
  int total;   // chunks of the group
};

__device__ __forceinline__ int wave_inclusive_sum(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int u = __shfl_up(v, o, kWave);
    if (lane >= o) v += u;
  }
  return v;
}

// The sum of two numbers of chunks, each up to 2^30.
constexpr uint32_t kMostChunks = 1u << 30;
__device__ __forceinline__ int plus(int a, int b) {
  return static_cast<int>(min(static_cast<uint32_t>(a) + static_cast<uint32_t>(b), kMostChunks));
}

__device__ __forceinline__ int wave_inclusive_chunks(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int u = __shfl_up(v, o, kWave);
    if (lane >= o) v = plus(v, u);
  }
  return v;
}

__device__ __forceinline__ void clamp_pair(int &lo, int &hi, int limit) {
  lo = lo < 0 ? 0 : (lo > limit ? limit : lo);
  hi = hi < lo ? lo : (hi > limit ? limit : hi);
}

// The groups base + 4 * lane + q, q = 0..3, of this lane: rows [lo, hi), n chunks of `size` rows; and
// the chunks of all lanes' groups up to this lane's last and in all.
struct Round {
  int lo[4], hi[4], n[4];
  int mine, incl, sum;
};

__device__ __forceinline__ Round round_of(const int32_t *off, int G, int limit, int size, int base) {
  Round r;
  const int g0 = base + 4 * static_cast<int>(threadIdx.x & 63);
  int o[5];
#pragma unroll
  for (int q = 0; q < 5; q++) o[q] = off[min(g0 + q, G)];
  r.mine = 0;
#pragma unroll
  for (int q = 0; q < 4; q++) {
    r.lo[q] = o[q];
    r.hi[q] = o[q + 1];
    clamp_pair(r.lo[q], r.hi[q], limit);
    r.n[q] = g0 + q < G ? (r.hi[q] - r.lo[q] + size - 1) / size : 0;
    r.mine = plus(r.mine, r.n[q]);
  }
  r.incl = wave_inclusive_chunks(r.mine);
  r.sum = __builtin_amdgcn_readlane(r.incl, kWave - 1);
  return r;
}

// Chunk `i` of a round's (i < r.sum), read out of the lane that has it (the first one, where sums stopped
// at 2^30; its index is one of the lane's chunks all the same).
__device__ __forceinline__ Chunk pick(const Round &r, int base, int i) {
  const int local = i - (r.incl - r.mine);
  const int src = __builtin_ctzll(__ballot(local >= 0 && local < r.mine));
  Chunk c = {};
  c.index = __builtin_amdgcn_readlane(local, src);
#pragma unroll
  for (int q = 0; q < 4; q++) {
    const int n = __builtin_amdgcn_readlane(r.n[q], src);
    if (c.total == 0) {
      if (c.index < n) {
        c.group = base + 4 * src + q;
        c.total = n;
        c.lo = __builtin_amdgcn_readlane(r.lo[q], src);
        c.hi = __builtin_amdgcn_readlane(r.hi[q], src);
      } else {
        c.index -= n;
      }
    }
  }
  return c;
}

// Chunks of all groups before group g (g <= G).
__device__ __forceinline__ int chunks_before(const int32_t *off, int g, int G, int limit, int size) {
  int sum = 0;
  for (int base = 0; base < g; base += 4 * kWave) {
    const Round r = round_of(off, G, limit, size, base);
    const int g0 = base + 4 * static_cast<int>(threadIdx.x & 63);
#pragma unroll
    for (int q = 0; q < 4; q++)
      if (g0 + q < g) sum = plus(sum, r.n[q]);
  }
  return __builtin_amdgcn_readlane(wave_inclusive_chunks(sum), kWave - 1);
}

// Chunk `i` of the concatenated chunks of all groups; false if there are not that many.
__device__ __forceinline__ bool find_chunk(const int32_t *off, int G, int limit, int size, int i, Chunk &c) {
  for (int base = 0; base < G; base += 4 * kWave) {
    const Round r = round_of(off, G, limit, size, base);
    if (i < r.sum) {
      c = pick(r, base, i);
      return true;
    }
    i -= r.sum;
  }
  return false;
}

// The chunk that `index(total)` names, a number that depends on the number of all chunks (negative:
// none); false if there is no such chunk.  Up to 256 groups' offsets are read once.
template <class F>
__device__ __forceinline__ bool find_chunk_of_all(const int32_t *off, int G, int limit, int size, F index, int &i, Chunk &c) {
  const Round first = round_of(off, G, limit, size, 0);
  int total = first.sum;
  for (int base = 4 * kWave; base < G; base += 4 * kWave) total = plus(total, round_of(off, G, limit, size, base).sum);
  i = index(total);
  if (i < 0) return false;
  if (i < first.sum) {
    c = pick(first, 0, i);
    return true;
  }
  return find_chunk(off, G, limit, size, i, c);
}

// Most chunks that R rows in G groups can hold (host): a group's last chunk may be short.
inline int64_t max_chunks(int64_t R, int64_t G, int64_t size) { return R / size + (R < G ? R : G); }

}  // namespace groups
}  // namespace moe
