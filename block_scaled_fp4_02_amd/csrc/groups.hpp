// Groups of consecutive rows given by offsets on the device (expert groups, sequences), cut
// into chunks: which group and rows does chunk number `i` hold?  Every wave works it out for
// itself, 256 groups per round (four per lane, their offsets loaded together), and the result
// is uniform over the wave.  Offsets are clamped to [0, limit] and made monotone pairwise, so
// bad values give wrong groups but never a row outside [0, limit).
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

__device__ __forceinline__ void clamp_pair(int &lo, int &hi, int limit) {
  lo = lo < 0 ? 0 : (lo > limit ? limit : lo);
  hi = hi < lo ? lo : (hi > limit ? limit : hi);
}

// Chunks of `size` rows held by the groups base + 4 * lane + q, q = 0..3, of this lane.
__device__ __forceinline__ void lane_chunks(const int32_t *off, int G, int limit, int size, int base, int (&n)[4]) {
  const int g0 = base + 4 * static_cast<int>(threadIdx.x & 63);
  int o[5];
#pragma unroll
  for (int q = 0; q < 5; q++) o[q] = off[min(g0 + q, G)];
#pragma unroll
  for (int q = 0; q < 4; q++) {
    int lo = o[q], hi = o[q + 1];
    clamp_pair(lo, hi, limit);
    n[q] = g0 + q < G ? (hi - lo + size - 1) / size : 0;
  }
}

// Chunks of all groups before group g (g <= G).
__device__ __forceinline__ int chunks_before(const int32_t *off, int g, int G, int limit, int size) {
  int sum = 0;
  for (int base = 0; base < g; base += 4 * kWave) {
    int n[4];
    lane_chunks(off, G, limit, size, base, n);
    const int g0 = base + 4 * static_cast<int>(threadIdx.x & 63);
#pragma unroll
    for (int q = 0; q < 4; q++)
      if (g0 + q < g) sum += n[q];
  }
  return __builtin_amdgcn_readlane(wave_inclusive_sum(sum), kWave - 1);
}

// Chunk `i` of the concatenated chunks of all groups; false if there are not that many.
__device__ __forceinline__ bool find_chunk(const int32_t *off, int G, int limit, int size, int i, Chunk &c) {
  int before = 0;
  for (int base = 0; base < G; base += 4 * kWave) {
    int n[4];
    lane_chunks(off, G, limit, size, base, n);
    const int mine = n[0] + n[1] + n[2] + n[3];
    const int incl = wave_inclusive_sum(mine);
    const int sum = __builtin_amdgcn_readlane(incl, kWave - 1);
    if (i < before + sum) {
      const int local = i - before - (incl - mine);
      const int src = __builtin_ctzll(__ballot(local >= 0 && local < mine));
      int l = __builtin_amdgcn_readlane(local, src);
      int g = base + 4 * src, total = 0;
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const int nq = __builtin_amdgcn_readlane(n[q], src);
        if (total == 0) {
          if (l < nq) {
            g = base + 4 * src + q;
            total = nq;
          } else {
            l -= nq;
          }
        }
      }
      int lo = __builtin_amdgcn_readfirstlane(off[g]), hi = __builtin_amdgcn_readfirstlane(off[g + 1]);
      clamp_pair(lo, hi, limit);
      c.group = g;
      c.lo = lo;
      c.hi = hi;
      c.index = l;
      c.total = total;
      return true;
    }
    before += sum;
  }
  return false;
}

// Chunks of all groups.
__device__ __forceinline__ int chunk_count(const int32_t *off, int G, int limit, int size) {
  return chunks_before(off, G, G, limit, size);
}

// Most chunks that R rows in G groups can hold (host): a group's last chunk may be short.
inline int64_t max_chunks(int64_t R, int64_t G, int64_t size) { return R / size + (R < G ? R : G); }

}  // namespace groups
}  // namespace moe
