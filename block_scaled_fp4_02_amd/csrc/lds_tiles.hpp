// Pieces that the grouped products with tiles in LDS share (fp8_gemm.hip, bf16_gemm.hip): copies from
// memory straight into LDS and the waits for them, the order of tiles over the XCDs, and wide stores.
#pragma once

#include "common.hpp"

namespace moe {
namespace lds {

typedef int int4x __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;

constexpr uint32_t kOob = 0x80000000u;   // an offset that no operand's range reaches

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
// ONCE: the bytes are read by this copy alone and need not stay in the caches.
template <bool ONCE = false>
__device__ __forceinline__ void copy16(const Buf &b, uint32_t lds, uint32_t voff) {
  if constexpr (ONCE)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen nt lds"
                 :
                 : "s"(lds), "v"(voff), "s"(descriptor(b))
                 : "memory");
  else
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

// copy16 if `yes` (uniform).  The branch is inside the statement so that the loop around it stays
// one block to the compiler, which otherwise runs out of registers.
__device__ __forceinline__ void copy16_if(bool yes, const Buf &b, uint32_t lds, uint32_t voff) {
  asm volatile("s_cmp_eq_u32 %3, 0\n\ts_cbranch_scc1 .Lnocopy%=\n\ts_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds\n.Lnocopy%=:"
               :
               : "s"(lds), "v"(voff), "s"(descriptor(b)), "s"(uniform(yes ? 1u : 0u))
               : "memory", "scc");
}

// Waits until at most `LATER` copies of this wave are under way and its LDS reads are done,
// then for the workgroup: after it every wave's older copies are in LDS, and no wave still
// reads the buffer that the stage before used.
template <int LATER>
__device__ __forceinline__ void arrive() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(LATER) : "memory");
}

// Between LDS writes and reads of different lanes of one wave, either way round.  LDS serves a wave in
// order, so no instruction is needed; the compiler, to which the lanes' addresses need not overlap,
// has to keep the order as well.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ uint2 bf16x4(const float4v &v) {
  return make_uint2(f32_to_bf16(v[0]) | (static_cast<uint32_t>(f32_to_bf16(v[1])) << 16),
                    f32_to_bf16(v[2]) | (static_cast<uint32_t>(f32_to_bf16(v[3])) << 16));
}

// STREAM: past the caches, which the operands of the other tiles keep (a large tile's launch writes
// far more than the next one reads soon).
template <bool STREAM>
__device__ __forceinline__ void store16(void *at, const uint4 &v) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  if (STREAM) __builtin_nontemporal_store(u32x4{v.x, v.y, v.z, v.w}, static_cast<u32x4 *>(at));
  else *static_cast<uint4 *>(at) = v;
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

}  // namespace lds
}  // namespace moe
