// FP8 rounding steps shared by the FP8 quantisers and the GEMM epilogue that quantises: block
// scale s = amax / 448, element code e4m3_rne(min(|x| / s, 448)) with the sign of x, every
// step one correctly rounded binary32 operation (callers compile these with contraction
// off).  A block whose maximum is 0, or so small that s underflows to 0, gets signed zeros.  A
// block that holds an infinity or a NaN gets scale NaN and codes 0: all its values are NaN.
#pragma once

#include <stdint.h>

#include "nvfp4_round.hpp"

namespace moe {

constexpr int kFp8Block = 128;   // elements (rows, tokens) that share one scale
constexpr float kFp8Max = 448.0f;

// Smallest scale that block_quotient serves.  Its remainder a - q s has to be exact, and E4M3's lowest
// rounding border is 2^-10: a quotient just below has steps of 2^-34 and a scale from 2^-92 on steps of
// at least 2^-115, so the remainder is a multiple of 2^-149, binary32's smallest number.  (Below that
// bound ties went to the wrong code now and then.  E2M1's lowest border is 2^-2, hence the lower bound
// of block_divisor.)
constexpr float kFp8FastFrom = 0x1p-92f;

// Block maxima are taken over the magnitudes' bits as integers: the order of non-negative
// floats, with infinity above every finite value and NaN above infinity.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

struct Fp8Block {
  BlockDivisor d;
  float scale;   // stored scale
  bool zero;     // codes are (signed) zeros
};

__device__ __forceinline__ Fp8Block fp8_block(uint32_t amax_bits) {
  Fp8Block b;
  const float amax = __uint_as_float(amax_bits);
  const bool bad = amax_bits >= 0x7f800000u;
  b.scale = bad ? __uint_as_float(0x7fc00000u) : amax / kFp8Max;
  b.zero = bad || b.scale == 0.f;
  b.d = block_divisor(b.zero ? 1.0f : b.scale, b.zero ? 0.f : amax);
  b.d.fast = b.d.fast && b.d.b >= kFp8FastFrom;
  return b;
}

// Signed quotient v / s clamped to the E4M3 range.  Both branches give the correctly rounded
// quotient as far as codes go (below 2^-11 the fast one may be a step off, which rounds to 0 all the
// same); the plain division serves scales near the ends of the binary32 range.
__device__ __forceinline__ float fp8_quotient(float v, const Fp8Block &b) {
  if (b.zero) return __builtin_copysignf(0.f, v);
  const float a = fabsf(v);
  const float u = b.d.fast ? block_quotient(a, b.d) : a / b.d.b;
  return __builtin_copysignf(fminf(u, kFp8Max), v);
}

// Four codes of already clamped quotients, the first in the low byte (hardware conversion,
// round to nearest even).
__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d) {
  int w = 0;
  w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  return static_cast<uint32_t>(w);
}

__device__ __forceinline__ uint32_t fp8_quantize4(float a, float b, float c, float d, const Fp8Block &s) {
  return fp8_pack4(fp8_quotient(a, s), fp8_quotient(b, s), fp8_quotient(c, s), fp8_quotient(d, s));
}

}  // namespace moe
