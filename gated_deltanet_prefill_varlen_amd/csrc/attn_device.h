// Matrix-core helpers of the attention over the paged 8-bit cache.
#pragma once

#include "cache_device.h"

namespace gdn {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896341f;

// Four codes of one dword as two dwords of bf16: exact (an int8 has 7 bits and
// a sign, an e4m3 value 4 significant bits; bf16 holds 8).
template <bool I8>
__device__ __forceinline__ void codes_to_bf16(uint32_t w, uint32_t* out) {
  if constexpr (I8) {
    float f[4];
    decode4<true>(w, f);   // the low halves of these fp32 are zero
    out[0] = __builtin_amdgcn_perm(__float_as_uint(f[1]), __float_as_uint(f[0]), 0x07060302);
    out[1] = __builtin_amdgcn_perm(__float_as_uint(f[3]), __float_as_uint(f[2]), 0x07060302);
  } else {
    out[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, false));
    out[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, true));
  }
}

// Eight codes as a matrix operand.
template <bool I8>
__device__ __forceinline__ bf16x8 codes_to_operand(uint32_t lo, uint32_t hi) {
  u32x4 r;
  uint32_t o[2];
  codes_to_bf16<I8>(lo, o);
  r.x = o[0];
  r.y = o[1];
  codes_to_bf16<I8>(hi, o);
  r.z = o[0];
  r.w = o[1];
  return __builtin_bit_cast(bf16x8, r);
}

// The first n bytes of a dword.
__device__ __forceinline__ uint32_t first_bytes(int n) { return n >= 4 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << (8 * n)) - 1; }

// Four codes with 0 for each NaN, whose places become bits at, at + 1, .. of *found.
template <bool I8>
__device__ __forceinline__ uint32_t without_nan(uint32_t w, int at, uint32_t* found) {
  if constexpr (I8) return w;
  const uint32_t nan = (((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7;
  *found |= ((nan * 0x10204080u) >> 28) << at;   // the four flags side by side
  return w & ~(nan * 0xFFu);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Value scales from 2^-100 to 2^122 meet probabilities in one fp32 product.
// A key whose scale is over 2^kLarge counts for the running maximum with what
// its scale is over: a softmax is the same against any measure, and against
// that one no probability times scale passes 2^kLarge, which leaves the sums of
// 2^30 keys with codes up to 448 room.  The measure is then above the largest
// score, but only where that key outweighs all others in the output.
constexpr float kLarge = 88.f;

// A page's factor of its scores.  Past fp32 it is the largest number: a score
// of 0 stays 0.
constexpr float kMostFactor = 0x1.fffffep127f;

}  // namespace gdn
