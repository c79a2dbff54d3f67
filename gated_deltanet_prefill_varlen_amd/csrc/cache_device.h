// Device helpers of the paged 8-bit key/value cache: its codes, its scales
// and its addresses.
#pragma once

#include "cache_internal.h"
#include "gdn_device.h"

namespace gdn {

// The smallest scale of a page; also a page's scale before its first token.
constexpr float kMinScale = 0x1p-100f;

// ---------------------------------------------------------------- codes --
// Four codes of one dword as fp32 (exact).
template <bool I8>
__device__ __forceinline__ void decode4(uint32_t w, float* f) {
  if constexpr (I8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = (float)(int8_t)(w >> (8 * i));
  } else {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
  }
}

// Four fp32 values already divided by their scale as codes: nearest, ties to
// even.  Values beyond the largest code (infinities only: the scale covers
// the others) saturate; NaN is e4m3's NaN, and 0 in int8.
template <bool I8>
__device__ __forceinline__ uint32_t encode4(const float* f) {
  float c[4];
  constexpr float top = I8 ? 127.f : 448.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = fminf(fmaxf(f[i], -top), top);
    if (f[i] != f[i]) c[i] = I8 ? 0.f : f[i];
  }
  if constexpr (I8) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w |= ((uint32_t)(int32_t)rintf(c[i]) & 0xFFu) << (8 * i);
    return w;
  } else {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], w, true);
  }
}

// Codes rounded again to a scale 1/ratio times theirs (ratio a power of two
// below 1).
template <bool I8>
__device__ __forceinline__ uint32_t recode4(uint32_t w, float ratio) {
  float f[4];
  decode4<I8>(w, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] *= ratio;
  return encode4<I8>(f);
}

// --------------------------------------------------------------- scales --
// The smallest power of two s with amax <= s * largest code, from the bits of
// amax (finite, >= 0): amax = m 2^a and the largest code = t 2^b, 1 <= m, t
// < 2, give 2^(a - b) while m <= t and twice that beyond.
template <bool I8>
__device__ __forceinline__ float scale_for(float amax) {
  constexpr uint32_t top = I8 ? 0x7E0000u : 0x600000u;   // fraction bits of 127 and 448
  constexpr int b = I8 ? 6 : 8;
  if (!(amax > 0x1p-94f)) return kMinScale;              // also every subnormal
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - b + ((u & 0x7FFFFFu) > top);
  return fmaxf(__uint_as_float((uint32_t)e << 23), kMinScale);
}

__device__ __forceinline__ float finite_abs(float x) {
  const float y = fabsf(x);
  return y < __builtin_inff() ? y : 0.f;   // NaN and infinities count as 0
}

// ------------------------------------------------------------- addresses --
// First byte of a (page, head)'s codes; the same in k and v.
__device__ __forceinline__ int64_t page_base(const CacheRef& c, int64_t page, int h) {
  return ((page * c.Hkv + h) * c.dim) << c.page_shift;
}

// ------------------------------------------------------------------ bf16 --
// Two fp32 as packed bf16, nearest even, NaN kept.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 f = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
}
__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

}  // namespace gdn
