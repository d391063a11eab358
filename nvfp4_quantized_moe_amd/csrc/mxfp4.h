// Microscaled 4-bit floats (MXFP4): E2M1 codes, two to a byte with the first in
// the low nibble, and for each 32 of them a power of two, held as its exponent
// + 127 in a byte (0xFF: every value of the block is NaN).
//
//   scale of a block  e = floor(log2 amax) - 2 (MX_SCALE_FLOOR: values in
//                     (6, 8) 2^e saturate) or the smallest e with amax <= 6 2^e
//                     (MX_SCALE_CEIL), at least -127
//   code              E2M1 nearest to x 2^-e, ties to the even code
//
// Both are exact: e comes from the maximum's exponent bits, and gfx950's
// conversions divide by the power of two and round once (all BF16 values at 12
// scales compared, the subnormal scale 2^-127 and saturation among them).
#pragma once
#include "common.h"

namespace nvfp4 {

constexpr int kMxBlock = 32;     // elements that share a scale
constexpr int kMxGroup = 128;    // rows of codes end on whole groups: four scales, one word
constexpr int kMxMaxK = 262144;  // elements along a row of codes

__device__ __forceinline__ int mx_padded(int n) { return (n + kMxGroup - 1) & ~(kMxGroup - 1); }

// A block's scale, as float32 bits, from those of its largest magnitude: the
// exponent field less 2, or one more where the fraction is above 1/2 (MX_SCALE_CEIL:
// `up` carries into the exponent there). Of BF16 values the low halves of `amax`
// may hold anything. The conversions read the exponent bits alone, 0 as 2^-127 and
// 255 as NaN; the field is the scale's code. Infinities and NaN: no scale holds them.
constexpr uint32_t kMxUpF32 = 0x3FFFFFu, kMxUpBf16 = 0x3F0000u;
__device__ __forceinline__ uint32_t mx_scale_bits(uint32_t amax, uint32_t up) {
  const int e = (int)((amax + up) & 0x7F800000u) - 0x01000000;
  return amax >= 0x7F800000u ? 0x7F800000u : (uint32_t)(e > 0 ? e : 0);
}

typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
// Larger magnitude, in each half, of two pairs of BF16 magnitudes.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a), __builtin_bit_cast(u16x2_t, b)));
}

// Two values to the byte SEL of a word of codes.
template <int SEL>
__device__ __forceinline__ uint32_t mx_encode2(uint32_t old, uint32_t bf16_pair, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(bf16x2_t, bf16_pair), scale, SEL);
}
template <int SEL>
__device__ __forceinline__ uint32_t mx_encode2(uint32_t old, float a, float b, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, a, b, scale, SEL);
}

// Eight values of a row as they are loaded: their largest magnitude (float32
// bits, the low half open for BF16) and their codes.
template <typename T>
struct MxVec8;
template <>
struct MxVec8<uint16_t> {
  static constexpr uint32_t kUp = kMxUpBf16;
  uint4 v;
  template <bool PAST>  // not to stay in the caches
  __device__ __forceinline__ void load(const uint16_t* p) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    const u32x4* at = reinterpret_cast<const u32x4*>(p);
    v = __builtin_bit_cast(uint4, PAST ? __builtin_nontemporal_load(at) : *at);
  }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ uint32_t amax() const {
    constexpr uint32_t m = 0x7FFF7FFFu;
    const uint32_t a = max_u16x2(max_u16x2(v.x & m, v.y & m), max_u16x2(v.z & m, v.w & m));
    return max(a, a << 16);
  }
  __device__ __forceinline__ uint32_t codes(float s) const {
    uint32_t w = mx_encode2<0>(0u, v.x, s);
    w = mx_encode2<1>(w, v.y, s);
    w = mx_encode2<2>(w, v.z, s);
    return mx_encode2<3>(w, v.w, s);
  }
};
template <>
struct MxVec8<float> {
  static constexpr uint32_t kUp = kMxUpF32;
  float4 a, b;
  template <bool>  // (two loads of every other 16 bytes: past the caches 52 us for 51)
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m = max(m, __float_as_uint((&a.x)[i]) & 0x7FFFFFFFu);
      m = max(m, __float_as_uint((&b.x)[i]) & 0x7FFFFFFFu);
    }
    return m;
  }
  __device__ __forceinline__ uint32_t codes(float s) const {
    uint32_t w = mx_encode2<0>(0u, a.x, a.y, s);
    w = mx_encode2<1>(w, a.z, a.w, s);
    w = mx_encode2<2>(w, b.x, b.y, s);
    return mx_encode2<3>(w, b.z, b.w, s);
  }
};

}  // namespace nvfp4
