// Reductions over the 64 lanes of a wave whose result every lane holds: four
// DPP steps inside each row of 16 lanes, then the gfx950 lane swaps across
// rows and halves. No LDS traffic, and one order of additions, so a float
// sum is reproducible.
#pragma once
#include "common.h"

namespace nvfp4 {

constexpr int kDppXor1 = 0xB1;         // quad_perm [1, 0, 3, 2]
constexpr int kDppXor2 = 0x4E;         // quad_perm [2, 3, 0, 1]
constexpr int kDppHalfMirror = 0x141;  // joins the quads of 8 lanes, once each quad holds one value
constexpr int kDppMirror = 0x140;      // joins the halves of 16 lanes, once each half holds one value

// (Every lane of these patterns has a source, so the value for lanes without one
// is never taken; as the constant 0 it lets the compiler fold the move into
// the operation that uses it.)
template <int CTRL>
__device__ __forceinline__ int dpp_i32(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
  return __builtin_bit_cast(float, dpp_i32<CTRL>(__builtin_bit_cast(int, v)));
}

// The two operands of the step across rows of 16 (or halves of 32): the value
// of the even row (lower half) and of the odd row (upper half), in all lanes.
typedef unsigned u32x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u32x2_t rows16(uint32_t v) { return __builtin_amdgcn_permlane16_swap(v, v, false, false); }
__device__ __forceinline__ u32x2_t rows32(uint32_t v) { return __builtin_amdgcn_permlane32_swap(v, v, false, false); }

template <typename Op>
__device__ __forceinline__ float wave_all_f32(float v, Op op) {
  v = op(v, dpp_f32<kDppXor1>(v));
  v = op(v, dpp_f32<kDppXor2>(v));
  v = op(v, dpp_f32<kDppHalfMirror>(v));
  v = op(v, dpp_f32<kDppMirror>(v));
  u32x2_t r = rows16(__float_as_uint(v));
  v = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
  r = rows32(__float_as_uint(v));
  return op(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float wave_all_sum(float v) {
  return wave_all_f32(v, [](float a, float b) { return a + b; });
}
template <typename Op>
__device__ __forceinline__ int wave_all_i32(int v, Op op) {
  v = op(v, dpp_i32<kDppXor1>(v));
  v = op(v, dpp_i32<kDppXor2>(v));
  v = op(v, dpp_i32<kDppHalfMirror>(v));
  v = op(v, dpp_i32<kDppMirror>(v));
  u32x2_t r = rows16((uint32_t)v);
  v = op((int)r[0], (int)r[1]);
  r = rows32((uint32_t)v);
  return op((int)r[0], (int)r[1]);
}
__device__ __forceinline__ int wave_all_min_i32(int v) {
  return wave_all_i32(v, [](int a, int b) { return min(a, b); });
}
// A float's bits in the order of signed integers; its own inverse. Maxima and
// minima of these take one instruction a step, with the lane move in it; those
// of floats three (the move and a quieting of its result apart).
__device__ __forceinline__ int ordered(float v) {
  const int b = __builtin_bit_cast(int, v);
  return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float from_ordered(int o) {
  return __builtin_bit_cast(float, o ^ ((o >> 31) & 0x7FFFFFFF));
}
__device__ __forceinline__ float wave_all_max(float v) {
  return from_ordered(wave_all_i32(ordered(v), [](int a, int b) { return max(a, b); }));
}
__device__ __forceinline__ double wave_all_max(double v) {
  for (int o = 1; o < 64; o <<= 1) v = fmax(v, __shfl_xor(v, o, 64));
  return v;
}
__device__ __forceinline__ double wave_all_sum(double v) {
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
  return v;
}

__device__ __forceinline__ float lane_value(float v, int lane) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}
__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint64_t u = (uint64_t)__builtin_bit_cast(int64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
  return __builtin_bit_cast(double, (int64_t)(((uint64_t)hi << 32) | lo));
}

// LDS written by some lanes of a wave and then read by others of the same
// wave: the hardware keeps a wave's LDS operations in order, this keeps the
// compiler from moving them across.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

}  // namespace nvfp4
