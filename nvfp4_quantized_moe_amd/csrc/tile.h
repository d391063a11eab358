// Pieces that the dense products' kernels share: the epilogue's arithmetic, the
// order of tiles, and loads that go straight to LDS.
#pragma once
#include <type_traits>

#include "common.h"

// Every rounding as it is written, here and in what follows the include.
#pragma clang fp contract(off)

namespace nvfp4 {

typedef int int4v __attribute__((ext_vector_type(4)));

// silu(g) u = g u / (1 + e^-g), by e^-|g|: e^-g itself would leave the range
// of float32 below g = -88 and take the result with it
__device__ __forceinline__ float silu_mul(float g, float u) {
  const float e = expf(-fabsf(g));
  return (g < 0.0f ? g * e : g) / (1.0f + e) * u;
}

// Tiles in runs of kTileGroup row tiles by all column tiles, so that the
// workgroups that run at one time share both operands' tiles; consecutive
// tiles go to one XCD (own L2). Returns (row tile, column tile).
constexpr int kTileGroup = 8;
__device__ __forceinline__ int2 tile_of_block(int bid, int mt, int nt) {
  const int total = mt * nt, whole = total / kXcds * kXcds;
  const int t = bid < whole ? (bid % kXcds) * (whole / kXcds) + bid / kXcds : bid;
  const int per = kTileGroup * nt, grp = t / per, rem = t - grp * per;
  const int rows = min(kTileGroup, mt - grp * kTileGroup);
  return make_int2(grp * kTileGroup + rem % rows, rem / rows);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}
constexpr int kOutOfRange = (int)0x80000000u;  // a buffer offset past every range: such loads give zeros

// 16 bytes per lane from memory to LDS, the lanes' side by side from `to` (the
// same for the whole wave) on.
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t r, int4v* to, int voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)to, 16, voff, soff, 0, 0);
}

// W = 8 or 4 outputs of one row, with the BF16 values to be added.
template <int W>
struct OutVec;
template <>
struct OutVec<8> {
  typedef uint32_t type __attribute__((ext_vector_type(4)));
};
template <>
struct OutVec<4> {
  typedef uint32_t type __attribute__((ext_vector_type(2)));
};
template <int W>
__device__ __forceinline__ typename OutVec<W>::type add_and_round(const float* o, typename OutVec<W>::type add) {
  typename OutVec<W>::type r;
#pragma unroll
  for (int e = 0; e < W / 2; ++e)
    r[e] = f32x2_to_bf16x2(o[2 * e] + __uint_as_float(add[e] << 16),
                           o[2 * e + 1] + __uint_as_float(add[e] & 0xFFFF0000u));
  return r;
}

// Waits until at most `left` of this wave's loads are in flight, then for all
// waves. The loads of a wave complete in order.
template <int LEFT>
__device__ __forceinline__ void wait_stage() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_s_waitcnt((LEFT & 15) | (LEFT >> 4) << 14 | 7 << 4);  // vmcnt(LEFT), lgkmcnt(0), no export count
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  __builtin_amdgcn_sched_barrier(0);
}

}  // namespace nvfp4
