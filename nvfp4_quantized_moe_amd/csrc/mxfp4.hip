// MXFP4 quantisation along rows, along columns or both, and its inverse.
//
// Codes of a matrix [R, C] are kept with C padded to whole groups of 128 (codes
// and scales of 0 behind the end):
//   q      uint8 [R, Cp / 2]
//   scale  uint8 [Cp / 128, R, 4]: the four scales of one row's group side by
//          side, the rows' next to each other, which is how the product reads
//          them (64 rows of a stage are 256 consecutive bytes; with a row's
//          scales in a run they are 64 lines)
// Along columns they are the codes of the transposed matrix, [C, Rp / 2], so
// that both operands of every product of a training step run along its K.
#include <type_traits>

#include "common.h"
#include "internal.h"
#include "mxfp4.h"
#include "wave.h"

namespace nvfp4 {

constexpr int kMxMaxM = 64 * 65535;

struct MxArgs {
  int M, K;
  uint8_t *q, *s;      // codes along the rows, [M, Kp / 2] and [Kp / 128, M, 4]
  uint8_t *qt, *st;    // codes along the columns, [K, Mp / 2] and [Mp / 128, K, 4]
  bool ceil;
};

// Along rows: a wave takes 512 columns of R rows, all R loads in flight; lane l
// holds columns 8 l .. 8 l + 7 of each, so four lanes share a scale.
template <typename T, int R>
__global__ __launch_bounds__(256) void mx_rows_kernel(const T* __restrict__ x, MxArgs g) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int Kp = mx_padded(g.K), c = blockIdx.y * 512 + lane * 8;
  const int r0 = (blockIdx.x * 4 + wave) * R;
  MxVec8<T> v[R];
#pragma unroll
  for (int i = 0; i < R; ++i)
    v[i].load(x + (size_t)min(r0 + i, g.M - 1) * g.K + min(c, g.K - 8));
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (c >= g.K) v[i].zero();
    int m = (int)v[i].amax();
    m = max(m, dpp_i32<kDppXor1>(m));
    m = max(m, dpp_i32<kDppXor2>(m));
    const uint32_t code = mx_scale_code((uint32_t)m, g.ceil);
    const uint32_t w = v[i].codes(mx_scale(code));
    const int r = r0 + i;
    if (r < g.M && c < Kp) {
      *reinterpret_cast<uint32_t*>(g.q + (size_t)r * (Kp / 2) + c / 2) = w;
      if ((lane & 3) == 0) g.s[((size_t)(c / kMxGroup) * g.M + r) * 4 + (c / kMxBlock) % 4] = (uint8_t)code;
    }
  }
}

// Four values of a row, as they are loaded.
template <typename T>
struct MxVec4;
template <>
struct MxVec4<uint16_t> {
  uint2 v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void zero() { v = make_uint2(0, 0); }
  __device__ __forceinline__ uint32_t amax() const {
    const uint32_t a = max_u16x2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu);
    const uint32_t lo = a << 16, hi = a & 0xFFFF0000u;
    return lo > hi ? lo : hi;
  }
  __device__ __forceinline__ uint32_t codes(float s) const { return mx_encode2<1>(mx_encode2<0>(0u, v.x, s), v.y, s); }
  // largest magnitudes of the four columns, running
  struct Max {
    uint32_t a = 0, b = 0;
    __device__ __forceinline__ void add(const MxVec4& o) {
      a = max_u16x2(a, o.v.x & 0x7FFF7FFFu);
      b = max_u16x2(b, o.v.y & 0x7FFF7FFFu);
    }
    __device__ __forceinline__ uint32_t get(int j) const {
      const uint32_t w = j < 2 ? a : b;
      return j & 1 ? w & 0xFFFF0000u : w << 16;
    }
  };
  // byte SEL of column j's codes: this row's value, then the next row's
  template <int SEL>
  static __device__ __forceinline__ uint32_t pair(uint32_t old, const MxVec4& lo, const MxVec4& hi, int j, float s) {
    const uint32_t l = j < 2 ? lo.v.x : lo.v.y, h = j < 2 ? hi.v.x : hi.v.y;
    return mx_encode2<SEL>(old, __builtin_amdgcn_perm(h, l, j & 1 ? 0x07060302u : 0x05040100u), s);
  }
};
template <>
struct MxVec4<float> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void zero() { v = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max(m, __float_as_uint((&v.x)[j]) & 0x7FFFFFFFu);
    return m;
  }
  __device__ __forceinline__ uint32_t codes(float s) const {
    return mx_encode2<1>(mx_encode2<0>(0u, v.x, v.y, s), v.z, v.w, s);
  }
  struct Max {
    uint32_t m[4] = {0, 0, 0, 0};
    __device__ __forceinline__ void add(const MxVec4& o) {
#pragma unroll
      for (int j = 0; j < 4; ++j) m[j] = max(m[j], __float_as_uint((&o.v.x)[j]) & 0x7FFFFFFFu);
    }
    __device__ __forceinline__ uint32_t get(int j) const { return m[j]; }
  };
  template <int SEL>
  static __device__ __forceinline__ uint32_t pair(uint32_t old, const MxVec4& lo, const MxVec4& hi, int j, float s) {
    return mx_encode2<SEL>(old, (&lo.v.x)[j], (&hi.v.x)[j], s);
  }
};

// Along columns (ROWS: and along rows, from the same registers): a wave holds 32
// rows of 256 columns, four columns to a lane, so that a lane has whole blocks
// of its columns. Four waves take the 128 rows of a group.
template <typename T, bool ROWS>
__global__ __launch_bounds__(256) void mx_columns_kernel(const T* __restrict__ x, MxArgs g) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 256 + lane * 4, r0 = blockIdx.y * kMxGroup + wave * kMxBlock;
  MxVec4<T> v[kMxBlock];
#pragma unroll
  for (int i = 0; i < kMxBlock; ++i)
    v[i].load(x + (size_t)min(r0 + i, g.M - 1) * g.K + min(c, g.K - 4));
  typename MxVec4<T>::Max top;
#pragma unroll
  for (int i = 0; i < kMxBlock; ++i) {
    if (c >= g.K || r0 + i >= g.M) v[i].zero();
    top.add(v[i]);
  }
  if (c < g.K) {
    const size_t pitch = (size_t)(mx_padded(g.M) / 2);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t code = mx_scale_code(top.get(j), g.ceil);
      const float s = mx_scale(code);
      uint32_t w[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const MxVec4<T>* at = v + 8 * p;
        w[p] = MxVec4<T>::template pair<0>(0u, at[0], at[1], j, s);
        w[p] = MxVec4<T>::template pair<1>(w[p], at[2], at[3], j, s);
        w[p] = MxVec4<T>::template pair<2>(w[p], at[4], at[5], j, s);
        w[p] = MxVec4<T>::template pair<3>(w[p], at[6], at[7], j, s);
      }
      *reinterpret_cast<uint4*>(g.qt + (size_t)(c + j) * pitch + r0 / 2) = make_uint4(w[0], w[1], w[2], w[3]);
      g.st[((size_t)blockIdx.y * g.K + c + j) * 4 + wave] = (uint8_t)code;
    }
  }
  if constexpr (ROWS) {
    const int Kp = mx_padded(g.K);
#pragma unroll
    for (int i = 0; i < kMxBlock; ++i) {
      int m = (int)v[i].amax();  // eight lanes share a block of the row
      m = max(m, dpp_i32<kDppXor1>(m));
      m = max(m, dpp_i32<kDppXor2>(m));
      m = max(m, dpp_i32<kDppHalfMirror>(m));
      const uint32_t code = mx_scale_code((uint32_t)m, g.ceil);
      const uint32_t w = v[i].codes(mx_scale(code));
      const int r = r0 + i;
      if (r < g.M && c < Kp) {
        *reinterpret_cast<uint16_t*>(g.q + (size_t)r * (Kp / 2) + c / 2) = (uint16_t)w;
        if ((lane & 7) == 0) g.s[((size_t)(c / kMxGroup) * g.M + r) * 4 + (c / kMxBlock) % 4] = (uint8_t)code;
      }
    }
  }
}

// Values of the codes, [R, cols] of the Kp columns: a thread takes eight of a
// row. Rows of any length: the store is 16 bytes at the type's own alignment.
template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Loose8 {
  uint32_t w[2 * sizeof(T)];
};
template <typename T>
__global__ __launch_bounds__(256) void mx_values_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ scale,
                                                        int R, int Kp, int cols, T* __restrict__ out) {
  const int c = (blockIdx.y * 64 + (threadIdx.x & 63)) * 8, r = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (r >= R || c >= cols) return;
  const uint32_t w = *reinterpret_cast<const uint32_t*>(q + (size_t)r * (Kp / 2) + c / 2);
  const float s = mx_scale(scale[((size_t)(c / kMxGroup) * R + r) * 4 + (c / kMxBlock) % 4]);
  Loose8<T> o;
  if constexpr (sizeof(T) == 2) {
    o.w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
    o.w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
    o.w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
    o.w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
  } else {
    const float2_t v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0), v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1);
    const float2_t v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2), v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3);
    const float f[8] = {v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
#pragma unroll
    for (int i = 0; i < 8; ++i) o.w[i] = __float_as_uint(f[i]);
  }
  T* to = out + (size_t)r * cols + c;
  if (c + 8 <= cols) {
    *reinterpret_cast<Loose8<T>*>(to) = o;
  } else {
    for (int i = 0; i < cols - c; ++i) {
      if constexpr (sizeof(T) == 2)
        to[i] = (uint16_t)(o.w[i >> 1] >> (16 * (i & 1)));
      else
        to[i] = __uint_as_float(o.w[i]);
    }
  }
}

}  // namespace nvfp4

using namespace nvfp4;

extern "C" int32_t mxfp4_padded(int32_t n) { return n < 0 || n > kMxMaxK ? -1 : (n + kMxGroup - 1) / kMxGroup * kMxGroup; }

extern "C" int mxfp4_quantize(const void* x, int32_t x_dtype, int32_t M, int32_t K, int32_t rule, uint8_t* q,
                              uint8_t* scale, uint8_t* q_t, uint8_t* scale_t, void* stream) {
  if (M < 0 || K <= 0 || K % 8 != 0 || K > kMxMaxK || M > kMxMaxM) return NVFP4_ERR_SHAPE;
  if ((x_dtype != NVFP4_DT_BF16 && x_dtype != NVFP4_DT_F32) || (rule != MX_SCALE_FLOOR && rule != MX_SCALE_CEIL))
    return NVFP4_ERR_ARG;
  if (M == 0) return NVFP4_OK;
  if (!x || !q != !scale || !q_t != !scale_t || (!q && !q_t)) return NVFP4_ERR_NULL;
  if (!nvfp4_aligned16(x) || !nvfp4_aligned16(q) || !nvfp4_aligned16(scale) || !nvfp4_aligned16(q_t) ||
      !nvfp4_aligned16(scale_t))
    return NVFP4_ERR_ALIGN;
  if (q_t && M > kMxMaxK) return NVFP4_ERR_SHAPE;  // along the columns, M is the length of a row of codes
  const MxArgs g = {M, K, q, scale, q_t, scale_t, rule == MX_SCALE_CEIL};
  const auto go = [&](auto xt) -> int {
    using T = decltype(xt);
    const T* at = reinterpret_cast<const T*>(x);
    if (!q_t) {
      const int cols = (K + 511) / 512;
      if ((int64_t)M * cols <= 8192)
        hipLaunchKernelGGL((mx_rows_kernel<T, 1>), dim3((M + 3) / 4, cols), dim3(256), 0, (hipStream_t)stream, at, g);
      else
        hipLaunchKernelGGL((mx_rows_kernel<T, 8>), dim3((M + 31) / 32, cols), dim3(256), 0, (hipStream_t)stream, at, g);
    } else {
      const dim3 grid((K + 255) / 256, (M + kMxGroup - 1) / kMxGroup);
      if (q)
        hipLaunchKernelGGL((mx_columns_kernel<T, true>), grid, dim3(256), 0, (hipStream_t)stream, at, g);
      else
        hipLaunchKernelGGL((mx_columns_kernel<T, false>), grid, dim3(256), 0, (hipStream_t)stream, at, g);
    }
    NVFP4_CHECK_LAUNCH();
    return NVFP4_OK;
  };
  return x_dtype == NVFP4_DT_BF16 ? go(uint16_t()) : go(float());
}

extern "C" int mxfp4_dequantize(const uint8_t* q, const uint8_t* scale, int32_t R, int32_t K, int32_t cols,
                                int32_t out_dtype, void* out, void* stream) {
  if (R < 0 || R > kMxMaxM || K < 0 || K > kMxMaxK || K % kMxGroup != 0 || cols < 0 || cols > K) return NVFP4_ERR_SHAPE;
  if (out_dtype != NVFP4_DT_BF16 && out_dtype != NVFP4_DT_F32) return NVFP4_ERR_ARG;
  if (R == 0 || cols == 0) return NVFP4_OK;
  if (!q || !scale || !out) return NVFP4_ERR_NULL;
  if (!nvfp4_aligned16(q) || !nvfp4_aligned16(scale) || !nvfp4_aligned16(out)) return NVFP4_ERR_ALIGN;
  const dim3 grid((R + 3) / 4, (cols + 511) / 512);
  if (out_dtype == NVFP4_DT_BF16)
    hipLaunchKernelGGL(mx_values_kernel<uint16_t>, grid, dim3(256), 0, (hipStream_t)stream, q, scale, R, K, cols,
                       reinterpret_cast<uint16_t*>(out));
  else
    hipLaunchKernelGGL(mx_values_kernel<float>, grid, dim3(256), 0, (hipStream_t)stream, q, scale, R, K, cols,
                       reinterpret_cast<float*>(out));
  NVFP4_CHECK_LAUNCH();
  return NVFP4_OK;
}
