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

// x of this size and more is read past the caches (PAST), which leaves them to the
// codes. It pays behind what writes x: after the layer norm both ways 4096 x 4096
// (33 MB) takes 31.8 us for the two [32.0 through the caches], 4096 x 7168 54.8
// [62.5], 8192 x 7168 111.6 [127.4], float32 4096 x 4096 59.9 [69.2]; along the rows
// 30.3 [30.3], 51.7 [54.8] and 98.4 [111.0] (float32 rows never: see MxVec8); below
// the limit, 2048 x 4096, 18.6 [18.5]. By itself in a loop over three inputs 8192 x
// 7168 takes 35.1 [40.3], 5.2 TB/s, rows 25.5 [29.5]; over six 42.5 [40.4], rows 25.6
// [29.6]; and on one input that the caches hold it takes longer (35.0 [28.3], 4096 x
// 4096 9.8 [9.7]).
constexpr int64_t kMxPastBytes = 32 << 20;

// Along rows: a wave takes 512 columns of R rows, all R loads in flight; lane l
// holds columns 8 l .. 8 l + 7 of each, so four lanes share a scale. Of four rows'
// scales each of them keeps one, so that all lanes store together: a byte store
// takes as long for 16 lanes as for 64. Eight rows from 32768 waves of one row on
// (8192 x 7168 BF16: 25.6 us, 5.8 TB/s [one row 29.1]; 16384 x 1024 8.2 [8.7]), one
// below (64 x 7168: 2.2 [eight rows 3.1], 1024 x 7168 5.0 [5.7], 2048 x 7168 7.8
// [8.1]; float32 2000 x 7168 13.3 [14.3], 12000 x 1024 11.7 [13.0]). (Wide float32
// rows gain from one row above it too, 8192 x 7168 47.2 for 51.0, short ones lose,
// 100000 x 264 24.4 for 22.1; one rule serves both types.) The values likewise,
// for codes that the caches still hold: 1024 x 7168 4.6 [4.8], 2048 x 7168 6.9 [6.8],
// at the limit 16384 x 1024 8.0 [7.9]; from memory eight rows are better throughout
// (6.0 [5.7], 9.9 [8.1] and 9.2 [10.9]).
constexpr int64_t kMxFewWaves = 32768;
template <typename T, int R, bool PAST>
__global__ __launch_bounds__(256) void mx_rows_kernel(const T* __restrict__ x, MxArgs g) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int Kp = mx_padded(g.K), across = (g.K + 511) / 512;
  const int c = (int)(blockIdx.x % across) * 512 + lane * 8, r0 = ((int)(blockIdx.x / across) * 4 + wave) * R;
  MxVec8<T> v[R];
#pragma unroll
  for (int i = 0; i < R; ++i)
    v[i].template load<PAST>(x + (size_t)min(r0 + i, g.M - 1) * g.K + min(c, g.K - 8));
  const uint32_t up = g.ceil ? MxVec8<T>::kUp : 0u;
  uint32_t keep = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (c >= g.K) v[i].zero();
    int m = (int)v[i].amax();
    m = max(m, dpp_i32<kDppXor1>(m));
    m = max(m, dpp_i32<kDppXor2>(m));
    const uint32_t scale = mx_scale_bits((uint32_t)m, up);
    const uint32_t w = v[i].codes(__uint_as_float(scale));
    const int r = r0 + i;
    if (r < g.M && c < Kp) *reinterpret_cast<uint32_t*>(g.q + (size_t)r * (Kp / 2) + c / 2) = w;
    keep = (lane & 3) == (i & 3) ? scale : keep;
    if ((i & 3) == 3 || i == R - 1) {
      const int from = r0 + (i & ~3) + (lane & 3);
      if ((lane & 3) <= (i & 3) && from < g.M && c < Kp)
        g.s[((size_t)(c / kMxGroup) * g.M + from) * 4 + (c / kMxBlock) % 4] = (uint8_t)(keep >> 23);
    }
  }
}

// Four values of a row, as they are loaded (PAST: not to stay in the caches).
template <typename T>
struct MxVec4;
template <>
struct MxVec4<uint16_t> {
  static constexpr uint32_t kUp = kMxUpBf16;
  uint2 v;
  template <bool PAST>
  __device__ __forceinline__ void load(const uint16_t* p) {
    const u32x2_t* at = reinterpret_cast<const u32x2_t*>(p);
    v = __builtin_bit_cast(uint2, PAST ? __builtin_nontemporal_load(at) : *at);
  }
  __device__ __forceinline__ void zero() { v = make_uint2(0, 0); }
  __device__ __forceinline__ uint32_t amax() const {
    const uint32_t a = max_u16x2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu);
    return max(a, a << 16);
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
  static constexpr uint32_t kUp = kMxUpF32;
  float4 v;
  template <bool PAST>
  __device__ __forceinline__ void load(const float* p) {
    const float4_t* at = reinterpret_cast<const float4_t*>(p);
    v = __builtin_bit_cast(float4, PAST ? __builtin_nontemporal_load(at) : *at);
  }
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

// Along columns (ROWS: and along rows, from the same registers): a workgroup takes
// 128 rows of 128 columns, a wave 32 of the rows, lane half h its rows 16 h ..
// 16 h + 15 and four columns to a lane, so that two lanes have whole blocks of
// their columns and eight share a block of a row. Codes and scales of the tile
// meet in LDS and leave in whole 64-byte runs: stored from the registers, 8 bytes
// here and there in 64 lines, the address unit was busy 84 % of the time
// (8192 x 7168 both ways: 48.5 us).
constexpr int kMxColPitch = 80;  // of a column's 64 bytes of codes in LDS, against bank conflicts
template <typename T, bool ROWS, bool PAST>
__global__ __launch_bounds__(256) void mx_columns_kernel(const T* __restrict__ x, MxArgs g) {
  constexpr int N = kMxBlock / 2;
  __shared__ __attribute__((aligned(16))) uint8_t cols[128 * kMxColPitch];  // [32 (c % 4) + c / 4][64 bytes]
  __shared__ __attribute__((aligned(16))) uint8_t rows[ROWS ? 128 * 64 : 16];
  __shared__ __attribute__((aligned(4))) uint8_t scales[2][128][4];         // of the columns, of the rows
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c0 = blockIdx.x * 128, m0 = blockIdx.y * kMxGroup;
  const int cl = (lane & 31) * 4, rl = wave * kMxBlock + (lane >> 5) * N, c = c0 + cl, r0 = m0 + rl;
  MxVec4<T> v[N];
  const T* from = x + min(c, g.K - 4);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i].template load<PAST>(from + (size_t)min(r0 + i, g.M - 1) * g.K);
  if (c0 + 128 > g.K || m0 + kMxGroup > g.M) {  // the same for the workgroup
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (c >= g.K || r0 + i >= g.M) v[i].zero();
  }
  const uint32_t up = g.ceil ? MxVec4<T>::kUp : 0u;
  typename MxVec4<T>::Max top;
#pragma unroll
  for (int i = 0; i < N; ++i) top.add(v[i]);
  if constexpr (ROWS) {
    uint32_t keep = 0;  // of eight rows' scales each of a block's lanes keeps one
#pragma unroll
    for (int i = 0; i < N; ++i) {
      int m = (int)v[i].amax();
      m = max(m, dpp_i32<kDppXor1>(m));
      m = max(m, dpp_i32<kDppXor2>(m));
      m = max(m, dpp_i32<kDppHalfMirror>(m));
      const uint32_t scale = mx_scale_bits((uint32_t)m, up);
      *reinterpret_cast<uint16_t*>(rows + (rl + i) * 64 + cl / 2) = (uint16_t)v[i].codes(__uint_as_float(scale));
      keep = (lane & 7) == (i & 7) ? scale : keep;
      if ((i & 7) == 7) scales[1][rl + i - 7 + (lane & 7)][(lane >> 3) & 3] = (uint8_t)(keep >> 23);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const u32x2_t halves = rows32(top.get(j));  // this lane's and that of the lane 32 on or back
    const uint32_t scale = mx_scale_bits(max(halves[0], halves[1]), up);
    const float s = __uint_as_float(scale);
    uint32_t w[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const MxVec4<T>* at = v + 8 * p;
      w[p] = MxVec4<T>::template pair<0>(0u, at[0], at[1], j, s);
      w[p] = MxVec4<T>::template pair<1>(w[p], at[2], at[3], j, s);
      w[p] = MxVec4<T>::template pair<2>(w[p], at[4], at[5], j, s);
      w[p] = MxVec4<T>::template pair<3>(w[p], at[6], at[7], j, s);
    }
    *reinterpret_cast<uint2*>(cols + (32 * j + (lane & 31)) * kMxColPitch + rl / 2) = make_uint2(w[0], w[1]);
    if (lane < 32) scales[0][cl + j][wave] = (uint8_t)(scale >> 23);
  }
  __syncthreads();
  const int t = threadIdx.x, part = (t & 3) * 16;
  const size_t col_pitch = (size_t)(mx_padded(g.M) / 2), row_pitch = (size_t)(mx_padded(g.K) / 2);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int at = t / 4 + 64 * i;
    if (c0 + at < g.K)
      *reinterpret_cast<uint4*>(g.qt + (c0 + at) * col_pitch + m0 / 2 + part) =
          *reinterpret_cast<const uint4*>(cols + (32 * (at & 3) + at / 4) * kMxColPitch + part);
    if (ROWS && m0 + at < g.M)
      *reinterpret_cast<uint4*>(g.q + (m0 + at) * row_pitch + c0 / 2 + part) =
          *reinterpret_cast<const uint4*>(rows + at * 64 + part);
  }
  if (t < 128) {
    if (c0 + t < g.K)
      reinterpret_cast<uint32_t*>(g.st)[(size_t)blockIdx.y * g.K + c0 + t] = *reinterpret_cast<const uint32_t*>(scales[0][t]);
  } else if (ROWS && m0 + t - 128 < g.M) {
    reinterpret_cast<uint32_t*>(g.s)[(size_t)blockIdx.x * g.M + m0 + t - 128] =
        *reinterpret_cast<const uint32_t*>(scales[1][t - 128]);
  }
}

// Values of the codes, [R, cols] of the Kp columns: a lane takes 16 bytes of
// values (eight or four columns) of N rows. Rows of any length: the store is 16
// bytes at the type's own alignment. 8192 x 7168 to BF16: 24 us, 6.2 TB/s. (Eight
// float32 values to a lane, in two stores of every other 16 bytes, took 70 us.)
template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Loose16 {
  uint32_t w[4];
};
template <typename T, int N>
__global__ __launch_bounds__(256) void mx_values_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ scale,
                                                        int R, int Kp, int cols, T* __restrict__ out) {
  constexpr int E = 16 / sizeof(T);
  const int across = (cols + 64 * E - 1) / (64 * E);
  const int c = ((int)(blockIdx.x % across) * 64 + (int)(threadIdx.x & 63)) * E;
  const int r0 = ((int)(blockIdx.x / across) * 4 + (int)(threadIdx.x >> 6)) * N;
  if (c >= cols) return;
  uint32_t w[N], code[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int r = min(r0 + i, R - 1);
    const uint8_t* from = q + (size_t)r * (Kp / 2) + c / 2;
    w[i] = E == 8 ? *reinterpret_cast<const uint32_t*>(from) : *reinterpret_cast<const uint16_t*>(from);
    code[i] = scale[((size_t)(c / kMxGroup) * R + r) * 4 + (c / kMxBlock) % 4];
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (r0 + i >= R) return;
    const float s = __uint_as_float(code[i] << 23);  // 0 is 2^-127, 255 NaN
    Loose16<T> o;
    if constexpr (sizeof(T) == 2) {
      o.w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], s, 0));
      o.w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], s, 1));
      o.w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], s, 2));
      o.w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i], s, 3));
    } else {
      const float2_t lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], s, 0), hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], s, 1);
      const float f[4] = {lo[0], lo[1], hi[0], hi[1]};
#pragma unroll
      for (int j = 0; j < 4; ++j) o.w[j] = __float_as_uint(f[j]);
    }
    T* to = out + (size_t)(r0 + i) * cols + c;
    if (c + E <= cols) {
      *reinterpret_cast<Loose16<T>*>(to) = o;
    } else {
#pragma unroll
      for (int j = 0; j < E - 1; ++j) {
        if (c + j >= cols) break;
        if constexpr (sizeof(T) == 2)
          to[j] = (uint16_t)(o.w[j >> 1] >> (16 * (j & 1)));
        else
          to[j] = __uint_as_float(o.w[j]);
      }
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
  if ((int64_t)((M + 31) / 32) * ((K + 511) / 512) >= (1 << 24)) return NVFP4_ERR_SHAPE;  // threads of a grid
  const MxArgs g = {M, K, q, scale, q_t, scale_t, rule == MX_SCALE_CEIL};
  const auto go = [&](auto xt) -> int {
    using T = decltype(xt);
    const T* at = reinterpret_cast<const T*>(x);
    const auto launch = [&](auto past) {
      constexpr bool PAST = decltype(past)::value;
      const dim3 grid((K + 127) / 128, (M + kMxGroup - 1) / kMxGroup), threads(256);
      const unsigned cols = (K + 511) / 512;
      if (q_t && q)
        hipLaunchKernelGGL((mx_columns_kernel<T, true, PAST>), grid, threads, 0, (hipStream_t)stream, at, g);
      else if (q_t)
        hipLaunchKernelGGL((mx_columns_kernel<T, false, PAST>), grid, threads, 0, (hipStream_t)stream, at, g);
      else if ((int64_t)M * cols < kMxFewWaves)
        hipLaunchKernelGGL((mx_rows_kernel<T, 1, false>), dim3((M + 3) / 4 * cols), threads, 0, (hipStream_t)stream, at, g);
      else
        hipLaunchKernelGGL((mx_rows_kernel<T, 8, PAST && sizeof(T) == 2>), dim3((M + 31) / 32 * cols), threads, 0,
                           (hipStream_t)stream, at, g);
    };
    if ((int64_t)M * K * (int64_t)sizeof(T) >= kMxPastBytes)
      launch(std::true_type());
    else
      launch(std::false_type());
    NVFP4_CHECK_LAUNCH();
    return NVFP4_OK;
  };
  return x_dtype == NVFP4_DT_BF16 ? go(uint16_t()) : go(float());
}

extern "C" int mxfp4_dequantize(const uint8_t* q, const uint8_t* scale, int32_t R, int32_t K, int32_t cols,
                                int32_t out_dtype, void* out, void* stream) {
  if (R < 0 || R > kMxMaxM || K < 0 || K > kMxMaxK || K % kMxGroup != 0 || cols < 0 || cols > K) return NVFP4_ERR_SHAPE;
  if (out_dtype != NVFP4_DT_BF16 && out_dtype != NVFP4_DT_F32) return NVFP4_ERR_ARG;
  const unsigned across = (unsigned)(((int64_t)cols * (out_dtype == NVFP4_DT_BF16 ? 2 : 4) + 1023) / 1024);
  if ((int64_t)((R + 31) / 32) * across >= (1 << 24)) return NVFP4_ERR_SHAPE;  // threads of a grid
  if (R == 0 || cols == 0) return NVFP4_OK;
  if (!q || !scale || !out) return NVFP4_ERR_NULL;
  if (!nvfp4_aligned16(q) || !nvfp4_aligned16(scale) || !nvfp4_aligned16(out)) return NVFP4_ERR_ALIGN;
  const auto by_size = [&](auto t) {
    using T = decltype(t);
    if ((int64_t)R * across < kMxFewWaves)
      hipLaunchKernelGGL((mx_values_kernel<T, 1>), dim3((R + 3) / 4 * across), dim3(256), 0, (hipStream_t)stream, q, scale,
                         R, K, cols, reinterpret_cast<T*>(out));
    else
      hipLaunchKernelGGL((mx_values_kernel<T, 8>), dim3((R + 31) / 32 * across), dim3(256), 0, (hipStream_t)stream, q,
                         scale, R, K, cols, reinterpret_cast<T*>(out));
  };
  if (out_dtype == NVFP4_DT_BF16)
    by_size(uint16_t());
  else
    by_size(float());
  NVFP4_CHECK_LAUNCH();
  return NVFP4_OK;
}
