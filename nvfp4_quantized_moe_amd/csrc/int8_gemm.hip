// Products of 8-bit integers with a scale per token and per output channel,
// for the dense expert that runs beside the routed ones:
//   q[m, k] = rne(x[m, k] / s_m), s_m = amax_k |x[m, k]| * (1 / 127)
//   C[m, n] = a_s[m] * b_s[n] * sum_k a_q[m, k] b_q[n, k]
// The sum is exact in int32 (K <= 65536: |sum| <= 2^30), so neither the order
// of K nor its split can change a result; the scales are applied to it in
// float32 and the output is rounded once.
#include <type_traits>

#include "common.h"
#include "internal.h"
#include "wave.h"

namespace nvfp4 {

typedef int int4v __attribute__((ext_vector_type(4)));
typedef int int16v __attribute__((ext_vector_type(16)));

constexpr int kInt8MaxK = 65536;

// ------------------------------------------------------------- row quantizer

// Nearest integer to the real quotient |x| / s, ties to even, at most 127.
// The float32 product |x| (1/s) is within 2^-22 relative of the quotient, so
// its floor t is off by one at most, and only next to an integer; the exact
// sign of |x| - (t + 1/2) s (one fma) then settles the rounding either way.
__device__ __forceinline__ int quantize_int8(float x, float s, float inv) {
  const float a = fabsf(x);
  const float t = floorf(a * inv);
  const float r = __builtin_fmaf(-(t + 0.5f), s, a);
  int n = (int)t;
  n += (r > 0.0f || (r == 0.0f && (n & 1))) ? 1 : 0;
  n = n > 127 ? 127 : n;
  return x < 0.0f ? -n : n;
}

template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&f)[16]);
template <>
__device__ __forceinline__ void load16<uint16_t>(const uint16_t* p, float (&f)[16]) {
  const uint4* v = reinterpret_cast<const uint4*>(p);
  const uint4 a = v[0], b = v[1];
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
template <>
__device__ __forceinline__ void load16<float>(const float* p, float (&f)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = reinterpret_cast<const float4*>(p)[i];
    f[4 * i] = v.x;
    f[4 * i + 1] = v.y;
    f[4 * i + 2] = v.z;
    f[4 * i + 3] = v.w;
  }
}

// One workgroup per row; thread i takes the 16-element chunks i, i + blockDim.x, ...
// The second pass over a row reads it from the cache.
template <typename T>
__global__ __launch_bounds__(256) void int8_rows_kernel(const T* __restrict__ x, int K, int8_t* __restrict__ q,
                                                        float* __restrict__ scale) {
  __shared__ float red[4];
  const size_t row = (size_t)blockIdx.x * K;
  const int n = K / 16;
  float m = 0.0f, f[16];
  for (int c = threadIdx.x; c < n; c += blockDim.x) {
    load16(x + row + c * 16, f);
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(f[i]));
  }
  m = wave_all_max(m);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  m = red[0];
  for (int w = 1; w < (int)blockDim.x / 64; ++w) m = fmaxf(m, red[w]);
  float s = m * (1.0f / 127.0f);
  if (threadIdx.x == 0) scale[blockIdx.x] = s;
  // rows of the smallest numbers are lifted by 2^100 (exactly, like their
  // scale), so that neither 1 / s nor the residual leaves the float32 range
  const float lift = s < 0x1p-100f ? 0x1p100f : 1.0f;
  s *= lift;
  const float inv = s > 0.0f ? 1.0f / s : 0.0f;
  for (int c = threadIdx.x; c < n; c += blockDim.x) {
    load16(x + row + c * 16, f);
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[j] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[j] |= (uint32_t)((s > 0.0f ? quantize_int8(f[4 * j + i] * lift, s, inv) : 0) & 0xFF) << (8 * i);
    }
    *reinterpret_cast<uint4*>(q + row + c * 16) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ------------------------------------------------------------------- product

constexpr int kInt8BK = 128;  // K bytes per stage: one 128-byte line per row

struct Int8Args {
  const int8_t* a;
  const float* a_s;
  const int8_t* b;
  const float* b_s;
  const uint16_t* add;  // BF16 [M, n_out] or NULL
  uint16_t* d;          // BF16 [M, n_out]
  int M, N, K, n_out;
};

// silu(g) u = g u / (1 + e^-g), by e^-|g|: e^-g itself would leave the range
// of float32 below g = -88 and take the result with it
__device__ __forceinline__ float silu_mul(float g, float u) {
  const float e = expf(-fabsf(g));
  return (g < 0.0f ? g * e : g) / (1.0f + e) * u;
}

// Weight row of row i of a column tile starting at output column n0. SILU:
// the rows alternate in runs of 32 between gate (row n) and up (row I + n), so
// that a wave holds both halves of an output in the same lane.
template <bool SILU>
__device__ __forceinline__ int tile_weight_row(int i, int n0, int half) {
  if (!SILU) return n0 + i;
  const int n = n0 + (i >> 6) * 32 + (i & 31);
  return (i & 32) ? half + n : n;
}

// Workgroup tile BM x BN of 2 x 2 waves. MFMA 32x32x32 with the weights as
// its first operand, so a lane holds four neighbouring output columns of one
// token. K stages of 128 bytes pass through registers into LDS (two buffers);
// a row's eight 16-byte chunks are stored at chunk ^ (row & 7), which spreads
// the 32 rows that a fragment read touches over all banks.
template <int BM, int BN, bool SILU>
__global__ __launch_bounds__(256) void int8_tile_kernel(Int8Args g) {
  constexpr int SM = BM / 64, SN = BN / 64;  // 32-wide subtiles per wave and side
  static_assert(!SILU || SN % 2 == 0, "gate and up halves in one wave");
  constexpr int PA = BM * 8 / 256, PB = BN * 8 / 256;  // 16-byte chunks per thread and stage
  __shared__ uint4 lds[2][(BM + BN) * 8];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave & 1, wn = wave >> 1;
  const int m0 = blockIdx.y * BM, n0 = blockIdx.x * (SILU ? BN / 2 : BN);
  const int half = g.N / 2;
  // rows past the end repeat the last one: their results are not stored
  const int8_t* pa[PA];
  const int8_t* pb[PB];
#pragma unroll
  for (int i = 0; i < PA; ++i) {
    const int row = (threadIdx.x + i * 256) >> 3;
    pa[i] = g.a + (size_t)min(m0 + row, g.M - 1) * g.K;
  }
#pragma unroll
  for (int i = 0; i < PB; ++i) {
    const int row = (threadIdx.x + i * 256) >> 3;
    pb[i] = g.b + (size_t)min(tile_weight_row<SILU>(row, n0, half), g.N - 1) * g.K;
  }
  const int kc = (threadIdx.x & 7) * 16;
  uint4 ra[PA], rb[PB];
  auto fetch = [&](int k0) {
    const bool in = k0 + kc < g.K;
#pragma unroll
    for (int i = 0; i < PA; ++i)
      ra[i] = in ? *reinterpret_cast<const uint4*>(pa[i] + k0 + kc) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < PB; ++i)
      rb[i] = in ? *reinterpret_cast<const uint4*>(pb[i] + k0 + kc) : make_uint4(0, 0, 0, 0);
  };
  auto place = [&](uint4* to) {
#pragma unroll
    for (int i = 0; i < PA; ++i) {
      const int row = (threadIdx.x + i * 256) >> 3;
      to[row * 8 + ((threadIdx.x & 7) ^ (row & 7))] = ra[i];
    }
#pragma unroll
    for (int i = 0; i < PB; ++i) {
      const int row = (threadIdx.x + i * 256) >> 3;
      to[(BM + row) * 8 + ((threadIdx.x & 7) ^ (row & 7))] = rb[i];
    }
  };
  int16v acc[SN][SM];
#pragma unroll
  for (int i = 0; i < SN; ++i)
#pragma unroll
    for (int j = 0; j < SM; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;
  const int stages = (g.K + kInt8BK - 1) / kInt8BK;
  fetch(0);
  place(lds[0]);
  __syncthreads();
  const int r = lane & 31, hi = lane >> 5;
  for (int s = 0; s < stages; ++s) {
    if (s + 1 < stages) fetch((s + 1) * kInt8BK);
    const uint4* at = lds[s & 1];
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      int4v fa[SM], fb[SN];
      const int c = ks * 2 + hi;
#pragma unroll
      for (int j = 0; j < SM; ++j)
        fa[j] = __builtin_bit_cast(int4v, at[(wm * 32 * SM + j * 32 + r) * 8 + (c ^ (r & 7))]);
#pragma unroll
      for (int i = 0; i < SN; ++i)
        fb[i] = __builtin_bit_cast(int4v, at[(BM + wn * 32 * SN + i * 32 + r) * 8 + (c ^ (r & 7))]);
#pragma unroll
      for (int i = 0; i < SN; ++i)
#pragma unroll
        for (int j = 0; j < SM; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[i], fa[j], acc[i][j], 0, 0, 0);
    }
    if (s + 1 < stages) place(lds[(s + 1) & 1]);
    __syncthreads();
  }
  // lane: token column r of a subtile, weight rows 8 q + 4 hi + 0..3 for q = 0..3
#pragma unroll
  for (int j = 0; j < SM; ++j) {
    const int m = m0 + wm * 32 * SM + j * 32 + r;
    if (m >= g.M) continue;
    const float as = g.a_s[m];
#pragma unroll
    for (int i = 0; i < SN; i += SILU ? 2 : 1) {
      const int col0 = SILU ? n0 + (wn * SN + i) / 2 * 32 : n0 + (wn * SN + i) * 32;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = col0 + 8 * q + 4 * hi;
        if (n >= g.n_out) continue;
        const float4 bs = *reinterpret_cast<const float4*>(g.b_s + n);
        float o[4];
        if constexpr (SILU) {
          const float4 us = *reinterpret_cast<const float4*>(g.b_s + half + n);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            o[e] = silu_mul((float)acc[i][j][4 * q + e] * (as * (&bs.x)[e]),
                            (float)acc[i + 1][j][4 * q + e] * (as * (&us.x)[e]));
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = (float)acc[i][j][4 * q + e] * (as * (&bs.x)[e]);
        }
        const size_t at = (size_t)m * g.n_out + n;
        if (g.add) {
          const uint2 v = *reinterpret_cast<const uint2*>(g.add + at);
          o[0] += __uint_as_float(v.x << 16);
          o[1] += __uint_as_float(v.x & 0xFFFF0000u);
          o[2] += __uint_as_float(v.y << 16);
          o[3] += __uint_as_float(v.y & 0xFFFF0000u);
        }
        *reinterpret_cast<uint2*>(g.d + at) = make_uint2(f32x2_to_bf16x2(o[0], o[1]), f32x2_to_bf16x2(o[2], o[3]));
      }
    }
  }
}

}  // namespace nvfp4

using namespace nvfp4;

extern "C" int int8_quantize_rows(const void* x, int32_t x_dtype, int32_t M, int32_t K, int8_t* q, float* scale,
                                  void* stream) {
  if (M < 0 || K <= 0 || K % 16 != 0 || K > kInt8MaxK) return NVFP4_ERR_SHAPE;
  if (x_dtype != NVFP4_DT_BF16 && x_dtype != NVFP4_DT_F32) return NVFP4_ERR_ARG;
  if (M == 0) return NVFP4_OK;
  if (!x || !q || !scale) return NVFP4_ERR_NULL;
  if (!nvfp4_aligned16(x) || !nvfp4_aligned16(q) || !nvfp4_aligned16(scale)) return NVFP4_ERR_ALIGN;
  int threads = (K / 16 + 63) / 64 * 64;
  if (threads > 256) threads = 256;
  if (x_dtype == NVFP4_DT_BF16)
    hipLaunchKernelGGL(int8_rows_kernel<uint16_t>, dim3(M), dim3(threads), 0, (hipStream_t)stream,
                       reinterpret_cast<const uint16_t*>(x), K, q, scale);
  else
    hipLaunchKernelGGL(int8_rows_kernel<float>, dim3(M), dim3(threads), 0, (hipStream_t)stream,
                       reinterpret_cast<const float*>(x), K, q, scale);
  NVFP4_CHECK_LAUNCH();
  return NVFP4_OK;
}

static int int8_gemm_check(int64_t M, int64_t N, int64_t K, int32_t epilogue) {
  if (epilogue != NVFP4_EPI_BF16 && epilogue != NVFP4_EPI_SILU_MUL) return NVFP4_ERR_ARG;
  if (M < 0 || N <= 0 || K <= 0 || K % 16 != 0 || K > kInt8MaxK) return NVFP4_ERR_SHAPE;
  if (N % (epilogue == NVFP4_EPI_SILU_MUL ? 16 : 8) != 0) return NVFP4_ERR_SHAPE;
  if ((M + 63) / 64 > 65535) return NVFP4_ERR_SHAPE;
  return NVFP4_OK;
}

template <bool SILU>
static int launch_int8(const Int8Args& g, hipStream_t stream) {
  // 128 x 128 tiles where they fill the 256 CUs, else 64 x 64 (64 x 128 for
  // SILU, whose waves need a gate and an up subtile)
  const int64_t big = (int64_t)((g.M + 127) / 128) * ((g.N + 127) / 128);
  if (big >= 256) {
    hipLaunchKernelGGL((int8_tile_kernel<128, 128, SILU>), dim3((g.N + 127) / 128, (g.M + 127) / 128), dim3(256), 0,
                       stream, g);
  } else {
    constexpr int BN = SILU ? 128 : 64;
    hipLaunchKernelGGL((int8_tile_kernel<64, BN, SILU>), dim3((g.N + BN - 1) / BN, (g.M + 63) / 64), dim3(256), 0,
                       stream, g);
  }
  NVFP4_CHECK_LAUNCH();
  return NVFP4_OK;
}

extern "C" int int8_gemm(const int8_t* a_q, const float* a_scale, const int8_t* b_q, const float* b_scale, int32_t M,
                         int32_t N, int32_t K, int32_t epilogue, const void* add_bf16, void* d_bf16, void* stream) {
  const int st = int8_gemm_check(M, N, K, epilogue);
  if (st) return st;
  if (M == 0) return NVFP4_OK;
  if (!a_q || !a_scale || !b_q || !b_scale || !d_bf16) return NVFP4_ERR_NULL;
  if (!nvfp4_aligned16(a_q) || !nvfp4_aligned16(a_scale) || !nvfp4_aligned16(b_q) || !nvfp4_aligned16(b_scale) ||
      !nvfp4_aligned16(add_bf16) || !nvfp4_aligned16(d_bf16))
    return NVFP4_ERR_ALIGN;
  const bool silu = epilogue == NVFP4_EPI_SILU_MUL;
  const Int8Args g = {a_q, a_scale, b_q, b_scale, reinterpret_cast<const uint16_t*>(add_bf16),
                      reinterpret_cast<uint16_t*>(d_bf16), M, N, K, silu ? N / 2 : N};
  return silu ? launch_int8<true>(g, (hipStream_t)stream) : launch_int8<false>(g, (hipStream_t)stream);
}

// ------------------------------------------------------------- dense expert

struct Int8FfnWs {
  size_t x_q, x_s, h, h_q, h_s, end;
};
static Int8FfnWs int8_ffn_layout(int64_t T, int64_t hidden, int64_t inter) {
  Int8FfnWs w;
  size_t p = 0;
  auto put = [&](size_t bytes) {
    const size_t at = p;
    p += nvfp4_align256(bytes);
    return at;
  };
  w.x_q = put((size_t)T * hidden);
  w.x_s = put((size_t)T * 4);
  w.h = put((size_t)T * inter * 2);
  w.h_q = put((size_t)T * inter);
  w.h_s = put((size_t)T * 4);
  w.end = p;
  return w;
}
static int int8_ffn_check(int32_t T, int32_t hidden, int32_t inter) {
  if (T < 0 || hidden <= 0 || inter <= 0 || hidden % 16 != 0 || inter % 16 != 0 || hidden > kInt8MaxK ||
      inter > kInt8MaxK || T > 64 * 65535)
    return NVFP4_ERR_SHAPE;
  return NVFP4_OK;
}

extern "C" size_t int8_ffn_ws_bytes(int32_t T, int32_t hidden, int32_t inter) {
  return int8_ffn_check(T, hidden, inter) ? 0 : int8_ffn_layout(T, hidden, inter).end;
}

extern "C" int int8_ffn_forward(const int8_t* w1_q, const float* w1_scale, const int8_t* w2_q, const float* w2_scale,
                                const void* x_bf16, int32_t T, int32_t hidden, int32_t inter, const void* add_bf16,
                                void* out_bf16, void* ws, size_t ws_bytes, void* stream) {
  int st = int8_ffn_check(T, hidden, inter);
  if (st) return st;
  if (T == 0) return NVFP4_OK;
  if (!w1_q || !w1_scale || !w2_q || !w2_scale || !x_bf16 || !out_bf16 || !ws) return NVFP4_ERR_NULL;
  if (!nvfp4_aligned16(w1_q) || !nvfp4_aligned16(w1_scale) || !nvfp4_aligned16(w2_q) || !nvfp4_aligned16(w2_scale) ||
      !nvfp4_aligned16(x_bf16) || !nvfp4_aligned16(add_bf16) || !nvfp4_aligned16(out_bf16) || !nvfp4_aligned16(ws))
    return NVFP4_ERR_ALIGN;
  const Int8FfnWs l = int8_ffn_layout(T, hidden, inter);
  if (ws_bytes < l.end) return NVFP4_ERR_WORKSPACE;
  char* base = reinterpret_cast<char*>(ws);
  int8_t* x_q = reinterpret_cast<int8_t*>(base + l.x_q);
  float* x_s = reinterpret_cast<float*>(base + l.x_s);
  int8_t* h_q = reinterpret_cast<int8_t*>(base + l.h_q);
  float* h_s = reinterpret_cast<float*>(base + l.h_s);
  st = int8_quantize_rows(x_bf16, NVFP4_DT_BF16, T, hidden, x_q, x_s, stream);
  if (st) return st;
  st = int8_gemm(x_q, x_s, w1_q, w1_scale, T, 2 * inter, hidden, NVFP4_EPI_SILU_MUL, nullptr, base + l.h, stream);
  if (st) return st;
  st = int8_quantize_rows(base + l.h, NVFP4_DT_BF16, T, inter, h_q, h_s, stream);
  if (st) return st;
  return int8_gemm(h_q, h_s, w2_q, w2_scale, T, hidden, inter, NVFP4_EPI_BF16, add_bf16, out_bf16, stream);
}
