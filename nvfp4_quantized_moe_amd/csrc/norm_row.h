// Rows of a norm in registers: their loads and stores, sums over a row, column
// weights, and the sums of a backward pass over rows; shared by the block's
// norms and the layer norm.
#pragma once
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "wave.h"

namespace nvfp4 {

constexpr int kNormMaxH = 16384;
constexpr int kNormMaxWaves = 16;
constexpr unsigned kGradThreads = 768;  // of a backward workgroup, at one chunk per thread

typedef uint32_t norm_u32x4_t __attribute__((ext_vector_type(4)));

template <typename T>
struct Vec8;  // eight elements as loaded
template <>
struct Vec8<uint16_t> {
  uint4 v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void load_past(const uint16_t* p) {  // not to stay in the caches
    v = __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const norm_u32x4_t*>(p)));
  }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t w = (&v.x)[i >> 1];
    return __uint_as_float((i & 1) ? (w & 0xFFFF0000u) : (w << 16));
  }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ float get(int i) const { return i < 4 ? (&a.x)[i] : (&b.x)[i - 4]; }
};
// Stores f[0..8) rounded to the type and leaves the stored values in f. PAST: past
// the caches (BF16 alone: of a lane's two stores of floats each fills every other
// 16 bytes).
template <bool PAST = false>
__device__ __forceinline__ uint4 store8(uint16_t* p, float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = f32x2_to_bf16x2(f[2 * i], f[2 * i + 1]);
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  const uint4 v = make_uint4(w[0], w[1], w[2], w[3]);
  if (p && PAST)
    __builtin_nontemporal_store(__builtin_bit_cast(norm_u32x4_t, v), reinterpret_cast<norm_u32x4_t*>(p));
  else if (p)
    *reinterpret_cast<uint4*>(p) = v;
  return v;
}
template <bool PAST = false>
__device__ __forceinline__ uint4 store8(float* p, float (&f)[8]) {
  if (p) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
  return make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ void load_weights8(const float* p, int at, float absent, float (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = absent;
  if (p) {
    Vec8<float> v;
    v.load(p + at);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = v.get(i);
  }
}

// A thread's place: `group` of the workgroup's row groups (whole waves), each
// with a row of its own, and `tid` of the `threads` of its group.
struct Place {
  int group, tid, threads;
};
__device__ __forceinline__ Place place_of(int threads) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = wave / (threads >> 6);
  return {group, (int)threadIdx.x - group * threads, threads};
}

// Sums of N values per thread over the row group, in every thread. A scratch
// array may be used again two calls later (in between, every wave has passed
// another call's barrier).
template <int N>
__device__ __forceinline__ void group_sums(const Place& at, float (&v)[N], float (*scratch)[N]) {
  const int waves = at.threads >> 6, first = at.group * waves;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_all_sum(v[i]);
  if (waves == 1) return;
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) scratch[threadIdx.x >> 6][i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.0f;
  for (int w = first; w < first + waves; ++w)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += scratch[w][i];
}

// Column weights of a thread's chunks: in registers for all rows, or (KEEP
// false, rows too wide for that) loaded at each use.
template <int CH, bool KEEP>
struct Columns {
  float w[KEEP ? CH : 1][8];
  const float* p;
  float absent;
  __device__ __forceinline__ void init(const Place& at, const float* from, float if_absent, int nchunk) {
    p = from;
    absent = if_absent;
    if constexpr (KEEP) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int ch = at.tid + c * at.threads;
        load_weights8(ch < nchunk ? p : nullptr, ch * 8, absent, w[c]);
      }
    }
  }
  __device__ __forceinline__ void get(const Place& at, int c, float (&o)[8]) const {
    if constexpr (KEEP) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = w[c][i];
    } else {
      load_weights8(p, (at.tid + c * at.threads) * 8, absent, o);
    }
  }
};

constexpr int kNormCus = 256;


// Column sums over the workgroups' partial rows: workgroup (b, s) adds 64
// columns of sum s of N. Its 16 waves take every 16th row, eight loads in flight,
// and are added in wave order (with 4 waves and one load in flight this took
// 20 us for 256 rows of 3 x 7168, now 5.4).
constexpr int kColumnWaves = 16;
template <int N>
__global__ __launch_bounds__(64 * kColumnWaves) void norm_columns_kernel(const float* __restrict__ partial, int rows,
                                                                         int H, float* out0, float* out1,
                                                                         float* out2) {
  __shared__ float sh[kColumnWaves][64];
  float* out = blockIdx.y == 0 ? out0 : blockIdx.y == 1 ? out1 : out2;
  if (!out) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (col < H) {
    const float* p = partial + (size_t)blockIdx.y * H + col;
    for (int r = wave; r < rows; r += 8 * kColumnWaves) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        v[u] = p[(size_t)min(r + u * kColumnWaves, rows - 1) * N * H];
#pragma unroll
      for (int u = 0; u < 8; ++u) s += r + u * kColumnWaves < rows ? v[u] : 0.0f;
    }
  }
  sh[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && col < H) {
    s = 0.0f;
    for (int w = 0; w < kColumnWaves; ++w) s += sh[w][lane];
    out[col] = s;
  }
}

}  // namespace nvfp4

// Threads for rows of H elements at CH chunks of 8 per thread: at most 512.
inline unsigned norm_threads(int32_t H, int ch) { return (unsigned)(((H / 8 + ch - 1) / ch + 63) / 64 * 64); }
// Workgroups that walk T rows: as many per CU as give it up to 16 waves. (More
// bring nothing where bytes count, 8192 x 7168: 93 us with 16 or 28, 98 with a
// workgroup per row; 4096 x 5120: 26.8, 29.6, 28.9; 2047 x 2888 float: 17.0,
// 19.5, 19.2. Small rows by themselves would be a little faster, 16384 x 2048:
// 43.3, 43.7, 40.6, larger ones not, 16384 x 4096: 102, 104, 125.)
inline unsigned norm_grid(int32_t T, unsigned threads) {
  const int per_cu = std::max(1, 16 / (int)(threads / 64));
  return (unsigned)std::min(T, nvfp4::kNormCus * per_cu);
}
// Chunks per thread: the fewest that 512 threads hold. Backward, one chunk only
// where two rows still share a workgroup of 768 threads: each thread's sums and
// weights of a second chunk cost less than a CU with a single row (16384 x
// 4096: 159 us instead of 180; 2047 x 2888 float: one chunk 32.9, two 34.5).
inline int norm_chunks(int32_t H) { return H <= 4096 ? 1 : H <= 8192 ? 2 : 4; }
inline int norm_grad_chunks(int32_t H) {
  return H <= 4096 && 2 * norm_threads(H, 1) > nvfp4::kGradThreads ? 2 : norm_chunks(H);
}
template <typename Fn>
inline int norm_by_chunks(int chunks, Fn fn) {
  if (chunks == 1) return fn(std::integral_constant<int, 1>());
  if (chunks == 2) return fn(std::integral_constant<int, 2>());
  return fn(std::integral_constant<int, 4>());
}

template <typename Fn>
inline int norm_by_types(int32_t x_dtype, int32_t res_dtype, Fn fn) {
  if (x_dtype == NVFP4_DT_BF16)
    return res_dtype == NVFP4_DT_BF16 ? fn(uint16_t(), uint16_t()) : fn(uint16_t(), float());
  return res_dtype == NVFP4_DT_BF16 ? fn(float(), uint16_t()) : fn(float(), float());
}

// One workgroup per CU, of as many row groups as give it 12 waves (8 with two
// chunks per thread, whose registers allow no more; 16384 x 2048 with 8 also at
// one chunk: 91 us instead of 84), fewer where the rows run out.
struct NormGradShape {
  unsigned row_threads, groups, grid;
};
inline NormGradShape norm_grad_shape(int32_t T, int32_t H) {
  const int ch = norm_grad_chunks(H);
  NormGradShape s;
  s.row_threads = norm_threads(H, ch);
  s.groups = (ch == 1 ? nvfp4::kGradThreads : 512) / s.row_threads;
  const unsigned rows = T < 1 ? 1 : (unsigned)T, want = (rows + nvfp4::kNormCus - 1) / nvfp4::kNormCus;
  if (s.groups > want) s.groups = want;
  if (s.groups < 1) s.groups = 1;
  const unsigned all = (rows + s.groups - 1) / s.groups;
  s.grid = all < (unsigned)nvfp4::kNormCus ? all : nvfp4::kNormCus;
  return s;
}
