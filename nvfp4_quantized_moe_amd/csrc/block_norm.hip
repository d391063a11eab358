// The norms around the expert FFN, fused with its gate and residual scale,
// and their gradients:
//   n  = x * rsqrt(mean x^2 + eps) * w_post        (or n = x)
//   r' = residual + scale * gate * n               stored in the residual's type
//   y  = r' * rsqrt(mean r'^2 + eps) * w_pre       from r' as stored; also as NVFP4
// One pass: a row's elements stay in registers between the two reductions.
//
// A workgroup owns whole rows; thread i holds the row's 8-element chunks i,
// i + blockDim.x, ... (16-byte loads). It walks the rows of its share with the
// next row's loads in flight and its columns' weights in registers: read
// again for every row, the three float32 vectors would be as many bytes from
// L2 as the row is from memory (8192 x 7168 BF16: 93 us, 5.05 TB/s, weights
// read again 108; backward 150 and 197). Sums are float32: the lanes of a wave by DPP,
// then the waves through LDS in wave order, so results repeat bit for bit.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "internal.h"
#include "quant_block.h"
#include "wave.h"

namespace nvfp4 {

constexpr int kNormMaxH = 16384;
constexpr int kNormMaxWaves = 16;
constexpr unsigned kGradThreads = 768;  // of a backward workgroup, at one chunk per thread

template <typename T>
struct Vec8;  // eight elements as loaded
template <>
struct Vec8<uint16_t> {
  uint4 v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const uint4*>(p); }
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
// Stores f[0..8) rounded to the type and leaves the stored values in f.
__device__ __forceinline__ uint4 store8(uint16_t* p, float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = f32x2_to_bf16x2(f[2 * i], f[2 * i + 1]);
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  const uint4 v = make_uint4(w[0], w[1], w[2], w[3]);
  if (p) *reinterpret_cast<uint4*>(p) = v;
  return v;
}
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

struct NormArgs {
  int T, H;
  const float* w_pre;    // NULL: no y
  const float* w_post;   // NULL: no norm of x
  const float* gate;     // [H], [T] or NULL
  int gate_tokens;       // gate is [T]
  float scale, eps;
};

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

template <typename X, typename R, int CH>
struct NormRow {  // a row's inputs as loaded
  Vec8<X> x[CH];
  Vec8<R> r[CH];
  __device__ __forceinline__ void load(const Place& at, const X* px, const R* pr, size_t row, int nchunk) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int ch = at.tid + c * at.threads;
      if (ch < nchunk) {
        x[c].load(px + row + ch * 8);
        if (pr) r[c].load(pr + row + ch * 8);
      }
    }
  }
};

constexpr int kNormCus = 256;

template <typename X, typename R, int CH, bool QUANT>
__global__ __launch_bounds__(512) void block_norm_kernel(const X* x, const R* residual, NormArgs a, R* residual_out,
                                                         X* y, const float* gs_in, uint8_t* y_q, uint8_t* y_sf) {
  // Every rounding as the formulas have it (one of g and g_row is 1), so that a
  // BF16 residual rounds as it does where they are computed step by step; a
  // float y made from it would show each that went the other way.
#pragma clang fp contract(off)
  constexpr bool KEEP = CH <= 2;
  __shared__ float scratch[4][kNormMaxWaves][1];
  __shared__ uint4 lut[QUANT ? kLutWords / 4 : 1];
  const int nchunk = a.H / 8;
  const Place at = {0, (int)threadIdx.x, (int)blockDim.x};
  float gs = 0.0f;
  if constexpr (QUANT) {
    gs = gs_in[0];
    build_threshold_lut(gs, reinterpret_cast<uint32_t*>(lut), threadIdx.x, blockDim.x);
    __syncthreads();
  }
  Columns<CH, KEEP> w_pre, w_post, gate;
  w_pre.init(at, a.w_pre, 1.0f, nchunk);
  w_post.init(at, a.w_post, 1.0f, nchunk);
  gate.init(at, a.gate_tokens ? nullptr : a.gate, 1.0f, nchunk);
  const float inv_h = 1.0f / (float)a.H;
  NormRow<X, R, CH> in;
  in.load(at, x, residual, (size_t)blockIdx.x * a.H, nchunk);
  int parity = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, parity ^= 2) {
    const size_t row = (size_t)t * a.H;
    const NormRow<X, R, CH> now = in;
    if (t + gridDim.x < a.T) in.load(at, x, residual, row + (size_t)gridDim.x * a.H, nchunk);
    float f[CH][8], s[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int ch = at.tid + c * at.threads;
      if (ch < nchunk) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          f[c][i] = now.x[c].get(i);
          s[0] += f[c][i] * f[c][i];
        }
      }
    }
    const float g_row = (a.gate && a.gate_tokens) ? a.gate[t] : 1.0f;
    float sig = 1.0f;
    if (a.w_post) {
      group_sums(at, s, scratch[parity]);
      sig = rsqrtf(s[0] * inv_h + a.eps);
    }
    s[0] = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int ch = at.tid + c * at.threads;
      if (ch < nchunk) {
        float w[8], g[8];
        w_post.get(at, c, w);
        gate.get(at, c, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          f[c][i] = a.scale * (f[c][i] * sig * w[i] * (g[i] * g_row));
          if (residual) f[c][i] = now.r[c].get(i) + f[c][i];
        }
        store8(residual_out + row + ch * 8, f[c]);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] += f[c][i] * f[c][i];
      }
    }
    if (!a.w_pre) continue;
    group_sums(at, s, scratch[parity + 1]);
    const float rho = rsqrtf(s[0] * inv_h + a.eps);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int ch = at.tid + c * at.threads;
      uint4 bits = make_uint4(0, 0, 0, 0);
      if (ch < nchunk) {
        float w[8];
        w_pre.get(at, c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[c][i] = f[c][i] * rho * w[i];
        bits = store8(y ? y + row + ch * 8 : nullptr, f[c]);
      }
      if constexpr (QUANT) {
        // a 16-element block is the chunks of two neighbouring lanes (an even
        // number of chunks in a row): the even lane takes the odd one's words
        const auto swap = [](uint32_t v) { return (uint32_t)dpp_i32<kDppXor1>((int)v); };
        const uint4 next = make_uint4(swap(bits.x), swap(bits.y), swap(bits.z), swap(bits.w));
        if (ch < nchunk && (threadIdx.x & 1) == 0) {
          const uint32_t w[8] = {bits.x, bits.y, bits.z, bits.w, next.x, next.y, next.z, next.w};
          uint2 packed;
          const uint32_t code = quantize_block16(w, quant_scale(gs), lut, &packed);
          const size_t blk = (row >> 4) + (ch >> 1);
          *reinterpret_cast<uint2*>(y_q + blk * 8) = packed;
          y_sf[blk] = (uint8_t)code;
        }
      }
    }
  }
}

// Backward of one row, with rn = r' rho, dn = d_y w_pre, xn = x sig:
//   d_r = d_r' + rho (dn - rn mean(dn rn)),  d_w_pre += d_y rn
//   db  = scale d_r,  d_gate = db n (summed over the row or the batch)
//   db' = db gate,    d_w_post += db' xn
//   d_x = sig (db' w_post - xn mean(db' w_post xn)),  or db' without w_post
// Two reductions per row (the second needs the first's result). The column
// sums d_w_pre, d_w_post, d_gate stay in registers over all rows of the
// thread; the workgroup's row groups add theirs in LDS, and it leaves one row
// of partial sums, which norm_columns_kernel adds in workgroup order. (With a
// workgroup for each row group, twice the partial rows: 2047 x 2888 took 36 us.)
template <typename X, typename R, int CH>
struct NormGradRow {
  Vec8<X> x[CH], y[CH];
  Vec8<R> r[CH], d[CH];
  __device__ __forceinline__ void load(const Place& at, const X* px, const X* py, const R* pr, const R* pd, size_t row,
                                       int nchunk) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int ch = at.tid + c * at.threads;
      if (ch < nchunk) {
        x[c].load(px + row + ch * 8);
        if (py) y[c].load(py + row + ch * 8);
        if (py) r[c].load(pr + row + ch * 8);
        if (pd) d[c].load(pd + row + ch * 8);
      }
    }
  }
};

template <typename X, typename R, int CH>
__global__ __launch_bounds__(CH == 1 ? kGradThreads : 512) void block_norm_backward_kernel(
    const X* d_y, const R* d_res_out, const X* x, const R* res_out, NormArgs a, int row_threads, X* d_x, R* d_res,
    float* d_gate_tokens, float* partial) {
  constexpr bool KEEP = CH <= 2;
  extern __shared__ float columns[];  // [groups / 2][3][H], with more than one row group
  __shared__ float scratch_a[2][kNormMaxWaves][3];
  __shared__ float scratch_b[2][kNormMaxWaves][2];
  const int nchunk = a.H / 8;
  const Place at = place_of(row_threads);
  const int groups = (int)blockDim.x / row_threads, step = (int)gridDim.x * groups;
  const float inv_h = 1.0f / (float)a.H;
  float c_pre[CH][8], c_post[CH][8], c_gate[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) c_pre[c][i] = c_post[c][i] = c_gate[c][i] = 0.0f;
  Columns<CH, KEEP> k_pre, k_post, k_gate;
  k_pre.init(at, a.w_pre, 0.0f, nchunk);
  k_post.init(at, a.w_post, 1.0f, nchunk);
  k_gate.init(at, a.gate_tokens ? nullptr : a.gate, 1.0f, nchunk);
  const X* py = a.w_pre ? d_y : nullptr;
  NormGradRow<X, R, CH> in;
  // all row groups make the same number of turns (they share the barriers); a
  // group without a row of its own repeats the last one and keeps nothing
  const int64_t first = (int64_t)blockIdx.x * groups;
  in.load(at, x, py, res_out, d_res_out, (size_t)min(first + at.group, (int64_t)a.T - 1) * a.H, nchunk);
  int parity = 0;
  for (int64_t t0 = first; t0 < a.T; t0 += step, parity ^= 1) {
    const bool mine = t0 + at.group < a.T;
    const int64_t t = mine ? t0 + at.group : a.T - 1, next = min(t0 + step + at.group, (int64_t)a.T - 1);
    const size_t row = (size_t)t * a.H;
    const NormGradRow<X, R, CH> now = in;
    if (KEEP && t0 + step < a.T) in.load(at, x, py, res_out, d_res_out, (size_t)next * a.H, nchunk);
    float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int ch = at.tid + c * at.threads;
      if (ch < nchunk) {
        if (a.w_pre) {
          float w[8];
          k_pre.get(at, c, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            s[0] += now.r[c].get(i) * now.r[c].get(i);
            s[1] += now.y[c].get(i) * w[i] * now.r[c].get(i);
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s[2] += now.x[c].get(i) * now.x[c].get(i);
      }
    }
    group_sums(at, s, scratch_a[parity]);
    const float rho = rsqrtf(s[0] * inv_h + a.eps);
    const float mean = s[1] * rho * inv_h;  // of dn rn
    const float sig = a.w_post ? rsqrtf(s[2] * inv_h + a.eps) : 1.0f;
    const float g_row = (a.gate && a.gate_tokens) ? a.gate[t] : 1.0f;
    float u[2] = {0.0f, 0.0f};
    float dxn[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int ch = at.tid + c * at.threads;
      if (ch < nchunk && mine) {
        float dr[8], w_pre[8], w_post[8], gate[8];
        k_pre.get(at, c, w_pre);
        k_post.get(at, c, w_post);
        k_gate.get(at, c, gate);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dr[i] = d_res_out ? now.d[c].get(i) : 0.0f;
          if (a.w_pre) {
            const float rn = now.r[c].get(i) * rho;
            dr[i] += rho * (now.y[c].get(i) * w_pre[i] - rn * mean);
            c_pre[c][i] += now.y[c].get(i) * rn;
          }
          const float xn = now.x[c].get(i) * sig;
          const float db = a.scale * dr[i];
          const float dg = db * xn * w_post[i];
          c_gate[c][i] += dg;
          u[1] += dg;
          const float dbg = db * (gate[i] * g_row);
          c_post[c][i] += dbg * xn;
          dxn[c][i] = dbg * w_post[i];
          u[0] += dxn[c][i] * xn;
        }
        store8(d_res + row + ch * 8, dr);
      }
    }
    if (a.w_post || d_gate_tokens) group_sums(at, u, scratch_b[parity]);
    if (d_gate_tokens && at.tid == 0 && mine) d_gate_tokens[t] = u[1];
    const float mx = a.w_post ? u[0] * inv_h : 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int ch = at.tid + c * at.threads;
      if (ch < nchunk && mine) {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          o[i] = a.w_post ? sig * (dxn[c][i] - now.x[c].get(i) * sig * mx) : dxn[c][i];
        store8(d_x + row + ch * 8, o);
      }
    }
    if (!KEEP && t0 + step < a.T) in.load(at, x, py, res_out, d_res_out, (size_t)next * a.H, nchunk);
  }
  // The row groups' column sums end in one group, which writes the workgroup's
  // partial sums, [workgroup][3][H]. Of up to twelve groups (one chunk per
  // thread) the upper half leaves its own in LDS and the lower half adds them,
  // again and again (8192 x 128: one group after the other 17.1 us, so 14.5);
  // of one or two the last adds the first's, which keeps the loop above as fast
  // as it is without (8192 x 7168: 151, in halves 154).
  if constexpr (CH == 1) {
    const auto each = [&](auto fn) {  // fn(place in [3][H], the eight sums there)
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int ch = at.tid + c * at.threads;
        if (ch < nchunk) {
          fn(ch * 8, c_pre[c]);
          fn(a.H + ch * 8, c_post[c]);
          fn(2 * a.H + ch * 8, c_gate[c]);
        }
      }
    };
    for (int n = groups; n > 1;) {
      const int keep = (n + 1) / 2;  // group keep + i adds to group i
      if (at.group >= keep && at.group < n)
        each([&](int place, float(&v)[8]) { store8(columns + (size_t)(at.group - keep) * 3 * a.H + place, v); });
      __syncthreads();
      if (at.group < n - keep)
        each([&](int place, float(&v)[8]) {
          Vec8<float> other;
          other.load(columns + (size_t)at.group * 3 * a.H + place);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] += other.get(e);
        });
      __syncthreads();
      n = keep;
    }
    if (at.group == 0)
      each([&](int place, float(&v)[8]) { store8(partial + (size_t)blockIdx.x * 3 * a.H + place, v); });
  } else {
    for (int g = 0; g < groups; ++g) {
      const bool last = g + 1 == groups;
      if (at.group == g) {
        // the last group writes the workgroup's partial sums: [workgroup][3][H]
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const int ch = at.tid + c * at.threads;
          if (ch < nchunk) {
            float* out = partial + (size_t)blockIdx.x * 3 * a.H + ch * 8;
            float(*v[3])[8] = {&c_pre[c], &c_post[c], &c_gate[c]};
#pragma unroll
            for (int i = 0; i < 3; ++i) {
              float* sum = columns + (size_t)i * a.H + ch * 8;
              if (g > 0) {
                Vec8<float> was;
                was.load(sum);
#pragma unroll
                for (int e = 0; e < 8; ++e) (*v[i])[e] += was.get(e);
              }
              store8(last ? out + (size_t)i * a.H : sum, *v[i]);
            }
          }
        }
      }
      if (!last) __syncthreads();
    }
  }
}

// Column sums over the workgroups' partial rows: workgroup (b, s) adds 64
// columns of sum s. Its 16 waves take every 16th row, eight loads in flight,
// and are added in wave order (with 4 waves and one load in flight this took
// 20 us for 256 rows of 3 x 7168, now 5.4).
constexpr int kColumnWaves = 16;
__global__ __launch_bounds__(64 * kColumnWaves) void norm_columns_kernel(const float* __restrict__ partial, int rows,
                                                                         int H, float* d_pre, float* d_post,
                                                                         float* d_gate) {
  __shared__ float sh[kColumnWaves][64];
  float* out = blockIdx.y == 0 ? d_pre : blockIdx.y == 1 ? d_post : d_gate;
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
        v[u] = p[(size_t)min(r + u * kColumnWaves, rows - 1) * 3 * H];
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

using namespace nvfp4;

static int norm_check(int32_t T, int32_t H, int32_t x_dtype, int32_t res_dtype, const float* gate, int32_t gate_mode) {
  if (T < 0 || H <= 0 || H % 8 != 0 || H > kNormMaxH) return NVFP4_ERR_SHAPE;
  if ((x_dtype != NVFP4_DT_BF16 && x_dtype != NVFP4_DT_F32) ||
      (res_dtype != NVFP4_DT_BF16 && res_dtype != NVFP4_DT_F32))
    return NVFP4_ERR_ARG;
  if (gate_mode != MOE_GATE_NONE && gate_mode != MOE_GATE_CHANNEL && gate_mode != MOE_GATE_TOKEN)
    return NVFP4_ERR_ARG;
  if (gate_mode != MOE_GATE_NONE && !gate && T > 0) return NVFP4_ERR_NULL;
  return NVFP4_OK;
}

// Threads for rows of H elements at CH chunks of 8 per thread: at most 512.
static unsigned norm_threads(int32_t H, int ch) { return (unsigned)(((H / 8 + ch - 1) / ch + 63) / 64 * 64); }
// Workgroups that walk T rows: as many per CU as give it up to 16 waves. (More
// bring nothing where bytes count, 8192 x 7168: 93 us with 16 or 28, 98 with a
// workgroup per row; 4096 x 5120: 26.8, 29.6, 28.9; 2047 x 2888 float: 17.0,
// 19.5, 19.2. Small rows by themselves would be a little faster, 16384 x 2048:
// 43.3, 43.7, 40.6, larger ones not, 16384 x 4096: 102, 104, 125.)
static unsigned norm_grid(int32_t T, unsigned threads) {
  const int per_cu = std::max(1, 16 / (int)(threads / 64));
  return (unsigned)std::min(T, kNormCus * per_cu);
}
// Chunks per thread: the fewest that 512 threads hold. Backward, one chunk only
// where two rows still share a workgroup of 768 threads: each thread's sums and
// weights of a second chunk cost less than a CU with a single row (16384 x
// 4096: 159 us instead of 180; 2047 x 2888 float: one chunk 32.9, two 34.5).
static int norm_chunks(int32_t H) { return H <= 4096 ? 1 : H <= 8192 ? 2 : 4; }
static int norm_grad_chunks(int32_t H) {
  return H <= 4096 && 2 * norm_threads(H, 1) > kGradThreads ? 2 : norm_chunks(H);
}
template <typename Fn>
static int norm_by_chunks(int chunks, Fn fn) {
  if (chunks == 1) return fn(std::integral_constant<int, 1>());
  if (chunks == 2) return fn(std::integral_constant<int, 2>());
  return fn(std::integral_constant<int, 4>());
}

template <typename Fn>
static int norm_by_types(int32_t x_dtype, int32_t res_dtype, Fn fn) {
  if (x_dtype == NVFP4_DT_BF16)
    return res_dtype == NVFP4_DT_BF16 ? fn(uint16_t(), uint16_t()) : fn(uint16_t(), float());
  return res_dtype == NVFP4_DT_BF16 ? fn(float(), uint16_t()) : fn(float(), float());
}

extern "C" int moe_block_norm(const void* x, int32_t x_dtype, const void* residual, int32_t res_dtype, int32_t T,
                              int32_t H, const float* w_pre, const float* w_post, const float* gate,
                              int32_t gate_mode, float scale, float eps, void* residual_out, void* y,
                              const float* gs_in, uint8_t* y_q, uint8_t* y_sf, void* stream) {
  const int st = norm_check(T, H, x_dtype, res_dtype, gate, gate_mode);
  if (st) return st;
  if (gs_in && H % 32 != 0) return NVFP4_ERR_SHAPE;
  if (gs_in && x_dtype != NVFP4_DT_BF16) return NVFP4_ERR_ARG;
  if (T == 0) return NVFP4_OK;
  if (!x || !residual_out || (w_pre && !y && !gs_in) || (gs_in && (!w_pre || !y_q || !y_sf))) return NVFP4_ERR_NULL;
  if (!nvfp4_aligned16(x) || !nvfp4_aligned16(residual) || !nvfp4_aligned16(residual_out) || !nvfp4_aligned16(y) ||
      !nvfp4_aligned16(w_pre) || !nvfp4_aligned16(w_post) || !nvfp4_aligned16(gate) || !nvfp4_aligned16(gs_in) ||
      !nvfp4_aligned16(y_q) || !nvfp4_aligned16(y_sf))
    return NVFP4_ERR_ALIGN;
  const NormArgs a = {T, H, w_pre, w_post, gate_mode == MOE_GATE_NONE ? nullptr : gate, gate_mode == MOE_GATE_TOKEN,
                      scale, eps};
  return norm_by_types(x_dtype, res_dtype, [&](auto xt, auto rt) -> int {
    using X = decltype(xt);
    using R = decltype(rt);
    auto go = [&](auto ch, auto quant) -> int {
      constexpr int CH = decltype(ch)::value;
      const unsigned threads = norm_threads(H, CH);
      hipLaunchKernelGGL((block_norm_kernel<X, R, CH, decltype(quant)::value>), dim3(norm_grid(T, threads)),
                         dim3(threads), 0, (hipStream_t)stream, reinterpret_cast<const X*>(x),
                         reinterpret_cast<const R*>(residual), a, reinterpret_cast<R*>(residual_out),
                         reinterpret_cast<X*>(y), gs_in, y_q, y_sf);
      NVFP4_CHECK_LAUNCH();
      return NVFP4_OK;
    };
    auto by_width = [&](auto quant) -> int {
      return norm_by_chunks(norm_chunks(H), [&](auto ch) { return go(ch, quant); });
    };
    if constexpr (std::is_same<X, uint16_t>::value)
      if (gs_in) return by_width(std::true_type());
    return by_width(std::false_type());
  });
}

// One workgroup per CU, of as many row groups as give it 12 waves (8 with two
// chunks per thread, whose registers allow no more; 16384 x 2048 with 8 also at
// one chunk: 91 us instead of 84), fewer where the rows run out.
struct NormGradShape {
  unsigned row_threads, groups, grid;
};
static NormGradShape norm_grad_shape(int32_t T, int32_t H) {
  const int ch = norm_grad_chunks(H);
  NormGradShape s;
  s.row_threads = norm_threads(H, ch);
  s.groups = (ch == 1 ? kGradThreads : 512) / s.row_threads;
  const unsigned rows = T < 1 ? 1 : (unsigned)T, want = (rows + kNormCus - 1) / kNormCus;
  if (s.groups > want) s.groups = want;
  if (s.groups < 1) s.groups = 1;
  const unsigned all = (rows + s.groups - 1) / s.groups;
  s.grid = all < (unsigned)kNormCus ? all : kNormCus;
  return s;
}

extern "C" size_t moe_block_norm_backward_ws_bytes(int32_t T, int32_t H) {
  if (T < 0 || H <= 0 || H % 8 != 0 || H > kNormMaxH) return 0;
  return (size_t)norm_grad_shape(T, H).grid * 3 * H * sizeof(float);
}

extern "C" int moe_block_norm_backward(const void* d_y, const void* d_residual_out, const void* x, int32_t x_dtype,
                                       const void* residual_out, int32_t res_dtype, int32_t T, int32_t H,
                                       const float* w_pre, const float* w_post, const float* gate, int32_t gate_mode,
                                       float scale, float eps, void* d_x, void* d_residual, float* d_w_pre,
                                       float* d_w_post, float* d_gate, void* ws, size_t ws_bytes, void* stream) {
  const int st = norm_check(T, H, x_dtype, res_dtype, gate, gate_mode);
  if (st) return st;
  if (T > 0 && (!x || !d_x || !d_residual || (w_pre && (!d_y || !residual_out)) || (!w_pre && !d_residual_out)))
    return NVFP4_ERR_NULL;
  if ((w_pre && !d_w_pre) || (w_post && !d_w_post) || (gate_mode == MOE_GATE_CHANNEL && !d_gate) ||
      (gate_mode == MOE_GATE_TOKEN && T > 0 && !d_gate) || !ws)
    return NVFP4_ERR_NULL;
  if (!nvfp4_aligned16(d_y) || !nvfp4_aligned16(d_residual_out) || !nvfp4_aligned16(x) ||
      !nvfp4_aligned16(residual_out) || !nvfp4_aligned16(w_pre) || !nvfp4_aligned16(w_post) ||
      !nvfp4_aligned16(gate) || !nvfp4_aligned16(d_x) || !nvfp4_aligned16(d_residual) || !nvfp4_aligned16(d_w_pre) ||
      !nvfp4_aligned16(d_w_post) || !nvfp4_aligned16(d_gate) || !nvfp4_aligned16(ws))
    return NVFP4_ERR_ALIGN;
  if (ws_bytes < moe_block_norm_backward_ws_bytes(T, H)) return NVFP4_ERR_WORKSPACE;
  const bool per_token = gate_mode == MOE_GATE_TOKEN;
  const NormArgs a = {T, H, w_pre, w_post, gate_mode == MOE_GATE_NONE ? nullptr : gate, per_token, scale, eps};
  const NormGradShape shape = norm_grad_shape(T, H);
  if (T > 0) {
    const int r = norm_by_types(x_dtype, res_dtype, [&](auto xt, auto rt) -> int {
      using X = decltype(xt);
      using R = decltype(rt);
      auto go = [&](auto ch) -> int {
        constexpr int CH = decltype(ch)::value;
        const size_t lds = (size_t)(shape.groups / 2) * 3 * H * sizeof(float);  // at most 48 KB: H * groups <= 8192
        hipLaunchKernelGGL((block_norm_backward_kernel<X, R, CH>), dim3(shape.grid),
                           dim3(shape.row_threads * shape.groups), lds, (hipStream_t)stream,
                           reinterpret_cast<const X*>(d_y), reinterpret_cast<const R*>(d_residual_out),
                           reinterpret_cast<const X*>(x), reinterpret_cast<const R*>(residual_out), a,
                           (int)shape.row_threads, reinterpret_cast<X*>(d_x),
                           reinterpret_cast<R*>(d_residual), per_token ? d_gate : nullptr,
                           reinterpret_cast<float*>(ws));
        NVFP4_CHECK_LAUNCH();
        return NVFP4_OK;
      };
      return norm_by_chunks(norm_grad_chunks(H), go);
    });
    if (r) return r;
  }
  // T = 0: the sums over no rows, zeros
  float* gate_cols = gate_mode == MOE_GATE_CHANNEL ? d_gate : nullptr;
  hipLaunchKernelGGL(norm_columns_kernel, dim3((H + 63) / 64, 3), dim3(64 * kColumnWaves), 0, (hipStream_t)stream,
                     reinterpret_cast<const float*>(ws), T > 0 ? (int)shape.grid : 0, H, w_pre ? d_w_pre : nullptr,
                     w_post ? d_w_post : nullptr, gate_cols);
  NVFP4_CHECK_LAUNCH();
  return NVFP4_OK;
}
