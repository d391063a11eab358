// Layer norm with the residual update in front of it, and its gradients:
//   r' = residual + scale * x              stored in the residual's type (or r' = x)
//   y  = (r' - mean) / sqrt(var + eps) * w + b     from r' as stored; also as MXFP4
// One pass: a row's elements stay in registers between its reductions, and
// workgroups walk their rows with the next row's loads in flight, as the block's
// norms do. What bounds it is reading and writing the rows: 8192 x 7168 BF16 takes
// 87 us, 5.4 TB/s, a copy's rate; 64 x 7168, two dependent row sums, 4.6.
//
// Mean and variance in two steps, so that a row far from 0 keeps its digits: m
// from the sum, then d = r' - m, whose sums give what the rounding of m left
// out, delta = mean(d), and var = mean(d^2) - delta^2 (delta is a few roundings
// of m, so nothing cancels).
#include <type_traits>

#include "common.h"
#include "internal.h"
#include "mxfp4.h"
#include "norm_row.h"
#include "wave.h"

// Every rounding as it is written, so that a stored r' is the one of the plain steps.
#pragma clang fp contract(off)

namespace nvfp4 {

struct LayerNormArgs {
  int T, H;
  const float *w, *b;  // NULL: 1, 0
  float scale, eps;
  uint8_t *q, *s;      // MXFP4 of y, [T, Hp / 2] and [Hp / 128, T, 4]; QUANT alone
  bool ceil;
};

// What the next operator reads (y, d_x) is left to the caches, the residual
// stream, which the next norm reads, goes past them: stored so at any size in
// BF16, loaded so (PAST) from kLayerPastBytes on, as a smaller one may still be
// there. 8192 x 7168 and the quantizer both ways behind it: 127 us with neither,
// 116 stored, 111 both; 2048 x 4096: 19.0, 18.6, 20.0; and a library product with
// 2048 columns behind 4096 x 7168: 143, 136, 136. All outputs past the caches are
// faster by themselves (88 for 92) and slower in front of a reader (4096 x 7168
// and the quantizer 66 for 60).
constexpr int64_t kLayerPastBytes = 32 << 20;
template <bool PAST, typename R>
__device__ __forceinline__ void load_stream(Vec8<R>& v, const R* p) {
  if constexpr (PAST && sizeof(R) == 2)
    v.load_past(p);
  else
    v.load(p);
}

template <typename X, typename R, int CH, bool RES, bool PAST>
struct LayerRow {  // a row's inputs as loaded
  Vec8<X> x[CH];
  Vec8<R> r[RES ? CH : 1];
  __device__ __forceinline__ void load(const Place& at, const X* px, const R* pr, size_t row, int nchunk) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int ch = at.tid + c * at.threads;
      if (ch < nchunk) {
        x[c].load(px + row + ch * 8);
        if constexpr (RES) load_stream<PAST>(r[c], pr + row + ch * 8);
      }
    }
  }
};

// The eight values of a chunk as stored, for the codes made of them.
__device__ __forceinline__ void as_stored(const float (&)[8], uint4 bits, MxVec8<uint16_t>& v) { v.v = bits; }
__device__ __forceinline__ void as_stored(const float (&f)[8], uint4, MxVec8<float>& v) {
  v.a = make_float4(f[0], f[1], f[2], f[3]);
  v.b = make_float4(f[4], f[5], f[6], f[7]);
}

template <typename X, typename R, int CH, bool RES, bool QUANT, bool PAST>
__global__ __launch_bounds__(512) void layer_norm_kernel(const X* x, const R* residual, LayerNormArgs a, R* residual_out,
                                                         X* y) {
  constexpr bool KEEP = CH <= 2;
  __shared__ float scratch_a[2][kNormMaxWaves][1];
  __shared__ float scratch_b[2][kNormMaxWaves][2];
  const int nchunk = a.H / 8;
  const Place at = {0, (int)threadIdx.x, (int)blockDim.x};
  Columns<CH, KEEP> w, b;
  w.init(at, a.w, 1.0f, nchunk);
  b.init(at, a.b, 0.0f, nchunk);
  const float inv_h = 1.0f / (float)a.H;
  LayerRow<X, R, CH, RES, PAST> in;
  in.load(at, x, residual, (size_t)blockIdx.x * a.H, nchunk);
  int parity = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, parity ^= 1) {
    const size_t row = (size_t)t * a.H;
    const LayerRow<X, R, CH, RES, PAST> now = in;
    if (t + gridDim.x < a.T) in.load(at, x, residual, row + (size_t)gridDim.x * a.H, nchunk);
    float f[CH][8], s[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int ch = at.tid + c * at.threads;
      if (ch < nchunk) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          f[c][i] = now.x[c].get(i);
          if constexpr (RES) f[c][i] = now.r[c].get(i) + a.scale * f[c][i];
        }
        if constexpr (RES) store8<true>(residual_out + row + ch * 8, f[c]);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] += f[c][i];
      }
    }
    group_sums(at, s, scratch_a[parity]);
    const float m = s[0] * inv_h;
    float u[2] = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int ch = at.tid + c * at.threads;
      if (ch < nchunk) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          f[c][i] -= m;
          u[0] += f[c][i];
          u[1] += f[c][i] * f[c][i];
        }
      }
    }
    group_sums(at, u, scratch_b[parity]);
    const float delta = u[0] * inv_h;
    const float rho = rsqrtf(fmaxf(u[1] * inv_h - delta * delta, 0.0f) + a.eps);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int ch = at.tid + c * at.threads;
      uint4 bits = make_uint4(0, 0, 0, 0);
      if (ch < nchunk) {
        float cw[8], cb[8];
        w.get(at, c, cw);
        b.get(at, c, cb);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[c][i] = (f[c][i] - delta) * rho * cw[i] + cb[i];
        bits = store8(y ? y + row + ch * 8 : nullptr, f[c]);
      }
      if constexpr (QUANT) {
        // four neighbouring lanes share a scale; chunks behind the row are zeros
        const int Hp = mx_padded(a.H);
        MxVec8<X> v;
        as_stored(f[c], bits, v);
        if (ch >= nchunk) v.zero();
        int top = (int)v.amax();
        top = max(top, dpp_i32<kDppXor1>(top));
        top = max(top, dpp_i32<kDppXor2>(top));
        const uint32_t scale = mx_scale_bits((uint32_t)top, a.ceil ? MxVec8<X>::kUp : 0u);
        const uint32_t codes = v.codes(__uint_as_float(scale));
        if (ch * 8 < Hp) {
          *reinterpret_cast<uint32_t*>(a.q + (size_t)t * (Hp / 2) + ch * 4) = codes;
          if ((ch & 3) == 0) a.s[((size_t)(ch / 16) * a.T + t) * 4 + (ch / 4) % 4] = (uint8_t)(scale >> 23);
        }
      }
    }
  }
}

// Backward of one row, with n = (r' - mean) rho, dn = d_y w:
//   d_r = d_r' + rho (dn - mean(dn) - n mean(dn n)),  d_x = scale d_r
//   d_w += d_y n,  d_b += d_y
// mean, rho and the two means of dn come from one row sum and four more behind
// it: mean(dn n) = rho (mean(dn d) - delta mean(dn)). The column sums stay in
// registers over all rows of the thread; the workgroup's row groups add theirs
// in LDS, halving, and it leaves one row of partial sums (8191 x 2888, BF16 with
// a float residual: 73 us, 5.2 TB/s, and 4.7 for the columns' sums).
template <typename X, typename R, int CH, bool PAST>
struct LayerGradRow {
  Vec8<X> y[CH];
  Vec8<R> r[CH], d[CH];
  __device__ __forceinline__ void load(const Place& at, const X* py, const R* pr, const R* pd, size_t row, int nchunk) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int ch = at.tid + c * at.threads;
      if (ch < nchunk) {
        y[c].load(py + row + ch * 8);
        load_stream<PAST>(r[c], pr + row + ch * 8);
        if (pd) load_stream<PAST>(d[c], pd + row + ch * 8);
      }
    }
  }
};

template <typename X, typename R, int CH, bool PAST>
__global__ __launch_bounds__(CH == 1 ? kGradThreads : 512) void layer_norm_backward_kernel(
    const X* d_y, const R* d_res_out, const R* r, LayerNormArgs a, int row_threads, X* d_x, R* d_res, float* partial) {
  constexpr bool KEEP = CH <= 2;
  extern __shared__ __align__(16) float columns[];  // [groups / 2][2][H], with more than one row group
  __shared__ float scratch_a[2][kNormMaxWaves][1];
  __shared__ float scratch_b[2][kNormMaxWaves][4];
  const int nchunk = a.H / 8;
  const Place at = place_of(row_threads);
  const int groups = (int)blockDim.x / row_threads, step = (int)gridDim.x * groups;
  const float inv_h = 1.0f / (float)a.H;
  float c_w[CH][8], c_b[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) c_w[c][i] = c_b[c][i] = 0.0f;
  Columns<CH, KEEP> k_w;
  k_w.init(at, a.w, 1.0f, nchunk);
  LayerGradRow<X, R, CH, PAST> in;
  // all row groups make the same number of turns (they share the barriers); a
  // group without a row of its own repeats the last one and keeps nothing
  const int64_t first = (int64_t)blockIdx.x * groups;
  in.load(at, d_y, r, d_res_out, (size_t)min(first + at.group, (int64_t)a.T - 1) * a.H, nchunk);
  int parity = 0;
  for (int64_t t0 = first; t0 < a.T; t0 += step, parity ^= 1) {
    const bool mine = t0 + at.group < a.T;
    const int64_t t = mine ? t0 + at.group : a.T - 1, next = min(t0 + step + at.group, (int64_t)a.T - 1);
    const size_t row = (size_t)t * a.H;
    const LayerGradRow<X, R, CH, PAST> now = in;
    if (KEEP && t0 + step < a.T) in.load(at, d_y, r, d_res_out, (size_t)next * a.H, nchunk);
    float s[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (at.tid + c * at.threads < nchunk)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] += now.r[c].get(i);
    group_sums(at, s, scratch_a[parity]);
    const float m = s[0] * inv_h;
    float u[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // of d, d^2, dn, dn d
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (at.tid + c * at.threads < nchunk) {
        float w[8];
        k_w.get(at, c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float d = now.r[c].get(i) - m, dn = now.y[c].get(i) * w[i];
          u[0] += d;
          u[1] += d * d;
          u[2] += dn;
          u[3] += dn * d;
        }
      }
    }
    group_sums(at, u, scratch_b[parity]);
    const float delta = u[0] * inv_h;
    const float rho = rsqrtf(fmaxf(u[1] * inv_h - delta * delta, 0.0f) + a.eps);
    const float mean_dn = u[2] * inv_h, mean_dn_n = rho * (u[3] * inv_h - delta * mean_dn);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int ch = at.tid + c * at.threads;
      if (ch < nchunk && mine) {
        float w[8], dr[8], dx[8];
        k_w.get(at, c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float n = ((now.r[c].get(i) - m) - delta) * rho, dy = now.y[c].get(i);
          c_w[c][i] += dy * n;
          c_b[c][i] += dy;
          dr[i] = rho * ((dy * w[i] - mean_dn) - n * mean_dn_n);
          if (d_res_out) dr[i] += now.d[c].get(i);
          dx[i] = a.scale * dr[i];
        }
        store8(d_x + row + ch * 8, dx);
        if (d_res) store8<true>(d_res + row + ch * 8, dr);
      }
    }
    if (!KEEP && t0 + step < a.T) in.load(at, d_y, r, d_res_out, (size_t)next * a.H, nchunk);
  }
  const auto each = [&](auto fn) {  // fn(place in [2][H], the eight sums there)
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int ch = at.tid + c * at.threads;
      if (ch < nchunk) {
        fn(ch * 8, c_w[c]);
        fn(a.H + ch * 8, c_b[c]);
      }
    }
  };
  for (int n = groups; n > 1;) {
    const int keep = (n + 1) / 2;  // group keep + i adds to group i
    if (at.group >= keep && at.group < n)
      each([&](int place, float(&v)[8]) { store8(columns + (size_t)(at.group - keep) * 2 * a.H + place, v); });
    __syncthreads();
    if (at.group < n - keep)
      each([&](int place, float(&v)[8]) {
        Vec8<float> other;
        other.load(columns + (size_t)at.group * 2 * a.H + place);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += other.get(e);
      });
    __syncthreads();
    n = keep;
  }
  if (at.group == 0)
    each([&](int place, float(&v)[8]) { store8(partial + (size_t)blockIdx.x * 2 * a.H + place, v); });
}

}  // namespace nvfp4

using namespace nvfp4;

// fn(std::true_type) where a BF16 residual of this size is loaded past the caches.
template <typename R, bool RES, typename Fn>
static int by_past(int32_t T, int32_t H, Fn fn) {
  if constexpr (RES && sizeof(R) == 2)
    if ((int64_t)T * H * 2 >= kLayerPastBytes) return fn(std::true_type());
  return fn(std::false_type());
}

static int layer_norm_check(int32_t T, int32_t H, int32_t x_dtype, int32_t res_dtype) {
  if (T < 0 || H <= 0 || H % 8 != 0 || H > kNormMaxH) return NVFP4_ERR_SHAPE;
  if ((x_dtype != NVFP4_DT_BF16 && x_dtype != NVFP4_DT_F32) || (res_dtype != NVFP4_DT_BF16 && res_dtype != NVFP4_DT_F32))
    return NVFP4_ERR_ARG;
  return NVFP4_OK;
}

extern "C" int moe_layer_norm(const void* x, int32_t x_dtype, const void* residual, int32_t res_dtype, int32_t T,
                              int32_t H, const float* w, const float* b, float scale, float eps, void* residual_out,
                              void* y, int32_t rule, uint8_t* y_q, uint8_t* y_scale, void* stream) {
  const int st = layer_norm_check(T, H, x_dtype, res_dtype);
  if (st) return st;
  const bool quant = y_q || y_scale;
  if (quant && rule != MX_SCALE_FLOOR && rule != MX_SCALE_CEIL) return NVFP4_ERR_ARG;
  if (T == 0) return NVFP4_OK;
  if (!residual && (scale != 1.0f || residual_out || res_dtype != x_dtype)) return NVFP4_ERR_ARG;
  if (!x || (!y && !quant) || (residual && !residual_out) || !y_q != !y_scale) return NVFP4_ERR_NULL;
  if (!nvfp4_aligned16(x) || !nvfp4_aligned16(residual) || !nvfp4_aligned16(residual_out) || !nvfp4_aligned16(y) ||
      !nvfp4_aligned16(w) || !nvfp4_aligned16(b) || !nvfp4_aligned16(y_q) || !nvfp4_aligned16(y_scale))
    return NVFP4_ERR_ALIGN;
  const LayerNormArgs a = {T, H, w, b, scale, eps, y_q, y_scale, rule == MX_SCALE_CEIL};
  const auto go = [&](auto xt, auto rt, auto res) -> int {
    using X = decltype(xt);
    using R = decltype(rt);
    constexpr bool RES = decltype(res)::value;
    return norm_by_chunks(norm_chunks(H), [&](auto ch) -> int {
      constexpr int CH = decltype(ch)::value;
      const unsigned threads = norm_threads(H, CH);
      const auto launch = [&](auto q) -> int {
        return by_past<R, RES>(T, H, [&](auto past) -> int {
          hipLaunchKernelGGL((layer_norm_kernel<X, R, CH, RES, decltype(q)::value, decltype(past)::value>),
                             dim3(norm_grid(T, threads)), dim3(threads), 0, (hipStream_t)stream,
                             reinterpret_cast<const X*>(x), reinterpret_cast<const R*>(residual), a,
                             reinterpret_cast<R*>(residual_out), reinterpret_cast<X*>(y));
          NVFP4_CHECK_LAUNCH();
          return NVFP4_OK;
        });
      };
      return quant ? launch(std::true_type()) : launch(std::false_type());
    });
  };
  if (!residual) return x_dtype == NVFP4_DT_BF16 ? go(uint16_t(), uint16_t(), std::false_type()) : go(float(), float(), std::false_type());
  return norm_by_types(x_dtype, res_dtype, [&](auto xt, auto rt) { return go(xt, rt, std::true_type()); });
}

extern "C" size_t moe_layer_norm_backward_ws_bytes(int32_t T, int32_t H) {
  if (T < 0 || H <= 0 || H % 8 != 0 || H > kNormMaxH) return 0;
  return (size_t)norm_grad_shape(T, H).grid * 2 * H * sizeof(float);
}

extern "C" int moe_layer_norm_backward(const void* d_y, int32_t x_dtype, const void* d_residual_out, const void* r,
                                       int32_t res_dtype, int32_t T, int32_t H, const float* w, float scale, float eps,
                                       void* d_x, void* d_residual, float* d_w, float* d_b, void* ws, size_t ws_bytes,
                                       void* stream) {
  const int st = layer_norm_check(T, H, x_dtype, res_dtype);
  if (st) return st;
  if (T > 0 && !d_residual && (scale != 1.0f || res_dtype != x_dtype)) return NVFP4_ERR_ARG;
  if ((T > 0 && (!d_y || !r || !d_x)) || !ws) return NVFP4_ERR_NULL;
  if (!nvfp4_aligned16(d_y) || !nvfp4_aligned16(d_residual_out) || !nvfp4_aligned16(r) || !nvfp4_aligned16(w) ||
      !nvfp4_aligned16(d_x) || !nvfp4_aligned16(d_residual) || !nvfp4_aligned16(d_w) || !nvfp4_aligned16(d_b) ||
      !nvfp4_aligned16(ws))
    return NVFP4_ERR_ALIGN;
  if (ws_bytes < moe_layer_norm_backward_ws_bytes(T, H)) return NVFP4_ERR_WORKSPACE;
  const LayerNormArgs a = {T, H, w, nullptr, scale, eps, nullptr, nullptr, false};
  const NormGradShape shape = norm_grad_shape(T, H);
  if (T > 0) {
    const int e = norm_by_types(x_dtype, res_dtype, [&](auto xt, auto rt) -> int {
      using X = decltype(xt);
      using R = decltype(rt);
      return norm_by_chunks(norm_grad_chunks(H), [&](auto ch) -> int {
        constexpr int CH = decltype(ch)::value;
        const size_t lds = (size_t)(shape.groups / 2) * 2 * H * sizeof(float);  // at most 32 KB: H * groups <= 8192
        return by_past<R, true>(T, H, [&](auto past) -> int {
          hipLaunchKernelGGL((layer_norm_backward_kernel<X, R, CH, decltype(past)::value>), dim3(shape.grid),
                             dim3(shape.row_threads * shape.groups), lds, (hipStream_t)stream,
                             reinterpret_cast<const X*>(d_y), reinterpret_cast<const R*>(d_residual_out),
                             reinterpret_cast<const R*>(r), a, (int)shape.row_threads, reinterpret_cast<X*>(d_x),
                             reinterpret_cast<R*>(d_residual), reinterpret_cast<float*>(ws));
          NVFP4_CHECK_LAUNCH();
          return NVFP4_OK;
        });
      });
    });
    if (e) return e;
  }
  if (!d_w && !d_b) return NVFP4_OK;
  // T = 0: the sums over no rows, zeros
  hipLaunchKernelGGL(norm_columns_kernel<2>, dim3((H + 63) / 64, 2), dim3(64 * kColumnWaves), 0, (hipStream_t)stream,
                     reinterpret_cast<const float*>(ws), T > 0 ? (int)shape.grid : 0, H, d_w, d_b, (float*)nullptr);
  NVFP4_CHECK_LAUNCH();
  return NVFP4_OK;
}
