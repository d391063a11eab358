// Products of 8-bit integers with a scale per token and per output channel,
// for the dense expert that runs beside the routed ones:
//   q[m, k] = rne(x[m, k] / s_m), s_m = amax_k |x[m, k]| * (1 / 127)
//   C[m, n] = a_s[m] * b_s[n] * sum_k a_q[m, k] b_q[n, k]
// The sum is exact in int32 (K <= 65536: |sum| <= 2^30), so neither the order
// of K nor its split can change a result; the scales are applied to it in
// float32 and the output is rounded once.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "internal.h"
#include "tile.h"
#include "wave.h"

// Every rounding as it is written (the fmas below are explicit): a token's
// outputs are the same whichever of the kernels computes them, so they do not
// depend on how many other tokens the call has.
#pragma clang fp contract(off)

namespace nvfp4 {

typedef int int16v __attribute__((ext_vector_type(16)));

constexpr int kInt8MaxK = 65536;
constexpr int kInt8MaxM = 64 * 65535;        // by 1024 threads still within a grid
constexpr int kInt8MaxN = (1 << 27) - 16;    // by 512 threads for 16 columns: fewer than 2^32

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

__device__ __forceinline__ void load8(const uint16_t* p, float (&f)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 v = reinterpret_cast<const float4*>(p)[i];
    f[4 * i] = v.x;
    f[4 * i + 1] = v.y;
    f[4 * i + 2] = v.z;
    f[4 * i + 3] = v.w;
  }
}

// Scale of a row from each thread's largest magnitude. Rows of the smallest
// numbers are lifted by 2^100 (exactly, like their scale), so that neither
// 1 / s nor the residual above leaves the float32 range.
struct RowScale {
  float stored, s, inv, lift;
};
__device__ __forceinline__ RowScale row_scale(float m, float* red) {
  m = wave_all_max(m);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  m = red[0];
  for (int w = 1; w < (int)blockDim.x / 64; ++w) m = fmaxf(m, red[w]);
  RowScale r;
  r.stored = m * (1.0f / 127.0f);
  r.lift = r.stored < 0x1p-100f ? 0x1p100f : 1.0f;
  r.s = r.stored * r.lift;
  r.inv = r.s > 0.0f ? 1.0f / r.s : 0.0f;
  return r;
}
// Codes of N values (a multiple of four), four to a word, the first in the low
// byte; zeros in a row of zeros. x (1/s) + 1.5 2^23 rounds to an integer n and
// leaves it, in two's complement, in the low mantissa bits. n is the nearest
// to x / s unless the remainder x - n s is about s / 2; where one of a
// thread's remainders is, all its codes go the exact way. (Exact for every
// element, 8192 x 7168 took 45 us.)
template <int N>
__device__ __forceinline__ void quantize_codes(const float* f, const RowScale& r, uint32_t* w) {
  constexpr float kMagic = 12582912.0f;
  float worst = 0.0f;
#pragma unroll
  for (int j = 0; j < N / 4; ++j) {
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = f[4 * j + i] * r.lift;
      const float m = __builtin_fmaf(x, r.inv, kMagic);
      worst = fmaxf(worst, fabsf(__builtin_fmaf(-(m - kMagic), r.s, x)));
      b[i] = __float_as_uint(m);
    }
    const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u), hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000C0Cu);
    w[j] = lo | hi;
  }
  if (worst >= r.s * 0.4999f) {
#pragma unroll
    for (int j = 0; j < N / 4; ++j) {
      w[j] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[j] |= (uint32_t)((r.s > 0.0f ? quantize_int8(f[4 * j + i] * r.lift, r.s, r.inv) : 0) & 0xFF) << (8 * i);
    }
  }
}

// One workgroup per row; thread i holds the row's 8-element chunks i, i +
// blockDim.x, ... between the maximum and the rounding. (8192 x 7168: with 16
// elements per thread, whose two loads each touch every line of 2 KB, 45 us;
// with the row read a second time from the cache 46 us.)
template <typename T, int CH>
__global__ __launch_bounds__(1024) void int8_rows_kernel(const T* __restrict__ x, int K, int8_t* __restrict__ q,
                                                         float* __restrict__ scale) {
  __shared__ float red[16];
  const size_t row = (size_t)blockIdx.x * K;
  const int n = K / 8;
  float m = 0.0f, f[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) load8(x + row + min((int)(threadIdx.x + c * blockDim.x), n - 1) * 8, f[c]);
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[c][i]));
  const RowScale rs = row_scale(m, red);
  if (threadIdx.x == 0) scale[blockIdx.x] = rs.stored;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int ch = threadIdx.x + c * blockDim.x;
    uint32_t w[2];
    quantize_codes<8>(f[c], rs, w);
    if (ch < n) *reinterpret_cast<uint2*>(q + row + ch * 8) = make_uint2(w[0], w[1]);
  }
}

// ------------------------------------------------------------------- product

struct Int8Args {
  const int8_t* a;
  const float* a_s;
  const int8_t* b;
  const float* b_s;
  const uint16_t* add;  // BF16 [M, n_out] or NULL
  uint16_t* d;          // BF16 [M, n_out]
  int M, N, K, n_out;
  int splits, k_split;  // K in `splits` parts of k_split bytes (a multiple of a stage)
  int32_t* part;        // their sums, int32 [splits][M][N], when splits > 1
};
enum { kInt8Bf16, kInt8Silu, kInt8Part };  // what a tile writes

// Workgroup tile BM x BN of WM x WN waves; MFMA 32x32x32 with the weights as
// its first operand, so a lane holds runs of four output columns of one token.
//
// K passes in stages of BK bytes through four LDS buffers, filled straight from
// memory (buffer loads to LDS pass no register) three stages ahead; the wait
// before a stage leaves the two younger stages in flight. Stages of 64 bytes
// where the tile fills the LDS; of 128 in the small tiles of few tokens, whose
// time is the number of stages (512 x 4096 x 7168: 39 -> 28 us). A row's
// 16-byte chunks are permuted by its number, which spreads the rows that
// eight lanes of a fragment read touch over all banks; the loads apply it to
// the address they read.
//
// SILU: the tile's weight rows alternate in runs of 32 between gate (row n)
// and up (row I + n), so that a wave holds both halves of an output.
template <int BM, int BN, int WM, int WN, int BK, int OUT>
__global__ __launch_bounds__(64 * WM * WN) void int8_tile_kernel(Int8Args g, int mt, int nt) {
  constexpr bool SILU = OUT == kInt8Silu;
  constexpr int TH = 64 * WM * WN;
  constexpr int SM = BM / WM / 32, SN = BN / WN / 32;  // 32 x 32 subtiles of a wave
  static_assert(!SILU || SN % 2 == 0, "gate and up halves in one wave");
  constexpr int CPR = BK / 16, KS = BK / 32;           // chunks of a row and MFMA steps of a stage
  constexpr int RPI = TH / CPR;                        // rows of one load instruction of the workgroup
  constexpr int PA = BM / RPI, PB = BN / RPI, PL = PA + PB;
  constexpr int BUF = (BM + BN) * CPR;                 // 16-byte chunks of a buffer: A rows, then B rows
  __shared__ int4v l0[BUF], l1[BUF], l2[BUF], l3[BUF];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WM, wn = wave / WM;
  const int2 tile = tile_of_block(blockIdx.x, mt, nt);
  const int m0 = tile.x * BM, n0 = tile.y * (SILU ? BN / 2 : BN), half = g.N / 2;
  // This thread's chunk of every load: row trow + RPI i of the tile (the last
  // row of the matrix again where there is none: its results are not stored),
  // K bytes tk of a stage. SILU: the rows of one load of a wave lie in one half,
  // by the wave (RPI a multiple of 64) or by the load (RPI 32).
  const auto swizzle = [](int row, int chunk) { return CPR == 8 ? chunk ^ (row & 7) : chunk ^ ((row >> 1) & 3); };
  const int trow = threadIdx.x / CPR, tk = swizzle(trow, threadIdx.x % CPR) * 16;
  static_assert(!SILU || RPI == 32 || RPI % 64 == 0, "the rows of a load of a wave lie in one half");
  const int a_rows = min(BM, g.M - m0), b_rows = min(SILU ? BN / 2 : BN, (SILU ? half : g.N) - n0);
  const bool up_wave = SILU && RPI != 32 && (wave * (64 / CPR) / 32) % 2 == 1;
  const __amdgpu_buffer_rsrc_t ra = buffer_rsrc(g.a + (size_t)m0 * g.K, (uint32_t)(a_rows * g.K));
  const __amdgpu_buffer_rsrc_t rb = buffer_rsrc(g.b + (size_t)(n0 + (up_wave ? half : 0)) * g.K, (uint32_t)(b_rows * g.K));
  const __amdgpu_buffer_rsrc_t ru = buffer_rsrc(g.b + (size_t)(n0 + half) * g.K, (uint32_t)(b_rows * g.K));
  int va[PA], vb[PB];
#pragma unroll
  for (int i = 0; i < PA; ++i) va[i] = min(trow + i * RPI, a_rows - 1) * g.K + tk;
#pragma unroll
  for (int i = 0; i < PB; ++i) {
    const int at = trow + i * RPI;  // in the tile
    const int row = SILU ? (at >> 6) * 32 + (at & 31) : at;
    vb[i] = min(row, b_rows - 1) * g.K + tk;
  }
  const int k_begin = (int)blockIdx.y * g.k_split, k_end = min(g.K, k_begin + g.k_split);
  auto fetch = [&](int k0, int4v* to) {
    const bool in = k0 + tk < k_end;     // zeros past the end of a row (or of this part of K)
    const int ks = k0 < k_end ? k0 : 0;  // the scalar offset stays inside the range
#pragma unroll
    for (int i = 0; i < PA; ++i)
      load_lds16(ra, to + wave * 64 + i * TH, in ? va[i] : kOutOfRange, ks);
#pragma unroll
    for (int i = 0; i < PB; ++i)
      load_lds16(SILU && RPI == 32 && i % 2 == 1 ? ru : rb, to + BM * CPR + wave * 64 + i * TH,
                 in ? vb[i] : kOutOfRange, ks);
  };
  int16v acc[SN][SM];
#pragma unroll
  for (int i = 0; i < SN; ++i)
#pragma unroll
    for (int j = 0; j < SM; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;
  const int r = lane & 31, hi = lane >> 5;
  int fa_at[KS], fb_at[KS];
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    const int c = swizzle(r, ks * 2 + hi);
    fa_at[ks] = (wm * 32 * SM + r) * CPR + c;
    fb_at[ks] = (BM + wn * 32 * SN + r) * CPR + c;
  }
  auto compute = [&](const int4v* at) {
    int4v fa[2][SM], fb[2][SN];
    auto read = [&](int ks) {
#pragma unroll
      for (int j = 0; j < SM; ++j) fa[ks & 1][j] = at[fa_at[ks] + j * 32 * CPR];
#pragma unroll
      for (int i = 0; i < SN; ++i) fb[ks & 1][i] = at[fb_at[ks] + i * 32 * CPR];
    };
    read(0);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      if (ks + 1 < KS) read(ks + 1);
#pragma unroll
      for (int i = 0; i < SN; ++i)
#pragma unroll
        for (int j = 0; j < SM; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[ks & 1][i], fa[ks & 1][j], acc[i][j], 0, 0, 0);
    }
  };
  const int stages = (k_end - k_begin + BK - 1) / BK;
  fetch(k_begin, l0);
  fetch(k_begin + BK, l1);
  fetch(k_begin + 2 * BK, l2);
  // Stage s: its own loads have arrived; every wave is past stage s - 1, whose
  // buffer takes the loads of stage s + 3 (zeros past the end of K). No branch
  // inside the loop: around the stages it leaves the compiler unsure which
  // buffer a load fills, and it waits for all of them before it reads any.
  auto stage = [&](int s, const int4v* cur, int4v* next) {
    wait_stage<2 * PL>();
    fetch(k_begin + (s + 3) * BK, next);
    compute(cur);
  };
  int s = 0;
  for (; s + 4 <= stages; s += 4) {
    stage(s, l0, l3);
    stage(s + 1, l1, l0);
    stage(s + 2, l2, l1);
    stage(s + 3, l3, l2);
  }
  if (s < stages) {
    stage(s, l0, l3);
    if (s + 1 < stages) {
      stage(s + 1, l1, l0);
      if (s + 2 < stages) stage(s + 2, l2, l1);
    }
  }
  wait_stage<0>();

  // Epilogue, each wave by itself: 32 tokens x 32 SN columns of sums through
  // LDS, so that a lane takes eight neighbouring columns of a token (four for
  // SILU) and its neighbours the rest of whole 64-byte lines. Stored
  // straight from the MFMA layout (8 bytes here and there in 32 rows), the
  // down product of 8192 tokens ran 30 us longer.
  constexpr int COLS = 32 * SN, PITCH = COLS + 4;
  constexpr int WPB = BUF * 16 / (32 * PITCH * 4);  // waves whose block fits one buffer
  static_assert(WPB * 4 >= WM * WN, "the LDS buffers hold every wave's block");
  int4v* const buf = wave / WPB == 0 ? l0 : wave / WPB == 1 ? l1 : wave / WPB == 2 ? l2 : l3;
  int* const sums = reinterpret_cast<int*>(buf) + (wave % WPB) * 32 * PITCH;
  constexpr int LPR = COLS / 8, RPS = 64 / LPR;  // lanes of a row, rows of a step
  const int col = lane % LPR;
  // output column and scales of this lane, the same for all its rows
  const int oc = SILU ? (col / 8) * 32 + (col % 8) * 4 : col * 8;  // within the wave's outputs
  const int n = n0 + wn * (SILU ? COLS / 2 : COLS) + oc;
  const bool n_ok = n < (OUT == kInt8Part ? g.N : g.n_out);
  float bs[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) bs[e] = 0.0f;
  if (n_ok && OUT != kInt8Part) {
    const float4 s0 = *reinterpret_cast<const float4*>(g.b_s + n);
    const float4 s1 = *reinterpret_cast<const float4*>(g.b_s + (SILU ? half + n : n + 4));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      bs[e] = (&s0.x)[e];
      bs[4 + e] = (&s1.x)[e];
    }
  }
  // where the lane's sums lie in a row: eight in a run, or four gate and the
  // four up sums 32 columns on
  const int c0 = SILU ? (col / 8) * 64 + (col % 8) * 4 : col * 8, c1 = SILU ? c0 + 32 : c0 + 4;
  // the rows' scales and the values to add are loaded one subtile ahead
  constexpr int STEPS = 32 / RPS, W = SILU ? 4 : 8;
  typedef typename OutVec<W>::type vec_t;
  float as[2][STEPS];
  vec_t add[2][STEPS];
  auto row_of = [&](int j, int st) { return m0 + wm * 32 * SM + j * 32 + st * RPS + lane / LPR; };
  auto load_rows = [&](int j) {
    if constexpr (OUT == kInt8Part) return;
#pragma unroll
    for (int st = 0; st < STEPS; ++st) as[j & 1][st] = g.a_s[min(row_of(j, st), g.M - 1)];
    if (g.add) {
#pragma unroll
      for (int st = 0; st < STEPS; ++st)
        add[j & 1][st] = *reinterpret_cast<const vec_t*>(g.add + (size_t)min(row_of(j, st), g.M - 1) * g.n_out +
                                                         (n_ok ? n : 0));
    } else {
#pragma unroll
      for (int st = 0; st < STEPS; ++st) add[j & 1][st] = vec_t(0u);
    }
  };
  load_rows(0);
#pragma unroll
  for (int j = 0; j < SM; ++j) {
#pragma unroll
    for (int i = 0; i < SN; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<int4v*>(sums + r * PITCH + i * 32 + 8 * q + 4 * hi) =
            int4v{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    wave_lds_fence();
    if (j + 1 < SM) load_rows(j + 1);
#pragma unroll
    for (int st = 0; st < STEPS; ++st) {
      const int row = st * RPS + lane / LPR, m = row_of(j, st);
      const int4v v0 = *reinterpret_cast<const int4v*>(sums + row * PITCH + c0);
      const int4v v1 = *reinterpret_cast<const int4v*>(sums + row * PITCH + c1);
      if constexpr (OUT == kInt8Part) {
        if (m < g.M && n_ok) {
          int32_t* to = g.part + ((size_t)blockIdx.y * g.M + m) * g.N + n;
          *reinterpret_cast<int4v*>(to) = v0;
          *reinterpret_cast<int4v*>(to + 4) = v1;
        }
        continue;
      }
      float o[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        o[e] = (float)v0[e] * (as[j & 1][st] * bs[e]);
        o[4 + e] = (float)v1[e] * (as[j & 1][st] * bs[4 + e]);
      }
      if constexpr (SILU) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = silu_mul(o[e], o[4 + e]);
      }
      if (m < g.M && n_ok)
        *reinterpret_cast<vec_t*>(g.d + (size_t)m * g.n_out + n) = add_and_round<W>(o, add[j & 1][st]);
    }
    wave_lds_fence();
  }
}

// Joins the parts of K: four outputs of row m from n on. Eight parts are in
// flight at once: they come from other XCDs' workgroups, through memory.
template <bool SILU>
__device__ __forceinline__ void join4(const Int8Args& g, int m, int n, float (&o)[4]) {
  const int half = g.N / 2;
  int4v s = int4v{0, 0, 0, 0}, u = int4v{0, 0, 0, 0};
  const int32_t* p = g.part + (size_t)m * g.N + n;
  const size_t step = (size_t)g.M * g.N;
  for (int i = 0; i < g.splits; i += 8) {
    int4v vs[8], vu[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int32_t* at = p + (size_t)min(i + j, g.splits - 1) * step;
      vs[j] = *reinterpret_cast<const int4v*>(at);
      if (SILU) vu[j] = *reinterpret_cast<const int4v*>(at + half);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < g.splits) {
        s += vs[j];
        if (SILU) u += vu[j];
      }
  }
  const float as = g.a_s[m];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    o[e] = (float)s[e] * (as * g.b_s[n + e]);
    if (SILU) o[e] = silu_mul(o[e], (float)u[e] * (as * g.b_s[half + n + e]));
  }
}

template <bool SILU>
__global__ __launch_bounds__(256) void int8_join_kernel(Int8Args g) {
  typedef OutVec<4>::type vec_t;
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (at >= (int64_t)g.M * g.n_out) return;
  const int m = (int)(at / g.n_out), n = (int)(at - (int64_t)m * g.n_out);
  vec_t add = vec_t(0u);
  if (g.add) add = *reinterpret_cast<const vec_t*>(g.add + at);
  float o[4];
  join4<SILU>(g, m, n, o);
  *reinterpret_cast<vec_t*>(g.d + at) = add_and_round<4>(o, add);
}

// The same for the dense expert's h, quantized in the same pass: workgroup m
// joins row m of up to kJoinRows outputs, four to a thread, rounds them to BF16
// and writes their codes and scale as int8_rows_kernel would from there.
// (64 x 2 x 2048 of 8 parts: 5.3 us; with four parts of eight values in flight
// and h by way of memory 7.0.)
constexpr int kJoinRows = 4096;
__global__ __launch_bounds__(1024) void int8_join_rows_kernel(Int8Args g, int8_t* __restrict__ q,
                                                              float* __restrict__ scale) {
  typedef OutVec<4>::type vec_t;
  __shared__ float red[16];
  const int m = blockIdx.x, n = threadIdx.x * 4;
  float f[4], top = 0.0f;
  join4<true>(g, m, min(n, g.n_out - 4), f);
  const vec_t h = add_and_round<4>(f, vec_t(0u));
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    f[2 * e] = __uint_as_float(h[e] << 16);
    f[2 * e + 1] = __uint_as_float(h[e] & 0xFFFF0000u);
    top = fmaxf(top, fmaxf(fabsf(f[2 * e]), fabsf(f[2 * e + 1])));
  }
  const RowScale rs = row_scale(top, red);
  if (threadIdx.x == 0) scale[m] = rs.stored;
  uint32_t w;
  quantize_codes<4>(f, rs, &w);
  if (n < g.n_out) *reinterpret_cast<uint32_t*>(q + (size_t)m * g.n_out + n) = w;
}

// Few tokens: the weights' bytes count, and every wave of the chip has to read
// some. A workgroup takes 16 weight rows (SILU: 8 gate and their 8 up rows) and
// 16 MT tokens; its eight waves split K; nothing is staged, a wave streams both
// operands' MFMA 16x16x64 fragments from memory (64 contiguous bytes of each of
// 16 rows per load) with the next group in flight, and the eight partial sums,
// exact integers, meet in LDS. Groups of two steps, one 128-byte line of each
// row: with four, 1 x 4096 x 7168 took 10.7 us, not 8.7 (3.4 TB/s; 1 x 16384 x
// 8192: 29.9, not 26.4: 5.1 TB/s), with one 10.4. What is left at small sizes
// is the launch (2 us) and the latency of a few dependent loads.
constexpr int kSkinnyWaves = 8;
template <int MT, bool SILU>
__global__ __launch_bounds__(64 * kSkinnyWaves, 2) void int8_skinny_kernel(Int8Args g) {
  constexpr int U = 2;                            // 64-byte steps of a group
  __shared__ int sums[kSkinnyWaves][MT][16][17];  // [wave][subtile][token][weight row], padded against conflicts
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, kq = (lane >> 4) * 16;
  const int m0 = blockIdx.y * 16 * MT, n0 = blockIdx.x * (SILU ? 8 : 16), half = g.N / 2;
  const int row = SILU ? (i < 8 ? n0 + i : half + n0 + i - 8) : min(n0 + i, g.N - 1);
  const int steps = (g.K + 63) / 64;
  const int per = ((steps + kSkinnyWaves - 1) / kSkinnyWaves + 1) & ~1;  // whole 128-byte lines per wave
  const int s0 = wave * per, s1 = min(s0 + per, steps);
  const int8_t* pb = g.b + (size_t)row * g.K;
  const int8_t* pa[MT];
  int4v acc[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    pa[j] = g.a + (size_t)min(m0 + 16 * j + i, g.M - 1) * g.K;
    acc[j] = int4v{0, 0, 0, 0};
  }
  int4v fa[2][U][MT], fb[2][U];
  auto load = [&](int s, int4v (&a)[U][MT], int4v (&b)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // past this wave's share or the row: some bytes of the row again, and
      // zeros for the weights (loads under a branch would leave one by one)
      const int k = (s + u) * 64 + kq, at = min(k, g.K - 16);
      const int4v w = *reinterpret_cast<const int4v*>(pb + at);
      b[u] = s + u < s1 && k < g.K ? w : int4v{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < MT; ++j) a[u][j] = *reinterpret_cast<const int4v*>(pa[j] + at);
    }
  };
  auto multiply = [&](const int4v (&a)[U][MT], const int4v (&b)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < MT; ++j) acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[u], a[u][j], acc[j], 0, 0, 0);
  };
  if (s0 < s1) load(s0, fa[0], fb[0]);
  for (int s = s0; s < s1; s += 2 * U) {
    if (s + U < s1) load(s + U, fa[1], fb[1]);
    multiply(fa[0], fb[0]);
    if (s + U >= s1) break;
    if (s + 2 * U < s1) load(s + 2 * U, fa[0], fb[0]);
    multiply(fa[1], fb[1]);
  }
  // lane: token i of a subtile, weight rows 4 (lane / 16) + 0..3
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int v = 0; v < 4; ++v) sums[wave][j][i][4 * (lane >> 4) + v] = acc[j][v];
  __syncthreads();
  constexpr int COLS = SILU ? 8 : 16;
  static_assert(MT * 16 * COLS <= 64 * kSkinnyWaves, "an output per thread");
  const int c = threadIdx.x % COLS, tok = threadIdx.x / COLS, m = m0 + tok, n = n0 + c;
  if (tok >= 16 * MT || m >= g.M || n >= g.n_out) return;
  int s = 0, u = 0;
#pragma unroll
  for (int w = 0; w < kSkinnyWaves; ++w) {
    s += sums[w][tok >> 4][tok & 15][c];
    if (SILU) u += sums[w][tok >> 4][tok & 15][c + 8];
  }
  const float as = g.a_s[m];
  float o = (float)s * (as * g.b_s[n]);
  if (SILU) o = silu_mul(o, (float)u * (as * g.b_s[half + n]));
  const size_t d = (size_t)m * g.n_out + n;
  o += g.add ? bf16_to_f32(g.add[d]) : 0.0f;  // 0 too, as the tiles do: it makes a -0 of the product 0
  g.d[d] = (uint16_t)f32_to_bf16(o);
}

}  // namespace nvfp4

using namespace nvfp4;

extern "C" int int8_quantize_rows(const void* x, int32_t x_dtype, int32_t M, int32_t K, int8_t* q, float* scale,
                                  void* stream) {
  if (M < 0 || M > kInt8MaxM || K <= 0 || K % 16 != 0 || K > kInt8MaxK) return NVFP4_ERR_SHAPE;
  if (x_dtype != NVFP4_DT_BF16 && x_dtype != NVFP4_DT_F32) return NVFP4_ERR_ARG;
  if (M == 0) return NVFP4_OK;
  if (!x || !q || !scale) return NVFP4_ERR_NULL;
  if (!nvfp4_aligned16(x) || !nvfp4_aligned16(q) || !nvfp4_aligned16(scale)) return NVFP4_ERR_ALIGN;
  const auto go = [&](auto xt, auto ch) -> int {
    using T = decltype(xt);
    constexpr int CH = decltype(ch)::value;
    const int threads = ((K / 8 + CH - 1) / CH + 63) / 64 * 64;
    hipLaunchKernelGGL((int8_rows_kernel<T, CH>), dim3(M), dim3(threads), 0, (hipStream_t)stream,
                       reinterpret_cast<const T*>(x), K, q, scale);
    NVFP4_CHECK_LAUNCH();
    return NVFP4_OK;
  };
  constexpr std::integral_constant<int, 2> two;
  constexpr std::integral_constant<int, 8> eight;  // rows of more than 1024 threads' two chunks
  if (x_dtype == NVFP4_DT_BF16) return K <= 16384 ? go(uint16_t(), two) : go(uint16_t(), eight);
  return K <= 16384 ? go(float(), two) : go(float(), eight);
}

static int int8_gemm_check(int64_t M, int64_t N, int64_t K, int32_t epilogue) {
  if (epilogue != NVFP4_EPI_BF16 && epilogue != NVFP4_EPI_SILU_MUL) return NVFP4_ERR_ARG;
  if (M < 0 || N <= 0 || K <= 0 || K % 16 != 0 || K > kInt8MaxK) return NVFP4_ERR_SHAPE;
  if (N % (epilogue == NVFP4_EPI_SILU_MUL ? 16 : 8) != 0) return NVFP4_ERR_SHAPE;
  if (M > kInt8MaxM || N > kInt8MaxN) return NVFP4_ERR_SHAPE;
  return NVFP4_OK;
}

template <int BM, int BN, int WM, int WN, int BK, int OUT>
static int launch_int8_tile(const Int8Args& g, hipStream_t stream) {
  const int mt = (g.M + BM - 1) / BM, nt = (g.N + BN - 1) / BN;
  if ((int64_t)mt * nt * (64 * WM * WN) >= (1ll << 32)) return NVFP4_ERR_SHAPE;  // threads of a grid
  hipLaunchKernelGGL((int8_tile_kernel<BM, BN, WM, WN, BK, OUT>), dim3((unsigned)mt * nt, g.splits),
                     dim3(64 * WM * WN), 0, stream, g, mt, nt);
  NVFP4_CHECK_LAUNCH();
  return NVFP4_OK;
}

template <int MT, bool SILU>
static int launch_int8_skinny(const Int8Args& g, hipStream_t stream) {
  const dim3 grid((g.N + 15) / 16, (g.M + 16 * MT - 1) / (16 * MT));
  hipLaunchKernelGGL((int8_skinny_kernel<MT, SILU>), grid, dim3(64 * kSkinnyWaves), 0, stream, g);
  NVFP4_CHECK_LAUNCH();
  return NVFP4_OK;
}

// Which kernel a product takes (us, weights from memory, the other side in
// brackets). The few-token kernel up to 16 tokens (16 x 4096 x 7168: 9.9 [tiles
// 14.9], 16 x 16384 x 8192: 36 [36]), and where its workgroups of 32 tokens by
// 16 rows do not outnumber the CUs (24 x 4096 x 7168: 11.9 [15.2]; 128 x 1024 x
// 1040: 3.5 [5.5]; with 448 of them, 32 x 7168 x 2048, it loses: 8.7 [7.2]),
// unless a long K meets too few of them (128 x 64 x 7168: 11.5 [9.3]).
constexpr int kSkinnyM = 16, kLongK = 4096;
static bool int8_few(int64_t M, int64_t N, int64_t K) {
  return M <= kSkinnyM || (((M + 31) / 32) * ((N + 15) / 16) <= 256 && (K < kLongK || N >= 4096));
}
// Parts of K for tiles: as many as bring 64 x 128 tiles to about one per CU,
// each of at least 512 bytes (33 x 4096 x 7168: 15.6 [undivided 27], 192: 21.5
// [29]), or one: with a short K the join costs more than it saves (32 x 7168 x
// 2048: 7.3 [divided 10.4]).
static int int8_parts(int64_t M, int64_t N, int64_t K) {
  const int64_t tiles = ((M + 63) / 64) * ((N + 127) / 128);
  const int64_t s = std::min<int64_t>(256 / tiles, K / 512);
  return s < 2 || K < kLongK ? 1 : (int)s;
}
static int int8_splits(int64_t M, int64_t N, int64_t K) { return int8_few(M, N, K) ? 1 : int8_parts(M, N, K); }
static Int8Args int8_args(const int8_t* a_q, const float* a_s, const int8_t* b_q, const float* b_s, int M, int N, int K,
                          int want, bool silu, const void* add, void* d, void* ws) {
  const int per = ((K + want - 1) / want + 127) / 128 * 128;
  return {a_q, a_s, b_q, b_s, reinterpret_cast<const uint16_t*>(add), reinterpret_cast<uint16_t*>(d), M, N, K,
          silu ? N / 2 : N, (K + per - 1) / per, per, reinterpret_cast<int32_t*>(ws)};
}
static size_t int8_part_bytes(int64_t M, int64_t N, int splits) { return splits > 1 ? (size_t)splits * M * N * 4 : 0; }

template <bool SILU>
static int launch_int8(const Int8Args& g, hipStream_t stream) {
  constexpr int OUT = SILU ? kInt8Silu : kInt8Bf16;
  if (g.splits > 1) {
    const int st = launch_int8_tile<64, 128, 2, 2, 128, kInt8Part>(g, stream);
    if (st) return st;
    hipLaunchKernelGGL(int8_join_kernel<SILU>, dim3((unsigned)(((int64_t)g.M * g.n_out / 4 + 255) / 256)), dim3(256), 0,
                       stream, g);
    NVFP4_CHECK_LAUNCH();
    return NVFP4_OK;
  }
  if (g.M <= kSkinnyM) return launch_int8_skinny<1, SILU>(g, stream);
  if (int8_few(g.M, g.N, g.K)) return launch_int8_skinny<2, SILU>(g, stream);
  // The tile whose rounds over the 256 CUs take least, by what one of each size
  // took at K = 7168 (us, in proportion to K): alone on its CU, or each of more.
  // (By the largest tile that still gives 192 CUs one, 2100 x 4096 x 7168 took
  // 100 us, not 83; 1536 x 7168 x 2048 34.8, not 31.7; 2900 x 3000 x 4096 58,
  // not 50.)
  const auto cost = [&](int bm, int bn, double alone, double each) {
    const int64_t tiles = (int64_t)((g.M + bm - 1) / bm) * ((g.N + bn - 1) / bn);
    return tiles <= 256 ? alone : each * (double)((tiles + 255) / 256);
  };
  constexpr int BN = SILU ? 128 : 64;
  const double large = cost(256, 256, 96.0, 96.0), middle = cost(128, 128, 49.0, 41.0);
  const double small = SILU ? cost(64, 128, 29.0, 26.0) : cost(64, 64, 24.0, 16.5);
  if (large <= middle && large <= small) return launch_int8_tile<256, 256, 2, 4, 64, OUT>(g, stream);
  if (middle <= small) return launch_int8_tile<128, 128, 2, 2, 64, OUT>(g, stream);
  return launch_int8_tile<64, BN, 2, 2, 128, OUT>(g, stream);
}

extern "C" size_t int8_gemm_ws_bytes(int32_t M, int32_t N, int32_t K) {
  if (int8_gemm_check(M, N, K, NVFP4_EPI_BF16)) return 0;
  return int8_part_bytes(M, N, int8_splits(M, N, K));
}

extern "C" int int8_gemm(const int8_t* a_q, const float* a_scale, const int8_t* b_q, const float* b_scale, int32_t M,
                         int32_t N, int32_t K, int32_t epilogue, const void* add_bf16, void* d_bf16, void* ws,
                         size_t ws_bytes, void* stream) {
  const int st = int8_gemm_check(M, N, K, epilogue);
  if (st) return st;
  if (M == 0) return NVFP4_OK;
  const int splits = int8_splits(M, N, K);
  const size_t need = int8_part_bytes(M, N, splits);
  if (!a_q || !a_scale || !b_q || !b_scale || !d_bf16 || (need && !ws)) return NVFP4_ERR_NULL;
  if (!nvfp4_aligned16(a_q) || !nvfp4_aligned16(a_scale) || !nvfp4_aligned16(b_q) || !nvfp4_aligned16(b_scale) ||
      !nvfp4_aligned16(add_bf16) || !nvfp4_aligned16(d_bf16) || !nvfp4_aligned16(ws))
    return NVFP4_ERR_ALIGN;
  if (ws_bytes < need) return NVFP4_ERR_WORKSPACE;
  const bool silu = epilogue == NVFP4_EPI_SILU_MUL;
  const Int8Args g = int8_args(a_q, a_scale, b_q, b_scale, M, N, K, splits, silu, add_bf16, d_bf16, ws);
  return silu ? launch_int8<true>(g, (hipStream_t)stream) : launch_int8<false>(g, (hipStream_t)stream);
}

// ------------------------------------------------------------- dense expert

// Parts of K of the up product. Past 16 tokens the join that a divided K needs
// quantizes h on the way, which is worth more than the few-token kernel.
static int int8_up_splits(int64_t T, int64_t hidden, int64_t inter) {
  return T <= kSkinnyM ? 1 : int8_parts(T, 2 * inter, hidden);
}
struct Int8FfnWs {
  size_t x_q, x_s, h, h_q, h_s, part, end;
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
  const size_t p1 = int8_part_bytes(T, 2 * inter, int8_up_splits(T, hidden, inter));
  const size_t p2 = int8_part_bytes(T, hidden, int8_splits(T, hidden, inter));
  w.part = put(p1 > p2 ? p1 : p2);
  w.end = p;
  return w;
}
static int int8_ffn_check(int32_t T, int32_t hidden, int32_t inter) {
  if (T < 0 || hidden <= 0 || inter <= 0 || hidden % 16 != 0 || inter % 16 != 0 || hidden > kInt8MaxK ||
      inter > kInt8MaxK || T > kInt8MaxM)
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
  const Int8Args up = int8_args(x_q, x_s, w1_q, w1_scale, T, 2 * inter, hidden, int8_up_splits(T, hidden, inter), true,
                                nullptr, base + l.h, base + l.part);
  if (up.splits > 1 && inter <= kJoinRows) {  // the join quantizes h as well
    st = launch_int8_tile<64, 128, 2, 2, 128, kInt8Part>(up, (hipStream_t)stream);
    if (st) return st;
    hipLaunchKernelGGL(int8_join_rows_kernel, dim3(T), dim3((inter / 4 + 63) / 64 * 64), 0, (hipStream_t)stream, up, h_q,
                       h_s);
    NVFP4_CHECK_LAUNCH();
  } else {
    st = launch_int8<true>(up, (hipStream_t)stream);
    if (st) return st;
    st = int8_quantize_rows(base + l.h, NVFP4_DT_BF16, T, inter, h_q, h_s, stream);
    if (st) return st;
  }
  const Int8Args down = int8_args(h_q, h_s, w2_q, w2_scale, T, hidden, inter, int8_splits(T, hidden, inter), false,
                                  add_bf16, out_bf16, base + l.part);
  return launch_int8<false>(down, (hipStream_t)stream);
}
