// Products of two MXFP4 matrices (mxfp4.h), C = A B^T of the values they stand
// for, with the dense expert's epilogues.
//
// gfx950's matrix unit takes this format as it is: one MFMA 32x32x64 (or
// 16x16x128) multiplies E2M1 operands of which each lane holds one block of 32
// and that block's scale, and adds in float32. A lane's 16 bytes are a block, so
// the scales cost one word per row and 128 elements and nothing is decoded. A
// byte does what it does in the 8-bit integer product, on twice the elements.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "common.h"
#include "internal.h"
#include "mxfp4.h"
#include "tile.h"
#include "wave.h"

namespace nvfp4 {

typedef int int8v __attribute__((ext_vector_type(8)));

constexpr int kMxGemmMaxM = 64 * 65535;
constexpr int kMxGemmMaxN = (1 << 27) - 16;  // by 512 threads for 16 columns: fewer than 2^32

struct MxGemmArgs {
  const uint8_t *a, *a_s;  // [M, K / 2], [K / 128, M, 4]
  const uint8_t *b, *b_s;  // [N, K / 2], [K / 128, N, 4]
  const void* add;         // of d's type and shape, or NULL
  void* d;                 // BF16 or float32 [M, n_out]
  int M, N, KB, n_out;     // KB: bytes of a row of codes
  int splits, k_split;     // K in `splits` parts of k_split bytes (a multiple of a stage)
  float* part;             // their sums, float32 [splits][M][N], when splits > 1
};
enum { kMxBf16, kMxSilu, kMxF32, kMxPart };  // what a tile writes

__device__ __forceinline__ int8v mx_operand(int4v v) { return int8v{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }
// D += A B^T on 32 x 64 codes each, with byte BYTE of a lane's word as its scale.
template <int BYTE>
__device__ __forceinline__ float16_t mx_mfma32(int4v a, int a_s, int4v b, int b_s, float16_t c) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_operand(a), mx_operand(b), c, 4, 4, BYTE, a_s, BYTE, b_s);
}

// silu(g) u = g u / (1 + e^-g), by e^-|g| as 2^(n + f), n the whole number next to
// -|g| log2 e and f the rest, from two parts of log2 e; by the hardware's power of
// two and reciprocal, one float32 step each, that is 8.4 half steps of float32 at
// any g. (From -|g| log2 e as it rounds it would be 64. The power of two ends at
// 2^-126: by itself it made 0 of every g below -87.3, whatever u; so e^-|g| has
// its digits down to 2^-149, as in silu_mul.) With the exact exponential and the
// division of silu_mul 8192 x 4096 x 1024 takes 43.4 us, so 38.3 [from -|g| log2 e
// as it rounds 36.6]; 8192 x 4096 x 7168 139.9, so 133.6 [131.6].
__device__ __forceinline__ float mx_silu_mul(float g, float u) {
  constexpr float kLog2e = 1.44269504f, kRest = 1.925963e-8f;
  const float a = fabsf(__builtin_amdgcn_fmed3f(g, -256.0f, 256.0f));  // e^-256 is 0
  const float n = rintf(-kLog2e * a);
  const float f = __builtin_fmaf(-kRest, a, __builtin_fmaf(-kLog2e, a, -n));
  const float e = __builtin_ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
  return (g < 0.0f ? g * e : g) * __builtin_amdgcn_rcpf(1.0f + e) * u;
}

// One word per lane from memory to LDS, side by side from `to` on.
__device__ __forceinline__ void load_lds4(__amdgpu_buffer_rsrc_t r, int* to, int voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)to, 4, voff, soff, 0, 0);
}

// 16 bytes of outputs of a row (8 for SILU), rounded to the output's type with
// what is to be added. PAST: stored past the caches.
template <int OUT>
struct MxOut {
  static constexpr int W = OUT == kMxSilu ? 4 : 8;
  typedef typename OutVec<W>::type vec;
  static __device__ __forceinline__ vec load(const void* add, size_t at) {
    return *reinterpret_cast<const vec*>(reinterpret_cast<const uint16_t*>(add) + at);
  }
  template <bool PAST>
  static __device__ __forceinline__ void store(void* d, size_t at, const float* o, vec add) {
    vec* to = reinterpret_cast<vec*>(reinterpret_cast<uint16_t*>(d) + at);
    const vec v = add_and_round<W>(o, add);
    if constexpr (PAST)
      __builtin_nontemporal_store(v, to);
    else
      *to = v;
  }
};
template <>
struct MxOut<kMxF32> {
  static constexpr int W = 4;
  typedef float4_t vec;
  static __device__ __forceinline__ vec load(const void* add, size_t at) {
    return *reinterpret_cast<const vec*>(reinterpret_cast<const float*>(add) + at);
  }
  template <bool PAST>
  static __device__ __forceinline__ void store(void* d, size_t at, const float* o, vec add) {
    vec* to = reinterpret_cast<vec*>(reinterpret_cast<float*>(d) + at);
    const vec v = {o[0] + add[0], o[1] + add[1], o[2] + add[2], o[3] + add[3]};
    if constexpr (PAST)
      __builtin_nontemporal_store(v, to);
    else
      *to = v;
  }
};

// Workgroup tile BM x BN of WM x WN waves, the weights as the MFMA's first
// operand, so a lane holds runs of four output columns of one token. K passes in
// stages of BK bytes through four LDS buffers, filled straight from memory three
// stages ahead; the wait before a stage leaves the two younger stages in flight.
// A row's 16-byte chunks are permuted by its number, which spreads the rows that
// sixteen lanes of a fragment read touch over all 64 banks (permuted for eight
// lanes and 32 banks, 43 % of the LDS cycles were conflicts). Behind a buffer's
// codes lie the stage's scales, one word per row and 64 bytes of codes.
//
// What bounds the large tile is power: on random codes the clock falls to 1.7 GHz
// (8192 x 4096 x 7168: 118 us, 4.1 PFLOP/s; zeros, at the same number of cycles,
// 90 us), where the matrix unit by itself does 6.0. Four waves of 128 x 128, with
// a third less to read from LDS, took 125; reads kept strictly ahead of a step's
// products 129.
//
// SILU: the tile's weight rows alternate in runs of 32 between gate (row n)
// and up (row I + n), so that a wave holds both halves of an output.
template <int BM, int BN, int WM, int WN, int BK, int OUT, bool PAST>
__global__ __launch_bounds__(64 * WM * WN) void mx_tile_kernel(MxGemmArgs g, int mt, int nt) {
  constexpr bool SILU = OUT == kMxSilu;
  constexpr int NW = WM * WN, TH = 64 * NW;
  constexpr int SM = BM / WM / 32, SN = BN / WN / 32;  // 32 x 32 subtiles of a wave
  static_assert(!SILU || SN % 2 == 0, "gate and up halves in one wave");
  constexpr int CPR = BK / 16, KS = BK / 32;           // chunks of a row and MFMA steps of a stage
  constexpr int RPI = TH / CPR;                        // rows of one load instruction of the workgroup
  constexpr int PA = BM / RPI, PB = BN / RPI;
  constexpr int BUF = (BM + BN) * CPR;                 // 16-byte chunks of a buffer: A rows, then B rows
  constexpr int DW = BK / 64;                          // scale words of a row of a stage
  constexpr int SL = (BM + BN) / 64 * DW;              // their loads, 64 rows each
  constexpr int PS = (SL + NW - 1) / NW;               // of each wave
  constexpr int PL = PA + PB + PS;
  __shared__ int4v l0[BUF + SL * 16], l1[BUF + SL * 16], l2[BUF + SL * 16], l3[BUF + SL * 16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WM, wn = wave / WM;
  const int2 tile = tile_of_block(blockIdx.x, mt, nt);
  const int m0 = tile.x * BM, n0 = tile.y * (SILU ? BN / 2 : BN), half = g.N / 2;
  // This thread's chunk of every load: row trow + RPI i of the tile (the last
  // row of the matrix again where there is none: its results are not stored),
  // K bytes tk of a stage. SILU: the rows of one load of a wave lie in one half,
  // by the wave (RPI a multiple of 64) or by the load (RPI 32).
  const auto swizzle = [](int row, int chunk) { return CPR == 8 ? chunk ^ ((row >> 1) & 7) : chunk ^ ((row >> 2) & 3); };
  const int trow = threadIdx.x / CPR, tk = swizzle(trow, threadIdx.x % CPR) * 16;
  static_assert(!SILU || RPI == 32 || RPI % 64 == 0, "the rows of a load of a wave lie in one half");
  const int a_rows = min(BM, g.M - m0), b_rows = min(SILU ? BN / 2 : BN, (SILU ? half : g.N) - n0);
  const bool up_wave = SILU && RPI != 32 && (wave * (64 / CPR) / 32) % 2 == 1;
  const __amdgpu_buffer_rsrc_t ra = buffer_rsrc(g.a + (size_t)m0 * g.KB, (uint32_t)(a_rows * g.KB));
  const __amdgpu_buffer_rsrc_t rb = buffer_rsrc(g.b + (size_t)(n0 + (up_wave ? half : 0)) * g.KB, (uint32_t)(b_rows * g.KB));
  const __amdgpu_buffer_rsrc_t ru = buffer_rsrc(g.b + (size_t)(n0 + half) * g.KB, (uint32_t)(b_rows * g.KB));
  int va[PA], vb[PB];
#pragma unroll
  for (int i = 0; i < PA; ++i) va[i] = min(trow + i * RPI, a_rows - 1) * g.KB + tk;
#pragma unroll
  for (int i = 0; i < PB; ++i) {
    const int at = trow + i * RPI;  // in the tile
    const int row = SILU ? (at >> 6) * 32 + (at & 31) : at;
    vb[i] = min(row, b_rows - 1) * g.KB + tk;
  }
  // The scale loads of this wave: word dw of 64 rows of one operand (waves
  // without one of their own repeat the last, so that all waves count alike).
  const int behind = max(g.KB / 64 - 1, 0);  // groups of 128 after the first
  const __amdgpu_buffer_rsrc_t sa = buffer_rsrc(g.a_s + (size_t)m0 * 4, (uint32_t)(((size_t)behind * g.M + a_rows) * 4));
  const __amdgpu_buffer_rsrc_t sb =
      buffer_rsrc(g.b_s + (size_t)n0 * 4, (uint32_t)(((size_t)behind * g.N + (SILU ? half : 0) + b_rows) * 4));
  int vs[PS], load_at[PS], load_dw[PS];
  bool of_a[PS];
#pragma unroll
  for (int i = 0; i < PS; ++i) {
    const int j = min(wave + i * NW, SL - 1), row = j % (SL / DW) * 64 + lane;
    load_at[i] = j * 64;
    load_dw[i] = j / (SL / DW);
    of_a[i] = j % (SL / DW) * 64 < BM;
    const int at = row - BM, n = SILU ? (at >> 6) * 32 + (at & 31) : at;
    vs[i] = (of_a[i] ? min(row, a_rows - 1) : min(n, b_rows - 1) + (SILU && (at & 32) ? half : 0)) * 4;
  }
  const int k_begin = (int)blockIdx.y * g.k_split, k_end = min(g.KB, k_begin + g.k_split);
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
#pragma unroll
    for (int i = 0; i < PS; ++i) {
      const int c = k0 / 64 + load_dw[i];
      const bool there = c * 64 < k_end;
      load_lds4(of_a[i] ? sa : sb, reinterpret_cast<int*>(to + BUF) + load_at[i], there ? vs[i] : kOutOfRange,
                there ? c * (of_a[i] ? g.M : g.N) * 4 : 0);
    }
  };
  float16_t acc[SN][SM];
#pragma unroll
  for (int i = 0; i < SN; ++i)
#pragma unroll
    for (int j = 0; j < SM; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
  const int r = lane & 31, hi = lane >> 5;
  int fa_at[KS], fb_at[KS];
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    const int c = swizzle(r, ks * 2 + hi);
    fa_at[ks] = (wm * 32 * SM + r) * CPR + c;
    fb_at[ks] = (BM + wn * 32 * SN + r) * CPR + c;
  }
  const int sa_at = wm * 32 * SM + r, sb_at = BM + wn * 32 * SN + r;
  int4v fa[2][SM], fb[2][SN];
  int wa[DW][SM], wb[DW][SN];  // scales of this lane's blocks: step ks in byte 2 (ks % 2) of word ks / 2
  auto read = [&](const int4v* at, int ks) {
#pragma unroll
    for (int j = 0; j < SM; ++j) fa[ks & 1][j] = at[fa_at[ks] + j * 32 * CPR];
#pragma unroll
    for (int i = 0; i < SN; ++i) fb[ks & 1][i] = at[fb_at[ks] + i * 32 * CPR];
  };
  int na[DW][SM], nb[DW][SN];  // the next stage's, as read
  auto read_scales = [&](const int4v* at) {
    const int* s = reinterpret_cast<const int*>(at + BUF);
#pragma unroll
    for (int d = 0; d < DW; ++d) {
#pragma unroll
      for (int j = 0; j < SM; ++j) na[d][j] = s[d * (BM + BN) + sa_at + j * 32];
#pragma unroll
      for (int i = 0; i < SN; ++i) nb[d][i] = s[d * (BM + BN) + sb_at + i * 32];
    }
  };
  auto take_scales = [&]() {
#pragma unroll
    for (int d = 0; d < DW; ++d) {
#pragma unroll
      for (int j = 0; j < SM; ++j) wa[d][j] = (int)((uint32_t)na[d][j] >> (8 * hi));
#pragma unroll
      for (int i = 0; i < SN; ++i) wb[d][i] = (int)((uint32_t)nb[d][i] >> (8 * hi));
    }
  };
  auto multiply = [&](int ks) {
#pragma unroll
    for (int i = 0; i < SN; ++i)
#pragma unroll
      for (int j = 0; j < SM; ++j)
        acc[i][j] = ks & 1 ? mx_mfma32<2>(fb[1][i], wb[ks / 2][i], fa[1][j], wa[ks / 2][j], acc[i][j])
                           : mx_mfma32<0>(fb[0][i], wb[ks / 2][i], fa[0][j], wa[ks / 2][j], acc[i][j]);
  };
  const int stages = (k_end - k_begin + BK - 1) / BK;
  fetch(k_begin, l0);
  fetch(k_begin + BK, l1);
  fetch(k_begin + 2 * BK, l2);
  wait_stage<2 * PL>();
  read_scales(l0);
  read(l0, 0);
  // Stage s, whose first fragments are on their way: each step reads the next
  // one's, the last those of stage s + 1, whose loads have then arrived for every
  // wave. All waves are past stage s - 1 there, so its buffer takes the loads of
  // stage s + 3 (zeros past the end of K). No branch inside the loop: around the
  // stages it leaves the compiler unsure which buffer a load fills, and it waits
  // for all of them before it reads any.
  auto stage = [&](int s, const int4v* cur, const int4v* after, int4v* fill) {
    take_scales();
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      if (ks + 1 < KS) {
        read(cur, ks + 1);
      } else {
        wait_stage<PL>();
        fetch(k_begin + (s + 3) * BK, fill);
        read_scales(after);
        read(after, 0);
      }
      multiply(ks);
    }
  };
  int s = 0;
  for (; s + 4 <= stages; s += 4) {
    stage(s, l0, l1, l3);
    stage(s + 1, l1, l2, l0);
    stage(s + 2, l2, l3, l1);
    stage(s + 3, l3, l0, l2);
  }
  if (s < stages) {
    stage(s, l0, l1, l3);
    if (s + 1 < stages) {
      stage(s + 1, l1, l2, l0);
      if (s + 2 < stages) stage(s + 2, l2, l3, l1);
    }
  }
  wait_stage<0>();

  // Epilogue, each wave by itself: 32 tokens x 32 SN columns of sums through
  // LDS, so that a lane takes 16 bytes of outputs of a token (8 for SILU) and its
  // neighbours the rest of whole 64-byte lines (with eight float32 outputs to a
  // lane, in two stores of every other 16 bytes, 4096 x 7168 x 4096 took 76 us, so
  // 74, and past the caches 104).
  typedef MxOut<OUT == kMxPart ? kMxF32 : OUT> Out;
  constexpr int COLS = 32 * SN, PITCH = COLS + 4, PER = SILU ? 8 : Out::W;  // PER: sums of a lane and row
  constexpr int WPB = BUF * 16 / (32 * PITCH * 4);                          // waves whose block fits one buffer
  static_assert(WPB * 4 >= NW, "the LDS buffers hold every wave's block");
  int4v* const buf = wave / WPB == 0 ? l0 : wave / WPB == 1 ? l1 : wave / WPB == 2 ? l2 : l3;
  float* const sums = reinterpret_cast<float*>(buf) + (wave % WPB) * 32 * PITCH;
  constexpr int LPR = COLS / PER, RPS = 64 / LPR;  // lanes of a row, rows of a step
  const int col = lane % LPR;
  // output column of this lane, the same for all its rows
  const int oc = SILU ? (col / 8) * 32 + (col % 8) * 4 : col * PER;  // within the wave's outputs
  const int n = n0 + wn * (SILU ? COLS / 2 : COLS) + oc;
  const bool n_ok = n < (OUT == kMxPart ? g.N : g.n_out);
  // where the lane's sums lie in a row: in a run, or four gate and the four up
  // sums 32 columns on
  const int c0 = SILU ? (col / 8) * 64 + (col % 8) * 4 : col * PER, c1 = SILU ? c0 + 32 : c0 + 4;
  // the values to add are loaded one subtile ahead
  constexpr int STEPS = 32 / RPS;
  typename Out::vec add[2][STEPS];
  auto row_of = [&](int j, int st) { return m0 + wm * 32 * SM + j * 32 + st * RPS + lane / LPR; };
  auto load_rows = [&](int j) {
#pragma unroll
    for (int st = 0; st < STEPS; ++st) add[j & 1][st] = typename Out::vec(0);
    if (OUT == kMxPart || !g.add) return;
#pragma unroll
    for (int st = 0; st < STEPS; ++st)
      add[j & 1][st] = Out::load(g.add, (size_t)min(row_of(j, st), g.M - 1) * g.n_out + (n_ok ? n : 0));
  };
  load_rows(0);
#pragma unroll
  for (int j = 0; j < SM; ++j) {
#pragma unroll
    for (int i = 0; i < SN; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<float4_t*>(sums + r * PITCH + i * 32 + 8 * q + 4 * hi) =
            float4_t{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    wave_lds_fence();
    if (j + 1 < SM) load_rows(j + 1);
#pragma unroll
    for (int st = 0; st < STEPS; ++st) {
      const int row = st * RPS + lane / LPR, m = row_of(j, st);
      float o[8];
      const float4_t v0 = *reinterpret_cast<const float4_t*>(sums + row * PITCH + c0);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = v0[e];
      if constexpr (PER == 8) {
        const float4_t v1 = *reinterpret_cast<const float4_t*>(sums + row * PITCH + c1);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[4 + e] = v1[e];
      }
      if constexpr (SILU) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = mx_silu_mul(o[e], o[4 + e]);
      }
      if (m >= g.M || !n_ok) continue;
      if constexpr (OUT == kMxPart)
        Out::template store<false>(g.part, ((size_t)blockIdx.y * g.M + m) * g.N + n, o, typename Out::vec(0));
      else
        Out::template store<PAST>(g.d, (size_t)m * g.n_out + n, o, add[j & 1][st]);
    }
    wave_lds_fence();
  }
}

// Joins the parts of K in their order, four outputs to a thread. Eight parts are
// in flight at once: they come from other XCDs' workgroups, through memory.
template <int OUT>
__global__ __launch_bounds__(256) void mx_join_kernel(MxGemmArgs g) {
  constexpr bool SILU = OUT == kMxSilu;
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (at >= (int64_t)g.M * g.n_out) return;
  const int m = (int)(at / g.n_out), n = (int)(at - (int64_t)m * g.n_out), half = g.N / 2;
  float4_t s = float4_t{0, 0, 0, 0}, u = float4_t{0, 0, 0, 0};
  const float* p = g.part + (size_t)m * g.N + n;
  const size_t step = (size_t)g.M * g.N;
  for (int i = 0; i < g.splits; i += 8) {
    float4_t vs[8], vu[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float* from = p + (size_t)min(i + j, g.splits - 1) * step;
      vs[j] = *reinterpret_cast<const float4_t*>(from);
      if (SILU) vu[j] = *reinterpret_cast<const float4_t*>(from + half);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < g.splits) {
        s += vs[j];
        if (SILU) u += vu[j];
      }
  }
  if constexpr (SILU) {
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = mx_silu_mul(s[e], u[e]);
  }
  if constexpr (OUT == kMxF32) {
    if (g.add) s += *reinterpret_cast<const float4_t*>(reinterpret_cast<const float*>(g.add) + at);
    *reinterpret_cast<float4_t*>(reinterpret_cast<float*>(g.d) + at) = s;
  } else {
    typedef OutVec<4>::type vec_t;
    vec_t add = vec_t(0u);
    if (g.add) add = *reinterpret_cast<const vec_t*>(reinterpret_cast<const uint16_t*>(g.add) + at);
    const float o[4] = {s[0], s[1], s[2], s[3]};
    *reinterpret_cast<vec_t*>(reinterpret_cast<uint16_t*>(g.d) + at) = add_and_round<4>(o, add);
  }
}

// Few tokens: the weights' bytes count, and every wave of the chip has to read
// some. A workgroup takes 16 weight rows (SILU: 8 gate and their 8 up rows) and
// 16 MT tokens; its eight waves split K; nothing is staged, a wave streams both
// operands' MFMA 16x16x128 fragments from memory (64 contiguous bytes of each of
// 16 rows per load) with the next group in flight, and the eight partial sums
// meet in LDS in the waves' order.
constexpr int kMxSkinnyWaves = 8;
template <int MT, int OUT>
__global__ __launch_bounds__(64 * kMxSkinnyWaves, 2) void mx_skinny_kernel(MxGemmArgs g) {
  constexpr bool SILU = OUT == kMxSilu;
  constexpr int U = 2;                                // 64-byte steps of a group (1 and 4: the same times)
  __shared__ float sums[kMxSkinnyWaves][MT][16][17];  // [wave][subtile][token][weight row], padded against conflicts
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, kq = lane >> 4;
  const int m0 = blockIdx.y * 16 * MT, n0 = blockIdx.x * (SILU ? 8 : 16), half = g.N / 2;
  const int row = SILU ? (i < 8 ? n0 + i : half + n0 + i - 8) : min(n0 + i, g.N - 1);
  const int steps = g.KB / 64;
  const int per = ((steps + kMxSkinnyWaves - 1) / kMxSkinnyWaves + 1) & ~1;  // whole 128-byte lines per wave
  const int s0 = wave * per, s1 = min(s0 + per, steps);
  const uint8_t* pb = g.b + (size_t)row * g.KB + kq * 16;
  const uint8_t* sb = g.b_s + (size_t)row * 4;
  const uint8_t *pa[MT], *sa[MT];
  float4_t acc[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int m = min(m0 + 16 * j + i, g.M - 1);
    pa[j] = g.a + (size_t)m * g.KB + kq * 16;
    sa[j] = g.a_s + (size_t)m * 4;
    acc[j] = float4_t{0, 0, 0, 0};
  }
  struct Group {
    int4v a[U][MT], b[U];
    uint32_t as[U][MT], bs[U];
  } f[2];
  auto load = [&](int s, Group& to) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // past this wave's share: its last step again, and zeros for the weights
      // (loads under a branch would leave one by one)
      const int at = min(s + u, s1 - 1);
      const int4v w = *reinterpret_cast<const int4v*>(pb + (size_t)at * 64);
      to.bs[u] = *reinterpret_cast<const uint32_t*>(sb + (size_t)at * g.N * 4);
      to.b[u] = s + u < s1 ? w : int4v{0, 0, 0, 0};
      if (s + u >= s1) to.bs[u] = 0;  // (a NaN there would not be undone by zeros)
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        to.a[u][j] = *reinterpret_cast<const int4v*>(pa[j] + (size_t)at * 64);
        to.as[u][j] = *reinterpret_cast<const uint32_t*>(sa[j] + (size_t)at * g.M * 4);
      }
    }
  };
  auto multiply = [&](const Group& from) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < MT; ++j)
        acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(from.b[u]), mx_operand(from.a[u][j]), acc[j], 4,
                                                                   4, 0, (int)(from.bs[u] >> (8 * kq)), 0,
                                                                   (int)(from.as[u][j] >> (8 * kq)));
  };
  if (s0 < s1) load(s0, f[0]);
  for (int s = s0; s < s1; s += 2 * U) {
    if (s + U < s1) load(s + U, f[1]);
    multiply(f[0]);
    if (s + U >= s1) break;
    if (s + 2 * U < s1) load(s + 2 * U, f[0]);
    multiply(f[1]);
  }
  // lane: token i of a subtile, weight rows 4 kq + 0..3
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int v = 0; v < 4; ++v) sums[wave][j][i][4 * kq + v] = acc[j][v];
  __syncthreads();
  constexpr int COLS = SILU ? 8 : 16;
  static_assert(MT * 16 * COLS <= 64 * kMxSkinnyWaves, "an output per thread");
  const int c = threadIdx.x % COLS, tok = threadIdx.x / COLS, m = m0 + tok, n = n0 + c;
  if (tok >= 16 * MT || m >= g.M || n >= g.n_out) return;
  float o = 0.0f, up = 0.0f;
#pragma unroll
  for (int w = 0; w < kMxSkinnyWaves; ++w) {
    o += sums[w][tok >> 4][tok & 15][c];
    if (SILU) up += sums[w][tok >> 4][tok & 15][c + 8];
  }
  if (SILU) o = mx_silu_mul(o, up);
  const size_t d = (size_t)m * g.n_out + n;
  if constexpr (OUT == kMxF32) {
    reinterpret_cast<float*>(g.d)[d] = o + (g.add ? reinterpret_cast<const float*>(g.add)[d] : 0.0f);
  } else {
    o += g.add ? bf16_to_f32(reinterpret_cast<const uint16_t*>(g.add)[d]) : 0.0f;
    reinterpret_cast<uint16_t*>(g.d)[d] = (uint16_t)f32_to_bf16(o);
  }
}

}  // namespace nvfp4

using namespace nvfp4;

static int mx_gemm_check(int64_t M, int64_t N, int64_t K, int32_t epilogue, int32_t d_dtype) {
  if ((epilogue != NVFP4_EPI_BF16 && epilogue != NVFP4_EPI_SILU_MUL) ||
      (d_dtype != NVFP4_DT_BF16 && d_dtype != NVFP4_DT_F32) ||
      (epilogue == NVFP4_EPI_SILU_MUL && d_dtype != NVFP4_DT_BF16))
    return NVFP4_ERR_ARG;
  if (M < 0 || N <= 0 || K < 0 || K % kMxGroup != 0 || K > kMxMaxK) return NVFP4_ERR_SHAPE;
  if (N % (epilogue == NVFP4_EPI_SILU_MUL ? 16 : 8) != 0) return NVFP4_ERR_SHAPE;
  if (M > kMxGemmMaxM || N > kMxGemmMaxN) return NVFP4_ERR_SHAPE;
  if (M * K >= (1ll << 36) || N * K >= (1ll << 36)) return NVFP4_ERR_SHAPE;  // a matrix's scales within 2^31 bytes
  return NVFP4_OK;
}

template <int BM, int BN, int WM, int WN, int BK, int OUT, bool PAST = false>
static int launch_mx_tile(const MxGemmArgs& g, hipStream_t stream) {
  const int mt = (g.M + BM - 1) / BM, nt = (g.N + BN - 1) / BN;
  if ((int64_t)mt * nt * (64 * WM * WN) >= (1ll << 32)) return NVFP4_ERR_SHAPE;  // threads of a grid
  hipLaunchKernelGGL((mx_tile_kernel<BM, BN, WM, WN, BK, OUT, PAST>), dim3((unsigned)mt * nt, g.splits),
                     dim3(64 * WM * WN), 0, stream, g, mt, nt);
  NVFP4_CHECK_LAUNCH();
  return NVFP4_OK;
}

template <int MT, int OUT>
static int launch_mx_skinny(const MxGemmArgs& g, hipStream_t stream) {
  const dim3 grid((g.N + 15) / 16, (g.M + 16 * MT - 1) / (16 * MT));
  hipLaunchKernelGGL((mx_skinny_kernel<MT, OUT>), grid, dim3(64 * kMxSkinnyWaves), 0, stream, g);
  NVFP4_CHECK_LAUNCH();
  return NVFP4_OK;
}

// Which kernel a product takes (us on the card, operands from memory, the other
// side in brackets; KB are bytes). Few tokens: one subtile of 16 tokens a
// workgroup up to 16 tokens (1 x 4096 x 7168: 5.3 [tiles 9.4]; 16 x 16384 x 8192:
// 16.7 [17.6]) or where that takes at most a workgroup per CU (32 x 1024 x 7168:
// 5.3 [two subtiles 7.1], 128 x 512 x 8192: 6.2 [parts of K 8.7]), two where that
// does (32 x 4096 x 7168: 6.8 [9.5], 64 x 2048 x 16384: 13.6 [parts 14.7]), unless
// a very long K meets few workgroups: their time grows with it.
constexpr int kMxSkinnyM = 16, kMxSkinnyKB = 8192;
static int mx_few(int64_t M, int64_t N, int64_t KB) {
  const int64_t across = (N + 15) / 16, one = (M + 15) / 16 * across, two = (M + 31) / 32 * across;
  if (M <= kMxSkinnyM) return KB > kMxSkinnyKB && one <= 128 ? 0 : 1;
  if (KB > kMxSkinnyKB) return 0;
  return one <= 256 ? 1 : two <= 256 ? 2 : 0;
}
// Outputs of the large tile that go past the caches: BF16 ones that would not stay
// there (16384 x 7168 x 2048, 235 MB: 136 us [142 through them], with a quantizer
// behind it 183 [204], a norm 332 [342]) and float32, a weight's gradient, which
// the next operator does not read. Smaller ones are read by what comes next: 8192
// x 7168 x 2048, 117 MB, and a norm 165 [158], although by itself 77 [82]; 4096 x
// 7168 x 4096 and a norm 108 [104].
constexpr int64_t kMxPastBytes = 128 << 20;

// Parts of K for tiles: as many as bring 64 x 128 tiles to about one per CU,
// each of at least 512 bytes (64 x 4096 x 16384: 11.7 + 3.8 [undivided 26]; 128
// x 1024 x 16384: 10.2 + 3.8 [18.3]), or one where K is short: the join costs
// more than it saves (64 x 4096 x 7168: 9.6 undivided).
static int mx_splits(int64_t M, int64_t N, int64_t KB) {
  if (mx_few(M, N, KB)) return 1;
  const int64_t tiles = ((M + 63) / 64) * ((N + 127) / 128);
  const int64_t s = std::min<int64_t>(256 / tiles, KB / 512);
  return s < 2 || KB < 4096 ? 1 : (int)s;
}
static size_t mx_part_bytes(int64_t M, int64_t N, int splits) { return splits > 1 ? (size_t)splits * M * N * 4 : 0; }

template <int OUT>
static int launch_mx(const MxGemmArgs& g, hipStream_t stream) {
  constexpr bool SILU = OUT == kMxSilu;
  if (g.splits > 1) {
    const int st = launch_mx_tile<64, 128, 2, 2, 128, kMxPart>(g, stream);
    if (st) return st;
    hipLaunchKernelGGL(mx_join_kernel<OUT>, dim3((unsigned)(((int64_t)g.M * g.n_out / 4 + 255) / 256)), dim3(256), 0,
                       stream, g);
    NVFP4_CHECK_LAUNCH();
    return NVFP4_OK;
  }
  const int few = mx_few(g.M, g.N, g.KB);
  if (few == 1) return launch_mx_skinny<1, OUT>(g, stream);
  if (few == 2) return launch_mx_skinny<2, OUT>(g, stream);
  // The tile that takes least, by what each took at K = 7168 (us, in proportion
  // to K), with r tiles for each of the 256 CUs: alone on a CU or, where all are
  // busy and the clock falls, by the tile.
  const auto rounds = [&](int bm, int bn) {
    return (double)((int64_t)((g.M + bm - 1) / bm) * ((g.N + bn - 1) / bn)) / 256.0;
  };
  const double rl = rounds(256, 256), rm = rounds(128, 128), rs = rounds(64, SILU ? 128 : 64);
  const double large = std::max(41.0 * std::ceil(rl), 61.0 * rl), middle = std::max(16.6 * std::ceil(rm), 1.8 + 19.2 * rm);
  const double small = SILU ? std::max(14.7 * std::ceil(rs), 15.2 * rs) : rs <= 1.0 ? 9.8 : 2.6 + 6.3 * rs;
  if (large <= middle && large <= small) {
    if (OUT == kMxF32 || (int64_t)g.M * g.n_out * 2 >= kMxPastBytes)
      return launch_mx_tile<256, 256, 2, 4, 64, OUT, true>(g, stream);
    if constexpr (OUT != kMxF32) return launch_mx_tile<256, 256, 2, 4, 64, OUT>(g, stream);
  }
  if (middle <= small) return launch_mx_tile<128, 128, 4, 2, 128, OUT>(g, stream);
  return launch_mx_tile<64, SILU ? 128 : 64, 2, 2, 128, OUT>(g, stream);
}

extern "C" size_t mxfp4_gemm_ws_bytes(int32_t M, int32_t N, int32_t K) {
  if (mx_gemm_check(M, N, K, NVFP4_EPI_BF16, NVFP4_DT_BF16) || M == 0) return 0;
  return mx_part_bytes(M, N, mx_splits(M, N, K / 2));
}

extern "C" int mxfp4_gemm(const uint8_t* a_q, const uint8_t* a_scale, const uint8_t* b_q, const uint8_t* b_scale,
                          int32_t M, int32_t N, int32_t K, int32_t epilogue, const void* add, int32_t d_dtype, void* d,
                          void* ws, size_t ws_bytes, void* stream) {
  const int st = mx_gemm_check(M, N, K, epilogue, d_dtype);
  if (st) return st;
  if (M == 0) return NVFP4_OK;
  const int want = mx_splits(M, N, K / 2);
  const size_t need = mx_part_bytes(M, N, want);
  if ((K > 0 && (!a_q || !a_scale || !b_q || !b_scale)) || !d || (need && !ws)) return NVFP4_ERR_NULL;
  if (!nvfp4_aligned16(a_q) || !nvfp4_aligned16(a_scale) || !nvfp4_aligned16(b_q) || !nvfp4_aligned16(b_scale) ||
      !nvfp4_aligned16(add) || !nvfp4_aligned16(d) || !nvfp4_aligned16(ws))
    return NVFP4_ERR_ALIGN;
  if (ws_bytes < need) return NVFP4_ERR_WORKSPACE;
  const bool silu = epilogue == NVFP4_EPI_SILU_MUL;
  const int KB = K / 2, per = std::max((KB + want - 1) / want + 127, 128) / 128 * 128;
  const MxGemmArgs g = {a_q, a_scale, b_q, b_scale, add, d, M, N, KB, silu ? N / 2 : N,
                        std::max((KB + per - 1) / per, 1), per, reinterpret_cast<float*>(ws)};
  if (silu) return launch_mx<kMxSilu>(g, (hipStream_t)stream);
  return d_dtype == NVFP4_DT_F32 ? launch_mx<kMxF32>(g, (hipStream_t)stream) : launch_mx<kMxBf16>(g, (hipStream_t)stream);
}
