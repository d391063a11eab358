// The expert layer for a few tokens, in two launches (a third joins parts of the
// down products where the layer is narrow) over the layer's packed NVFP4 weights
// (nvfp4_pack_weights):
//   h[t, e]  = bf16(silu(gs_g W_gate x[t]) * (gs_u W_up x[t]))  for the experts e of token t on this rank
//   out[t]   = bf16(sum_e w[t, e] gs_2 W_down h[t, e] [+ add[t]])
// with BF16 activations as they are and sums in float32. What bounds it is the
// bytes of the experts that the tokens chose; x, h and out are small. So
// nothing is quantized, sorted or gathered beforehand: every workgroup finds
// its expert in the choices themselves, and every wave streams weight chunks
// from memory to registers and multiplies them there.
//
// What bounds the rest is instructions and the loads of the tokens, so an expert
// with up to eight tokens (most, in a decode step) is handled so that each weight
// costs least. An E2M1 code is exact in BF16, and a block of 16 shares one E4M3
// scale: a matrix step covers one block, MFMA 32x32x16 BF16 with the tokens as
// first operand and 32 weight rows as second, from codes turned to BF16 two at a
// time, and its sums are added to the running ones times the rows' scales. A lane
// of the result holds one weight row, so one scale, and four tokens: four
// multiply-adds for what takes 24 instructions where every weight is multiplied
// by its scale before the step. The tokens' operands come through LDS, by loads
// that pass no register, one for four tokens: read by every lane from memory they
// kept the address unit busy for longer than the weights. More tokens are handled
// by scaled weights and direct loads, as their own multiply-adds would cost more.
// (64 tokens on 48 x 7168 x 2048, up and down: 102 + 61 us, all that way 105 + 82;
// with an expert's tokens in one place, not in those of a half of the batch, whose
// weights were read again: 79 + 46, 5.0 and 4.4 TB/s.)
//
// A packed chunk's lane halves hold 64 of 128 K elements each. A swap between the
// halves brings the two words of a block side by side.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "few_lds.h"
#include "internal.h"
#include "tile.h"
#include "wave.h"

namespace nvfp4 {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kFewMaxT = 64, kFewMaxK = 64, kFewMaxL = 4096;
constexpr int kFewChunk = 2304, kFewScales = 2048;  // bytes of 32 rows x 128 columns, and where their scales start
constexpr int kUpWaves = 4;

struct FewArgs {
  const uint16_t* x;     // BF16 [T, H]
  const int32_t* ids;    // [T, k] global
  const float* weight;   // [T, k]
  const uint8_t *w1, *w2;
  const float *gs1, *gs2;
  uint16_t* h;           // BF16 [T * k, I], row t k + j of the first j with that expert
  float* partial;        // [parts][T, H], with more than one part
  const uint16_t* add;   // BF16 [T, H] or NULL
  uint16_t* out;
  int T, k, L, start, H, I, dual, parts;
};

__device__ __forceinline__ void few_store(const FewArgs& g, size_t at, float4_t o) {
  typedef OutVec<4>::type vec_t;
  vec_t add = vec_t(0u);
  if (g.add) add = *reinterpret_cast<const vec_t*>(g.add + at);
  const float f[4] = {o[0], o[1], o[2], o[3]};
  *reinterpret_cast<vec_t*>(g.out + at) = add_and_round<4>(f, add);
}
__device__ __forceinline__ int local_expert(const FewArgs& g, int id) {
  const int64_t e = (int64_t)id - g.start;
  return e >= 0 && e < g.L ? (int)e : -1;
}

// The experts that some token chose, as every workgroup finds them in the choices
// by itself: a bitmap in LDS, taken in ascending order.
struct Choices {
  struct Found {
    uint32_t bits[kFewMaxL / 32];
    int before[kFewMaxL / 32 + 1];  // experts in the words before, and in all
  };
  const Found* s;
  const int16_t* ids;  // the choices as local experts, -1: not here
  const float* weights;
  int k, T, words;
  __device__ __forceinline__ void find(const FewArgs& g, Found& to, int16_t* local, float* weights_lds) {
    s = &to;
    ids = local;
    weights = weights_lds;
    k = g.k;
    T = g.T;
    words = (g.L + 31) / 32;
    const int n = T * k;
    for (int i = threadIdx.x; i < words; i += blockDim.x) to.bits[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      const int e = local_expert(g, g.ids[i]);
      local[i] = (int16_t)e;
      if (weights_lds) weights_lds[i] = g.weight[i];
      if (e >= 0) atomicOr(&to.bits[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    if (threadIdx.x < 64) {  // two words to a lane, at most 128
      const int at = threadIdx.x * 2;
      const int c = at < words ? __popc(to.bits[at]) : 0, sum = c + (at + 1 < words ? __popc(to.bits[at + 1]) : 0);
      int scan = sum;
      for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(scan, o, 64);
        if ((int)threadIdx.x >= o) scan += v;
      }
      to.before[at] = scan - sum;
      to.before[at + 1] = scan - sum + c;
      if (threadIdx.x == 63) to.before[128] = scan;
    }
    __syncthreads();
  }
  __device__ __forceinline__ int count() const { return s->before[128]; }
  // The a-th of them, by all lanes of a wave: one each for the words and for the bits.
  __device__ __forceinline__ int expert(int a) const {
    const int lane = threadIdx.x & 63;
    int lo = -1;  // the last word with before <= a
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = 64 * h + lane;
      lo += __popcll(__ballot(at < words && s->before[min(at, words - 1)] <= a));
    }
    const uint32_t b = s->bits[lo], below = (1u << (lane & 31)) - 1;
    const bool here = (b >> (lane & 31) & 1u) && __popc(b & below) == a - s->before[lo];
    return __builtin_amdgcn_readfirstlane(lo * 32 + __ffsll((long long)__ballot(here)) - 1);
  }
  // The first choice of this lane's token that is expert e (-1: none), and (WEIGHT)
  // the token's weight on it: a token that lists an expert twice has both weights.
  // Four choices at a time are on their way from LDS.
  template <bool WEIGHT>
  __device__ __forceinline__ int choice(int e, float& weight) const {
    const int t = threadIdx.x & 63, row = min(t, T - 1) * k;
    int first = -1;
    weight = 0.0f;
    for (int j = 0; j < k; j += 4) {
      int id[4];
      float w[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {  // past the end the last one again
        id[u] = ids[row + min(j + u, k - 1)];
        if constexpr (WEIGHT) w[u] = weights[row + min(j + u, k - 1)];
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        first = first < 0 && id[u] == e ? j + u : first;
        if constexpr (WEIGHT) weight += id[u] == e && j + u < k ? w[u] : 0.0f;
      }
    }
    return t < T ? first : -1;
  }
};

// An expert's n tokens in order: lane p holds the p-th (and its first choice that is
// the expert, and its weight on it); lanes from n on the first again, with j = -1.
struct Mine {
  int n, t, j;
  float w;
};
template <bool WEIGHT>
__device__ __forceinline__ Mine tokens_of(const Choices& ch, int e) {
  float weight;
  const int lane = threadIdx.x & 63, j = ch.choice<WEIGHT>(e, weight);
  const uint64_t chose = __ballot(j >= 0), below = (1ull << lane) - 1;
  Mine m;
  m.n = __popcll(chose);
  // each lane hands its token to the lane of its rank, those without one behind
  const int rank = j >= 0 ? __popcll(chose & below) : m.n + __popcll(~chose & below);
  const int both = __builtin_amdgcn_ds_permute(rank * 4, lane << 8 | (j & 255));
  m.t = (lane < m.n ? both : __builtin_amdgcn_readfirstlane(both)) >> 8;
  m.j = lane < m.n ? both & 255 : -1;
  m.w = WEIGHT ? __shfl(weight, m.t, 64) : 0.0f;
  return m;
}
// 32 of them, from `from` on, in lanes 0..31 and again in 32..63.
__device__ __forceinline__ Mine part_of(const Mine& m, int from) {
  const int p = from + (int)(threadIdx.x & 31);
  return {m.n, __shfl(m.t, p, 64), __shfl(m.j, p, 64), __shfl(m.w, p, 64)};
}

// Loads of a wave's stages. `in` says whether the stage exists: where it does
// not they take an offset out of range, which moves nothing; a branch around
// them would leave the compiler unsure what is in flight, and it would wait for
// all of it.
__device__ __forceinline__ u32x4_t load16(__amdgpu_buffer_rsrc_t r, int voff, int soff) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, 0);
}
// One lane's part of a chunk, and (direct) its BF16 operands with their scales.
struct Chunk {
  u32x4_t q[2];
  uint32_t s;
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, int soff, int lane, bool in) {
    const int at = in ? lane * 16 : kOutOfRange, scales = in ? lane * 4 : kOutOfRange;
    q[0] = load16(r, at, soff);
    q[1] = load16(r, at, soff + 1024);
    s = __builtin_amdgcn_raw_buffer_load_b32(r, scales, soff + kFewScales, 0);
  }
  template <int STEP>
  __device__ __forceinline__ bf16x8_t operand() const {
    const uint32_t w = q[STEP / 4][STEP % 4];
    const float f = __builtin_amdgcn_cvt_f32_fp8((int)s, STEP / 2);
    return __builtin_bit_cast(bf16x8_t, u32x4_t{pair<0>(w, f), pair<1>(w, f), pair<2>(w, f), pair<3>(w, f)});
  }

 private:
  template <int SEL>
  static __device__ __forceinline__ uint32_t pair(uint32_t w, float f) {  // at most 6 significant bits: exact
    const float2_t v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, SEL);
    return __builtin_amdgcn_perm(__float_as_uint(v[1] * f), __float_as_uint(v[0] * f), 0x07060302u);
  }
};

// ---- more than eight tokens: direct loads, scaled weights as first operand

// Lane half g holds the elements [64 g, 64 g + 64) of its row, eight to a step.
struct Tokens {
  u32x4_t v[8];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, int voff, int soff, bool in) {
    const int at = in ? voff : kOutOfRange;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = load16(r, at + 16 * i, soff);
  }
};
template <int STEP = 0>
__device__ __forceinline__ void multiply(const Chunk& c, const Tokens& t, float16_t& acc) {
  acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(c.operand<STEP>(), __builtin_bit_cast(bf16x8_t, t.v[STEP]), acc, 0, 0, 0);
  if constexpr (STEP < 7) multiply<STEP + 1>(c, t, acc);
}

// ---- up to eight tokens: through LDS, scales behind the step

// A stage's tokens in LDS: 256 bytes each, a token's 16-byte pieces permuted by its
// number, so that the tokens' pieces of one step lie in different banks.
struct FewLoad {  // this lane's piece of each load of four tokens
  int at[2];
  __device__ __forceinline__ void init(int offset, int n) {  // offset: of the token that lane p holds
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int r = 4 * g + lane / 16, from = __shfl(offset, r, 64);
      at[g] = r < n ? from + ((lane & 15) ^ r) * 16 : kOutOfRange;
    }
  }
  template <int NG>
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, int4v* to, int soff, bool in) const {
#pragma unroll
    for (int g = 0; g < NG; ++g) load_lds16(r, to + 64 * g, in ? at[g] : kOutOfRange, soff);
  }
};
// acc += tokens x chunk: register i of a lane is weight row lane % 32 and token
// 4 (lane / 32) + i.
__device__ __forceinline__ float16_t block_product(int4v tok, uint32_t codes) {
  const u32x4_t w = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, 1.0f, 0)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, 1.0f, 1)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, 1.0f, 2)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, 1.0f, 3))};
  float16_t zero;
#pragma unroll
  for (int v = 0; v < 16; ++v) zero[v] = 0.0f;
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, tok), __builtin_bit_cast(bf16x8_t, w), zero, 0,
                                                 0, 0);
}
struct FewTokens {
  int4v lo[4], hi[4];  // pieces of the lower half's blocks and of the upper half's
  // piece: this lane's token's place in the stage, and its number
  __device__ __forceinline__ void read(const int4v* stage, int r) {
    const int half = (threadIdx.x & 63) >> 5;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      lo[b] = stage[r * 16 + ((2 * b + half) ^ r)];
      hi[b] = stage[r * 16 + ((8 + 2 * b + half) ^ r)];
    }
  }
};
__device__ __forceinline__ void multiply(const Chunk& c, const FewTokens& t, float4_t& acc) {
  const u32x2_t s = rows32(c.s);  // scales of the lower half's blocks, and of the upper half's
  float16_t p[2];
  const auto add = [&](const float16_t& v, float scale) {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(scale, v[i], acc[i]);
  };
#define FEW_BLOCK(B)                                                                                             \
  {                                                                                                              \
    const u32x2_t w = __builtin_amdgcn_permlane32_swap(c.q[B / 2][2 * (B % 2)], c.q[B / 2][2 * (B % 2) + 1], false, \
                                                       false);                                                   \
    const float16_t lo = block_product(t.lo[B], w[0]);                                                           \
    if (B > 0) add(p[1], __builtin_amdgcn_cvt_f32_fp8((int)s[1], B > 0 ? B - 1 : 0));                            \
    const float16_t hi = block_product(t.hi[B], w[1]);                                                           \
    add(lo, __builtin_amdgcn_cvt_f32_fp8((int)s[0], B));                                                         \
    p[1] = hi;                                                                                                   \
    __builtin_amdgcn_sched_barrier(0); /* more products at a time would not fit the registers */                 \
  }
  FEW_BLOCK(0) FEW_BLOCK(1) FEW_BLOCK(2) FEW_BLOCK(3)
#undef FEW_BLOCK
  add(p[1], __builtin_amdgcn_cvt_f32_fp8((int)s[1], 3));
}

// Until no load of this wave is in flight: those of stages that do not exist write
// to LDS too, and neither the next run nor another workgroup may find them there.
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_s_waitcnt(15 << 8 | 7 << 4);  // vmcnt(0) alone
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Where the tokens of a stage wait in LDS, eight for each wave; an array for each
// stage of the ring, so that the compiler can tell their loads apart.
template <int W>
struct alignas(16) Ring {
  int4v at[W][128];
};

// The sums of 32 gate and the 32 up rows over a wave's K stages, left in
// sums[gate, up][token][row].
struct UpStages {
  __amdgpu_buffer_rsrc_t w, x;
  int from, up, stages;  // bytes of the gate rows' first chunk, from there to the up rows', K stages
  int lane, wave;
  Chunk gate[3], ups[3];
  __device__ __forceinline__ void load_w(int s, int d) {
    const bool in = s < stages;
    const int at = in ? from + s * kFewChunk : 0;
    gate[d].load(w, at, lane, in);
    ups[d].load(w, at + up, lane, in);
  }
};
template <int NG>
__device__ __forceinline__ void up_few(UpStages& u, int offset, int n, int4v* r0, int4v* r1, int4v* r2, float (*sums)[32][36]) {
  constexpr int W = kUpWaves;
  FewLoad tok;
  tok.init(offset, n);
  const int r = min(u.lane & 31, n - 1);
  float4_t acc[2] = {float4_t{0, 0, 0, 0}, float4_t{0, 0, 0, 0}};
  const auto slot = [&](int d) { return d == 0 ? r0 : d == 1 ? r1 : r2; };
  const auto load = [&](int s, int d) {
    tok.template load<NG>(u.x, slot(d), s < u.stages ? s * 256 : 0, s < u.stages);
    u.load_w(s, d);
  };
  const auto compute = [&](int d) {
    FewTokens t;
    t.read(slot(d), r);
    multiply(u.gate[d], t, acc[0]);
    multiply(u.ups[d], t, acc[1]);
  };
  load(u.wave, 0);
  load(u.wave + W, 1);
  int s = u.wave;
  for (; s + 2 * W < u.stages; s += 3 * W) {
#pragma unroll
    for (int d = 0; d < 3; ++d) {
      load(s + (d + 2) * W, (d + 2) % 3);
      compute(d);
    }
  }
  if (s < u.stages) compute(0);
  if (s + W < u.stages) compute(1);
  wait_loads();
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[p][4 * (u.lane >> 5) + i][u.lane & 31] = acc[p][i];
}
__device__ __forceinline__ void up_many(UpStages& u, int offset, float (*sums)[32][36]) {
  constexpr int W = kUpWaves;
  Tokens tok[2];
  float16_t acc[2];
#pragma unroll
  for (int v = 0; v < 16; ++v) acc[0][v] = acc[1][v] = 0.0f;
  const auto load_x = [&](int s, int d) { tok[d].load(u.x, offset, s < u.stages ? s * 256 : 0, s < u.stages); };
  // the tokens of the next stage before the weights of the one behind it: loads
  // are waited for in order
  const auto step = [&](int s, int d) {
    load_x(s + W, (d + 1) % 2);
    u.load_w(s + 2 * W, (d + 2) % 3);
    multiply(u.gate[d % 3], tok[d % 2], acc[0]);
    multiply(u.ups[d % 3], tok[d % 2], acc[1]);
  };
  u.load_w(u.wave, 0);
  load_x(u.wave, 0);
  u.load_w(u.wave + W, 1);
  int s = u.wave;
  for (; s + 5 * W < u.stages; s += 6 * W) {
#pragma unroll
    for (int d = 0; d < 6; ++d) step(s + d * W, d);
  }
#pragma unroll
  for (int d = 0; d < 5; ++d) {
    if (s + d * W >= u.stages) break;
    step(s + d * W, d);
  }
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<float4_t*>(&sums[p][u.lane & 31][8 * q + 4 * (u.lane >> 5)]) =
          float4_t{acc[p][4 * q], acc[p][4 * q + 1], acc[p][4 * q + 2], acc[p][4 * q + 3]};
}

// A workgroup: 32 gate and their 32 up rows of one expert. Its waves share out the
// K stages, and their sums meet in LDS in the waves' order. More than 32 tokens are
// two parts, one after the other.
__global__ __launch_bounds__(64 * kUpWaves) void few_up_kernel(FewArgs g) {
  __shared__ Choices::Found found;
  __shared__ Ring<kUpWaves> r0, r1, r2;
  __shared__ float sums[kUpWaves][2][32][36];  // [wave][gate, up][token][row]
  __shared__ int place[32];                    // of the part's tokens in h
  extern __shared__ int16_t ids[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Choices ch;
  ch.find(g, found, ids, nullptr);
  const int pairs = g.I / 32, a = blockIdx.x / pairs, sub = blockIdx.x % pairs;
  if (a >= ch.count()) return;
  const int e = ch.expert(a), stages = g.H / 128, matrix = 2 * pairs * stages * kFewChunk;
  const Mine m = tokens_of<false>(ch, e);
  const int n = __builtin_amdgcn_readfirstlane(m.n);
  const float ag = g.dual ? g.gs1[2 * e] : g.gs1[e], au = g.dual ? g.gs1[2 * e + 1] : ag;
  UpStages u;
  u.w = buffer_rsrc(g.w1 + (size_t)e * matrix, (uint32_t)matrix);
  u.x = buffer_rsrc(g.x, (uint32_t)(g.T * g.H * 2));
  u.from = sub * stages * kFewChunk;
  u.up = pairs * stages * kFewChunk;
  u.stages = stages;
  u.lane = lane;
  u.wave = wave;
  for (int part = 0; part < n; part += 32) {
    const Mine mp = part_of(m, part);
    if (n <= 4)
      up_few<1>(u, m.t * g.H * 2, n, r0.at[wave], r1.at[wave], r2.at[wave], sums[wave]);
    else if (n <= 8)
      up_few<2>(u, m.t * g.H * 2, n, r0.at[wave], r1.at[wave], r2.at[wave], sums[wave]);
    else
      up_many(u, mp.t * g.H * 2 + 128 * (lane >> 5), sums[wave]);
    if (threadIdx.x < 32) place[threadIdx.x] = mp.j >= 0 ? mp.t * g.k + mp.j : -1;
    __syncthreads();
    const int token = threadIdx.x >> 3, row = (threadIdx.x & 7) * 4, slot = place[token];
    if (slot >= 0) {
      float4_t g4 = float4_t{0, 0, 0, 0}, u4 = float4_t{0, 0, 0, 0};
#pragma unroll
      for (int v = 0; v < kUpWaves; ++v) {
        g4 += *reinterpret_cast<const float4_t*>(&sums[v][0][token][row]);
        u4 += *reinterpret_cast<const float4_t*>(&sums[v][1][token][row]);
      }
      float o[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) o[v] = silu_mul(ag * g4[v], au * u4[v]);
      *reinterpret_cast<uint2*>(g.h + (size_t)slot * g.I + sub * 32 + row) =
          make_uint2(f32x2_to_bf16x2(o[0], o[1]), f32x2_to_bf16x2(o[2], o[3]));
    }
    __syncthreads();  // the next part's sums take the same place
  }
}

// A wave's run of K stages [s0, s1) of an expert's down rows.
struct DownStages {
  __amdgpu_buffer_rsrc_t w, h;
  int from, s0, s1, lane;
  __device__ __forceinline__ void load_w(Chunk& c, int s) const { c.load(w, s < s1 ? from + s * kFewChunk : 0, lane, s < s1); }
};
template <int NG>
__device__ __forceinline__ float4_t down_few(const DownStages& u, int offset, int n, int4v* r0, int4v* r1, int4v* r2,
                                             int4v* r3, int4v* r4) {
  constexpr int D = kDownStages;
  FewLoad tok;
  tok.init(offset, n);
  const int r = min(u.lane & 31, n - 1);
  float4_t acc = float4_t{0, 0, 0, 0};
  Chunk c[D];
  const auto slot = [&](int d) { return d == 0 ? r0 : d == 1 ? r1 : d == 2 ? r2 : d == 3 ? r3 : r4; };
  const auto load = [&](int s, int d) {
    tok.template load<NG>(u.h, slot(d), s < u.s1 ? s * 256 : 0, s < u.s1);
    u.load_w(c[d], s);
  };
  const auto compute = [&](int d) {
    FewTokens t;
    t.read(slot(d), r);
    multiply(c[d], t, acc);
  };
#pragma unroll
  for (int d = 0; d + 1 < D; ++d) load(u.s0 + d, d);
  int s = u.s0;
  for (; s + D <= u.s1; s += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      load(s + d + D - 1, (d + D - 1) % D);
      compute(d);
    }
  }
#pragma unroll
  for (int d = 0; d + 1 < D; ++d)
    if (s + d < u.s1) compute(d);
  wait_loads();
  return acc;
}
__device__ __forceinline__ float16_t down_many(const DownStages& u, int offset) {
  float16_t acc;
#pragma unroll
  for (int v = 0; v < 16; ++v) acc[v] = 0.0f;
  Chunk c[3];
  Tokens tok[2];
  const auto load_h = [&](int s, int d) { tok[d].load(u.h, offset, s < u.s1 ? s * 256 : 0, s < u.s1); };
  const auto step = [&](int s, int d) {
    load_h(s + 1, (d + 1) % 2);
    u.load_w(c[(d + 2) % 3], s + 2);
    multiply(c[d % 3], tok[d % 2], acc);
  };
  u.load_w(c[0], u.s0);
  load_h(u.s0, 0);
  u.load_w(c[1], u.s0 + 1);
  int s = u.s0;
  for (; s + 6 <= u.s1; s += 6) {
#pragma unroll
    for (int d = 0; d < 6; ++d) step(s + d, d);
  }
#pragma unroll
  for (int d = 0; d < 5; ++d) {
    if (s + d >= u.s1) break;
    step(s + d, d);
  }
  return acc;
}

// A workgroup: 32 rows of the down weights of every expert chosen, or one of
// `parts` equal runs of the (expert, K stage) sequence. Its waves take equal runs;
// each adds what its experts give, times their weights, to a tile of its own in
// LDS, and the tiles are added in the waves' order. RING: up to eight tokens of an
// expert go through LDS, where that fits beside the tiles.
template <bool RING>
__global__ __launch_bounds__(64 * kDownWaves) void few_down_kernel(FewArgs g) {
  constexpr int W = kDownWaves, PITCH = kDownPitch;
  static_assert((sizeof(Choices::Found) + 15) / 16 * 16 == kFoundBytes && sizeof(Ring<W>) == kRingBytes, "as the host counts");
  __shared__ Choices::Found found;
  __shared__ Ring<RING ? W : 1> r0, r1, r2, r3, r4;
  extern __shared__ __align__(16) float lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float* const tiles = lds;                                              // [wave][T][PITCH]
  float* const weights = lds + W * g.T * PITCH;                          // [T][k]
  int16_t* const ids = reinterpret_cast<int16_t*>(weights + g.T * g.k);  // [T][k]
  for (int i = lane; i < g.T * PITCH; i += 64) tiles[wave * g.T * PITCH + i] = 0.0f;
  Choices ch;
  ch.find(g, found, ids, weights);
  float* const mine = tiles + wave * g.T * PITCH;
  const int stages = g.I / 128, matrix = (g.H / 32) * stages * kFewChunk;
  DownStages u;
  u.h = buffer_rsrc(g.h, (uint32_t)(g.T * g.k * g.I * 2));
  u.from = (int)blockIdx.x * stages * kFewChunk;
  u.lane = lane;
  const int64_t total = (int64_t)ch.count() * stages;
  const int run = (int)blockIdx.y * W + wave, runs = g.parts * W;
  const int end = (int)(total * (run + 1) / runs);
  for (int at = (int)(total * run / runs); at < end; at += u.s1 - u.s0) {
    const int a = at / stages;
    u.s0 = at - a * stages;
    u.s1 = min(stages, u.s0 + end - at);
    const int e = ch.expert(a);
    const Mine m = tokens_of<true>(ch, e);
    const int n = __builtin_amdgcn_readfirstlane(m.n);
    const float gs = g.gs2[e];
    const int row = m.t * g.k + m.j, first = __builtin_amdgcn_readfirstlane(row);
    u.w = buffer_rsrc(g.w2 + (size_t)e * matrix, (uint32_t)matrix);
    if (RING && n <= 8) {
      const float4_t acc =
          n <= 4 ? down_few<1>(u, row * g.I * 2, n, r0.at[wave], r1.at[wave], r2.at[wave], r3.at[wave], r4.at[wave])
                 : down_few<2>(u, row * g.I * 2, n, r0.at[wave], r1.at[wave], r2.at[wave], r3.at[wave], r4.at[wave]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int p = 4 * (lane >> 5) + i;  // the expert's p-th token, which lane p knows
        const float pw = __shfl(m.w, p, 64);
        const int pt = __shfl(m.t, p, 64);
        if (p < n) mine[pt * PITCH + (lane & 31)] += pw * (gs * acc[i]);
      }
    } else {
      for (int part = 0; part < n; part += 32) {
        const Mine mp = part_of(m, part);
        const float16_t acc = down_many(u, (mp.j >= 0 ? mp.t * g.k + mp.j : first) * g.I * 2 + 128 * (lane >> 5));
        if (mp.j < 0) continue;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float4_t* to = reinterpret_cast<float4_t*>(mine + mp.t * PITCH + 8 * q + 4 * (lane >> 5));
          float4_t v = *to;
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] += mp.w * (gs * acc[4 * q + i]);
          *to = v;
        }
      }
    }
    wave_lds_fence();
  }
  __syncthreads();
  for (int i = threadIdx.x; i < g.T * 8; i += 64 * W) {
    const int t = i >> 3, row = (i & 7) * 4;
    float4_t o = float4_t{0, 0, 0, 0};
#pragma unroll
    for (int v = 0; v < W; ++v) o += *reinterpret_cast<const float4_t*>(tiles + (v * g.T + t) * PITCH + row);
    const size_t to = (size_t)t * g.H + blockIdx.x * 32 + row;
    if (g.parts > 1)
      *reinterpret_cast<float4_t*>(g.partial + (size_t)blockIdx.y * g.T * g.H + to) = o;
    else
      few_store(g, to, o);
  }
}

// Adds the parts in their order, four outputs to a thread.
__global__ __launch_bounds__(256) void few_join_kernel(FewArgs g) {
  const size_t at = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4, n = (size_t)g.T * g.H;
  if (at >= n) return;
  float4_t o = float4_t{0, 0, 0, 0};
  for (int p = 0; p < g.parts; ++p) o += *reinterpret_cast<const float4_t*>(g.partial + p * n + at);
  few_store(g, at, o);
}

}  // namespace nvfp4

using namespace nvfp4;

static int few_check(int32_t T, int32_t k, int32_t hidden, int32_t inter, int32_t L) {
  if (T < 0 || T > kFewMaxT || k < 1 || k > kFewMaxK || L < 1 || L > kFewMaxL) return NVFP4_ERR_SHAPE;
  if (hidden <= 0 || inter <= 0 || hidden % 128 != 0 || inter % 128 != 0) return NVFP4_ERR_SHAPE;
  if ((int64_t)2 * inter * hidden / 32 * 18 >= (1ll << 31) || (int64_t)inter / 32 * kFewMaxT * kFewMaxK >= (1ll << 23))
    return NVFP4_ERR_SHAPE;  // an expert's weights as in the layer; threads of a grid
  return NVFP4_OK;
}
// Parts of the down products' sequence: as many as bring its workgroups to one per
// CU, each wave to at least eight chunks where every choice is another expert; one
// otherwise, since the join is a launch more. (Down and join, us [one
// part]: 8 tokens of 8 experts each, 64 x 4096 x 1024: 24.7 + 4.8 [37]; 64 tokens,
// 48 x 1024 x 1024: 16.4 + 4.7 [53]; 16 tokens, 32 x 512 x 512: 13.2 + 4.0 [19].)
static int few_parts(int T, int k, int hidden, int inter, int L) {
  const int64_t chunks = (int64_t)std::min(T * k, L) * (inter / 128);
  return (int)std::max<int64_t>(1, std::min<int64_t>(256 / std::min(256, hidden / 32), chunks / (8 * kDownWaves)));
}
static size_t few_h_bytes(int T, int k, int inter) { return nvfp4_align256((size_t)T * k * inter * 2); }

extern "C" int32_t nvfp4_moe_few_max_tokens(void) { return kFewMaxT; }

extern "C" size_t nvfp4_moe_few_ws_bytes(int32_t T, int32_t k, int32_t hidden, int32_t inter, int32_t num_local) {
  if (few_check(T, k, hidden, inter, num_local)) return 0;
  const int parts = few_parts(T, k, hidden, inter, num_local);
  return few_h_bytes(T, k, inter) + (parts > 1 ? (size_t)parts * T * hidden * 4 : 0);
}

extern "C" int nvfp4_moe_forward_few(const nvfp4_moe_weights* w, const void* x_bf16, int32_t T, const int32_t* topk_ids,
                                     const float* topk_w, int32_t k, int32_t expert_start, const void* add_bf16,
                                     void* out_bf16, void* ws, size_t ws_bytes, void* stream) {
  if (!w) return NVFP4_ERR_NULL;
  const int st = few_check(T, k, w->hidden, w->inter, w->num_local);
  if (st) return st;
  if (w->w1_dual_gs != 0 && w->w1_dual_gs != 1) return NVFP4_ERR_ARG;
  if (T == 0) return NVFP4_OK;
  if (!w->w1 || !w->w1_gs || !w->w2 || !w->w2_gs || !x_bf16 || !topk_ids || !topk_w || !out_bf16 || !ws)
    return NVFP4_ERR_NULL;
  if (!nvfp4_aligned16(w->w1) || !nvfp4_aligned16(w->w2) || !nvfp4_aligned16(x_bf16) || !nvfp4_aligned16(add_bf16) ||
      !nvfp4_aligned16(out_bf16) || !nvfp4_aligned16(ws))
    return NVFP4_ERR_ALIGN;
  if (ws_bytes < nvfp4_moe_few_ws_bytes(T, k, w->hidden, w->inter, w->num_local)) return NVFP4_ERR_WORKSPACE;
  const int parts = few_parts(T, k, w->hidden, w->inter, w->num_local);
  char* const base = reinterpret_cast<char*>(ws);
  const FewArgs g = {reinterpret_cast<const uint16_t*>(x_bf16), topk_ids, topk_w, w->w1, w->w2, w->w1_gs, w->w2_gs,
                     reinterpret_cast<uint16_t*>(base), reinterpret_cast<float*>(base + few_h_bytes(T, k, w->inter)),
                     reinterpret_cast<const uint16_t*>(add_bf16), reinterpret_cast<uint16_t*>(out_bf16), T, k,
                     w->num_local, expert_start, w->hidden, w->inter, w->w1_dual_gs, parts};
  const int experts = std::min(T * k, w->num_local);  // chosen ones, at most
  hipLaunchKernelGGL(few_up_kernel, dim3((unsigned)experts * (w->inter / 32)), dim3(64 * kUpWaves),
                     (size_t)(T * k * 2 + 15) / 16 * 16, (hipStream_t)stream, g);
  NVFP4_CHECK_LAUNCH();
  const dim3 down(w->hidden / 32, parts), threads(64 * kDownWaves);
  const FewDownLds lds = few_down_lds(T, k);
  if (lds.ring)
    hipLaunchKernelGGL(few_down_kernel<true>, down, threads, lds.bytes, (hipStream_t)stream, g);
  else  // many choices for many tokens
    hipLaunchKernelGGL(few_down_kernel<false>, down, threads, lds.bytes, (hipStream_t)stream, g);
  NVFP4_CHECK_LAUNCH();
  if (parts > 1) {
    hipLaunchKernelGGL(few_join_kernel, dim3((unsigned)(((size_t)T * w->hidden / 4 + 255) / 256)), dim3(256), 0,
                       (hipStream_t)stream, g);
    NVFP4_CHECK_LAUNCH();
  }
  return NVFP4_OK;
}
