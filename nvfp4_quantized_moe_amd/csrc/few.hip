// The expert layer for a few tokens, in two launches over the packed NVFP4
// weights of the layer (moe_forward's, nvfp4_pack_weights):
//   h[t, e]  = bf16(silu(gs_g W_gate x[t]) * (gs_u W_up x[t]))  for the experts e of token t on this rank
//   out[t]   = bf16(sum_e w[t, e] gs_2 W_down h[t, e] [+ add[t]])
// with BF16 activations as they are and sums in float32. What bounds it is the
// bytes of the experts that the tokens chose; x, h and out are small. So
// nothing is quantized, sorted or gathered beforehand: every workgroup finds
// its expert in the choices themselves, and every wave streams weight chunks
// from memory to registers and multiplies them there.
//
// E2M1 x E4M3 has at most 6 significant bits, so a weight without its global
// scale is exact in BF16: two values decode to float32 in one instruction, are
// multiplied by the block's scale and meet in one word. MFMA 32x32x16 BF16
// with the weights' 32 rows as first operand and 32 tokens as second; a chunk's
// lanes hold 64 of 128 K elements each (lane half g the range [64 g, 64 g + 64)),
// and the tokens' operand is read in the same order.
#include <algorithm>

#include "common.h"
#include "internal.h"
#include "tile.h"
#include "wave.h"

namespace nvfp4 {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kFewMaxT = 64, kFewMaxK = 64, kFewMaxL = 4096;
constexpr int kFewChunk = 2304, kFewScales = 2048;  // bytes of 32 rows x 128 columns, and where their scales start
constexpr int kUpWaves = 4, kDownWaves = 8;
constexpr int kUpDepth = 3, kDownDepth = 4;

struct FewArgs {
  const uint16_t* x;     // BF16 [T, H]
  const int32_t* ids;    // [T, k] global
  const float* weight;   // [T, k]
  const uint8_t *w1, *w2;
  const float *gs1, *gs2;
  uint16_t* h;           // BF16 [T * k, I], row t k + j of the first j with that expert
  const uint16_t* add;   // BF16 [T, H] or NULL
  uint16_t* out;
  int T, k, L, start, H, I, dual;
};

// An item is an expert and 32 tokens (the lower or the upper half of the batch)
// of which at least one chose it. Bit 2 e + half of a bitmap in LDS says which
// there are; they are taken in ascending order.
struct Items {
  uint32_t bits[2 * kFewMaxL / 32];
  int before[2 * kFewMaxL / 32 + 1];  // items in the words before, and in all
};
__device__ __forceinline__ int local_expert(const FewArgs& g, int id) {
  const int64_t e = (int64_t)id - g.start;
  return e >= 0 && e < g.L ? (int)e : -1;
}
// Fills the bitmap, and ids with the choices as local experts (-1: not here).
__device__ __forceinline__ void find_items(const FewArgs& g, Items& s, int16_t* ids) {
  const int words = (2 * g.L + 31) / 32, n = g.T * g.k;
  for (int i = threadIdx.x; i < words; i += blockDim.x) s.bits[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int e = local_expert(g, g.ids[i]);
    ids[i] = (int16_t)e;
    if (e >= 0) {
      const int b = 2 * e + (i >= 32 * g.k ? 1 : 0);
      atomicOr(&s.bits[b >> 5], 1u << (b & 31));
    }
  }
  __syncthreads();
  if (threadIdx.x < 64) {  // four words to a lane, at most 256
    int sum = 0, c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = threadIdx.x * 4 + i;
      c[i] = sum;
      sum += at < words ? __popc(s.bits[at]) : 0;
    }
    int scan = sum;
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(scan, o, 64);
      if ((int)threadIdx.x >= o) scan += v;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s.before[threadIdx.x * 4 + i] = scan - sum + c[i];
    if (threadIdx.x == 63) s.before[256] = scan;
  }
  __syncthreads();
}
// The a-th item (a < their number): 2 e + half. The same for a whole wave.
__device__ __forceinline__ int item_at(const Items& s, int a, int words) {
  int lo = 0, hi = words - 1;  // the last word with before <= a
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.before[mid] <= a) lo = mid; else hi = mid - 1;
  }
  uint32_t b = s.bits[lo];
  for (int i = a - s.before[lo]; i > 0; --i) b &= b - 1;
  return lo * 32 + __ffs((int)b) - 1;
}
// This lane's token of an item (lane % 32 of its half), its first choice that is
// the expert (-1: none).
__device__ __forceinline__ int choice_of(const FewArgs& g, const int16_t* ids, int e, int t) {
  int first = -1;
  if (t < g.T)
    for (int j = g.k - 1; j >= 0; --j) first = ids[t * g.k + j] == e ? j : first;
  return first;
}

// Loads of a wave's stages. `in` says whether the stage exists: where it does
// not they take an offset out of range, which moves nothing; a branch around
// them would leave the compiler unsure what is in flight, and it would wait for
// all of it.
__device__ __forceinline__ u32x4_t load16(__amdgpu_buffer_rsrc_t r, int voff, int soff) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, 0);
}
// One lane's part of a chunk, and its BF16 operands.
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
  static __device__ __forceinline__ uint32_t pair(uint32_t w, float f) {
    const float2_t v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, SEL);
    return __builtin_amdgcn_perm(__float_as_uint(v[1] * f), __float_as_uint(v[0] * f), 0x07060302u);  // exact
  }
};
// The tokens' operands of a chunk: eight runs of eight elements.
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

// A workgroup: 32 gate and their 32 up rows of one item's expert. Its waves share
// out the K stages, and their sums meet in LDS in the waves' order.
__global__ __launch_bounds__(64 * kUpWaves) void few_up_kernel(FewArgs g) {
  __shared__ Items items;
  __shared__ float sums[kUpWaves][2][32][36];  // [wave][gate, up][token][row]
  extern __shared__ int16_t ids[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  find_items(g, items, ids);
  const int pairs = g.I / 32, a = blockIdx.x / pairs, sub = blockIdx.x % pairs;
  if (a >= items.before[256]) return;
  const int item = item_at(items, a, (2 * g.L + 31) / 32);
  const int e = item >> 1, t = (item & 1) * 32 + (lane & 31), j = choice_of(g, ids, e, t);
  const uint64_t chose = __ballot(j >= 0);
  const int some = __builtin_ctzll(chose) + (item & 1) * 32;  // lanes without a token repeat one
  const int stages = g.H / 128;
  const __amdgpu_buffer_rsrc_t rx = buffer_rsrc(g.x, (uint32_t)(g.T * g.H * 2));
  const int matrix = 2 * pairs * stages * kFewChunk, from = sub * stages * kFewChunk, up = pairs * stages * kFewChunk;
  const __amdgpu_buffer_rsrc_t rw = buffer_rsrc(g.w1 + (size_t)e * matrix, (uint32_t)matrix);
  const int at_x = (j >= 0 ? t : some) * g.H * 2 + 128 * (lane >> 5);
  float16_t acc[2];
#pragma unroll
  for (int v = 0; v < 16; ++v) acc[0][v] = acc[1][v] = 0.0f;
  struct Stage {
    Chunk gate, up;
    Tokens tok;
  } st[kUpDepth];
  auto load = [&](int s, Stage& to) {
    const bool in = s < stages;
    const int at = in ? from + s * kFewChunk : 0;
    to.gate.load(rw, at, lane, in);
    to.up.load(rw, at + up, lane, in);
    to.tok.load(rx, at_x, in ? s * 256 : 0, in);
  };
  auto compute = [&](const Stage& it) {
    multiply(it.gate, it.tok, acc[0]);
    multiply(it.up, it.tok, acc[1]);
  };
#pragma unroll
  for (int d = 0; d < kUpDepth - 1; ++d) load(wave + d * kUpWaves, st[d]);
  int s = wave;
  for (; s + (kUpDepth - 1) * kUpWaves < stages; s += kUpDepth * kUpWaves) {
#pragma unroll
    for (int d = 0; d < kUpDepth; ++d) {
      load(s + (d + kUpDepth - 1) * kUpWaves, st[(d + kUpDepth - 1) % kUpDepth]);
      compute(st[d]);
    }
  }
#pragma unroll
  for (int d = 0; d < kUpDepth - 1; ++d)
    if (s + d * kUpWaves < stages) compute(st[d]);
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<float4_t*>(&sums[wave][p][lane & 31][8 * q + 4 * (lane >> 5)]) =
          float4_t{acc[p][4 * q], acc[p][4 * q + 1], acc[p][4 * q + 2], acc[p][4 * q + 3]};
  __syncthreads();
  const int token = threadIdx.x >> 3, row = (threadIdx.x & 7) * 4;
  const int tt = (item & 1) * 32 + token, jj = choice_of(g, ids, e, tt);
  if (jj < 0) return;
  float4_t gate = float4_t{0, 0, 0, 0}, ups = float4_t{0, 0, 0, 0};
#pragma unroll
  for (int v = 0; v < kUpWaves; ++v) {
    gate += *reinterpret_cast<const float4_t*>(&sums[v][0][token][row]);
    ups += *reinterpret_cast<const float4_t*>(&sums[v][1][token][row]);
  }
  const float ag = g.dual ? g.gs1[2 * e] : g.gs1[e], au = g.dual ? g.gs1[2 * e + 1] : ag;
  float o[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) o[v] = silu_mul(ag * gate[v], au * ups[v]);
  *reinterpret_cast<uint2*>(g.h + ((size_t)tt * g.k + jj) * g.I + sub * 32 + row) =
      make_uint2(f32x2_to_bf16x2(o[0], o[1]), f32x2_to_bf16x2(o[2], o[3]));
}

// A workgroup: 32 rows of the down weights of every item. Its waves take equal
// runs of the (item, K stage) sequence; each adds what its items give, times
// their weights, to a tile of its own in LDS, and the tiles are added in the
// waves' order.
__global__ __launch_bounds__(64 * kDownWaves) void few_down_kernel(FewArgs g) {
  __shared__ Items items;
  extern __shared__ float lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int PITCH = 36;
  float* const tiles = lds;                                             // [wave][T][PITCH]
  float* const weight = lds + kDownWaves * g.T * PITCH;                 // [T][k]
  int16_t* const ids = reinterpret_cast<int16_t*>(weight + g.T * g.k);  // [T][k]
  for (int i = threadIdx.x; i < kDownWaves * g.T * PITCH; i += 64 * kDownWaves) tiles[i] = 0.0f;
  for (int i = threadIdx.x; i < g.T * g.k; i += 64 * kDownWaves) weight[i] = g.weight[i];
  find_items(g, items, ids);
  float* const mine = tiles + wave * g.T * PITCH;
  const __amdgpu_buffer_rsrc_t rh = buffer_rsrc(g.h, (uint32_t)(g.T * g.k * g.I * 2));
  const int stages = g.I / 128, words = (2 * g.L + 31) / 32;
  const int64_t total = (int64_t)items.before[256] * stages;
  int64_t u = total * wave / kDownWaves;
  const int64_t end = total * (wave + 1) / kDownWaves;
  while (u < end) {
    const int a = (int)(u / stages), s0 = (int)(u - (int64_t)a * stages);
    const int s1 = (int)min((int64_t)stages, s0 + (end - u));
    u += s1 - s0;
    const int item = item_at(items, a, words);
    const int e = item >> 1, t = (item & 1) * 32 + (lane & 31), j = choice_of(g, ids, e, t);
    const uint64_t chose = __ballot(j >= 0);
    const int first = __builtin_ctzll(chose);
    const int row = j >= 0 ? t * g.k + j : -1, some = __shfl(row, first, 64);
    const int matrix = (g.H / 32) * stages * kFewChunk, from = (int)blockIdx.x * stages * kFewChunk;
    const __amdgpu_buffer_rsrc_t rw = buffer_rsrc(g.w2 + (size_t)e * matrix, (uint32_t)matrix);
    const int at_h = (row >= 0 ? row : some) * g.I * 2 + 128 * (lane >> 5);
    float16_t acc;
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[v] = 0.0f;
    struct Stage {
      Chunk c;
      Tokens tok;
    } st[kDownDepth];
    auto load = [&](int s, Stage& to) {
      const bool in = s < s1;
      to.c.load(rw, in ? from + s * kFewChunk : 0, lane, in);
      to.tok.load(rh, at_h, in ? s * 256 : 0, in);
    };
#pragma unroll
    for (int d = 0; d < kDownDepth - 1; ++d) load(s0 + d, st[d]);
    int s = s0;
    for (; s + kDownDepth <= s1; s += kDownDepth) {
#pragma unroll
      for (int d = 0; d < kDownDepth; ++d) {
        load(s + d + kDownDepth - 1, st[(d + kDownDepth - 1) % kDownDepth]);
        multiply(st[d].c, st[d].tok, acc);
      }
    }
#pragma unroll
    for (int d = 0; d < kDownDepth - 1; ++d)
      if (s + d < s1) multiply(st[d].c, st[d].tok, acc);
    if (j >= 0) {  // a token that lists an expert twice has both weights
      float wt = 0.0f;
      for (int i = j; i < g.k; ++i) wt += ids[t * g.k + i] == e ? weight[t * g.k + i] : 0.0f;
      const float gs = g.gs2[e];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float4_t* at = reinterpret_cast<float4_t*>(mine + t * PITCH + 8 * q + 4 * (lane >> 5));
        float4_t v = *at;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += wt * (gs * acc[4 * q + i]);
        *at = v;
      }
    }
    wave_lds_fence();
  }
  __syncthreads();
  for (int i = threadIdx.x; i < g.T * 8; i += 64 * kDownWaves) {
    const int t = i >> 3, row = (i & 7) * 4;
    float4_t o = float4_t{0, 0, 0, 0};
#pragma unroll
    for (int v = 0; v < kDownWaves; ++v) o += *reinterpret_cast<const float4_t*>(tiles + (v * g.T + t) * PITCH + row);
    const size_t at = (size_t)t * g.H + blockIdx.x * 32 + row;
    typedef OutVec<4>::type vec_t;
    vec_t add = vec_t(0u);
    if (g.add) add = *reinterpret_cast<const vec_t*>(g.add + at);
    const float f[4] = {o[0], o[1], o[2], o[3]};
    *reinterpret_cast<vec_t*>(g.out + at) = add_and_round<4>(f, add);
  }
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

extern "C" int32_t nvfp4_moe_few_max_tokens(void) { return kFewMaxT; }

extern "C" size_t nvfp4_moe_few_ws_bytes(int32_t T, int32_t k, int32_t hidden, int32_t inter, int32_t num_local) {
  if (few_check(T, k, hidden, inter, num_local)) return 0;
  return nvfp4_align256((size_t)T * k * inter * 2);
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
  const FewArgs g = {reinterpret_cast<const uint16_t*>(x_bf16), topk_ids, topk_w, w->w1, w->w2, w->w1_gs, w->w2_gs,
                     reinterpret_cast<uint16_t*>(ws), reinterpret_cast<const uint16_t*>(add_bf16),
                     reinterpret_cast<uint16_t*>(out_bf16), T, k, w->num_local, expert_start, w->hidden, w->inter,
                     w->w1_dual_gs};
  const int items = std::min(T * k, (T > 32 ? 2 : 1) * w->num_local);  // at most
  hipLaunchKernelGGL(few_up_kernel, dim3((unsigned)items * (w->inter / 32)), dim3(64 * kUpWaves),
                     (size_t)(T * k * 2 + 15) / 16 * 16, (hipStream_t)stream, g);
  NVFP4_CHECK_LAUNCH();
  const size_t lds = (size_t)kDownWaves * T * 36 * 4 + (size_t)T * k * 6;
  hipLaunchKernelGGL(few_down_kernel, dim3(w->hidden / 32), dim3(64 * kDownWaves), lds, (hipStream_t)stream, g);
  NVFP4_CHECK_LAUNCH();
  return NVFP4_OK;
}
