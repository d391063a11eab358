// The routing gate in front of the layer: scores of a token's logits, the k
// highest, their weights; the balance loss over these choices with per-expert
// counts; and the gradient of both with respect to the logits.
//
// Score of a logit x: softmax over the row, 1 / (1 + e^-x), or
// sqrt(log(1 + e^x)). The choice goes by key = score + bias (float64 order,
// see gate_topk_kernel), the weight by the score alone.
//
// One wave owns one token in every kernel here: lane l holds logits l,
// l + 64, ... (any E and any row alignment give coalesced loads), row
// reductions are register-only (wave.h), and a workgroup needs no barrier.
#include <type_traits>

#include "common.h"
#include "internal.h"
#include "wave.h"

namespace nvfp4 {

constexpr int kGateWaves = 4;      // tokens per workgroup
constexpr int kGateMaxExperts = 1024;
constexpr int kGateMaxK = 64;      // lane j holds choice j
constexpr float kInf = __builtin_inff();

template <typename T>
__device__ __forceinline__ float load_logit(const T* p, size_t i);
template <>
__device__ __forceinline__ float load_logit<float>(const float* p, size_t i) {
  return p[i];
}
template <>
__device__ __forceinline__ float load_logit<uint16_t>(const uint16_t* p, size_t i) {
  return bf16_to_f32(p[i]);
}
__device__ __forceinline__ void store_logit(float* p, size_t i, float v) { p[i] = v; }
__device__ __forceinline__ void store_logit(uint16_t* p, size_t i, float v) { p[i] = (uint16_t)f32_to_bf16(v); }

// The lane's logits of row `row`; -inf past E. The index is clamped rather than
// the load masked: fewer instructions, and all loads leave together.
template <typename L, int VPT>
__device__ __forceinline__ void load_row(const L* logits, size_t row, int E, float (&x)[VPT]) {
  const int lane = threadIdx.x & 63;
  const L* p = logits + row;
#pragma unroll
  for (int v = 0; v < VPT; ++v) x[v] = load_logit(p, (uint32_t)min(v * 64 + lane, E - 1));
  if (E < VPT * 64) {
#pragma unroll
    for (int v = 0; v < VPT; ++v)
      if (v * 64 + lane >= E) x[v] = -kInf;
  }
}

// Scores that depend on one logit alone (x = -inf gives 0).
__device__ __forceinline__ float sigmoid_score(float x) { return 1.0f / (1.0f + expf(-x)); }
__device__ __forceinline__ double sigmoid_score(double x) {  // e^-x itself would end at x = -709, not -745
  const double e = exp(-fabs(x));
  return (x < 0.0 ? e : 1.0) / (1.0 + e);
}
// sqrt(log(1 + e^x)) with the large term outside the logarithm. Far below 0
// it equals e^(x/2) to the last bit, and e^x itself would underflow first.
__device__ __forceinline__ float sqrt_softplus(float x) {
  return x < -20.0f ? expf(0.5f * x) : sqrtf(fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x))));
}
__device__ __forceinline__ double sqrt_softplus(double x) {
  return x < -40.0 ? exp(0.5 * x) : sqrt(fmax(x, 0.0) + log1p(exp(-fabs(x))));
}
template <typename F>
__device__ __forceinline__ F pointwise_score(F x, int score) {
  return score == MOE_SCORE_SIGMOID ? sigmoid_score(x) : sqrt_softplus(x);
}
// derivative of a pointwise score s = score(x); the sigmoid's from e^-|x|,
// since 1 - s has lost its digits where s is near 1
__device__ __forceinline__ float score_slope(float x, float s, int score) {
  if (score == MOE_SCORE_SIGMOID) {
    const float e = expf(-fabsf(x));
    return e / ((1.0f + e) * (1.0f + e));
  }
  return x < -20.0f ? 0.5f * s : 0.5f * sigmoid_score(x) / s;
}

// Far below 0 a score is e^(x tail_power) to float32's last bit, and soon leaves
// float32. Scores that are divided by their sum, a sum that shows all of them to
// lie there, are taken relative to the largest instead; down to where float64
// ends (below, they count as 0).
__device__ __forceinline__ float tail_power(int score) { return score == MOE_SCORE_SIGMOID ? 1.0f : 0.5f; }
__device__ __forceinline__ bool in_tail(float sum, int score) {  // every logit below -19: e^-19 < 2^-27
  return sum < (score == MOE_SCORE_SIGMOID ? 0x1p-28f : 0x1p-14f);
}
constexpr float kTailEnd = -708.0f;

// The same scores where they are summed or multiplied into a gradient rather
// than compared: hardware exponential, logarithm, root and reciprocal, each
// within one or two float32 steps of what it is given: e^x through 2^(x log2 e)
// has |x| half steps more, log(1 + t) the rounding of 1 + t (64 half steps of the
// result at t = 2^-6, fewer above).
constexpr float kLog2e = 1.44269504f, kLn2 = 0.69314718f;
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }
__device__ __forceinline__ float fast_log1p(float t) {  // t >= 0
  // below 2^-6 the series (next term t^4 / 5 < 2^-26): 1 + t has rounded t away
  return t < 0x1p-6f ? t * (1.0f - t * (0.5f - t * (1.0f / 3.0f - t * 0.25f)))
                     : __builtin_amdgcn_logf(1.0f + t) * kLn2;
}
// score and (with SLOPE) slope; both 0 at x = -inf
template <bool SLOPE>
__device__ __forceinline__ float fast_sigmoid(float x, float* slope) {
  const float e = fast_exp(-fabsf(x)), r = __builtin_amdgcn_rcpf(1.0f + e);
  if (SLOPE) *slope = e * r * r;
  return x < 0.0f ? e * r : r;
}
template <bool SLOPE>
__device__ __forceinline__ float fast_sqrt_softplus(float x, float* slope) {
  const float e = fast_exp(-fabsf(x));
  const bool low = x < -20.0f;
  const float s = low ? fast_exp(0.5f * x) : __builtin_amdgcn_sqrtf(fmaxf(x, 0.0f) + fast_log1p(e));
  if (SLOPE) {
    const float r = __builtin_amdgcn_rcpf(1.0f + e);
    *slope = low ? 0.5f * s : 0.5f * (x < 0.0f ? e * r : r) * __builtin_amdgcn_rcpf(s);
  }
  return s;
}

// e^x within two float32 steps: the hardware's 2^t at t = x log2 e, corrected
// by what the product's rounding (and that of log2 e) left out. Past +-88,
// the edge of float32, e^x stays what it is there.
__device__ __forceinline__ float near_exp(float x) {
  x = fminf(fmaxf(x, -88.0f), 88.0f);
  const float t = x * kLog2e;
  const float rest = __builtin_fmaf(x, 1.92596299e-8f, __builtin_fmaf(x, kLog2e, -t));  // log2 e - kLog2e
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e * kLn2, rest, e);
}
// Bits of a key in the order of unsigned integers (-0 as 0).
__device__ __forceinline__ uint32_t order_bits(float key) {
  const uint32_t bits = __float_as_uint(key + 0.0f);
  return bits ^ ((uint32_t)((int32_t)bits >> 31) | 0x80000000u);
}

struct GateShape {
  int T, E, k, score;
  int n_group, topk_group, group_size;
  int renormalize;
  float scale;
};

// What a float key may be off by beside its relative error: scores below 2^-126
// become 0 (a sum of two of them, or with a bias, then loses its order).
constexpr float kLostScore = 0x1p-120f;

// Float key of every logit of the lane: the logits themselves when the order
// of scores is theirs (no bias, one group). *bmax: the lane's largest |bias| of
// an expert that can be chosen.
template <int VPT>
__device__ __forceinline__ void gate_keys(const float (&x)[VPT], const float* bias, const GateShape& g,
                                          float (&key)[VPT], float* bmax) {
  const int lane = threadIdx.x & 63;
  *bmax = 0.0f;
  if (!bias && g.n_group == 1) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) key[v] = x[v];
    return;
  }
  if (g.score == MOE_SCORE_SOFTMAX) {
    float top = -kInf, sum = 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) top = fmaxf(top, x[v]);
    top = wave_all_max(top);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      key[v] = x[v] > -kInf ? near_exp(x[v] - top) : 0.0f;
      sum += key[v];
    }
    sum = 1.0f / wave_all_sum(sum);
#pragma unroll
    for (int v = 0; v < VPT; ++v) key[v] *= sum;
  } else if (g.score == MOE_SCORE_SIGMOID) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) key[v] = __builtin_amdgcn_rcpf(1.0f + near_exp(-x[v]));
  } else {
#pragma unroll
    for (int v = 0; v < VPT; ++v) key[v] = fast_sqrt_softplus<false>(x[v], nullptr);
  }
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const float b = bias ? bias[min(v * 64 + lane, g.E - 1)] : 0.0f;
    key[v] = x[v] > -kInf ? key[v] + b : -kInf;
    *bmax = fmaxf(*bmax, key[v] > -kInf ? fabsf(b) : 0.0f);
  }
}

// The same in float64, one logit at a time. For softmax, of a row whose
// highest logit and 1 / (sum of e^(x - highest)) are given. (Not inlined: the
// constants of three float64 functions would take registers of the whole
// kernel, which hardly ever calls them; 16384 x 512 in groups took 49 us
// instead of 24.)
struct ExactRow {
  double top, inv;
};
static __device__ __attribute__((noinline)) double exact_key(float x, float bias, ExactRow r, int score) {
  const double s = score == MOE_SCORE_SOFTMAX ? exp((double)x - r.top) * r.inv : pointwise_score((double)x, score);
  return x > -kInf ? s + (double)bias : (double)-kInf;
}
template <typename L>
__device__ __forceinline__ ExactRow exact_row(const L* logits, size_t row, const GateShape& g) {
  ExactRow r = {0.0, 0.0};
  if (g.score != MOE_SCORE_SOFTMAX) return r;
  const int lane = threadIdx.x & 63;
  float top = -kInf;
#pragma unroll 1
  for (int e = lane; e < g.E; e += 64) top = fmaxf(top, load_logit(logits, row + e));
  r.top = wave_all_max(top);
  double sum = 0.0;
#pragma unroll 1
  for (int e = lane; e < g.E; e += 64)
    sum += fmax(exact_key(load_logit(logits, row + e), 0.0f, {r.top, 1.0}, MOE_SCORE_SOFTMAX), 0.0);  // 0 at -inf
  r.inv = 1.0 / wave_all_sum(sum);
  return r;
}

// Which groups stay: a group's value is the sum of its two highest keys; the
// topk_group highest values stay, ties to the lower group. Bit per * i of
// *stays is group i's. Tells how far apart the last kept and the first dropped
// value are, and their size, in *gap and *size (float keys: whether float64
// could decide otherwise). keys: LDS, E of them, this wave's own.
template <typename F>
__device__ __forceinline__ int choose_groups(const F* keys, const GateShape& g, uint64_t* stays, F* gap, F* size) {
  const int lane = threadIdx.x & 63;
  const F inf = (F)kInf;
  int per = 64;  // lanes per group: a power of two, per * n_group <= 64
  while (per * g.n_group > 64) per >>= 1;
  const int mine = lane / per, sub = lane % per;
  F a = -inf, b = -inf;  // the two highest of this lane's share, a >= b
  if (mine < g.n_group)
    for (int i = sub; i < g.group_size; i += 4 * per) {  // four reads in flight
      F v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = keys[mine * g.group_size + min(i + u * per, g.group_size - 1)];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const F w = i + u * per < g.group_size ? v[u] : -inf;
        b = fmax(b, fmin(a, w));
        a = fmax(a, w);
      }
    }
  for (int o = 1; o < per; o <<= 1) {
    const F a2 = __shfl_xor(a, o, 64), b2 = __shfl_xor(b, o, 64);
    b = fmax(fmax(b, b2), fmin(a, a2));
    a = fmax(a, a2);
  }
  const F value = a + (b > -inf ? b : (F)0);  // -inf when nothing in the group can be chosen
  int rank = 0;
  if constexpr (sizeof(F) == 4) {  // one comparison: the value's bits above the group
    const uint32_t order = order_bits(value);
    const uint64_t mine64 = ((uint64_t)order << 32) | (uint32_t)(63 - mine);
    for (int j = 0; j < g.n_group; ++j) {
      const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)order, j * per);
      rank += (((uint64_t)o << 32) | (uint32_t)(63 - j)) > mine64 ? 1 : 0;
    }
  } else {
    for (int j = 0; j < g.n_group; ++j) {
      const F o = lane_value(value, j * per);
      rank += (o > value || (o == value && j < mine)) ? 1 : 0;
    }
  }
  const bool there = mine < g.n_group;
  *stays = __ballot(there && rank < g.topk_group);
  // the lanes of the last kept and the first dropped group (the latter is there if any is)
  const uint64_t last = __ballot(there && rank == g.topk_group - 1), first = __ballot(there && rank == g.topk_group);
  const F lowest = lane_value(value, __ffsll((unsigned long long)last) - 1);
  const F highest = first ? lane_value(value, __ffsll((unsigned long long)first) - 1) : -inf;
  *gap = lowest - highest;
  *size = fmax(fabs(lowest), fabs(highest));
  return per;
}

// Doubles of a wave's part of LDS: E float64 keys, or a float per lane and
// register (64 VPT <= 2 E, but for E < 32).
__host__ __device__ __forceinline__ int gate_keys_stride(int E) { return E < 32 ? 32 : E; }

// The whole row's float64 keys, in LDS (E of them, this wave's own).
template <typename L>
__device__ __forceinline__ void exact_keys(const L* logits, size_t row, const float* bias, const GateShape& g,
                                           double* keys) {
  const ExactRow r = exact_row(logits, row, g);
#pragma unroll 1
  for (int e = threadIdx.x & 63; e < g.E; e += 64)
    keys[e] = exact_key(load_logit(logits, row + e), bias ? bias[e] : 0.0f, r, g.score);
  wave_lds_fence();
}

// Drops the float keys of the groups that do not stay, by float64 keys where
// the last kept and the first dropped value are too close: a value is a sum of
// two keys, each score + bias, |bias| <= bmax.
template <typename L, int VPT>
__device__ __forceinline__ void keep_groups(const L* logits, size_t row, const float* bias, float (&key)[VPT],
                                            const GateShape& g, float tol, float bmax, double* lds) {
  const int lane = threadIdx.x & 63;
  float* const keys = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int v = 0; v < VPT; ++v) keys[v * 64 + lane] = key[v];  // the wave's part holds 64 VPT floats
  wave_lds_fence();
  uint64_t stays;
  float gap, size;
  const uint32_t per = choose_groups(keys, g, &stays, &gap, &size);
  if (g.topk_group < g.n_group && !(gap > 4.0f * tol * (size + 2.0f * wave_all_max(bmax)) + kLostScore)) {
    double gap64, size64;
    wave_lds_fence();
    exact_keys(logits, row, bias, g, lds);
    choose_groups(lds, g, &stays, &gap64, &size64);
  }
  const uint32_t magic = ((1u << 20) + (uint32_t)g.group_size - 1u) / (uint32_t)g.group_size;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    // e / group_size: exact for e, group_size <= 1024
    const uint32_t grp = ((uint32_t)(v * 64 + lane) * magic) >> 20;
    if (!((stays >> ((grp * per) & 63u)) & 1u)) key[v] = -kInf;
  }
  wave_lds_fence();
}

// The `want` highest keys, one wave maximum at a time, ties to the lowest
// expert: lane j < want gets the j-th (id -1 when none is left).
template <int VPT>
__device__ __forceinline__ void pick_by_rounds(float (&key)[VPT], int want, int* id, float* at) {
  const int lane = threadIdx.x & 63;
  *id = -1;
  *at = -kInf;
  for (int r = 0; r < want; ++r) {
    float top = -kInf;
#pragma unroll
    for (int v = 0; v < VPT; ++v) top = fmaxf(top, key[v]);
    top = wave_all_max(top);
    if (!(top > -kInf)) break;
    int e = 0x7FFFFFFF;
#pragma unroll
    for (int v = VPT - 1; v >= 0; --v)
      if (key[v] == top) e = v * 64 + lane;
    e = wave_all_min_i32(e);
#pragma unroll
    for (int v = 0; v < VPT; ++v)
      if (v * 64 + lane == e) key[v] = -kInf;
    if (lane == r) {
      *id = e;
      *at = top;
    }
  }
}

// The `want` highest keys for k <= 16, without a chain of wave maxima. The
// wave's lanes fall into `groups` >= k runs; the lowest of the runs' maxima is
// at most the groups-th highest key, so the keys from it on (about 17 of 384
// for 8 runs) hold the k highest. They are compacted in expert order, one per
// lane, and each counts those before it. Returns false, having done nothing,
// when more than 64 remain (many equal keys); *all tells whether the want-th is
// among them. (16384 x 384 and k = 8: 20 us, by rounds 29; k = 16: 25 and
// 37; k = 2: 7.1 and 7.1. Past 16 the runs would be single lanes.)
constexpr int kFastK = 16;
struct Picked {  // a compacted key with its expert
  float key;
  int32_t id;
};
// The lowest of the runs' maxima, from each lane's maximum.
__device__ __forceinline__ float lowest_run(float highest, int k) {
  // steps 1, 2, 4, 8, 16, 32 of the reduction: maxima inside a run, then minima over the runs
  const auto step = [](bool inside, int a, int b) { return inside ? max(a, b) : min(a, b); };
  int m = ordered(highest);
  m = max(m, dpp_i32<kDppXor1>(m));
  m = max(m, dpp_i32<kDppXor2>(m));
  m = step(k <= 8, m, dpp_i32<kDppHalfMirror>(m));
  m = step(k <= 4, m, dpp_i32<kDppMirror>(m));
  u32x2_t r = rows16((uint32_t)m);
  m = step(k <= 2, (int)r[0], (int)r[1]);
  r = rows32((uint32_t)m);
  return from_ordered(step(k <= 1, (int)r[0], (int)r[1]));
}
// How many of the n lanes' keys come before this lane's: a higher key, or the
// same in a lower lane.
__device__ __forceinline__ int rank_of(float key, int n) {
  const int lane = threadIdx.x & 63;
  // one comparison, of the key's bits (in an order of integers; 0 past n, before
  // none) above the place; four lanes a turn
  const uint32_t order = lane < n ? order_bits(key) : 0u;
  const uint64_t mine = ((uint64_t)order << 32) | (uint32_t)(63 - lane);
  int rank = 0;
  for (int j = 0; j < n; j += 4) {  // n <= 64
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)order, j + u);
      rank += (((uint64_t)o << 32) | (uint32_t)(63 - j - u)) > mine ? 1 : 0;
    }
  }
  return rank;
}
__device__ __forceinline__ int rank_of(double key, int n) {
  const int lane = threadIdx.x & 63;
  int rank = 0;
  for (int j = 0; j < n; ++j) {
    const double other = lane_value(key, j);
    rank += other > key || (other == key && j < lane) ? 1 : 0;
  }
  return rank;
}
template <int VPT>
__device__ __forceinline__ bool pick_by_count(const float (&key)[VPT], int k, int want, Picked* lds, int* id, float* at,
                                              bool* all) {
  const int lane = threadIdx.x & 63;
  float m = key[0];
#pragma unroll
  for (int v = 1; v < VPT; ++v) m = fmaxf(m, key[v]);
  m = lowest_run(m, k);
  uint64_t mine[VPT];
  int n = 0;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    mine[v] = __ballot(key[v] >= m && key[v] > -kInf);
    n += __popcll(mine[v]);
  }
  if (n > 64) return false;
  int before = 0;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    if ((mine[v] >> lane) & 1u) lds[before + __popcll(mine[v] & ((1ull << lane) - 1ull))] = {key[v], v * 64 + lane};
    before += __popcll(mine[v]);
  }
  wave_lds_fence();
  const Picked c = lds[lane];  // past n: left over, never counted
  const int rank = rank_of(c.key, n);
  wave_lds_fence();
  if (lane < n && rank < want) lds[rank] = c;
  wave_lds_fence();
  const int have = min(n, want);
  const Picked got = lds[lane];
  *id = lane < have ? got.id : -1;
  *at = lane < have ? got.key : -kInf;
  *all = n >= want;
  wave_lds_fence();
  return true;
}

// Whether some key is within slack of `key0` that is not of the logit x0 and the bias b0.
template <int VPT>
__device__ __forceinline__ bool others_near(const float (&x)[VPT], const float (&key)[VPT], const float* bias, int E,
                                            float key0, float slack, float x0, float b0) {
  const int lane = threadIdx.x & 63;
  bool found = false;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const float b = bias ? bias[min(v * 64 + lane, E - 1)] : 0.0f;
    found |= fabsf(key[v] - key0) <= slack && !(x[v] == x0 && b == b0);
  }
  return __ballot(found) != 0;
}

// The k highest by float64 keys, where the k highest float keys (lane j: the
// j-th, expert *id) are within `slack` of keys that may belong before them:
// the experts down to the k-th key - slack, one exact key per lane; or, if
// these are more than 64, the whole row's keys in LDS, one maximum at a time.
template <typename L, int VPT>
__device__ __forceinline__ void pick_exact(const L* logits, size_t row, const float* bias, const GateShape& g,
                                           const float (&key)[VPT], float at, float slack, Picked* picked,
                                           double* keys, int* id) {
  const int lane = threadIdx.x & 63;
  const float from = lane_value(at, g.k - 1) - slack;  // of -inf: all there are
  int n = 0;
#pragma unroll
  for (int v = 0; v < VPT; ++v) n += __popcll(__ballot(key[v] >= from && key[v] > -kInf));
  if (n <= 64) {
    int before = 0;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const uint64_t mine = __ballot(key[v] >= from && key[v] > -kInf);
      if ((mine >> lane) & 1u) picked[before + __popcll(mine & ((1ull << lane) - 1ull))].id = v * 64 + lane;
      before += __popcll(mine);
    }
    wave_lds_fence();
    const int e = lane < n ? picked[lane].id : 0;
    const double key64 =
        exact_key(load_logit(logits, row + e), bias ? bias[e] : 0.0f, exact_row(logits, row, g), g.score);
    const int rank = rank_of(key64, n);
    wave_lds_fence();
    if (lane < n && rank < g.k) picked[rank].id = e;
    wave_lds_fence();
    *id = lane < min(n, g.k) ? picked[lane].id : -1;
    return;
  }
  exact_keys(logits, row, bias, g, keys);
#pragma unroll
  for (int v = 0; v < VPT; ++v)  // the dropped groups
    if (v * 64 + lane < g.E && !(key[v] > -kInf)) keys[v * 64 + lane] = -kInf;
  *id = -1;
#pragma unroll 1
  for (int j = 0; j < g.k; ++j) {
    double top = -kInf;
    int first = 0x7FFFFFFF;  // this lane's first expert with its highest key
#pragma unroll 1
    for (int e = lane; e < g.E; e += 64) {  // each lane reads and writes its own
      const double k64 = keys[e];
      if (k64 > top) {
        top = k64;
        first = e;
      }
    }
    const double best = wave_all_max(top);
    if (!(best > (double)-kInf)) break;
    const int e = wave_all_min_i32(top == best ? first : 0x7FFFFFFF);
    if (lane == j) *id = e;
    if (lane == (e & 63)) keys[e] = -kInf;
  }
}

// The weights of the choices (lane j < k: expert id, its logit xl) and the stores.
template <int VPT>
__device__ __forceinline__ void write_choices(const float (&x)[VPT], const GateShape& g, int id, float xl, size_t t,
                                              int32_t* ids, float* w) {
  const int lane = threadIdx.x & 63;
  const bool on = lane < g.k && id >= 0;
  if (!on) xl = -kInf;
  float s;
  if (g.score == MOE_SCORE_SOFTMAX) {
    if (g.renormalize) {  // the softmax over the choices alone: nothing of the row's sum is left in it
      const float top = wave_all_max(xl);
      s = on ? near_exp(xl - top) : 0.0f;
    } else {
      float top = -kInf, sum = 0.0f;
#pragma unroll
      for (int v = 0; v < VPT; ++v) top = fmaxf(top, x[v]);
      top = wave_all_max(top);
#pragma unroll
      for (int v = 0; v < VPT; ++v) sum += x[v] > -kInf ? near_exp(x[v] - top) : 0.0f;
      sum = wave_all_sum(sum);
      s = on ? expf(xl - top) / sum : 0.0f;
    }
  } else {
    s = on ? pointwise_score(xl, g.score) : 0.0f;
  }
  if (g.renormalize) {
    float sum = wave_all_sum(s);
    if (in_tail(sum, g.score)) {
      const float top = wave_all_max(xl);
      s = on && top >= kTailEnd ? near_exp(tail_power(g.score) * (xl - top)) : 0.0f;
      sum = wave_all_sum(s);
    }
    s = sum > 0.0f ? s * __builtin_amdgcn_rcpf(sum) : 0.0f;
  }
  if (lane < g.k) {
    ids[t * g.k + lane] = on ? id : -1;
    w[t * g.k + lane] = s * g.scale;
  }
}

// One wave per token. The order of the choices is that of the keys in
// float64; float32 keys decide it wherever two neighbours are further apart
// than their rounding (2^-20 of the scores for the sigmoid; 2^-17 for softmax,
// whose argument x - max is rounded first, and for sqrt-softplus, from the
// hardware's logarithm) or are the same sum of the same numbers. Where they are
// not, float64 keys decide: those of the candidates, one per lane (of every
// expert, 16384 x 384 by sqrt-softplus took 33 us instead of 20).
//
// Bound by the instructions of choosing: 16384 x 256 BF16 with bias and 8
// groups takes 19.1 us, 570 vector instructions a token, waiting for 38 % of
// its waves' cycles (its 8 MB take 1.8 us); 16384 x 384 by the logits alone 10.9.
// Waves on a SIMD, as many as the registers of the common path allow: eight
// (8192 x 256 in groups 12.0 us, with seven 12.3; 16384 x 384 by sqrt-softplus
// with bias 19.5, 20.0), six with 8 logits per lane (16384 x 512 by the logits
// 12.5, with eight 15.7), four with 16 (16384 x 1024 by the sigmoid with bias
// 32.5, with five 52).
// k of one or two with a bias or groups: the threshold of k runs often passes
// fewer than k + 1 keys, and such rows take the float64 keys (16384 x 384 by
// sqrt-softplus with bias: k = 1 23.0 us, 2 22.1, 4 19.6, 8 20.4).
template <typename L, int VPT>
__global__ __launch_bounds__(64 * kGateWaves, VPT <= 6 ? 8 : VPT <= 8 ? 6 : 4) void gate_topk_kernel(const L* __restrict__ logits,
                                                                    const float* __restrict__ bias,
                                                                    const uint8_t* __restrict__ mask, GateShape g,
                                                                    int32_t* __restrict__ ids, float* __restrict__ w) {
  extern __shared__ double lds[];  // unless the keys are the logits: [kGateWaves][gate_keys_stride(E)]
  __shared__ Picked picked[kGateWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kGateWaves + wave;
  if (t >= g.T) return;
  if (mask && mask[t] == 0) {
    if (lane < g.k) {
      ids[t * g.k + lane] = -1;
      w[t * g.k + lane] = 0.0f;
    }
    return;
  }
  const size_t row = (size_t)t * g.E;
  float x[VPT];
  load_row(logits, row, g.E, x);

  const bool by_logit = !bias && g.n_group == 1;
  float key[VPT];
  int id;
  float at;
  float bmax;
  gate_keys(x, bias, g, key, &bmax);
  double* const keys = lds + (size_t)wave * gate_keys_stride(g.E);
  const float tol = g.score == MOE_SCORE_SIGMOID ? 0x1p-20f : 0x1p-17f;
  if (g.n_group > 1) keep_groups(logits, row, bias, key, g, tol, bmax, keys);
  const int want = by_logit ? g.k : min(g.k + 1, 64);
  bool all = true;
  const bool counted = g.k <= kFastK && pick_by_count(key, g.k, want, picked[wave], &id, &at, &all);
  if (!counted) pick_by_rounds(key, want, &id, &at);
  float xl = at;
  if (!by_logit) {
    xl = load_logit(logits, row + max(id, 0));
    const float bl = bias ? bias[max(id, 0)] : 0.0f;
    const float next = __shfl_down(at, 1, 64), xn = __shfl_down(xl, 1, 64), bn = __shfl_down(bl, 1, 64);
    const int idn = __shfl_down(id, 1, 64);
    const bool same = xl == xn && bl == bn;
    const float size = fabsf(at) + fabsf(next) + fabsf(bl) + fabsf(bn);
    const bool close = lane + 1 < g.k && idn >= 0 && !same && !(at - next > 2.0f * tol * size + kLostScore);
    // Between the last choice and what is left out the largest bias counts, not
    // those of the two neighbours: further down lie keys whose biases have
    // cancelled large scores. (Every lane asks with its own largest.)
    const float kth = lane_value(at, g.k - 1), left = lane_value(at, min(g.k, 63));
    const bool last = left > -kInf && !(kth - left > 4.0f * tol * (fabsf(kth) + 2.0f * bmax) + kLostScore);
    const bool doubt = __ballot(close) != 0 || want == g.k || !all;  // !all: the first key left out is unknown
    if (doubt || __ballot(last) != 0) {
      const float slack = 4.0f * tol * (fabsf(kth) + 2.0f * wave_all_max(bmax)) + kLostScore;
      // Copies of one logit and bias on both sides of the border: the lower ids
      // were taken, unless some other key is as near.
      const bool copies = (__ballot(same) >> (g.k - 1)) & 1u;
      if (doubt || !copies || others_near(x, key, bias, g.E, kth, slack, lane_value(xl, g.k - 1), lane_value(bl, g.k - 1))) {
        if (!counted) {  // the rounds took the picked keys out
          for (int j = 0; j < want; ++j) {
            const int e = __builtin_amdgcn_readlane(id, j);
            const float k32 = lane_value(at, j);
#pragma unroll
            for (int v = 0; v < VPT; ++v)
              if (v * 64 + lane == e) key[v] = k32;
          }
        }
        pick_exact(logits, row, bias, g, key, at, slack, picked[wave], keys, &id);
        xl = load_logit(logits, row + max(id, 0));
      }
    }
  }
  write_choices(x, g, id, xl, (size_t)t, ids, w);
}

// ---------------------------------------------------------------- balance loss
//
// Per sequence b with N_b live tokens (mask nonzero, some logit above -inf):
//   share P_be = (1/N_b) sum_t q_te,   f_be = counts_be / (N_b k),
//   L = mean over the sequences with N_b > 0 of E sum_e f_be P_be,
//   z = mean over all live tokens of logsumexp(x_t)^2,
// with q the score divided by its row sum. Three launches: workgroups own runs
// of at most `chunk` tokens of one sequence and leave partial sums (slots, no
// float atomics: the result does not depend on the order they finish in); the
// second joins them per sequence and column block; the third adds the terms
// (a single workgroup of the second does it itself).

struct BalanceShape {
  int T, E, k, B, score;
  int chunk, max_chunks;
};
struct BalanceWs {
  float* q;          // [max_chunks][E] sums of q
  int32_t* counts;   // [max_chunks][E]
  double* z;         // [max_chunks] sums of logsumexp^2
  int32_t* live;     // [max_chunks]
  double* term;      // [B][column blocks] this sequence's share of L before the mean
  double* z_seq;     // [B]
};

struct Span {
  int seq, begin, end;  // tokens [begin, end) of sequence seq; empty when there is no such chunk
};
__device__ __forceinline__ int2 seq_bounds(const int32_t* cu, int s, int T) {
  if (!cu) return make_int2(0, T);
  const int b = min(max(cu[s], 0), T);
  return make_int2(b, max(b, min(cu[s + 1], T)));
}
// Chunk number i over all sequences in order (wave-uniform).
__device__ Span find_chunk(const int32_t* cu, const BalanceShape& g, int i) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int base = 0; base < g.B; base += 64) {
    const int s = base + lane;
    const int2 r = s < g.B ? seq_bounds(cu, s, g.T) : make_int2(0, 0);
    const int n = (r.y - r.x + g.chunk - 1) / g.chunk;
    int incl = n;
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(incl, o, 64);
      if (lane >= o) incl += v;
    }
    const uint64_t past = __ballot(before + incl > i);
    if (past) {
      const int l = __ffsll((unsigned long long)past) - 1;
      const int first = before + __shfl(incl - n, l, 64);
      const int begin = __shfl(r.x, l, 64) + (i - first) * g.chunk;
      return {base + l, begin, min(begin + g.chunk, __shfl(r.y, l, 64))};
    }
    before += __shfl(incl, 63, 64);
  }
  return {0, 0, 0};
}

// Normalized scores of a row (lane l: experts l, l + 64, ...). Returns false
// for a row without a logit above -inf. top: the highest logit, part: 1 / sum of
// e^(x - top), lse: log of the sum of e^x, inv: 1 / sum of the scores, 0 for 0;
// p[v] = e^(x - top) part, which a common offset of a row's logits leaves as it
// is (e^(x - lse) would take on the rounding of lse at the offset's size).
// slope[v]: of the pointwise scores, with SLOPE.
struct RowSums {
  float top, part, lse, inv;
};
template <bool SLOPE, int VPT>
__device__ __forceinline__ bool row_scores(const float (&x)[VPT], int score, float (&q)[VPT], float (&p)[VPT],
                                           float (&slope)[VPT], RowSums* r) {
  float top = -kInf;
#pragma unroll
  for (int v = 0; v < VPT; ++v) top = fmaxf(top, x[v]);
  top = wave_all_max(top);
  if (!(top > -kInf)) return false;
  float es = 0.0f;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    p[v] = fast_exp(x[v] - top);  // 0 at -inf
    es += p[v];
  }
  es = wave_all_sum(es);
  r->lse = top + __builtin_amdgcn_logf(es) * kLn2;
  r->top = top;
  r->part = __builtin_amdgcn_rcpf(es);
#pragma unroll
  for (int v = 0; v < VPT; ++v) p[v] *= r->part;
  if (score == MOE_SCORE_SOFTMAX) {
    r->inv = 1.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) q[v] = p[v];
    return true;
  }
  float sum = 0.0f;
  if (score == MOE_SCORE_SIGMOID) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) q[v] = fast_sigmoid<SLOPE>(x[v], &slope[v]);
  } else {
#pragma unroll
    for (int v = 0; v < VPT; ++v) q[v] = fast_sqrt_softplus<SLOPE>(x[v], &slope[v]);
  }
#pragma unroll
  for (int v = 0; v < VPT; ++v) sum += q[v];
  sum = wave_all_sum(sum);
  if (in_tail(sum, score)) {
    sum = 0.0f;
    const float power = tail_power(score);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      q[v] = top >= kTailEnd ? fast_exp(power * (x[v] - top)) : 0.0f;
      if (SLOPE) slope[v] = power * q[v];
      sum += q[v];
    }
    sum = wave_all_sum(sum);
  }
  r->inv = sum > 0.0f ? __builtin_amdgcn_rcpf(sum) : 0.0f;
#pragma unroll
  for (int v = 0; v < VPT; ++v) q[v] *= r->inv;
  return true;
}

// A wave's tokens one after the other, their scores summed in its registers in
// float32, 64 tokens at most in a row, then in LDS in float64 (a chunk of the
// largest batches gives a wave 16384 tokens); choices counted by LDS atomics on
// whole numbers.
// (16384 x 384 float: 12.6 us, 2 TB/s; about half of it issues the 230 vector
// instructions a token, the rest is the launch and the first row's latency.)
template <typename L, int VPT>
__global__ __launch_bounds__(64 * kGateWaves) void balance_partial_kernel(const L* __restrict__ logits,
                                                                          const int32_t* __restrict__ ids,
                                                                          const uint8_t* __restrict__ mask,
                                                                          const int32_t* __restrict__ cu,
                                                                          BalanceShape g, BalanceWs ws) {
  extern __shared__ double lds[];
  double* q_sh = lds;                                                   // [kGateWaves][E]
  int32_t* hist = reinterpret_cast<int32_t*>(q_sh + kGateWaves * g.E);  // [E]
  __shared__ double z_sh[kGateWaves];
  __shared__ int n_sh[kGateWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int e = threadIdx.x; e < g.E; e += blockDim.x) hist[e] = 0;
  const Span span = find_chunk(cu, g, (int)blockIdx.x);
  if (span.begin >= span.end) return;  // whole workgroup
  __syncthreads();
  float acc[VPT];
#pragma unroll
  for (int v = 0; v < VPT; ++v) acc[v] = 0.0f;
  double z = 0.0;
  int n = 0;
  float next[VPT];
  int next_id = -1, next_on = 0;
  const auto load = [&](int t) {
    load_row(logits, (size_t)t * g.E, g.E, next);
    next_id = ids[(size_t)t * g.k + min(lane, g.k - 1)];
    next_on = mask ? mask[t] : 1;
  };
  if (span.begin + wave < span.end) load(span.begin + wave);
  constexpr int kRun = 64 * kGateWaves;
  for (int from = span.begin; from < span.end; from += kRun) {
    const int to = min(from + kRun, span.end);
    for (int t = from + wave; t < to; t += kGateWaves) {  // with the next row's loads in flight
      float x[VPT], q[VPT], p[VPT], unused[VPT];
#pragma unroll
      for (int v = 0; v < VPT; ++v) x[v] = next[v];
      const int id = lane < g.k ? next_id : -1, on = next_on;
      load(min(t + kGateWaves, span.end - 1));
      if (!on) continue;
      RowSums r;
      if (!row_scores<false>(x, g.score, q, p, unused, &r)) continue;
      if (id >= 0 && id < g.E) atomicAdd(&hist[id], 1);
#pragma unroll
      for (int v = 0; v < VPT; ++v) acc[v] += q[v];
      z += (double)r.lse * (double)r.lse;
      ++n;
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      if (v * 64 + lane < g.E) {  // this lane's alone until the barrier
        double* const sum = q_sh + wave * g.E + v * 64 + lane;
        *sum = from > span.begin ? *sum + (double)acc[v] : (double)acc[v];
      }
      acc[v] = 0.0f;
    }
  }
  if (lane == 0) {
    z_sh[wave] = z;
    n_sh[wave] = n;
  }
  __syncthreads();
  const size_t at = (size_t)blockIdx.x * g.E;
  for (int e = threadIdx.x; e < g.E; e += blockDim.x) {
    double s = q_sh[e];
    for (int w = 1; w < kGateWaves; ++w) s += q_sh[w * g.E + e];
    ws.q[at + e] = (float)s;
    ws.counts[at + e] = hist[e];
  }
  if (threadIdx.x == 0) {
    double zs = 0.0;
    int ns = 0;
    for (int w = 0; w < kGateWaves; ++w) {
      zs += z_sh[w];
      ns += n_sh[w];
    }
    ws.z[blockIdx.x] = zs;
    ws.live[blockIdx.x] = ns;
  }
}

// Workgroup (c, b): experts [COLS c, COLS (c + 1)) of sequence b. A wave takes
// 64 / COLS chunks at a time, eight steps in flight.
template <int COLS, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void balance_join_kernel(const int32_t* __restrict__ cu, BalanceShape g,
                                                                  BalanceWs ws, int32_t* __restrict__ counts,
                                                                  int32_t* __restrict__ tokens,
                                                                  float* __restrict__ loss) {
  __shared__ double q_sh[WAVES][COLS], z_sh[WAVES];
  __shared__ int c_sh[WAVES][COLS], n_sh[WAVES];
  constexpr int SUB = 64 / COLS, STEP = WAVES * SUB;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int b = blockIdx.y, e = blockIdx.x * COLS + lane % COLS;
  // this sequence's chunks: [first, end)
  int first = 0;
  if (cu) {
    for (int base = 0; base < b; base += 64) {
      const int s = base + lane;
      int v = 0;
      if (s < b) {
        const int2 r = seq_bounds(cu, s, g.T);
        v = (r.y - r.x + g.chunk - 1) / g.chunk;
      }
      for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
      first += v;
    }
  }
  const int2 range = seq_bounds(cu, b, g.T);
  const int end = min(first + (range.y - range.x + g.chunk - 1) / g.chunk, g.max_chunks);
  double q = 0.0;
  int cnt = 0;
  for (int c0 = first + wave * SUB + lane / COLS; c0 < end; c0 += 8 * STEP) {
    float v[8];
    int n[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const size_t at = (size_t)min(c0 + u * STEP, end - 1) * g.E + min(e, g.E - 1);
      v[u] = ws.q[at];
      n[u] = ws.counts[at];
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const bool in = c0 + u * STEP < end;
      q += in ? (double)v[u] : 0.0;
      cnt += in ? n[u] : 0;
    }
  }
  for (int o = COLS; o < 64; o <<= 1) {
    q += __shfl_xor(q, o, 64);
    cnt += __shfl_xor(cnt, o, 64);
  }
  int n = 0;
  double z = 0.0;
  for (int c = first + (int)threadIdx.x; c < end; c += blockDim.x) {
    n += ws.live[c];
    z += ws.z[c];
  }
  for (int o = 1; o < 64; o <<= 1) n += __shfl_xor(n, o, 64);
  z = wave_all_sum(z);
  if (lane < COLS) {
    q_sh[wave][lane] = q;
    c_sh[wave][lane] = cnt;
  }
  if (lane == 0) {
    n_sh[wave] = n;
    z_sh[wave] = z;
  }
  __syncthreads();
  if (wave != 0) return;
  n = 0;
  z = q = 0.0;
  cnt = 0;
  for (int w = 0; w < WAVES; ++w) {
    n += n_sh[w];
    z += z_sh[w];
    q += q_sh[w][lane % COLS];
    cnt += c_sh[w][lane % COLS];
  }
  const bool mine = lane < COLS && e < g.E;
  if (mine) counts[(size_t)b * g.E + e] = cnt;
  const double sum = wave_all_sum(mine ? (double)cnt * q : 0.0);
  if (lane == 0) {
    ws.term[(size_t)b * gridDim.x + blockIdx.x] = n > 0 ? sum * g.E / ((double)n * n * g.k) : 0.0;
    if (blockIdx.x == 0) {
      tokens[b] = n;
      ws.z_seq[b] = z;
    }
    if (gridDim.x * gridDim.y == 1) {  // nothing else to add up
      tokens[1] = n;
      tokens[2] = n > 0;
      loss[0] = n > 0 ? (float)(sum * g.E / ((double)n * n * g.k)) : 0.0f;
      loss[1] = n > 0 ? (float)(z / n) : 0.0f;
    }
  }
}

// The two losses from the sequences' terms, one workgroup: 2.2 us for 24
// sequences of 384 experts, nearly all of it the launch.
constexpr int kLossWaves = 4;
__global__ __launch_bounds__(64 * kLossWaves) void balance_loss_kernel(BalanceShape g, BalanceWs ws, int cols,
                                                                       int32_t* __restrict__ tokens,
                                                                       float* __restrict__ loss) {
  __shared__ double d_sh[2][kLossWaves];
  __shared__ int n_sh[2][kLossWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double term = 0.0, z = 0.0;
  int total = 0, seqs = 0;
  for (int64_t i = threadIdx.x; i < (int64_t)g.B * cols; i += blockDim.x) term += ws.term[i];
  for (int s = threadIdx.x; s < g.B; s += blockDim.x) {
    const int m = tokens[s];
    total += m;
    seqs += m > 0;
    z += ws.z_seq[s];
  }
  for (int o = 1; o < 64; o <<= 1) {
    total += __shfl_xor(total, o, 64);
    seqs += __shfl_xor(seqs, o, 64);
  }
  term = wave_all_sum(term);
  z = wave_all_sum(z);
  if (lane == 0) {
    d_sh[0][wave] = term;
    d_sh[1][wave] = z;
    n_sh[0][wave] = total;
    n_sh[1][wave] = seqs;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  term = z = 0.0;
  total = seqs = 0;
  for (int w = 0; w < kLossWaves; ++w) {
    term += d_sh[0][w];
    z += d_sh[1][w];
    total += n_sh[0][w];
    seqs += n_sh[1][w];
  }
  tokens[g.B] = total;
  tokens[g.B + 1] = seqs;
  loss[0] = seqs > 0 ? (float)(term / seqs) : 0.0f;
  loss[1] = total > 0 ? (float)(z / total) : 0.0f;
}

// -------------------------------------------------------------------- gradient
//
// dL/dx of one token, from the gradient of its weights and (or) of the two
// losses:
//   weights  w_j = c s_j / S:  ds_j = (c dw_j - sum_m c dw_m s_m / S) / S, or c dw_j
//            without renormalization; softmax weights renormalized are the
//            softmax over the choices, dx_j = w_j (c dw_j - sum_m c dw_m w_m)
//   balance  dq_e = g0 E counts_be / (B' N_b^2 k), then ds_e = (dq_e - sum dq q) / sum s
//   z        2 g1 lse p_e / N
// and dx_e = s'(x_e) ds_e, or p_e (ds_e - sum ds p) for softmax.
// (16384 x 384 float, both losses: 16 us, 3.1 TB/s of logits and gradients;
// three quarters of it issue the 420 vector instructions a token.)
struct GateGradArgs {
  const int32_t* ids;
  const float* d_w;      // NULL: no gradient through the weights
  const float* d_loss;   // NULL: none through the losses
  const int32_t* counts;
  const int32_t* tokens;
  const int32_t* cu;
  const uint8_t* mask;
  int T, E, k, B, score, renormalize;
  float scale;
};

template <typename L, int VPT>
__global__ __launch_bounds__(64 * kGateWaves) void gate_backward_kernel(const L* __restrict__ logits, GateGradArgs a,
                                                                        L* __restrict__ d_logits) {
  extern __shared__ double lds[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kGateWaves + wave;
  if (t >= a.T) return;
  float* direct = reinterpret_cast<float*>(lds) + (size_t)wave * a.E;
  const size_t row = (size_t)t * a.E;
  float x[VPT], dx[VPT];
#pragma unroll
  for (int v = 0; v < VPT; ++v) dx[v] = 0.0f;
  if (!(a.mask && a.mask[t] == 0)) {
    const bool softmax = a.score == MOE_SCORE_SOFTMAX;
    bool row_softmax = a.d_w && softmax && !a.renormalize;
    // (the row's loads first: the search below is a chain of its own)
    if (a.d_loss || row_softmax) load_row(logits, row, a.E, x);  // else only the chosen logits matter
    // sequence of the token; -1: it lies in none and the losses do not see it
    int seq = a.d_loss ? 0 : -1;
    if (a.d_loss && a.cu) {
      int lo = 0, hi = a.B + 1;  // cu entries <= t
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid] <= (int)t) lo = mid + 1;
        else hi = mid;
      }
      seq = lo - 1 < a.B ? lo - 1 : -1;
    }
    bool in_loss = seq >= 0;
    float q[VPT], p[VPT], slope[VPT];
    RowSums r = {0.0f, 1.0f, 0.0f, 1.0f};
    int32_t chosen[VPT];
    if (in_loss) {
#pragma unroll
      for (int v = 0; v < VPT; ++v) chosen[v] = a.counts[(size_t)seq * a.E + min(v * 64 + lane, a.E - 1)];
    }
    if (in_loss || row_softmax) {
      if (!row_scores<true>(x, a.score, q, p, slope, &r)) in_loss = row_softmax = false;  // not one choice either
    }
    float inner = 0.0f;  // softmax: sum over the row of (gradient of p) p
    if (a.d_w) {
      const int id = lane < a.k ? a.ids[(size_t)t * a.k + lane] : -1;
      const bool on = id >= 0 && id < a.E;
      const float xl = on ? load_logit(logits, row + id) : -kInf;
      const bool some = on && xl > -kInf;
      const float c = some ? a.scale * a.d_w[(size_t)t * a.k + lane] : 0.0f;
      float d;  // dx of this choice, apart from the softmax row term
      if (softmax && a.renormalize) {
        const float m = wave_all_max(some ? xl : -kInf);
        float e = some ? expf(xl - m) : 0.0f;
        e = e / fmaxf(wave_all_sum(e), 1.0f);  // the largest is e^0; 1 also where nothing is chosen
        d = e * (c - wave_all_sum(c * e));
      } else {
        float s = !some ? 0.0f : softmax ? expf(xl - r.top) * r.part : pointwise_score(xl, a.score);
        float ds = c, slope_l = some && !softmax ? score_slope(xl, s, a.score) : 0.0f;
        if (a.renormalize) {
          float sum = wave_all_sum(s);
          if (in_tail(sum, a.score)) {
            const float top = wave_all_max(some ? xl : -kInf), power = tail_power(a.score);
            s = some && top >= kTailEnd ? expf(power * (xl - top)) : 0.0f;
            slope_l = power * s;
            sum = wave_all_sum(s);
          }
          // by the weights' quotients s / sum: of a single choice exactly 1, and its gradient 0
          const float dot = wave_all_sum(c * (s / sum));
          ds = some && sum > 0.0f ? (c - dot) / sum : 0.0f;
        }
        if (softmax) {
          d = s * ds;
          inner = wave_all_sum(d);
        } else {
          d = some ? ds * slope_l : 0.0f;
        }
      }
      // an expert listed twice gets both gradients: every lane of it holds the sum
      float all = 0.0f;
      for (int j = 0; j < a.k; ++j) {
        const int other = __builtin_amdgcn_readlane(id, j);
        const float dj = lane_value(d, j);
        all += other == id ? dj : 0.0f;
      }
#pragma unroll
      for (int v = 0; v < VPT; ++v)
        if (v * 64 + lane < a.E) direct[v * 64 + lane] = 0.0f;
      wave_lds_fence();
      if (on) direct[id] = all;
      wave_lds_fence();
#pragma unroll
      for (int v = 0; v < VPT; ++v)
        if (v * 64 + lane < a.E) dx[v] = direct[v * 64 + lane];
    }
    float dq[VPT];
    float zc = 0.0f;
    if (in_loss) {
      const float n = (float)a.tokens[seq];
      const float f0 = a.d_loss[0] * (float)a.E / ((float)a.tokens[a.B + 1] * n * n * (float)a.k);
      float dot = 0.0f;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        dq[v] = f0 * (float)chosen[v];
        dot += dq[v] * q[v];  // q is 0 past E
      }
      dot = wave_all_sum(dot);
      zc = 2.0f * a.d_loss[1] * r.lse / (float)a.tokens[a.B];
      if (softmax) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) dx[v] += p[v] * (dq[v] - dot - inner + zc);
      } else {
#pragma unroll
        for (int v = 0; v < VPT; ++v) dx[v] += (dq[v] - dot) * r.inv * slope[v] + zc * p[v];
      }
    } else if (row_softmax) {
#pragma unroll
      for (int v = 0; v < VPT; ++v) dx[v] -= p[v] * inner;
    }
  }
#pragma unroll
  for (int v = 0; v < VPT; ++v)
    if (v * 64 + lane < a.E) store_logit(d_logits, row + v * 64 + lane, dx[v]);
}

}  // namespace nvfp4

using namespace nvfp4;

static int gate_check(const void* logits, int32_t dtype, int32_t T, int32_t E, int32_t k, int32_t score) {
  if (T < 0 || E < 1 || E > kGateMaxExperts || k < 1 || k > kGateMaxK || k > E) return NVFP4_ERR_SHAPE;
  if ((int64_t)T * k >= (1ll << 30) || T >= (1 << 26)) return NVFP4_ERR_SHAPE;  // 64 threads a token: a grid's limit
  if (dtype != NVFP4_DT_BF16 && dtype != NVFP4_DT_F32) return NVFP4_ERR_ARG;
  if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID && score != MOE_SCORE_SQRT_SOFTPLUS)
    return NVFP4_ERR_ARG;
  if (T > 0 && !logits) return NVFP4_ERR_NULL;
  if (T > 0 && !nvfp4_aligned16(logits)) return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

// Values per lane for E experts: the kernels are built for these.
template <typename Fn>
static int gate_by_width(int32_t E, Fn fn) {
  const int need = (E + 63) / 64;
  if (need <= 1) return fn(std::integral_constant<int, 1>());
  if (need <= 2) return fn(std::integral_constant<int, 2>());
  if (need <= 4) return fn(std::integral_constant<int, 4>());
  if (need <= 6) return fn(std::integral_constant<int, 6>());
  if (need <= 8) return fn(std::integral_constant<int, 8>());
  return fn(std::integral_constant<int, 16>());
}

extern "C" int moe_gate_topk(const void* logits, int32_t logits_dtype, const float* bias, const uint8_t* token_mask,
                             int32_t T, int32_t E, int32_t k, int32_t score, int32_t n_group, int32_t topk_group,
                             int32_t renormalize, float scale, int32_t* topk_ids, float* topk_w, void* stream) {
  const int st = gate_check(logits, logits_dtype, T, E, k, score);
  if (st) return st;
  if (n_group < 1 || n_group > 64 || E % n_group != 0 || topk_group < 1 || topk_group > n_group)
    return NVFP4_ERR_SHAPE;
  if (k > topk_group * (E / n_group)) return NVFP4_ERR_SHAPE;
  if (renormalize != 0 && renormalize != 1) return NVFP4_ERR_ARG;
  if (T == 0) return NVFP4_OK;
  if (!topk_ids || !topk_w) return NVFP4_ERR_NULL;
  if (!nvfp4_aligned16(topk_ids) || !nvfp4_aligned16(topk_w) || !nvfp4_aligned16(bias) ||
      !nvfp4_aligned16(token_mask))
    return NVFP4_ERR_ALIGN;
  const GateShape g = {T, E, k, score, n_group, topk_group, E / n_group, renormalize, scale};
  const unsigned grid = (unsigned)((T + kGateWaves - 1) / kGateWaves);
  const size_t lds = n_group > 1 || bias ? (size_t)kGateWaves * gate_keys_stride(E) * sizeof(double) : 0;
  return gate_by_width(E, [&](auto vpt) -> int {
    constexpr int VPT = decltype(vpt)::value;
    if (logits_dtype == NVFP4_DT_F32)
      hipLaunchKernelGGL((gate_topk_kernel<float, VPT>), dim3(grid), dim3(64 * kGateWaves), lds, (hipStream_t)stream,
                         reinterpret_cast<const float*>(logits), bias, token_mask, g, topk_ids, topk_w);
    else
      hipLaunchKernelGGL((gate_topk_kernel<uint16_t, VPT>), dim3(grid), dim3(64 * kGateWaves), lds,
                         (hipStream_t)stream, reinterpret_cast<const uint16_t*>(logits), bias, token_mask, g,
                         topk_ids, topk_w);
    NVFP4_CHECK_LAUNCH();
    return NVFP4_OK;
  });
}

// Tokens of one partial sum: 8, and more for batches of over 8192 tokens, so
// that the partial rows (8 E bytes each) stay a small part of the logits'
// bytes. (The whole call, 2048 x 384: 8 tokens 10.9 us, 16 11.6, 32 13.6;
// 16384 x 384 in 4 sequences: 16 tokens 16.2, 32 16.7.)
static int balance_chunk(int32_t T) {
  const int per = ((T + 1023) / 1024 + kGateWaves - 1) / kGateWaves * kGateWaves;
  return per < 8 ? 8 : per;
}
static size_t balance_layout(int32_t T, int32_t E, int32_t B, BalanceShape* g, char* base, BalanceWs* ws) {
  const int chunk = balance_chunk(T);
  const int max_chunks = (T + chunk - 1) / chunk + B;  // every sequence may end inside a chunk
  const int cols = (E + 15) / 16;  // column blocks, at most
  size_t p = 0;
  auto put = [&](size_t bytes) {
    char* at = base + p;
    p += nvfp4_align256(bytes);
    return at;
  };
  BalanceWs w;
  w.q = reinterpret_cast<float*>(put((size_t)max_chunks * E * 4));
  w.counts = reinterpret_cast<int32_t*>(put((size_t)max_chunks * E * 4));
  w.z = reinterpret_cast<double*>(put((size_t)max_chunks * 8));
  w.live = reinterpret_cast<int32_t*>(put((size_t)max_chunks * 4));
  w.term = reinterpret_cast<double*>(put((size_t)B * cols * 8));
  w.z_seq = reinterpret_cast<double*>(put((size_t)B * 8));
  if (g) {
    g->chunk = chunk;
    g->max_chunks = max_chunks;
  }
  if (ws) *ws = w;
  return p;
}

static bool balance_sizes_ok(int32_t T, int32_t E, int32_t B) {
  return T >= 0 && T < (1 << 30) && E >= 1 && E <= kGateMaxExperts && B >= 1 && B <= 65535;
}

extern "C" size_t moe_balance_loss_ws_bytes(int32_t T, int32_t E, int32_t B) {
  return balance_sizes_ok(T, E, B) ? balance_layout(T, E, B, nullptr, nullptr, nullptr) : 0;
}

extern "C" int moe_balance_loss(const void* logits, int32_t logits_dtype, const int32_t* topk_ids,
                                const uint8_t* token_mask, const int32_t* cu_seqlens, int32_t B, int32_t T, int32_t E,
                                int32_t k, int32_t score, float* loss, int32_t* counts, int32_t* tokens, void* ws,
                                size_t ws_bytes, void* stream) {
  const int st = gate_check(logits, logits_dtype, T, E, k, score);
  if (st) return st;
  if (!balance_sizes_ok(T, E, B) || (!cu_seqlens && B != 1)) return NVFP4_ERR_SHAPE;
  if ((T > 0 && !topk_ids) || !loss || !counts || !tokens || !ws) return NVFP4_ERR_NULL;
  if (!nvfp4_aligned16(topk_ids) || !nvfp4_aligned16(token_mask) || !nvfp4_aligned16(cu_seqlens) ||
      !nvfp4_aligned16(loss) || !nvfp4_aligned16(counts) || !nvfp4_aligned16(tokens) || !nvfp4_aligned16(ws))
    return NVFP4_ERR_ALIGN;
  BalanceShape g = {T, E, k, B, score, 0, 0};
  BalanceWs w;
  if (ws_bytes < balance_layout(T, E, B, &g, reinterpret_cast<char*>(ws), &w)) return NVFP4_ERR_WORKSPACE;
  const size_t lds = (size_t)(kGateWaves * 8 + 4) * E;
  return gate_by_width(E, [&](auto vpt) -> int {
    constexpr int VPT = decltype(vpt)::value;
    if (logits_dtype == NVFP4_DT_F32)
      hipLaunchKernelGGL((balance_partial_kernel<float, VPT>), dim3(g.max_chunks), dim3(64 * kGateWaves), lds,
                         (hipStream_t)stream, reinterpret_cast<const float*>(logits), topk_ids, token_mask,
                         cu_seqlens, g, w);
    else
      hipLaunchKernelGGL((balance_partial_kernel<uint16_t, VPT>), dim3(g.max_chunks), dim3(64 * kGateWaves), lds,
                         (hipStream_t)stream, reinterpret_cast<const uint16_t*>(logits), topk_ids, token_mask,
                         cu_seqlens, g, w);
    NVFP4_CHECK_LAUNCH();
    // Long sequences: more workgroups and waves over the same chunks (the whole
    // call, 16384 x 384: one sequence 17.3 us [otherwise 29.5], 4 sequences 16.1
    // [18.0]; short ones lose, 24 sequences: 21.5 [15.3]). By the mean length, as
    // the lengths are on the device: one sequence of 16016 tokens beside 23 of 16
    // takes 32.6 us, alone 19.9 (logits from memory).
    const bool tall = T / B >= 64 * g.chunk;
    const int cols = tall ? (E + 15) / 16 : (E + 63) / 64;
    if (tall)
      hipLaunchKernelGGL((balance_join_kernel<16, 16>), dim3(cols, B), dim3(1024), 0, (hipStream_t)stream, cu_seqlens,
                         g, w, counts, tokens, loss);
    else
      hipLaunchKernelGGL((balance_join_kernel<64, 4>), dim3(cols, B), dim3(256), 0, (hipStream_t)stream, cu_seqlens, g,
                         w, counts, tokens, loss);
    NVFP4_CHECK_LAUNCH();
    if (cols * B == 1) return NVFP4_OK;
    hipLaunchKernelGGL(balance_loss_kernel, dim3(1), dim3(64 * kLossWaves), 0, (hipStream_t)stream, g, w, cols, tokens,
                       loss);
    NVFP4_CHECK_LAUNCH();
    return NVFP4_OK;
  });
}

extern "C" int moe_gate_backward(const void* logits, int32_t logits_dtype, const int32_t* topk_ids,
                                 const uint8_t* token_mask, int32_t T, int32_t E, int32_t k, int32_t score,
                                 int32_t renormalize, float scale, const float* d_topk_w, const float* d_loss,
                                 const int32_t* counts, const int32_t* tokens, const int32_t* cu_seqlens, int32_t B,
                                 void* d_logits, void* stream) {
  const int st = gate_check(logits, logits_dtype, T, E, k, score);
  if (st) return st;
  if (renormalize != 0 && renormalize != 1) return NVFP4_ERR_ARG;
  if (T > 0 && !d_topk_w && !d_loss) return NVFP4_ERR_NULL;
  if (d_loss && (!balance_sizes_ok(T, E, B) || (!cu_seqlens && B != 1))) return NVFP4_ERR_SHAPE;
  if (T == 0) return NVFP4_OK;
  if (!d_logits || (d_topk_w && !topk_ids) || (d_loss && (!counts || !tokens))) return NVFP4_ERR_NULL;
  if (!nvfp4_aligned16(topk_ids) || !nvfp4_aligned16(token_mask) || !nvfp4_aligned16(d_topk_w) ||
      !nvfp4_aligned16(d_loss) || !nvfp4_aligned16(counts) || !nvfp4_aligned16(tokens) ||
      !nvfp4_aligned16(cu_seqlens) || !nvfp4_aligned16(d_logits))
    return NVFP4_ERR_ALIGN;
  const GateGradArgs a = {topk_ids, d_topk_w, d_loss, counts, tokens, cu_seqlens, token_mask,
                          T, E, k, B, score, renormalize, scale};
  const unsigned grid = (unsigned)((T + kGateWaves - 1) / kGateWaves);
  const size_t lds = d_topk_w ? (size_t)kGateWaves * E * 4 : 0;
  return gate_by_width(E, [&](auto vpt) -> int {
    constexpr int VPT = decltype(vpt)::value;
    if (logits_dtype == NVFP4_DT_F32)
      hipLaunchKernelGGL((gate_backward_kernel<float, VPT>), dim3(grid), dim3(64 * kGateWaves), lds,
                         (hipStream_t)stream, reinterpret_cast<const float*>(logits), a,
                         reinterpret_cast<float*>(d_logits));
    else
      hipLaunchKernelGGL((gate_backward_kernel<uint16_t, VPT>), dim3(grid), dim3(64 * kGateWaves), lds,
                         (hipStream_t)stream, reinterpret_cast<const uint16_t*>(logits), a,
                         reinterpret_cast<uint16_t*>(d_logits));
    NVFP4_CHECK_LAUNCH();
    return NVFP4_OK;
  });
}
