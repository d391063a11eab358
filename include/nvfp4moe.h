/*
 * nvfp4moe — NVFP4 mixture-of-experts expert FFN on AMD Instinct MI355X (gfx950).
 *
 * C ABI of libnvfp4moe.so. The layer runs in six steps (tests history of the
 * nvfp4-megamoe-kernel project, moe_pipeline commit): quantize the BF16
 * activation to NVFP4; L1 grouped GEMM (gate+up); SiLU(gate)*up, re-quantized;
 * L2 grouped GEMM (down_proj); weighted scatter back to token rows.
 *
 * NVFP4 storage used throughout:
 *   - values: E2M1 nibbles, bit 3 = sign, bits 2:0 index {0,0.5,1,1.5,2,3,4,6};
 *     two per byte along K, element 2j in the low nibble of byte j;
 *     a [rows, K] tensor is stored as uint8 [rows, K/2], row-major;
 *   - block scales: one E4M3 (float8_e4m3fn) bit pattern per 16 consecutive
 *     K elements, uint8 [rows, K/16], row-major, never negative, at most 448;
 *   - global scale: float32 gs = amax / 2688 (= 6 * 448) per tensor;
 *     value = E2M1(nibble) * E4M3(scale) * gs.
 * BF16 tensors are passed as raw 16-bit patterns (void*).
 *
 * Conventions for every entry point:
 *   - Pointers are device pointers unless marked (host). The caller owns all
 *     memory; the library never allocates or frees memory, holds no data from
 *     one call to the next, and reads no environment variables. Its only
 *     process-wide state is launch sizes that depend on the device alone (CU
 *     count times resident workgroups per CU), queried on the first call on
 *     each device and kept per device, and the device array (with its address
 *     per device) that nvfp4_quantize_noalloc uses in place of a workspace.
 *   - Calls are asynchronous on `stream` (a hipStream_t; NULL = the default
 *     stream) and never synchronize with the host.
 *   - Every entry point that launches work returns an int: NVFP4_OK (0) or
 *     one of the nvfp4_status codes below (declared int so that the ABI does
 *     not depend on the size of an enum).
 *   - Arguments are validated on the host before anything is launched; a
 *     rejected call returns a nonzero status and launches nothing. A launch
 *     failure returns NVFP4_ERR_HIP (the error is taken with hipGetLastError,
 *     without synchronizing).
 *   - Data-dependent conditions are not errors: expert ids outside this
 *     rank's range are dropped, and zero local slots give a zero output.
 *   - Device pointers must be 16-byte aligned; floating-point inputs finite.
 *   - Calls that share no output buffers may run concurrently.
 */
#ifndef NVFP4MOE_H
#define NVFP4MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  NVFP4_OK = 0,
  NVFP4_ERR_NULL = 1,       /* a required pointer is NULL */
  NVFP4_ERR_SHAPE = 2,      /* a size is negative, zero where it must not be, or not a multiple it must be */
  NVFP4_ERR_ALIGN = 3,      /* a device pointer is not 16-byte aligned */
  NVFP4_ERR_WORKSPACE = 4,  /* workspace smaller than the matching *_ws_bytes() */
  NVFP4_ERR_HIP = 5,        /* a kernel launch failed */
  NVFP4_ERR_ARG = 6         /* an enum or option value is unknown */
} nvfp4_status;

/* Static description of a status code (host). */
const char* nvfp4_status_string(int status);

/* Library version as major*10000 + minor*100 + patch (host). */
int nvfp4moe_version(void);

/* ---------------------------------------------------------------- quantize
 * Activation/weight quantizer (nvfp4_mega_moe.py history: overflow-fix commit,
 * alpha commit and three-quantizer-bugs commit; tests history: packing along K).
 *
 * x_bf16 holds B independent tensors, each [M, K] BF16 row-major
 * (B*M*K elements). Tensor b gets its own global scale:
 *   amax_b = max |x_b|   (or amax_in[b] when amax_in != NULL)
 *   gs_b   = RN_f32(amax_b / 2688)                         -> gs_out[b]
 * and for every row and 16-element block with bmax = max |x| in the block:
 *   sf     = nearest E4M3 to bmax / (6 gs_b), ties to even, saturating at 448
 *   nibble = sign bit of x | nearest E2M1 magnitude index of |x| / (E4M3(sf) gs_b),
 *            ties to the even index, saturating at 6; magnitude 0 where sf == 0
 * Both roundings are decided exactly (as on the real quotient). amax == 0 gives
 * gs = 0, sf = 0 and magnitude 0.
 *   q  : uint8 [B, M, K/2]    sf : uint8 [B, M, K/16]    gs_out : float [B]
 *   amax_in : float [B] or NULL (device; the h path passes the L1 epilogue's amax)
 *   ws : scratch of at least nvfp4_quantize_ws_bytes(B, M, K) bytes: the
 *        per-workgroup amax partials, a fixed number per tensor, so the size
 *        depends on B alone (M and K are accepted for a stable signature)
 * Requires B >= 1, M >= 0, K > 0, K % 32 == 0.
 */
size_t nvfp4_quantize_ws_bytes(int64_t B, int64_t M, int64_t K);
int nvfp4_quantize(const void* x_bf16, int64_t B, int64_t M, int64_t K, const float* amax_in,
                   uint8_t* q, uint8_t* sf, float* gs_out, void* ws, size_t ws_bytes, void* stream);

/* nvfp4_quantize for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc):
 * the same arguments, results, kernels and launches without the workspace.
 * The amax partials live in a device array of the library, 256 KB on each
 * device it runs on (allocated when the library's code is loaded there, kept
 * until the process ends); its address is taken on the first call on a device.
 * The call allocates and frees nothing. Calls on one device share that array,
 * so calls that overlap on one device (concurrent streams, threads) race;
 * with amax_in != NULL the array is not used. Requires B <= 128 (more tensors
 * return NVFP4_ERR_WORKSPACE) and otherwise what nvfp4_quantize requires.
 */
int nvfp4_quantize_noalloc(const void* x_bf16, int64_t B, int64_t M, int64_t K, const float* amax_in,
                           uint8_t* q, uint8_t* sf, float* gs_out, void* stream);

/* Quantize with fixed global scales (nvfp4_cutedsl.py history, page 2,
 * static-scale commit: a warmup pass measures gs once; afterwards activations
 * are quantized with that gs and no max reduction). As nvfp4_quantize with
 * gs_b = gs_in[b] (device float [B], finite and >= 0; 0 gives all zeros), no
 * amax pass and no workspace. Where |x| exceeds 2688 * gs_b the block scale
 * saturates at 448 and magnitudes at 6. One launch.
 * Requires 1 <= B <= 65535, M >= 0, K > 0, K % 32 == 0.
 */
int nvfp4_quantize_static(const void* x_bf16, int64_t B, int64_t M, int64_t K, const float* gs_in,
                          uint8_t* q, uint8_t* sf, void* stream);

/* ------------------------------------------------------------------- route
 * Slot routing for one rank's share of experts (nvfp4_mega_moe.py history:
 * local-expert-id commit; src history: one 1-D slot order for both GEMMs;
 * nvfp4_cutedsl.py history: bincount/cumsum int32 offsets and sort by expert).
 *
 * topk_ids int32 [T, k] are global expert ids; local = id - expert_start is
 * kept when 0 <= local < num_local and dropped otherwise. S = number of kept
 * (t, j) pairs. Slots are ordered by (local expert, t*k + j):
 *   counts      int32 [num_local]     kept pairs per local expert
 *   offsets     int32 [num_local + 1] exclusive prefix sum; offsets[num_local] = S
 *   slot_token  int32 [T*k]  token of slot s, -1 for s >= S
 *   slot_expert int32 [T*k]  local expert of slot s, -1 for s >= S
 *   slot_weight float [T*k]  topk_w of slot s, 0 for s >= S
 *   token_slot  int32 [T*k]  slot of pair t*k + j, -1 when dropped
 *   tile_table  int32 [nvfp4_tile_table_len(T*k, num_local, tile_m)]
 *               [0] = n tiles; then n pairs (expert, first slot): expert e
 *               contributes ceil(counts[e] / tile_m) tiles starting at
 *               offsets[e], offsets[e] + tile_m, ... in expert order.
 * ws: at least moe_route_ws_bytes(T, k, num_local) bytes.
 * Requires T >= 0, 1 <= k <= 64, 1 <= num_local <= 4096, tile_m a multiple of 16 in [16, 256],
 * T*k < 2^30.
 */
size_t moe_route_ws_bytes(int32_t T, int32_t k, int32_t num_local);
int64_t nvfp4_tile_table_len(int64_t slot_capacity, int32_t num_local, int32_t tile_m);
int moe_route_slots(const int32_t* topk_ids, const float* topk_w, int32_t T, int32_t k,
                    int32_t expert_start, int32_t num_local, int32_t tile_m,
                    int32_t* counts, int32_t* offsets, int32_t* slot_token, int32_t* slot_expert,
                    float* slot_weight, int32_t* token_slot, int32_t* tile_table,
                    void* ws, size_t ws_bytes, void* stream);

/* -------------------------------------------------------------------- gate
 * The routing gate in front of moe_route_slots: expert ids and weights from
 * router logits [T, E] (row-major, BF16 or float; each finite, or -inf for an
 * expert the token must not use). E <= 1024, 1 <= k <= min(E, 64), T < 2^26,
 * T*k < 2^30. In this section and the next outputs and workspaces
 * overlap neither inputs nor each other, except where it is said.
 *
 *   score  MOE_SCORE_SOFTMAX        s = softmax over the row
 *          MOE_SCORE_SIGMOID        s = 1 / (1 + e^-x)
 *          MOE_SCORE_SQRT_SOFTPLUS  s = sqrt(log(1 + e^x))
 *   key    s + bias[e] (float [E] or NULL), compared as float64 numbers; with
 *          neither bias nor groups the logit itself (the same order)
 *   groups the experts form n_group runs of E / n_group (n_group <= 64). A
 *          group's value is the sum of its two highest keys (one key where it
 *          has one); the topk_group highest groups stay (ties: lower group).
 *          k <= topk_group * E / n_group.
 *   choice the k highest keys of the row, highest first, ties to the lower id:
 *            topk_ids int32 [T, k],
 *            topk_w   float [T, k] = scale * s, or with renormalize = 1
 *                     scale * s / (sum of the k scores), 0 if that sum is 0.
 *          A score that is divided by a sum of scores, here and in the balance
 *          loss, may lie far below float32's range; where all logits of the sum
 *          are under -708, about where float64 ends, it counts as 0.
 * Where fewer than k experts can be chosen the rest is id -1, weight 0 (and
 * dropped by moe_route_slots). token_mask (uint8 [T] or NULL): tokens with
 * mask 0 get ids -1 and weights 0, and their logits are not used (any bits).
 * One launch.
 */
enum { NVFP4_DT_BF16 = 0, NVFP4_DT_F32 = 1 };
enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1, MOE_SCORE_SQRT_SOFTPLUS = 2 };
int moe_gate_topk(const void* logits, int32_t logits_dtype, const float* bias, const uint8_t* token_mask,
                  int32_t T, int32_t E, int32_t k, int32_t score, int32_t n_group, int32_t topk_group,
                  int32_t renormalize, float scale, int32_t* topk_ids, float* topk_w, void* stream);

/* Balance loss of the choices, and how often each expert was chosen.
 * cu_seqlens int32 [B + 1] (device, nondecreasing, within [0, T]): sequence b
 * is tokens [cu[b], cu[b+1]); tokens in no sequence do not count. NULL with
 * B = 1: all T tokens. B <= 65535. A token is live when its mask is not 0 and
 * one of its logits is above -inf; N_b = live tokens of sequence b.
 *   counts int32 [B, E]   pairs (t, j) of live tokens with topk_ids[t, j] = e
 *                         (ids outside [0, E) are skipped)
 *   tokens int32 [B + 2]  N_0 .. N_{B-1}, their sum N, and the number B' of
 *                         sequences with N_b > 0
 *   loss   float [2]      [0] mean over those sequences of
 *                             E * sum_e (counts_be / (N_b k)) * (sum_t q_te / N_b),
 *                             q = s / (row sum of s)
 *                         [1] mean over the N live tokens of logsumexp(x_t)^2
 *                         (0 where there is nothing to average)
 * ws: at least moe_balance_loss_ws_bytes(T, E, B) bytes (0 for sizes that are
 * refused). Two or three launches; the result does not depend on their timing.
 */
size_t moe_balance_loss_ws_bytes(int32_t T, int32_t E, int32_t B);
int moe_balance_loss(const void* logits, int32_t logits_dtype, const int32_t* topk_ids, const uint8_t* token_mask,
                     const int32_t* cu_seqlens, int32_t B, int32_t T, int32_t E, int32_t k, int32_t score,
                     float* loss, int32_t* counts, int32_t* tokens, void* ws, size_t ws_bytes, void* stream);

/* Gradient of the logits, d_logits [T, E] (the logits' type, every element
 * written), as the sum of
 *   - the gradient through the weights, when d_topk_w (float [T, k]) is given:
 *     topk_ids, score, renormalize and scale as in moe_gate_topk; the choice
 *     itself is constant. Ids outside [0, E) take no part; an expert listed
 *     twice gets both gradients;
 *   - the gradient of the losses, when d_loss (float [2], device) is given:
 *     d_loss[i] times that of loss[i], with counts, tokens, cu_seqlens and B
 *     from moe_balance_loss of the same logits, ids and mask (the counts are
 *     constant; topk_ids may be NULL when d_topk_w is).
 * At least one of the two is needed. Rows of masked tokens are 0. One launch.
 */
int moe_gate_backward(const void* logits, int32_t logits_dtype, const int32_t* topk_ids, const uint8_t* token_mask,
                      int32_t T, int32_t E, int32_t k, int32_t score, int32_t renormalize, float scale,
                      const float* d_topk_w, const float* d_loss, const int32_t* counts, const int32_t* tokens,
                      const int32_t* cu_seqlens, int32_t B, void* d_logits, void* stream);

/* ------------------------------------------------------- norms of the block
 * The residual update behind one block and the norm in front of the next, in
 * one pass (around this layer: x its output, y its next input):
 *   n  = x * rsqrt(mean(x^2) + eps) * w_post     (w_post NULL: n = x)
 *   r' = residual + scale * gate * n             -> residual_out, rounded once
 *   y  = r' * rsqrt(mean(r'^2) + eps) * w_pre    -> y, from r' as stored
 * x, y [T, H] of x_dtype; residual (NULL: zeros), residual_out [T, H] of
 * res_dtype (NVFP4_DT_*, any combination); w_pre, w_post float [H]; gate float
 * [H] (MOE_GATE_CHANNEL), [T] (MOE_GATE_TOKEN) or unused (MOE_GATE_NONE, 1).
 * w_pre NULL: no y. residual_out may be residual, y may be x. Sums in float32.
 * gs_in (float [1], device) writes y as NVFP4 too: y_q uint8 [T, H/2], y_sf
 * uint8 [T, H/16], exactly what nvfp4_quantize_static makes of the BF16 y; it
 * needs w_pre, x_dtype BF16 and H % 32 == 0, and y may then be NULL.
 * Requires T >= 0, 0 < H <= 16384, H % 8 == 0. One launch.
 */
enum { MOE_GATE_NONE = 0, MOE_GATE_CHANNEL = 1, MOE_GATE_TOKEN = 2 };
int moe_block_norm(const void* x, int32_t x_dtype, const void* residual, int32_t res_dtype, int32_t T, int32_t H,
                   const float* w_pre, const float* w_post, const float* gate, int32_t gate_mode, float scale,
                   float eps, void* residual_out, void* y, const float* gs_in, uint8_t* y_q, uint8_t* y_sf,
                   void* stream);

/* Its gradients. d_y [T, H] of x_dtype (needed with w_pre), d_residual_out
 * [T, H] of res_dtype (the gradient of r' from elsewhere; NULL: zeros; needed
 * without w_pre); x and residual_out as moe_block_norm read and left them (the
 * rounding of r' counts as the identity).
 *   d_x [T, H] of x_dtype, d_residual [T, H] of res_dtype (may be d_y and
 *   d_residual_out where the types agree); float d_w_pre [H] (with w_pre),
 *   d_w_post [H] (with w_post), d_gate [H] or [T] (by gate_mode).
 * ws: at least moe_block_norm_backward_ws_bytes(T, H) bytes. Sums over tokens
 * have a fixed order. Two launches.
 */
size_t moe_block_norm_backward_ws_bytes(int32_t T, int32_t H);
int moe_block_norm_backward(const void* d_y, const void* d_residual_out, const void* x, int32_t x_dtype,
                            const void* residual_out, int32_t res_dtype, int32_t T, int32_t H, const float* w_pre,
                            const float* w_post, const float* gate, int32_t gate_mode, float scale, float eps,
                            void* d_x, void* d_residual, float* d_w_pre, float* d_w_post, float* d_gate, void* ws,
                            size_t ws_bytes, void* stream);

/* Layer norm with the residual update in front of it, for blocks that centre:
 *   r' = residual + scale * x                        -> residual_out, rounded once
 *   y  = (r' - mean r') * rsqrt(var r' + eps) * w + b    -> y, from r' as stored
 * x, y [T, H] of x_dtype; residual, residual_out [T, H] of res_dtype (any
 * combination); w, b float [H] (NULL: 1, 0). residual NULL: r' = x, which is not
 * written (residual_out NULL, scale 1, res_dtype x_dtype). residual_out may be
 * residual, y may be x. var is the mean squared deviation; sums in float32, of
 * deviations from the mean, so rows far from 0 keep their digits.
 * y_q, y_scale (both or neither) take y as MXFP4 too, exactly what mxfp4_quantize
 * makes of the stored y by `rule` (MX_SCALE_*): [T, Hp/2], [Hp/128, T, 4], Hp =
 * mxfp4_padded(H); y may then be NULL (its values are those it would have). An
 * infinity or NaN in a row makes all of its y NaN.
 * Requires T >= 0, 0 < H <= 16384, H % 8 == 0. One launch.
 */
int moe_layer_norm(const void* x, int32_t x_dtype, const void* residual, int32_t res_dtype, int32_t T, int32_t H,
                   const float* w, const float* b, float scale, float eps, void* residual_out, void* y, int32_t rule,
                   uint8_t* y_q, uint8_t* y_scale, void* stream);

/* Its gradients. d_y [T, H] of x_dtype; r [T, H] of res_dtype, the r' that was
 * normalized; d_residual_out [T, H] of res_dtype (the gradient of r' from
 * elsewhere; NULL: zeros). The rounding of r' counts as the identity.
 *   d_residual [T, H] of res_dtype, d_x = scale * d_residual [T, H] of x_dtype
 *   (may be d_residual_out and d_y where the types agree); without a residual
 *   d_residual is NULL, and scale and types as there
 *   float d_w [H], d_b [H]; NULL where not wanted
 * ws: at least moe_layer_norm_backward_ws_bytes(T, H) bytes. Sums over tokens
 * have a fixed order. Two launches.
 */
size_t moe_layer_norm_backward_ws_bytes(int32_t T, int32_t H);
int moe_layer_norm_backward(const void* d_y, int32_t x_dtype, const void* d_residual_out, const void* r,
                            int32_t res_dtype, int32_t T, int32_t H, const float* w, float scale, float eps, void* d_x,
                            void* d_residual, float* d_w, float* d_b, void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------- weight packing
 * Offline weight preparation, step three (after quantize and fold): the
 * grouped GEMM reads weights in a packed order that matches its MFMA operand
 * fragments, so that every load instruction of a wave reads one contiguous
 * 1 KB (or 256 B) block. Packing is a byte permutation of (q, sf); nothing is
 * rounded. (Layout of this library's own design; the NVFP4 values and scales
 * are those of nvfp4_quantize.)
 *
 * Input: B matrices, q uint8 [B, N, K/2] and sf uint8 [B, N, K/16], row-major.
 * Output: packed uint8 [B][N/32][K/128][2304], one 2304-byte chunk per
 * (matrix b, 32-row subtile t, 128-element K stage c):
 *   chunk[h*1024 + 16*l + i] = q [b, 32t + l%32, 64c + 32*(l/32) + 16h + i]
 *                                           h in {0,1}, l in [0,64), i in [0,16)
 *   chunk[2048 + 4*l + i]    = sf[b, 32t + l%32, 8c + 4*(l/32) + i]        i in [0,4)
 * Size: nvfp4_packed_bytes(B, N, K) = B * N * K * 9/16 bytes (same as q + sf).
 * Requires B >= 0, N % 32 == 0, K % 128 == 0; nvfp4_packed_bytes returns -1 otherwise.
 */
int64_t nvfp4_packed_bytes(int64_t B, int64_t N, int64_t K);
int nvfp4_pack_weights(const uint8_t* q, const uint8_t* sf, int64_t B, int64_t N, int64_t K,
                       uint8_t* packed, void* stream);

/* ------------------------------------------------------------ grouped GEMM
 * NVFP4 x NVFP4 grouped GEMM over slot rows (nvfp4_mega_moe.py history: alpha
 * commit; src history: 1-D slot ids, gather only for L1; tests history:
 * [expert0 | expert1 | ...] row layout for the 2-D x 3-D grouped GEMM).
 *
 * For every tile (e, r0) of tile_table and every slot row s in
 * [r0, min(r0 + tile_m, offsets[e+1])):
 *   a = a_row_index ? a_row_index[s] : s          (L1 gathers token rows)
 *   G[s, n] = alpha_e * sum_k A_hat[a, k] * W_hat_e[n, k],  alpha_e = RN_f32(a_gs[0] * b_gs[e])
 * with A_hat, W_hat the exact dequantized values without global scale and the
 * sum in float32.
 *   a_q uint8 [*, K/2], a_sf uint8 [*, K/16] (row-major NVFP4);
 *   b_packed: the L expert matrices W_e [N, K] packed by nvfp4_pack_weights (B = L);
 *   a_gs float [1]; b_gs float [L]; offsets int32 [L+1]; tile_table as from moe_route_slots
 *   with the same tile_m; rows_cap = capacity of the row arrays (tile_table holds at
 *   most nvfp4_tile_table_len(rows_cap, L, tile_m) entries).
 * epilogue NVFP4_EPI_BF16:        d = BF16 [rows_cap, N], d[s, n] = RN_bf16(G[s, n]).
 * epilogue NVFP4_EPI_SILU_MUL:    N = 2*I (gate rows [0, I), up rows [I, 2I) of W_e;
 *   nvfp4_cutedsl.py history, intermediate-split commit), d = BF16 [rows_cap, I],
 *   g = RN_bf16(G[s, n]), u = RN_bf16(G[s, I + n]), d[s, n] = RN_bf16(silu(g) * u)
 *   with silu(g) = g / (1 + exp(-g)) in float32; amax_out[0] is raised (atomic max)
 *   to max |d| over the rows written, so the caller sets it to 0 first.
 * epilogue NVFP4_EPI_SILU_MUL_DUAL: as NVFP4_EPI_SILU_MUL for an L1 weight whose gate and
 *   up halves keep their own global scales (no nvfp4_fold_scales): b_gs is float [L, 2]
 *   = (gs_gate, gs_up) and the gate columns take alpha = RN_f32(a_gs[0] * b_gs[e][0]), the up
 *   columns RN_f32(a_gs[0] * b_gs[e][1]) (the alpha commit's global-scale treatment applied to
 *   each half, instead of the finalize_weights fold).
 * Activation row indices must satisfy (row + 1) * K/2 < 2^31, as must rows_cap * K/2,
 * N * K * 9/16 and 256 * N (32-bit buffer offsets); NVFP4_ERR_SHAPE otherwise.
 * Only rows of listed tiles are written. Requires K % 128 == 0, N % 64 == 0
 * (N % 128 == 0 for NVFP4_EPI_SILU_MUL), 1 <= L, tile_m 32 (decode-shaped
 * batches), 64, 96 (prefill-shaped) or 128 (large groups).
 */
enum { NVFP4_EPI_BF16 = 0, NVFP4_EPI_SILU_MUL = 1, NVFP4_EPI_SILU_MUL_DUAL = 2 };
int nvfp4_grouped_gemm(const uint8_t* a_q, const uint8_t* a_sf, const int32_t* a_row_index,
                       const float* a_gs, const uint8_t* b_packed, const float* b_gs,
                       const int32_t* offsets, const int32_t* tile_table, int32_t num_local,
                       int32_t rows_cap, int32_t N, int32_t K, int32_t tile_m, int32_t epilogue,
                       void* d, float* amax_out, void* stream);

/* L1 with h written as NVFP4: the NVFP4_EPI_SILU_MUL (dual_gs = 0) or
 * NVFP4_EPI_SILU_MUL_DUAL (dual_gs = 1) GEMM, whose BF16 h[s, n] is quantized
 * in the epilogue with the fixed global scale out_gs[0] (device float [1]) by
 * exactly the rules of nvfp4_quantize_static: d_q uint8 [rows_cap, N/4],
 * d_sf uint8 [rows_cap, N/32] (h = [rows_cap, N/2] row-major, 16-column
 * blocks). This fuses the re-quantization of h into L1 once gs_h is fixed
 * (nvfp4_cutedsl.py history, static-scale commit); no BF16 h and no amax are
 * written. Same shapes, tile heights and limits as nvfp4_grouped_gemm with
 * N % 128 == 0; d_q 16-byte aligned.
 */
int nvfp4_grouped_gemm_silu_nvfp4(const uint8_t* a_q, const uint8_t* a_sf, const int32_t* a_row_index,
                                  const float* a_gs, const uint8_t* b_packed, const float* b_gs, int32_t dual_gs,
                                  const int32_t* offsets, const int32_t* tile_table, int32_t num_local,
                                  int32_t rows_cap, int32_t N, int32_t K, int32_t tile_m, const float* out_gs,
                                  uint8_t* d_q, uint8_t* d_sf, void* stream);

/* ------------------------------------------------- 8-bit integer products
 * Row quantizer: for each row m of x [M, K] (BF16 or float, row-major)
 *   scale[m] = RN_f32(max_k |x[m, k]| * RN_f32(1 / 127))
 *   q[m, k]  = the integer nearest to x[m, k] / scale[m], ties to even (as on
 *              the real quotient), at most 127 in size; 0 where scale is 0.
 * x finite; q int8 [M, K]; scale float [M]. For activations a row is a token,
 * for weights [N, K] an output channel. K % 16 == 0, 0 < K <= 65536,
 * M <= 64 * 65535. One launch. In this section outputs and
 * workspaces overlap neither inputs nor each other, except where it is said.
 */
int int8_quantize_rows(const void* x, int32_t x_dtype, int32_t M, int32_t K, int8_t* q, float* scale, void* stream);

/* G[m, n] = a_scale[m] * b_scale[n] * sum_k a_q[m, k] * b_q[n, k], the sum
 * exact, the rest in float32. a_q int8 [M, K] with a_scale float [M], b_q int8
 * [N, K] with b_scale float [N], all row-major.
 * epilogue NVFP4_EPI_BF16:     d BF16 [M, N], d = RN_bf16(G [+ add]); N % 8 == 0
 * epilogue NVFP4_EPI_SILU_MUL: gate rows [0, I), up rows [I, 2I) of b_q, N = 2I:
 *   d BF16 [M, I], d = RN_bf16(silu(G[m, n]) * G[m, I + n] [+ add]); I % 8 == 0
 * add: BF16 of d's shape, or NULL; may be d itself. K % 16 == 0, K <= 65536,
 * M <= 64 * 65535, N <= 2^27 - 16. ws: at least int8_gemm_ws_bytes(M, N, K) bytes (the sums of
 * the parts of K where few tokens split it; 0 otherwise, then ws may be NULL).
 * A token's outputs have the same bits whichever other tokens M holds. One
 * launch, or two with parts.
 */
size_t int8_gemm_ws_bytes(int32_t M, int32_t N, int32_t K);
int int8_gemm(const int8_t* a_q, const float* a_scale, const int8_t* b_q, const float* b_scale, int32_t M, int32_t N,
              int32_t K, int32_t epilogue, const void* add_bf16, void* d_bf16, void* ws, size_t ws_bytes,
              void* stream);

/* Dense (shared) expert FFN in 8-bit integers: quantize x, the gate+up product
 * with the SiLU epilogue into BF16 h, quantize h, the down product, and add:
 *   out[t] = RN_bf16(w2 (silu(w1_gate x[t]) * (w1_up x[t])) + add[t])
 * w1_q int8 [2I, H] (gate rows, then up rows) with w1_scale [2I]; w2_q int8
 * [H, I] with w2_scale [H]; x, out BF16 [T, H]; add BF16 [T, H] (such as the
 * output of nvfp4_moe_forward; may be out) or NULL. H % 16 == 0, I % 16 == 0,
 * both <= 65536, T <= 64 * 65535. ws: at least int8_ffn_ws_bytes(T, H, I).
 * Exactly what the functions above give in sequence. Four to six launches.
 */
size_t int8_ffn_ws_bytes(int32_t T, int32_t hidden, int32_t inter);
int int8_ffn_forward(const int8_t* w1_q, const float* w1_scale, const int8_t* w2_q, const float* w2_scale,
                     const void* x_bf16, int32_t T, int32_t hidden, int32_t inter, const void* add_bf16,
                     void* out_bf16, void* ws, size_t ws_bytes, void* stream);

/* --------------------------------------- microscaled 4-bit floats (MXFP4)
 * E2M1 codes, two to a byte (the first in the low nibble), and for each 32
 * elements of a row one power of two, a byte holding its exponent + 127 (0xFF:
 * the block's values are NaN). A matrix [R, C] is kept with C padded to
 * Cp = mxfp4_padded(C), whole groups of 128, with codes and scales of 0:
 *   q uint8 [R, Cp/2];  scale uint8 [Cp/128, R, 4], scale[c, r, i] that of the
 *   elements [128c + 32i, +32) of row r
 * (row-major scales uint8 [R, Cp/32] are their view [R, Cp/128, 4] with the first
 * two axes exchanged).
 */
enum { MX_SCALE_FLOOR = 0, MX_SCALE_CEIL = 1 };
int32_t mxfp4_padded(int32_t n);  /* -1 outside [0, 262144] */

/* Quantizer of x [M, K] (BF16 or float, row-major), along its rows (q, scale:
 * [M, Kp/2], [Kp/128, M, 4]), along its columns (q_t, scale_t: the transposed
 * matrix, [K, Mp/2], [Mp/128, K, 4]), or both from one read; the pair that is not
 * wanted is NULL. Of a block with largest magnitude a > 0:
 *   MX_SCALE_FLOOR: e = floor(log2 a) - 2; values above 6 * 2^e become 6 * 2^e
 *   MX_SCALE_CEIL:  the smallest e with a <= 6 * 2^e
 * but at least -127 (also for a = 0); q = E2M1 nearest to x / 2^e, ties to the
 * even code, both exactly. A block with an infinity or NaN gets the scale 0xFF.
 * K % 8 == 0, 0 < K <= 262144; M <= 64 * 65535, along the columns <= 262144.
 * Outputs overlap neither x nor each other. One launch.
 */
int mxfp4_quantize(const void* x, int32_t x_dtype, int32_t M, int32_t K, int32_t rule, uint8_t* q, uint8_t* scale,
                   uint8_t* q_t, uint8_t* scale_t, void* stream);

/* out [R, cols] (BF16 or float) = the values of the first cols columns of q
 * [R, K/2], scale [K/128, R, 4]. Every one of them has its value in BF16 except
 * those past its range, which become infinite. K % 128 == 0, K <= 262144, cols <= K,
 * R <= 64 * 65535, R * cols below 2^38 (float 2^37). One launch.
 */
int mxfp4_dequantize(const uint8_t* q, const uint8_t* scale, int32_t R, int32_t K, int32_t cols, int32_t out_dtype,
                     void* out, void* stream);

/* G[m, n] = sum_k A[m, k] B[n, k] of the values of a_q [M, K/2], a_scale
 * [K/128, M, 4] and b_q [N, K/2], b_scale [K/128, N, 4]; products exact, sums in
 * float32 (a product under its normal numbers, 2^-126, may count as 0).
 * epilogue NVFP4_EPI_BF16:     d [M, N] of d_dtype, d = RN(G [+ add]); N % 8 == 0
 * epilogue NVFP4_EPI_SILU_MUL: gate rows [0, I), up rows [I, 2I) of B, N = 2I:
 *   d BF16 [M, I], d = RN(silu(G[m, n]) * G[m, I + n] [+ add]); I % 8 == 0;
 *   silu(g) = g / (1 + e^-g) by e^-|g| in float32: under 2^-126 (|g| > 87.3)
 *   with fewer digits, from |g| = 104 on 0
 * add: of d's type and shape, or NULL; may be d itself. K % 128 == 0, K <= 262144
 * (K = 0: d = add, or 0), M <= 64 * 65535, N <= 2^27 - 16, M * K and N * K below
 * 2^36. ws: at least mxfp4_gemm_ws_bytes(M, N, K) bytes (sums of the parts of K
 * where few tokens split it; 0 otherwise, then ws may be NULL). The order of a
 * sum depends on M, N and K alone, so calls repeat bit for bit. One launch, or
 * two with parts. Outputs and workspaces overlap neither inputs nor each other,
 * except where it is said.
 */
size_t mxfp4_gemm_ws_bytes(int32_t M, int32_t N, int32_t K);
int mxfp4_gemm(const uint8_t* a_q, const uint8_t* a_scale, const uint8_t* b_q, const uint8_t* b_scale, int32_t M,
               int32_t N, int32_t K, int32_t epilogue, const void* add, int32_t d_dtype, void* d, void* ws,
               size_t ws_bytes, void* stream);

/* ------------------------------------------------------- weighted scatter
 * out[t, :] = RN_bf16( sum over j = 0..k-1 with token_slot[t*k+j] >= 0 of
 *                      topk_w[t, j] * y[token_slot[t*k+j], :] ), float32, increasing j;
 * 0 for tokens with no local pair (nvfp4_cutedsl.py history: scatter with routing
 * weights; made order-fixed). y BF16 [*, H]; out BF16 [T, H]; H % 8 == 0.
 */
int moe_weighted_scatter(const void* y_bf16, const int32_t* token_slot, const float* topk_w,
                         int32_t T, int32_t k, int32_t H, void* out_bf16, void* stream);

/* ---------------------------------------------------------- scale folding
 * Offline weight preparation (nvfp4_cutedsl.py history, finalize_weights commit):
 * gate and up carry their own global scales; both are brought to
 * gs1[e] = max(gs_gate[e], gs_up[e]) by rewriting the block scales of the half
 * with the smaller scale: ratio = RN_f32(gs_p / gs1), sf' = E4M3 nearest-even,
 * saturating, of RN_f32(E4M3(sf) * ratio). Equal scales leave sf unchanged.
 *   w1_sf uint8 [L, 2I, K/16] in place; gs_gate, gs_up float [L]; gs1 float [L] out.
 */
int nvfp4_fold_scales(uint8_t* w1_sf, const float* gs_gate, const float* gs_up, float* gs1,
                      int32_t num_local, int32_t inter, int32_t K, void* stream);

/* ------------------------------------------------------------ whole layer
 * One rank's share of the MoE expert FFN (nvfp4_mega_moe.py history:
 * expert-parallel note — the layer writes a local partial output and the
 * caller reduces across ranks). Steps, all on `stream`, no host sync:
 *   quantize x (own gs) -> route -> L1 grouped GEMM with the SiLU*up epilogue
 *   (alpha = gs_x * w1_gs[e]) -> re-quantize h (gs_h from the epilogue's amax)
 *   -> L2 grouped GEMM (alpha = gs_h * w2_gs[e]) -> weighted scatter.
 * Weights (host struct of device pointers), L = num_local, each packed by
 * nvfp4_pack_weights from its row-major NVFP4 form:
 *   w1: W1 [L, 2I, H] packed (B = L, N = 2I, K = H), w1_gs [L]
 *       gate rows [0,I), up rows [I,2I), gate/up scales folded to one gs (nvfp4_fold_scales);
 *       or, with w1_dual_gs = 1, unfolded scales and w1_gs [L, 2] = (gs_gate, gs_up)
 *   w2: W2 [L, H, I] packed (B = L, N = H, K = I),   w2_gs [L]
 * x_bf16 [T, H]; topk_ids int32 [T, k] global ids; topk_w float [T, k];
 * out_bf16 [T, H] (tokens with no local expert get zeros).
 * ws: at least nvfp4_moe_ws_bytes(...) bytes; its regions (nvfp4_moe_ws_layout)
 * hold the intermediates after the call. Requires H % 128 == 0, I % 128 == 0,
 * T*k < 2^30, and T*H/2, T*k*I/2, 2I*H*9/16, 512*I and 256*H below 2^31.
 */
typedef struct {
  int32_t num_local, hidden, inter;
  const uint8_t* w1;
  const float* w1_gs;
  const uint8_t* w2;
  const float* w2_gs;
  int32_t w1_dual_gs;  /* 0: w1_gs [L] (folded); 1: w1_gs [L, 2] (gate, up) */
} nvfp4_moe_weights;

enum {
  NVFP4_WS_X_Q = 0, NVFP4_WS_X_SF, NVFP4_WS_SCALARS, NVFP4_WS_COUNTS, NVFP4_WS_OFFSETS,
  NVFP4_WS_SLOT_TOKEN, NVFP4_WS_SLOT_EXPERT, NVFP4_WS_SLOT_WEIGHT, NVFP4_WS_TOKEN_SLOT,
  NVFP4_WS_TILES, NVFP4_WS_ROUTE_SCRATCH, NVFP4_WS_H, NVFP4_WS_H_Q, NVFP4_WS_H_SF, NVFP4_WS_Y,
  NVFP4_WS_QUANT_SCRATCH, NVFP4_WS_END, NVFP4_WS_NREGIONS
};
/* Scalars region (float[4]): [0] gs_x, [1] amax_h, [2] gs_h, [3] reserved. */

/* Byte offset of every workspace region (host array of NVFP4_WS_NREGIONS entries;
 * entry NVFP4_WS_END is the total size). Returns the total size. */
size_t nvfp4_moe_ws_layout(int32_t T, int32_t k, int32_t hidden, int32_t inter, int32_t num_local,
                           int32_t tile_m, size_t* offsets_out);
size_t nvfp4_moe_ws_bytes(int32_t T, int32_t k, int32_t hidden, int32_t inter, int32_t num_local);
/* GEMM row-tile height the layer uses for a given batch: 32 when decode-shaped, 96 when
 * prefill-shaped (slot capacity T*k of at least 64 rows per local expert). */
int32_t nvfp4_moe_tile_m(int32_t T, int32_t k, int32_t num_local);
int nvfp4_moe_forward(const nvfp4_moe_weights* w, const void* x_bf16, int32_t T,
                      const int32_t* topk_ids, const float* topk_w, int32_t k, int32_t expert_start,
                      void* out_bf16, void* ws, size_t ws_bytes, void* stream);

/* nvfp4_moe_forward with per-stage timing: the same launches, with HIP events
 * recorded on `stream` between them, so that the caller can time each step of
 * the real layer. events: host array of NVFP4_NSTAGES + 1 hipEvent_t the caller
 * created (timing enabled); events[0] is recorded before the first launch and
 * events[i + 1] after the launches of stage i:
 *   NVFP4_STAGE_AMAX_ROUTE  a1, amax of x, sharing its launch with a3: the whole
 *                           route when T*k <= 1024, else the per-chunk histograms
 *   NVFP4_STAGE_QUANT_X     a2, block quantization of x; when T*k > 1024 its launch
 *                           also runs the rest of a3 (scan, slot scatter, tile table)
 *   NVFP4_STAGE_ROUTE       no launch of its own (events back to back), except for
 *                           very large routes (more than 65536 histogram entries:
 *                           ceil(T*k / 1024) x num_local), which take separate scan
 *                           and scatter launches here
 *   NVFP4_STAGE_L1          a4 + a5, L1 grouped GEMM with the SiLU*up epilogue
 *   NVFP4_STAGE_QUANT_H     a6, re-quantization of h
 *   NVFP4_STAGE_L2          a7, L2 grouped GEMM
 *   NVFP4_STAGE_SCATTER     a8, weighted scatter
 * A NULL entry skips that record; a NULL events array returns NVFP4_ERR_NULL,
 * a failed event record NVFP4_ERR_HIP. Arguments and results as
 * nvfp4_moe_forward.
 */
enum {
  NVFP4_STAGE_AMAX_ROUTE = 0, NVFP4_STAGE_QUANT_X, NVFP4_STAGE_ROUTE, NVFP4_STAGE_L1, NVFP4_STAGE_QUANT_H,
  NVFP4_STAGE_L2, NVFP4_STAGE_SCATTER, NVFP4_NSTAGES
};
int nvfp4_moe_forward_stage_events(const nvfp4_moe_weights* w, const void* x_bf16, int32_t T,
                                   const int32_t* topk_ids, const float* topk_w, int32_t k, int32_t expert_start,
                                   void* out_bf16, void* ws, size_t ws_bytes, void* const* events, void* stream);

/* The layer with fixed global scales (nvfp4_cutedsl.py history, page 2,
 * static-scale commit: warmup measures gs for the L1 input and for the L1
 * output; inference quantizes with them, no max reduction, no host sync).
 * gs_in: device float [2] = (gs_x, gs_h), e.g. the scalars [0] and [2] that
 * nvfp4_moe_forward leaves in its workspace for a calibration batch. Steps:
 * nvfp4_quantize_static of x with gs_x -> route -> L1 whose epilogue writes h
 * as NVFP4 with gs_h (nvfp4_grouped_gemm_silu_nvfp4) -> L2 (alpha = gs_h *
 * w2_gs[e]) -> weighted scatter. Decode-shaped batches (nvfp4_moe_tile_m ==
 * 32) write BF16 h and quantize it with gs_h in a launch of its own instead.
 * With the gs values nvfp4_moe_forward measured for the same inputs, the
 * output equals nvfp4_moe_forward's bit for bit. Same arguments, workspace
 * and limits as nvfp4_moe_forward; the SCALARS region is left unspecified.
 */
int nvfp4_moe_forward_static(const nvfp4_moe_weights* w, const void* x_bf16, int32_t T,
                             const int32_t* topk_ids, const float* topk_w, int32_t k, int32_t expert_start,
                             const float* gs_in, void* out_bf16, void* ws, size_t ws_bytes, void* stream);

/* The layer for at most nvfp4_moe_few_max_tokens() = 64 tokens, in two launches
 * (three for narrow layers) on the same weights, with activations as they are
 * (BF16, not quantized):
 *   h_e    = RN_bf16(silu(G) * U), G and U = w1_gs[e] (gate and up) times the
 *            products of x[t] with the gate and up rows of W1_e
 *   out[t] = RN_bf16(sum over the experts e of token t on this rank of
 *            topk_w[t, e] * w2_gs[e] * W2_e h_e [+ add[t]])
 * sums in float32, each expert with the sum of its weights where a token lists
 * it twice. add BF16 [T, H] (such as the dense expert's output; may be out) or
 * NULL. Ids outside [expert_start, expert_start + L) take no part. The order of
 * the sums depends on what the tokens chose, so a call repeats bit for bit, but
 * a token's last bits may differ with the others in the batch.
 * ws: at least nvfp4_moe_few_ws_bytes(...) bytes; h comes first, BF16 [T, k, I],
 * a row for each choice on this rank (the first of an expert listed twice).
 * out may be x or add; ws overlaps nothing. 1 <= k <= 64, 1 <= L <= 4096,
 * H % 128 == 0, I % 128 == 0, I < 65536, 2I*H*9/16 below 2^31.
 */
int32_t nvfp4_moe_few_max_tokens(void);
size_t nvfp4_moe_few_ws_bytes(int32_t T, int32_t k, int32_t hidden, int32_t inter, int32_t num_local);
int nvfp4_moe_forward_few(const nvfp4_moe_weights* w, const void* x_bf16, int32_t T, const int32_t* topk_ids,
                          const float* topk_w, int32_t k, int32_t expert_start, const void* add_bf16, void* out_bf16,
                          void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* NVFP4MOE_H */
