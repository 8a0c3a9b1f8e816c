/*
 * fm_ops.h -- C ABI of the E4M3 block-scaled operators: the pieces of a
 * transformer layer whose linears run on E4M3 codes with one fp32 scale per
 * block of 128, for the backbone that fills the prefix cache of
 * fm_expert.h (its K and V, after fm_rope_axes, are what fm_set_prefix takes)
 * or any decoder beside it.  fm_expert.h's W8A8 path keeps one scale per row;
 * these operators keep one per 128 inputs of a row (activations) and one per
 * 128 x 128 block (weights).
 *
 *   fm_add_rmsnorm_e4m3         residual add + RMS norm -> codes + scales
 *   fm_gated_e4m3               SwiGLU / GELU gate (or nothing) -> codes + scales
 *   fm_quantize_weight_e4m3_b128  bf16 weight -> codes + block scales (set-up)
 *   fm_gemm_e4m3_b128           codes x codes -> bf16 or fp32, optional bias
 *   fm_rope_axes                RoPE with a position axis per frequency, fused
 *                               q|k|v rows -> q, k, v
 *
 * Conventions (beside those of fm_expert.h):
 *   * No handle and no workspace: every pointer is the caller's device memory
 *     on the CURRENT device (host memory and memory of another device are
 *     refused), unless marked "host".  Nothing is kept between calls (but the
 *     timeouts that fm_ops_sync reports), so calls on several threads and streams are
 *     independent.
 *   * Stream-ordered, asynchronous, capturable in a CUDA graph.
 *   * Matrices are row-major; ld* is the distance between rows in elements and
 *     at least the row's width (any value when there is one row or none).
 *     Rows of the vectorised operands start on 16-byte boundaries: the base
 *     pointer is 16-byte aligned and ld x element size a multiple of 16 (for
 *     the exceptions see each call).
 *   * Zero rows are a no-op.  Rows and columns outside the stated extents
 *     (strides wider than the row, rows behind the last) are never written.
 *   * An output must not overlap an input or another output, except where
 *     the call says so.
 *   * Scales: for a group with largest magnitude a, with a' = max(a, 2^-100):
 *     s = a' / 448 and codes = E4M3(y * (448 / a')) (fp32, nearest-even,
 *     saturating); s = 1 and codes 0 for an all-zero group.  The value is
 *     code * s.  A NaN element gets a NaN code (0x7F) and does not count for
 *     a; a group with an infinite element gets s = +inf and NaN or zero codes.
 *   * On error the call returns a non-zero fm_status before it launches
 *     anything and fm_last_error(NULL) says why.
 */
#ifndef FM_OPS_H
#define FM_OPS_H

#include <stddef.h>
#include <stdint.h>

#include "fm_expert.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum fm_dtype {
  FM_BF16 = 0,
  FM_F32 = 1
} fm_dtype;

typedef enum fm_act {
  FM_ACT_NONE = 0,          /* u = x                                             */
  FM_ACT_SILU = 1,          /* u = gate / (1 + exp(-gate)) * up                  */
  FM_ACT_GELU_TANH = 2      /* u = gate/2 (1 + tanh(sqrt(2/pi) (gate + 0.044715 gate^3))) * up */
} fm_act;

/* h = x + residual (fp32; h = x when residual is NULL),
 * y = h (mean(h^2) + eps)^-1/2 (gain + gain_offset), in fp32 from the
 * unrounded h; codes and scales of y per row and 128 columns.
 *   x: [rows, d] of x_type; residual: [rows, d] of h_type or NULL; gain: bf16
 *   [d] or NULL (all ones); gain_offset: 0, or 1 for gains stored around zero.
 *   h_out: [rows, d] of h_type or NULL (not written); it may be `residual`
 *   itself (same pointer and stride), or x itself when the types agree.
 *   codes: [rows, d] bytes; scales: fp32 [rows, ceil(d/128)], any stride.
 * d: a multiple of 16, 16 .. 16384.  eps >= 0 (a zero row with eps = 0 gives
 * NaN).  The sum of squares is fp32: a row whose sum passes 3.4e38 (one h of
 * 1.9e19) gets zero codes, and with eps = 0 one of |h| below 1e-23 NaN codes. */
fm_status fm_add_rmsnorm_e4m3(const void *x, fm_dtype x_type, int64_t ldx, const void *residual,
                              fm_dtype h_type, int64_t ldr, const uint16_t *gain, float gain_offset,
                              float eps, int rows, int d, void *h_out, int64_t ldh, uint8_t *codes,
                              int64_t ldc, float *scales, int64_t lds, void *stream);

/* u = act(x[:, :f]) * x[:, f:2f] in fp32 (act FM_ACT_NONE: u = x[:, :f]);
 * codes and scales of u per row and 128 columns.  u is good to 13 roundings of
 * fp32 (GELU's to 8 |t| more, t < 0 its exponent sqrt(8/pi) (gate + 0.044715
 * gate^3)), far negative gates included.
 *   x: [rows, 2f] (FM_ACT_NONE: [rows, f]) of x_type, gate first.
 *   codes: [rows, f]; scales: fp32 [rows, ceil(f/128)], any stride.
 * f: a multiple of 16, 16 .. 2^20. */
fm_status fm_gated_e4m3(const void *x, fm_dtype x_type, int64_t ldx, fm_act act, int rows, int f,
                        uint8_t *codes, int64_t ldc, float *scales, int64_t lds, void *stream);

/* Codes [n, k] and scales [ceil(n/128), ceil(k/128)] of a bf16 weight [n, k],
 * one scale per 128 x 128 block; codes = E4M3(w / s) (fp32 division, as the
 * per-row weight recipe of FM_W_FP8_E4M3), s as above.  ldw, ldc, lds and the
 * pointers need only their element's alignment. */
fm_status fm_quantize_weight_e4m3_b128(const uint16_t *w, int64_t ldw, int n, int k, uint8_t *codes,
                                       int64_t ldc, float *scales, int64_t lds, void *stream);

/* out[i, j] = sum_g sa[i, g] sw[j/128, g] sum_{c in group g} a[i, c] w[j, c]
 *             (+ bias[j]),  groups of 128 consecutive inputs (the last may be
 * shorter).  E4M3 products and fp32 sums inside a group on the tensor cores,
 * fp32 scaling (by sa sw, rounded to fp32 first: it has to lie in fp32's range)
 * and summing over the groups, one rounding to out_type.
 *   a: codes [m, k]; sa: fp32 [m, ceil(k/128)]; w: codes [n, k]; sw: fp32
 *   [ceil(n/128), ceil(k/128)]; bias: bf16 [n] or NULL; out: [m, n].
 * k: a multiple of 16, at least 16 (a and w rows on 16-byte boundaries); m
 * and n any.  sa, sw, bias and out need only their element's alignment.  The
 * same call gives the same bits; where k is split between blocks (and so the
 * order of the fp32 sums over the groups) is chosen by m, n, k, the alignment of
 * a, w and out and the device's number of multiprocessors.  A device-side wait that exceeds its bound leaves its
 * part of `out` unspecified and is reported by fm_ops_sync. */
fm_status fm_gemm_e4m3_b128(const uint8_t *a, int64_t lda, const float *sa, int64_t ldsa,
                            const uint8_t *w, int64_t ldw, const float *sw, int64_t ldsw,
                            const uint16_t *bias, int m, int n, int k, void *out, fm_dtype out_type,
                            int64_t ldo, void *stream);

/* Rotate-half RoPE with several position axes, fused with the split of q|k|v
 * rows.  Pair j < n_pairs of a head is (element j, element j + n_pairs), its
 * angle positions[pair_axis[j]][row] * pair_freq[j] (radians, reduced in 64
 * bits); the pair (lo, hi) becomes (lo cos - hi sin, hi cos + lo sin), computed
 * in fp32 and rounded once.  Elements from 2 n_pairs on, and v, are copied.
 *   x: [rows, (n_q + 2 n_kv) head_dim] of `type`: n_q query heads, n_kv key
 *   heads, n_kv value heads (without v_out only the q and k columns are read).
 *   positions: int32 [n_axes, rows], any values, axes ldp elements apart.
 *   pair_axis (host): n_pairs axis numbers; pair_freq (host): n_pairs finite
 *   frequencies in radians per position.
 *   q_out: [rows, n_q head_dim], k_out and v_out: [rows, n_kv head_dim], of
 *   `type`, each with its own stride; each may be NULL (not written), and may be
 *   its own columns of x (in place: same pointer and stride).
 * n_q, n_kv 0 .. 1024; head_dim even, 2 .. 256; 1 <= n_pairs <= head_dim / 2; 1 <= n_axes <= 8.
 * Pointers and strides need only their element's alignment; a thread moves 8,
 * 4, 2 or 1 elements at a time, the most that head_dim, n_pairs and the rows'
 * alignment allow. */
fm_status fm_rope_axes(const void *x, fm_dtype type, int64_t ldx, int rows, int n_q, int n_kv,
                       int head_dim, const int32_t *positions, int64_t ldp, int n_axes,
                       const uint8_t *pair_axis, const double *pair_freq, int n_pairs, void *q_out,
                       int64_t ldq, void *k_out, int64_t ldk, void *v_out, int64_t ldv, void *stream);

/* Wait for `stream` (of the current device; one that is being captured is
 * refused), then report (FM_ERR_TIMEOUT) whether any fm_gemm_e4m3_b128 of this
 * device, on whatever stream, has given up a wait since the calling thread's
 * previous fm_ops_sync on it (the thread's first: since the library was loaded).
 * Every thread is told, and told once: after a report the products that the
 * device ended since the thread's previous call are all in doubt, those of other
 * streams too. */
fm_status fm_ops_sync(void *stream);

/* Test hook for failure detection: in the fm_gemm_e4m3_b128 calls that this
 * thread makes from now on (graphs keep what they were captured with) `role`
 * gives up when it has done `group` groups of 128 inputs, and every other wait
 * of the pipeline after `spin_cycles` SM clock cycles (0: the default of about
 * 2 s).  Such a call ends early where it has more groups than that: its `out` is
 * unspecified and fm_ops_sync reports FM_ERR_TIMEOUT; the device context stays
 * usable.  The roles are the loading and the multiplying warps of a cluster's
 * first and second block (many rows: the two multiplying warps of a pair).
 * FM_ERR_INVALID_ARG for another role or a negative number. */
typedef enum fm_stall {
  FM_STALL_NONE = 0,
  FM_STALL_TMA0 = 1,
  FM_STALL_TMA1 = 2,
  FM_STALL_MMA0 = 3,
  FM_STALL_MMA1 = 4
} fm_stall;
fm_status fm_ops_test_stall(fm_stall role, int group, long long spin_cycles);

#ifdef __cplusplus
}
#endif
#endif /* FM_OPS_H */
