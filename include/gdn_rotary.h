/*
 * gdn_rotary.h — what queries and keys go through between their projection and the layers of gdn.h
 * and gdn_linear.h: the norm of every head and the rotation by the token's position, with their
 * gradients. In the same library (libgdn.so).
 *
 * The rotation. Of a head's D values the first R (even, 0 <= R <= D) are R / 2 pairs, pair i turned
 * by theta = p * freqs[i] at a token of position p; the values from R on are copied:
 *
 *     (x, y) -> amplitude * (x cos theta - y sin theta,  x sin theta + y cos theta)
 *
 * Pair i is (x_i, x_{i + R/2}) (half layout, interleaved = 0) or (x_{2i}, x_{2i+1}) (interleaved =
 * 1). The angle is formed in 64 bits and reduced before it is rounded, so positions of millions lose
 * nothing (for |theta| up to 2^31 its error is below 2^-20). Scalings for long contexts are a choice
 * of freqs and amplitude.
 * The norm. x -> x * w / sqrt(mean x^2 + eps) over the head's D values; w one weight per value, or per
 * value and head. The unit length of the gated delta rule's q and k, x / sqrt(sum x^2 + e), is the
 * weight D^-1/2 with eps = e / D.
 *
 * The conventions of gdn.h hold for every call (asynchronous on `stream`, arguments validated on the
 * host before anything is enqueued, nothing synchronises, allocates or reads the environment, every
 * call may be captured into a HIP graph, the same call on the same inputs gives the same bits), with
 * two differences for q, k, their gradients and outputs:
 *  - Strides. They are [B][T][H][D] with the last index dense. `..._strides` gives the other three
 *    strides (sequence, token, head) in elements, none negative, as a host array of 3 read during the
 *    call; NULL means the dense tensor. So views of a packed projection, and heads before tokens, are
 *    taken as they are. An output's elements must be distinct, and must not be another argument's
 *    except where a call says so (interleaved views, such as the q and k parts of one packed tensor,
 *    are told apart).
 *  - Alignment is that of an element. Vectors of 16 bytes are used where pointers, strides, R and D
 *    allow them.
 * Sizes: Hq >= 1; Hk >= 0, and with Hk = 0 there is no k (its pointers are ignored); Hq + Hk <= 16384;
 * 1 <= D <= 512; B * T < 2^31; GDN_OK for B == 0 or T == 0.
 * Positions. `positions` int32 [B][T] in device memory, dense; NULL counts every sequence's tokens from 0.
 * `freqs` float64 [R/2] in device memory, in radians per position, finite; NULL if R == 0.
 * Lengths. `lengths` (int32 [B] in device memory, or NULL) gives the tokens of each sequence, clamped
 * to [0, T]: inputs past it are not read, outputs past it are written as zeros.
 * Arithmetic is fp32 (16-bit inputs widen exactly); outputs round to nearest even once. A row whose sum of
 * squares passes fp32's range counts as infinitely long (its norm gives zeros), squares below 2^-126 lose
 * digits and below 2^-149 count as zeros (with eps = 0 a row of such values has no norm: infinities), and an
 * infinity in a row makes NaNs of that row alone.
 */
#ifndef GDN_ROTARY_H
#define GDN_ROTARY_H

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * gdn_rope — the rotation of q and k.
 *   q      dtype [B][T][Hq][D]    k      dtype [B][T][Hk][D]    (strided)
 *   q_out  dtype [B][T][Hq][D]    k_out  dtype [B][T][Hk][D]    (strided), written; each may be its input
 *                                 itself (same pointer and strides: in place)
 * Errors: GDN_ERR_INVALID_ARGUMENT, GDN_ERR_UNSUPPORTED (D > 512, Hq + Hk > 16384, B * T >= 2^31), GDN_ERR_HIP.
 */
gdn_status gdn_rope(int64_t B, int32_t T, int32_t Hq, int32_t Hk, int32_t D, int32_t R,
                    gdn_dtype dtype, const void* q, const int64_t* q_strides, const void* k,
                    const int64_t* k_strides, const int32_t* positions, const double* freqs,
                    float amplitude, int32_t interleaved, const int32_t* lengths, void* q_out,
                    const int64_t* q_out_strides, void* k_out, const int64_t* k_out_strides,
                    void* stream);

/* gdn_rope_backward — the gradients of q and k from those of q_out and k_out: the transposed rotation,
 * with gdn_rope's arguments (dq, dk in place of q, k). Errors: as gdn_rope. */
gdn_status gdn_rope_backward(int64_t B, int32_t T, int32_t Hq, int32_t Hk, int32_t D, int32_t R,
                             gdn_dtype dtype, const void* dq, const int64_t* dq_strides,
                             const void* dk, const int64_t* dk_strides, const int32_t* positions,
                             const double* freqs, float amplitude, int32_t interleaved,
                             const int32_t* lengths, void* q_out, const int64_t* q_out_strides,
                             void* k_out, const int64_t* k_out_strides, void* stream);

/*
 * gdn_qk_norm_rope — the norm of every head of q and k, then the rotation (R = 0: the norm alone), in
 * one pass; gdn_rope's arguments, and
 *   q_weight  fp32 [D], or [Hq][D] where per_head is not 0, or NULL (1)
 *   k_weight  fp32 [D], or [Hk][D], or NULL
 *   eps       >= 0. A row of zeros gives zeros where eps > 0.
 * Errors: as gdn_rope.
 */
gdn_status gdn_qk_norm_rope(int64_t B, int32_t T, int32_t Hq, int32_t Hk, int32_t D, int32_t R,
                            gdn_dtype dtype, const void* q, const int64_t* q_strides, const void* k,
                            const int64_t* k_strides, const float* q_weight, const float* k_weight,
                            int32_t per_head, float eps, const int32_t* positions,
                            const double* freqs, float amplitude, int32_t interleaved,
                            const int32_t* lengths, void* q_out, const int64_t* q_out_strides,
                            void* k_out, const int64_t* k_out_strides, void* stream);

/* gdn_qk_norm_rope_backward_workspace_size — bytes of device workspace gdn_qk_norm_rope_backward needs
 * for these sizes where a weight's gradient is wanted. Errors: GDN_ERR_INVALID_ARGUMENT, GDN_ERR_UNSUPPORTED. */
gdn_status gdn_qk_norm_rope_backward_workspace_size(int64_t B, int32_t T, int32_t Hq, int32_t Hk,
                                                    int32_t D, size_t* bytes);

/*
 * gdn_qk_norm_rope_backward — gradients of gdn_qk_norm_rope from dq, dk, those of q_out and k_out. With
 * r = 1 / sqrt(mean x^2 + eps), n = x r and g the transposed rotation of the gradient:
 *
 *     dx = r (g w - n mean(g w n))      dw = sum of g n over the rows (of each head where per_head is not 0)
 *
 *   dq, dk, q, k       dtype, strided; q, k, the weights and the rest as the forward call's
 *   q_out, k_out       dtype, strided, written: the gradients of q and k (each may be dq, dk itself)
 *   dq_weight          fp32, the weight's shape, written, or NULL if not wanted; dk_weight likewise
 *   workspace          device buffer of workspace_bytes, needed where dq_weight or dk_weight is not NULL;
 *                      contents on entry do not matter; must not overlap any other argument. Two calls
 *                      in flight at once (also two captured graphs) need two workspaces.
 * The sums over rows are taken in a fixed order (no atomics), 0 for B == 0 or T == 0.
 * Errors: as gdn_rope; GDN_ERR_INVALID_ARGUMENT also for a small workspace.
 */
gdn_status gdn_qk_norm_rope_backward(
    int64_t B, int32_t T, int32_t Hq, int32_t Hk, int32_t D, int32_t R, gdn_dtype dtype,
    const void* dq, const int64_t* dq_strides, const void* dk, const int64_t* dk_strides,
    const void* q, const int64_t* q_strides, const void* k, const int64_t* k_strides,
    const float* q_weight, const float* k_weight, int32_t per_head, float eps,
    const int32_t* positions, const double* freqs, float amplitude, int32_t interleaved,
    const int32_t* lengths, void* q_out, const int64_t* q_out_strides, void* k_out,
    const int64_t* k_out_strides, float* dq_weight, float* dk_weight, void* workspace,
    size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_ROTARY_H */
