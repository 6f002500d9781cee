/*
 * gdn_linear.h — linear attention with a decay for each head, its gradients, and the layer norm
 * of a layer's output: the companions of gdn.h, in the same library (libgdn.so).
 *
 * The operation. For each sequence b and head h the library keeps a state S of dv x dk values
 * (the layout of gdn.h: rows indexed by the value dimension) and, for each token t in order,
 *
 *     S_t = decay_h * S_{t-1} + v_t k_t^T
 *     o_t = S_t (scale * q_t)
 *
 * which is the gated delta rule of gdn.h without its correction term and with one decay per head.
 * The decay is fixed for the call: any finite value is taken as given (0 forgets everything
 * before the token, 1 keeps everything; beyond 1 the state grows, and a prompt's results are
 * defined while the decay's powers up to its length stay within fp32's range).
 *
 * The conventions of gdn.h hold for every call: dense row-major device buffers of the current
 * device, 16-byte aligned, owned by the caller; asynchronous on `stream`; arguments validated on
 * the host before anything is enqueued; GDN_OK for B == 0 or T == 0 (the pointers of empty
 * tensors may then be NULL); gdn_last_error() explains a failure; dk == dv, one of 16, 32, 64,
 * 128; B * H * 8 * dk < 2^32 and T < 2^30. Nothing synchronises, allocates or reads the environment, and every
 * call may be captured into a HIP graph. Results do not depend on timing: the same call on the
 * same inputs gives the same bits.
 *
 * Heads. q and k have Hk heads, v and o have H, a multiple of Hk: head h reads q/k head
 * h / (H / Hk), and dq, dk are the sums over the heads that share one.
 * Lengths. `lengths` (int32 [B] in device memory, or NULL) gives the tokens of each sequence,
 * clamped to [0, T]; NULL means T for all. Inputs past a sequence's length are not read, its
 * state is the one after its last token (unchanged where the length is 0), and outputs past it
 * (rows of o, dq, dk, dv) are written as zeros.
 * Arithmetic is fp32 throughout (16-bit inputs widen exactly; sums and states stay fp32 until
 * they are stored; 16-bit outputs round to nearest even once). Prompts and gradients take their
 * factors apart into bf16 parts on the matrix cores, of which at most 2^-26 of a term is lost; of
 * values below 2^-109 bits under 2^-133 are lost, and an infinity (or a value that rounds to one in
 * bf16, from 2^128 (1 - 2^-9)) may come out as a NaN.
 */
#ifndef GDN_LINEAR_H
#define GDN_LINEAR_H

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * gdn_linear_attn_decode_step — the recurrent form: T new tokens (one, or a few drafted ones) of
 * every sequence, token by token on the state in registers.
 *
 *   q, k     act_dtype [B][T][Hk][dk]    read only (may alias each other)
 *   v        act_dtype [B][T][H][dv]     read only
 *   decay    fp32 [H]
 *   lengths  int32 [B] or NULL
 *   state    state_dtype [B][H][dv][dk]  read and updated IN PLACE
 *   o        act_dtype [B][T][H][dv]     written; must not overlap any other argument
 * Errors: GDN_ERR_INVALID_ARGUMENT (also for Hk < 1 or H not a multiple of Hk),
 *         GDN_ERR_UNSUPPORTED, GDN_ERR_HIP (see gdn.h).
 */
gdn_status gdn_linear_attn_decode_step(int64_t B, int32_t T, int32_t H, int32_t Hk, int32_t dk,
                                       int32_t dv, const void* q, const void* k, const void* v,
                                       gdn_dtype act_dtype, const float* decay,
                                       const int32_t* lengths, void* state,
                                       gdn_dtype state_dtype, void* o, float scale, void* stream);

/* gdn_linear_attn_prefill_workspace_size — bytes of device workspace gdn_linear_attn_prefill needs
 * for these sizes (it may be 0: a NULL workspace is then accepted).
 * Errors: GDN_ERR_INVALID_ARGUMENT (bytes NULL, bad size), GDN_ERR_UNSUPPORTED (head dims). */
gdn_status gdn_linear_attn_prefill_workspace_size(int64_t B, int32_t T, int32_t H, int32_t dk,
                                                  int32_t dv, size_t* bytes);

/*
 * gdn_linear_attn_prefill — the same operation over a prompt of T tokens: arguments and result of
 * gdn_linear_attn_decode_step, up to the order of fp32 sums. A NaN or infinity in a token's q, k
 * or v can also reach the earlier outputs of its own chunk (64 tokens of bf16, 32 of fp16
 * and fp32); other heads and sequences are unaffected.
 *
 *   workspace        device buffer of at least gdn_linear_attn_prefill_workspace_size(...) bytes;
 *                    contents on entry do not matter; must not overlap any other argument. Two
 *                    calls in flight at once (also two captured graphs) need two workspaces.
 *   workspace_bytes  its size in bytes
 * Errors: as gdn_linear_attn_decode_step; GDN_ERR_INVALID_ARGUMENT also for a small workspace.
 */
gdn_status gdn_linear_attn_prefill(int64_t B, int32_t T, int32_t H, int32_t Hk, int32_t dk,
                                   int32_t dv, const void* q, const void* k, const void* v,
                                   gdn_dtype act_dtype, const float* decay,
                                   const int32_t* lengths, void* state, gdn_dtype state_dtype,
                                   void* o, float scale, void* workspace, size_t workspace_bytes,
                                   void* stream);

/* gdn_linear_attn_backward_workspace_size — bytes of device workspace gdn_linear_attn_backward needs
 * for these sizes, with every optional output. Errors: as the prefill's. */
gdn_status gdn_linear_attn_backward_workspace_size(int64_t B, int32_t T, int32_t H, int32_t Hk,
                                                   int32_t dk, int32_t dv, size_t* bytes);

/*
 * gdn_linear_attn_backward — gradients of the operation (prompt or decode form) from the gradient
 * `d_o` of o and `dstate` of the state after the last token:
 *
 *     R_t = decay R_{t+1} + scale do_t q_t^T   (the adjoint of S_t; dstate enters at the last token)
 *     dq_t = scale S_t^T do_t    dk_t = R_t^T v_t    dv_t = R_t k_t
 *     dstate0 = decay R_0        ddecay_h = sum over b and t of <R_t, S_{t-1}>
 *
 * The states S_t are recomputed from state0, k and v; nothing has to be kept from the forward call
 * but its inputs (state0 is the state BEFORE it: the forward call updates its own in place).
 *
 *   q, k, v, decay, lengths, scale, act_dtype  as the forward call's
 *   state0    state_dtype [B][H][dv][dk], or NULL for a zero state
 *   d_o       act_dtype [B][T][H][dv]
 *   dstate    state_dtype [B][H][dv][dk], or NULL for zero
 *   dq, dk    act_dtype [B][T][Hk][dk], written      dv_out  act_dtype [B][T][H][dv], written
 *   dstate0   state_dtype [B][H][dv][dk], written, or NULL if not wanted
 *   ddecay    fp32 [H], written, or NULL if not wanted
 * With T == 0 (or a length of 0) dstate0 is dstate and ddecay 0; with B == 0 ddecay is 0.
 * Outputs must not overlap each other or any input. A NaN or infinity in a token's inputs can also
 * reach other tokens of its own chunk.
 * Errors: as gdn_linear_attn_prefill.
 */
gdn_status gdn_linear_attn_backward(int64_t B, int32_t T, int32_t H, int32_t Hk, int32_t dk,
                                    int32_t dv, const void* q, const void* k, const void* v,
                                    gdn_dtype act_dtype, const float* decay,
                                    const int32_t* lengths, const void* state0,
                                    const void* d_o, const void* dstate, gdn_dtype state_dtype,
                                    void* dq, void* dk_out, void* dv_out, void* dstate0,
                                    float* ddecay, float scale, void* workspace,
                                    size_t workspace_bytes, void* stream);

/*
 * gdn_layer_norm — layer norm over the last dimension of x [rows][C], with an affine per group of
 * rows: row r uses weight and bias row r mod G. G = 1 is the plain layer norm; x = o [B][T][H][dv]
 * with rows = B T H, G = H, C = dv normalises every head's output with that head's own affine.
 *
 *     y = (x - mean) * rstd * weight + bias,   mean = sum x / C,  rstd = 1 / sqrt(sum (x - mean)^2 / C + eps)
 *
 *   x       dtype [rows][C]       weight, bias  fp32 [G][C] or NULL (1 and 0)
 *   y       dtype [rows][C], written (may be x itself: in place)
 *   mean, rstd  fp32 [rows], written, or both NULL if not wanted (backward needs them)
 * rows must be a multiple of G; any C >= 1; rows * C < 2^60, G * C < 2^31. A row of up to 32 KiB is summed
 * in fp32, a lane's terms first and then a tree; a longer one in 64 bits.
 * Errors: GDN_ERR_INVALID_ARGUMENT, GDN_ERR_HIP. rows == 0 is a valid no-op.
 */
gdn_status gdn_layer_norm(int64_t rows, int32_t G, int32_t C, const void* x, gdn_dtype dtype,
                          const float* weight, const float* bias, void* y, float* mean,
                          float* rstd, float eps, void* stream);

/* gdn_layer_norm_backward_workspace_size — bytes of device workspace gdn_layer_norm_backward needs
 * for these sizes when dweight or dbias is wanted. Errors: GDN_ERR_INVALID_ARGUMENT. */
gdn_status gdn_layer_norm_backward_workspace_size(int64_t rows, int32_t G, int32_t C, size_t* bytes);

/*
 * gdn_layer_norm_backward — gradients of gdn_layer_norm from the gradient dy of y and the kept
 * statistics, with n = (x - mean) rstd and g = dy * weight:
 *
 *     dx = rstd (g - mean_C(g) - n mean_C(g n))   dweight = sum over rows of dy n   dbias = sum of dy
 *
 *   dy, x   dtype [rows][C]     weight  fp32 [G][C] or NULL (1)     mean, rstd  fp32 [rows]
 *   dx      dtype [rows][C], written (may be dy itself)
 *   dweight, dbias  fp32 [G][C], written, each NULL if not wanted
 * The sums over rows are taken in a fixed order (no atomics). With rows == 0, dweight and dbias
 * are written as zeros.
 * Errors: GDN_ERR_INVALID_ARGUMENT (also a small workspace where dweight or dbias is wanted), GDN_ERR_HIP.
 */
gdn_status gdn_layer_norm_backward(int64_t rows, int32_t G, int32_t C, const void* dy,
                                   const void* x, gdn_dtype dtype, const float* weight,
                                   const float* mean, const float* rstd, void* dx,
                                   float* dweight, float* dbias, void* workspace,
                                   size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_LINEAR_H */
