/*
 * gdn_scan.h — a gated linear recurrence with one value of state for each channel, and its gradients:
 * the diagonal companion of gdn_linear.h, in the same library (libgdn.so).
 *
 * The operation. For each sequence b and channel c the library keeps one value h and, for each token t
 * in order, with the token's gates a_t, b_t of that channel,
 *
 *     alpha_t = exp(-rate_c * softplus(a_t))        beta_t = sigmoid(b_t), or 1 - alpha_t without b
 *     h_t = alpha_t * h_{t-1} + beta_t * x_t        o_t = h_t
 *
 * (alpha and beta as in gdn_conv_gate_decode, with a rate.) softplus(a) = ln(1 + e^a), of an infinite a
 * fp32's largest value; rate any finite value: 0 keeps the state for ever, below 0 it grows. 1 - alpha is
 * formed without cancellation, so decays next to 1 keep their distance from it, and of a state that a token
 * forgets what is left keeps fp32's own steps (decays, and products of the decays of 64 tokens, may count as 0
 * below 2^-126). Where states grow, prompts and gradients stay finite as long as the states and adjoints do,
 * also where the product of 64 decays, or one of them, is past fp32's range (over states of 0, say); a
 * channel goes through such tokens one by one, at 1 to 2 us a token.
 *
 * The conventions of gdn.h hold for every call: asynchronous on `stream`, arguments validated on the host
 * before anything is enqueued, GDN_OK for B == 0 or T == 0, gdn_last_error() explains a failure. Nothing
 * synchronises, allocates or reads the environment, every call may be captured into a HIP graph, and the
 * same call on the same inputs gives the same bits. One difference: x, a, b, their gradients, o and d_o are
 * [B][T][C] with the last index dense and `..._strides` (a host array of 2, read during the call: sequence,
 * token, in elements, none negative; NULL means dense), aligned to an element; so views of one packed projection
 * are taken as they are. An output's elements must be distinct and must not be another argument's
 * (interleaved views of one tensor are told apart); o may not be x.
 * Sizes: C >= 1; B * C < 2^31; T < 2^30; B * T * C < 2^60;
 * B * ceil(T / 64) * ceil(C / 64) < 2^31.
 * Lengths. `lengths` (int32 [B] in device memory, or NULL) gives the tokens of each sequence, clamped
 * to [0, T]: inputs past it are not read, outputs past it (rows of o, dx, da, db) are written as zeros, and the
 * state is the one after the last token.
 * Arithmetic is fp32 (16-bit inputs widen exactly, states stay fp32 until they are stored, 16-bit outputs
 * round to nearest even once). A NaN or infinity stays within its own sequence and channel, and may reach
 * that channel's earlier outputs of the same 64 tokens.
 */
#ifndef GDN_SCAN_H
#define GDN_SCAN_H

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Tokens from one kept state (`checkpoints`) to the next. */
#define GDN_SCAN_CHECKPOINT 64

/*
 * gdn_gated_scan_decode_step — T new tokens (one, or a few drafted ones) of every sequence.
 *   x, a     act_dtype [B][T][C] (strided)
 *   b        act_dtype [B][T][C] (strided) or NULL (beta = 1 - alpha)
 *   rate     fp32 [C] or NULL (1)
 *   lengths  int32 [B] or NULL
 *   state    state_dtype [B][C], dense, read and updated IN PLACE
 *   o        act_dtype [B][T][C] (strided), written
 * Errors: GDN_ERR_INVALID_ARGUMENT, GDN_ERR_UNSUPPORTED, GDN_ERR_HIP (see gdn.h).
 */
gdn_status gdn_gated_scan_decode_step(int64_t B, int32_t T, int32_t C, const void* x,
                                      const int64_t* x_strides, const void* a,
                                      const int64_t* a_strides, const void* b,
                                      const int64_t* b_strides, gdn_dtype act_dtype,
                                      const float* rate, const int32_t* lengths, void* state,
                                      gdn_dtype state_dtype, void* o, const int64_t* o_strides,
                                      void* stream);

/* gdn_gated_scan_prefill_workspace_size — bytes of device workspace gdn_gated_scan_prefill needs for
 * these sizes (it may be 0: a NULL workspace is then accepted). Errors: GDN_ERR_INVALID_ARGUMENT, GDN_ERR_UNSUPPORTED. */
gdn_status gdn_gated_scan_prefill_workspace_size(int64_t B, int32_t T, int32_t C, size_t* bytes);

/*
 * gdn_gated_scan_prefill — the same operation over a prompt, split along its tokens: arguments and
 * result of gdn_gated_scan_decode_step, up to the order of fp32 operations, and
 *   checkpoints      fp32 [B][ceil(T / 64)][C], dense, written, or NULL if not wanted: the state after the
 *                    first min(64 j, length) tokens, for gdn_gated_scan_backward
 *   workspace        device buffer of at least gdn_gated_scan_prefill_workspace_size(...) bytes; contents
 *                    on entry do not matter; must not overlap any other argument. Two calls in flight
 *                    at once (also two captured graphs) need two workspaces.
 *   workspace_bytes  its size in bytes
 * Errors: as gdn_gated_scan_decode_step; GDN_ERR_INVALID_ARGUMENT also for a small workspace.
 */
gdn_status gdn_gated_scan_prefill(int64_t B, int32_t T, int32_t C, const void* x,
                                  const int64_t* x_strides, const void* a, const int64_t* a_strides,
                                  const void* b, const int64_t* b_strides, gdn_dtype act_dtype,
                                  const float* rate, const int32_t* lengths, void* state,
                                  gdn_dtype state_dtype, void* o, const int64_t* o_strides,
                                  float* checkpoints, void* workspace, size_t workspace_bytes,
                                  void* stream);

/* gdn_gated_scan_backward_workspace_size — bytes of device workspace gdn_gated_scan_backward needs for
 * these sizes, with every optional input and output. Errors: as the prefill's. */
gdn_status gdn_gated_scan_backward_workspace_size(int64_t B, int32_t T, int32_t C, size_t* bytes);

/*
 * gdn_gated_scan_backward — gradients of the operation (prompt or decode form) from the gradient `d_o` of
 * o and `dstate` of the state after the last token:
 *
 *     g_t = do_t + alpha_{t+1} g_{t+1}          (dstate enters as alpha_{t+1} g_{t+1} after the last token)
 *     dx_t = beta_t g_t         db_t = g_t x_t beta_t (1 - beta_t)
 *     e_t = alpha_t g_t (x_t [without b] - h_{t-1})     the gradient of rate * softplus(a_t)
 *     da_t = e_t rate sigmoid(a_t)              drate = sum over b and t of e_t softplus(a_t)
 *     dstate0 = alpha_1 g_1
 *
 *   x, a, b, rate, lengths, act_dtype  as the forward call's
 *   state0       state_dtype [B][C], the state BEFORE the forward call, or NULL for zeros
 *   checkpoints  fp32 [B][ceil(T / 64)][C] as the forward call wrote them, or NULL: the states are then
 *                made again from state0, x, a and b (with checkpoints state0 is not read)
 *   d_o          act_dtype [B][T][C] (strided)     dstate  state_dtype [B][C] or NULL for zero
 *   dx, da       act_dtype [B][T][C] (strided), written      db  likewise, NULL exactly where b is
 *   dstate0      state_dtype [B][C], written, or NULL if not wanted
 *   drate        fp32 [C], written, or NULL if not wanted
 * Sums over sequences and tokens are taken in a fixed order. With T == 0 (or a length of 0) dstate0 is dstate
 * and drate 0; with B == 0 drate is 0.
 * Errors: as gdn_gated_scan_prefill.
 */
gdn_status gdn_gated_scan_backward(
    int64_t B, int32_t T, int32_t C, const void* x, const int64_t* x_strides, const void* a,
    const int64_t* a_strides, const void* b, const int64_t* b_strides, gdn_dtype act_dtype,
    const float* rate, const int32_t* lengths, const void* state0, const float* checkpoints,
    const void* d_o, const int64_t* d_o_strides, const void* dstate, gdn_dtype state_dtype, void* dx,
    const int64_t* dx_strides, void* da, const int64_t* da_strides, void* db,
    const int64_t* db_strides, void* dstate0, float* drate, void* workspace, size_t workspace_bytes,
    void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_SCAN_H */
