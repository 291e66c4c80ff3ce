/*
 * mamba_gdr.h -- C ABI of the gated delta rule: the sequence layer whose state
 * update first takes back what the state already answers for a key.  It stands
 * beside mamba_ssd_fwd (mamba_scan.h): the same decay per head, the same
 * (B, H*P, N) state, the same sequence-fastest layout, and the conventions of
 * that header (device pointers, host checks before any launch, status codes,
 * the caller's workspace, graph capture) hold for every call here.
 *
 * What the calls compute, per value head h of P channels with state S (P x N)
 * and key head g = h / (H / G):
 *     delta_t = softplus(delta_raw[b,h,t] + delta_bias[h]),  a_t = exp(A[h] delta_t)
 *     b_t     = sigmoid(beta_raw[b,h,t])
 *     S' = a_t S_(t-1);   u_t = b_t (v_t - S' k_t);   S_t = S' + u_t k_t^T
 *     y_t = scale * S_t q_t
 * With MAMBA_FLAG_QK_NORM, q_t and k_t are first divided by
 * sqrt(their sum of squares + 1e-6).  Without it the keys are taken as they are:
 * the update is a contraction only while b_t |k_t|^2 <= 2.
 *
 * Arguments shared by the calls
 *   q, k        : (B, G*N, L) in_dtype, channel g*N + n; one key head serves the
 *                 H / G value heads g*(H/G) .. (g+1)*(H/G) - 1.
 *   v           : (B, H*P, L) in_dtype, channel h*P + p.
 *   delta, beta : (B, H, L) in_dtype, raw (before bias and softplus / sigmoid).
 *   q_stride, k_stride, v_stride : elements from one batch row to the next (at
 *                 least the row's own size), so that q, k and v may be channel
 *                 ranges of one convolution's output.
 *   A           : (H) fp32.  delta_bias : (H) fp32 or NULL (zeros).
 *   states      : (B, H*P, N) fp32.
 *   lengths     : (B) int32 on the device, or NULL (every row has L tokens).
 *                 Row b ends after lengths[b] tokens (values are held to 0 .. L):
 *                 what its inputs hold behind that is not looked at, be it NaN,
 *                 its outputs and gradients there are zero, and its final state is
 *                 the one after lengths[b] tokens.
 *
 * Sizes: 1 <= N <= 128; B, H, G, P, L >= 1; H a multiple of G; B*H*P*L and
 * B*G*N*L < 2^46; and no launch of 2^32 threads or more: B*H*ceil(P/4) < 2^26 for one token (four times
 * that with vector accesses); B*H*ceil(P/64)*ceil(L/32) < 2^23 is enough for sequences.
 * in_dtype and the output dtypes may each be MAMBA_F32 or
 * MAMBA_BF16.  Alignment: every array to its element size (16 bytes, and sizes that
 * are multiples of a vector, select vector accesses); workspaces 256 bytes.
 * A NaN or an infinity among the inputs of a token leaves the outputs of the tokens
 * before it as they are; from that token on, every output and state that it reaches
 * is NaN or infinite.  (Numbers beyond 3.38e38 count as infinite.)  In the backward pass
 * any gradient of such a batch row may be NaN, dA and ddelta_bias with it.  An infinite
 * delta or beta is not meant: a step of infinite length forgets the state (A < 0), and the
 * gates and all gradients take their limits.
 * State, gates and sums are fp32 or better.  The results are deterministic (sums in a
 * fixed order, no atomics): the same call gives the same bits, and what the other rows of
 * the batch hold has no influence on a row.  How many rows there are has: in mamba_gdr_fwd
 * B, like every other size, takes part in the choice between token by token and chunks
 * and of the segments of L, and those agree to fp32 rounding only.  mamba_gdr_update and
 * mamba_gdr_bwd give a row the same bits in a batch of any size.
 */
#ifndef MAMBA_GDR_H_
#define MAMBA_GDR_H_

#include "mamba_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MAMBA_FLAG_QK_NORM 0x4u          /* unit-length queries and keys */

/*
 * Bytes of workspace mamba_gdr_fwd needs (sizes only; callable without a GPU);
 * 0 when it needs none, (size_t)-1 for an invalid or unsupported shape.
 */
size_t mamba_gdr_workspace_size(int64_t B, int64_t H, int64_t G, int64_t P, int64_t N, int64_t L,
                                mamba_dtype_t in_dtype);

/*
 * The rule over whole sequences.
 *   initial_state : (B, H*P, N) fp32 or NULL (zeros).
 *   y             : (B, H*P, L) out_dtype, written.
 *   final_state   : (B, H*P, N) fp32, written, or NULL.
 */
int mamba_gdr_fwd(const void* q, const void* k, const void* v, const void* delta, const void* beta,
                  const float* A, const float* delta_bias, const float* initial_state,
                  const int32_t* lengths, void* y, float* final_state,
                  int64_t B, int64_t H, int64_t G, int64_t P, int64_t N, int64_t L,
                  int64_t q_stride, int64_t k_stride, int64_t v_stride, float scale,
                  mamba_dtype_t in_dtype, mamba_dtype_t out_dtype, unsigned flags,
                  void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * One token for every batch row, on a pool of states updated in place.
 *   state : (n_slots, H*P, N) fp32.
 *   slots : (B) int32 on the device: the state of row b is state[slots[b]]; NULL
 *           takes state[b] (then n_slots >= B is required).  A row whose slot is
 *           negative or not below n_slots is empty: its y is zero and no state is
 *           read or written for it.  A slot named by two rows of one call leaves
 *           that state unspecified (the rows run at the same time).
 *   q, k  : (B, G*N); v : (B, H*P); delta, beta : (B, H); y : (B, H*P) out_dtype,
 *           written.  No workspace is used.
 */
int mamba_gdr_update(float* state, const int32_t* slots, const void* q, const void* k, const void* v,
                     const void* delta, const void* beta, const float* A, const float* delta_bias, void* y,
                     int64_t B, int64_t H, int64_t G, int64_t P, int64_t N, int64_t n_slots,
                     int64_t q_stride, int64_t k_stride, int64_t v_stride, float scale,
                     mamba_dtype_t in_dtype, mamba_dtype_t out_dtype, unsigned flags, hipStream_t stream);

/*
 * Bytes of workspace mamba_gdr_bwd needs (sizes only; callable without a GPU),
 * (size_t)-1 for an invalid or unsupported shape.  With Pp and Np, P and N rounded up to
 * 64, it holds per value head and chunk of 32 tokens 19 KiB of operands and factors, 256 Pp
 * bytes of updates and gradients of v and 5 Pp Np bytes of states; where a key head has
 * more than one value head or P > 64, 256 Np bytes per key head and chunk; and a padded last
 * chunk of q, k, v and dy per row.  160 heads of 128 x 128, two to a key head, L = 2048: 1.55 GB.
 */
size_t mamba_gdr_bwd_workspace_size(int64_t B, int64_t H, int64_t G, int64_t P, int64_t N, int64_t L,
                                    mamba_dtype_t in_dtype, mamba_dtype_t grad_dtype);

/*
 * Gradients of mamba_gdr_fwd for a gradient dy of y and, optionally, dfinal_state of
 * the final state.  Nothing of the forward pass is kept: the states are recomputed.
 *   dy             : (B, H*P, L) grad_dtype.
 *   dfinal_state   : (B, H*P, N) fp32 or NULL (zeros).
 *   dq, dk         : (B, G*N, L) grad_dtype, written (summed over the value heads of a key
 *                    head, and through the normalisation with MAMBA_FLAG_QK_NORM).
 *   dv             : (B, H*P, L) grad_dtype, written.
 *   ddelta, dbeta  : (B, H, L) grad_dtype, written: gradients of the raw values.
 *   dA, ddelta_bias : (H) fp32, written (summed over batch rows and tokens), also when
 *                    delta_bias is NULL.
 *   dinitial_state : (B, H*P, N) fp32, written, or NULL.
 * All outputs are overwritten, dense, and zero for tokens behind a row's end.
 */
int mamba_gdr_bwd(const void* q, const void* k, const void* v, const void* delta, const void* beta,
                  const float* A, const float* delta_bias, const float* initial_state,
                  const int32_t* lengths, const void* dy, const float* dfinal_state,
                  void* dq, void* dk, void* dv, void* ddelta, void* dbeta, float* dA, float* ddelta_bias,
                  float* dinitial_state,
                  int64_t B, int64_t H, int64_t G, int64_t P, int64_t N, int64_t L,
                  int64_t q_stride, int64_t k_stride, int64_t v_stride, float scale,
                  mamba_dtype_t in_dtype, mamba_dtype_t grad_dtype, unsigned flags,
                  void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Test and diagnostic knobs, process-wide like mamba_set_test_knobs: how a call is
 * carried out, never what it computes (to fp32 rounding).  A workspace size asked
 * for before a change does not fit a call after it.
 *   kernel   : 0 the planner's choice; 1 token by token; 2 in chunks.
 *   segments : > 0: mamba_gdr_fwd in chunks cuts L into this many segments (at most one
 *              per chunk of 32 tokens); 0: the planner decides.
 * Returns MAMBA_ERR_SHAPE for other values.
 */
int mamba_gdr_set_test_knobs(int kernel, int64_t segments);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA_GDR_H_ */
