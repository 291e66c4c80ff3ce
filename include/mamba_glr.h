/*
 * mamba_glr.h -- C ABI of the gated linear recurrence: the sequence layer that
 * keeps one number per channel, with a decay and an input gate taken from the
 * token.  It stands beside mamba_scan_fwd (mamba_scan.h), which keeps N numbers
 * per channel: the same sequence-fastest layout, the same output gate, and the
 * conventions of that header (device pointers, host checks before any launch,
 * status codes, the caller's workspace, graph capture) hold for every call here.
 *
 * What the calls compute, per batch row b and channel d:
 *     s_t = sigmoid(r[b,d,t] + r_bias[d])
 *     a_t = exp(A[d] s_t),  n_t = sqrt(1 - a_t^2)
 *     g_t = sigmoid(i[b,d,t] + i_bias[d])        (1 without i)
 *     h_t = a_t h_(t-1) + n_t g_t x[b,d,t]
 *     y_t = h_t z_t sigmoid(z_t)                 (h_t without z)
 * n_t keeps the variance of h at that of the gated inputs, whatever the decay.
 * With MAMBA_FLAG_BLEND the state is blended with the input, a_t = 1 - s_t and
 * n_t = s_t (A is not used): the gate of "Mamba 与状态空间模型" section 06,
 * theorem 1, h <- (1 - g) h + g x.
 *
 * Arguments shared by the calls
 *   x, r     : (B, D, L) in_dtype.  i, z : (B, D, L) in_dtype or NULL.
 *   x_stride, r_stride, i_stride, z_stride : elements from one batch row to the
 *              next (at least D*L), so that the inputs may be channel ranges of one
 *              projection's output.  Those of absent inputs are not looked at.
 *   A        : (D) fp32, below zero; NULL with MAMBA_FLAG_BLEND.  (A = 0 keeps the state
 *              and takes no input; the gradient of A is infinite there, and comes out as very
 *              large numbers.  A below -2e38, -inf too, counts as -2e38: nothing of the state is kept.
 *              A > 0 gives NaN.)
 *   r_bias, i_bias : (D) fp32 or NULL (zeros).  An infinite one holds its gate open or closed.
 *   states   : (B, D) fp32.
 *   lengths  : (B) int32 on the device, or NULL (every row has L tokens).
 *              Row b ends after lengths[b] tokens (values are held to 0 .. L):
 *              what its inputs hold behind that is not looked at, be it NaN,
 *              its outputs and gradients there are zero, and its final state is
 *              the one after lengths[b] tokens (of none: the initial state, whatever the
 *              channel's parameters hold).
 *
 * Sizes: B, D, L >= 1; B*D*L < 2^46, strides < 2^46 / B; and no launch of 2^32 threads or more:
 * B*D*(ceil(L/512) + ceil(L/2048)) < 2^26 is enough (mamba_glr_update: B*ceil(D/256) < 2^24).  in_dtype and the
 * output dtypes may each be MAMBA_F32 or MAMBA_BF16.  Alignment: every array to its element
 * size; workspaces 256 bytes.
 * A NaN among the inputs of a token leaves the outputs of the tokens before it as they are;
 * from that token on, every output and state that it reaches is NaN.  So does an infinite x or z, with
 * NaN or infinities; an infinite r or i is a gate wholly open or closed.  In the backward pass any
 * gradient of such a channel may be NaN, in the batch row that holds it, and that channel's sums.
 * State, gates and sums are fp32.  The results are deterministic (sums in a fixed order, no
 * atomics): the same call gives the same bits.  Past 256 tokens, B, like every other size, takes part in
 * the choice of how a row is cut over waves and segments, and those agree to fp32 rounding only.
 */
#ifndef MAMBA_GLR_H_
#define MAMBA_GLR_H_

#include "mamba_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MAMBA_FLAG_BLEND 0x8u            /* a = 1 - s, n = s */

/*
 * Bytes of workspace mamba_glr_fwd needs (sizes only; callable without a GPU);
 * 0 when it needs none, (size_t)-1 for an invalid shape.
 */
size_t mamba_glr_workspace_size(int64_t B, int64_t D, int64_t L);

/*
 * The recurrence over whole sequences.
 *   initial_state : (B, D) fp32 or NULL (zeros).
 *   y             : (B, D, L) out_dtype, written, dense.
 *   final_state   : (B, D) fp32, written, or NULL.  Not the initial state's array: where a row is
 *                   cut into segments, some read the one while another writes the other.
 */
int mamba_glr_fwd(const void* x, const void* r, const void* i, const void* z, const float* A,
                  const float* r_bias, const float* i_bias, const float* initial_state,
                  const int32_t* lengths, void* y, float* final_state, int64_t B, int64_t D, int64_t L,
                  int64_t x_stride, int64_t r_stride, int64_t i_stride, int64_t z_stride,
                  mamba_dtype_t in_dtype, mamba_dtype_t out_dtype, unsigned flags,
                  void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * One token for every batch row, on a pool of states updated in place.
 *   state : (n_slots, D) fp32.
 *   slots : (B) int32 on the device: the state of row b is state[slots[b]]; NULL
 *           takes state[b] (then n_slots >= B is required).  A row whose slot is
 *           negative or not below n_slots is empty: its y is zero and no state is
 *           read or written for it.  A slot named by two rows of one call leaves
 *           that state unspecified (the rows run at the same time).
 *   x, r, i, z : (B, D); y : (B, D) out_dtype, written.  No workspace is used.
 */
int mamba_glr_update(float* state, const int32_t* slots, const void* x, const void* r, const void* i,
                     const void* z, const float* A, const float* r_bias, const float* i_bias, void* y,
                     int64_t B, int64_t D, int64_t n_slots, int64_t x_stride, int64_t r_stride,
                     int64_t i_stride, int64_t z_stride, mamba_dtype_t in_dtype, mamba_dtype_t out_dtype,
                     unsigned flags, hipStream_t stream);

/* Bytes of workspace mamba_glr_bwd needs, (size_t)-1 for an invalid shape. */
size_t mamba_glr_bwd_workspace_size(int64_t B, int64_t D, int64_t L);

/*
 * Gradients of mamba_glr_fwd for a gradient dy of y and, optionally, dfinal_state of
 * the final state.  Nothing of the forward pass is kept: the states are recomputed.
 *   dy              : (B, D, L) grad_dtype, dense.
 *   dfinal_state    : (B, D) fp32 or NULL (zeros).
 *   dx, dr, di, dz  : (B, D, L) grad_dtype, written, dense; di and dz NULL where i and z are
 *                     (required otherwise).
 *   dA, dr_bias, di_bias : (D) fp32, written (summed over batch rows and tokens), also where the
 *                     bias is NULL; dA NULL with MAMBA_FLAG_BLEND, di_bias NULL without i.
 *   dinitial_state  : (B, D) fp32, written, or NULL.
 */
int mamba_glr_bwd(const void* x, const void* r, const void* i, const void* z, const float* A,
                  const float* r_bias, const float* i_bias, const float* initial_state,
                  const int32_t* lengths, const void* dy, const float* dfinal_state, void* dx, void* dr,
                  void* di, void* dz, float* dA, float* dr_bias, float* di_bias, float* dinitial_state,
                  int64_t B, int64_t D, int64_t L, int64_t x_stride, int64_t r_stride, int64_t i_stride,
                  int64_t z_stride, mamba_dtype_t in_dtype, mamba_dtype_t grad_dtype, unsigned flags,
                  void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Test and diagnostic knobs, process-wide like mamba_set_test_knobs: how a call is
 * carried out, never what it computes (to fp32 rounding).  A workspace size asked
 * for before a change does not fit a call after it.
 *   waves    : > 0: at most this many waves of a workgroup on a row, 1 .. 16 (a wave takes 512 tokens at a
 *              time); 0: the planner decides.
 *   segments : > 0: L is cut into this many segments (at most one per 8 tokens; in mamba_glr_bwd
 *              at least as many as its waves need); 0: the planner decides.
 * Returns MAMBA_ERR_SHAPE for other values.
 */
int mamba_glr_set_test_knobs(int waves, int64_t segments);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA_GLR_H_ */
