/*
 * mamba_norm.h -- C ABI of the layer norm over channels: the norm in front of a
 * block, and the norm per head of a layer's output with an output gate, which
 * mamba_gdr_fwd leaves to what follows it (mamba_ssd_fwd and mamba_glr_fwd take a z of
 * their own, in front of the norm, or none).  The conventions of mamba_scan.h hold.
 *
 * For every token (b, t) and group of Dg = D / groups consecutive channels:
 *     xh = (x - mean) / sqrt(var + eps)          (var: the mean of (x - mean)^2)
 *     y  = (xh weight[d] + bias[d]) z sigmoid(z)  (without the gate where z is NULL)
 * With MAMBA_FLAG_RMS, xh = x / sqrt(mean of x^2 + eps).
 *
 *   x      : (B, D, L) in_dtype.  z : (B, D, L) in_dtype or NULL.  L = 1 is the
 *            token-major form: (rows, D), channels consecutive.
 *   x_stride, z_stride : elements from one batch row to the next (at least D*L).
 *   weight : (D) fp32 or NULL (ones).  bias : (D) fp32 or NULL (zeros).
 *
 * Sizes: B, D, L >= 1; D a multiple of groups; B*D*L < 2^46, strides < 2^46 / B; and no launch of 2^32
 * threads or more: D < 2^27, B*groups*ceil(L/32) < 2^22 and B*D*ceil(L/64) < 2^29 are enough.
 * in_dtype and the output dtypes may each be MAMBA_F32 or MAMBA_BF16.  eps >= 0.  Alignment: every array to
 * its element size; workspaces 256 bytes.  Statistics and sums are fp32; the variance is taken
 * around the mean, or around one of the numbers for a few of them, never as a difference of large squares.  (The mean is
 * rounded to fp32, so x - mean is off by 2^-24 of a large offset; numbers more than 1e17 from the mean may overflow the variance.)  A NaN
 * or an infinity stays in its own token and group (dweight and dbias aside).  Deterministic: sums in a
 * fixed order, no atomics: the same call gives the same bits.  B takes part in how channel-major groups of more
 * than 256 channels are cut, which agrees to fp32 rounding; token-major rows and smaller groups have the
 * same bits in a batch of any size (dweight and dbias aside).
 */
#ifndef MAMBA_NORM_H_
#define MAMBA_NORM_H_

#include "mamba_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MAMBA_FLAG_RMS 0x10u             /* no mean taken off */

/*
 * Bytes of workspace mamba_layer_norm_fwd needs (sizes only; callable without a GPU); 0 when it
 * needs none, (size_t)-1 for an invalid shape.
 */
size_t mamba_layer_norm_workspace_size(int64_t B, int64_t D, int64_t L, int64_t groups);

/* y : (B, D, L) out_dtype, written, dense. */
int mamba_layer_norm_fwd(const void* x, const void* z, const float* weight, const float* bias, void* y,
                         int64_t B, int64_t D, int64_t L, int64_t groups, int64_t x_stride,
                         int64_t z_stride, float eps, mamba_dtype_t in_dtype, mamba_dtype_t out_dtype,
                         unsigned flags, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace mamba_layer_norm_bwd needs, (size_t)-1 for an invalid shape. */
size_t mamba_layer_norm_bwd_workspace_size(int64_t B, int64_t D, int64_t L, int64_t groups);

/*
 * Gradients for a gradient dy of y; the statistics are recomputed.
 *   dy            : (B, D, L) grad_dtype, dense.
 *   dx, dz        : (B, D, L) grad_dtype, written, dense; dz NULL where z is (required otherwise).
 *   dweight, dbias : (D) fp32, written (summed over batch rows and tokens), also where weight or
 *                   bias is NULL.
 */
int mamba_layer_norm_bwd(const void* x, const void* z, const float* weight, const float* bias,
                         const void* dy, void* dx, void* dz, float* dweight, float* dbias, int64_t B,
                         int64_t D, int64_t L, int64_t groups, int64_t x_stride, int64_t z_stride,
                         float eps, mamba_dtype_t in_dtype, mamba_dtype_t grad_dtype, unsigned flags,
                         void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA_NORM_H_ */
