/*
 * mamba_state_cache.h -- C ABI of the 8-bit state cache: rows of fixed-size
 * per-request state (of the scan, the convolution, the SSD layer or the gated
 * delta rule, laid out flat) kept in a quarter of their fp32 size while the
 * request waits or its prefix is shared, and read back when it runs.  The
 * conventions of mamba_scan.h hold.
 *
 * A cached row of n numbers is n signed bytes and, for every 32 consecutive
 * numbers (the last group may be shorter), one byte e8: the numbers stand for
 * code * 2^(e8 - 127).  Writing takes the smallest power with
 * 127 * 2^(e8 - 127) >= max|x| of the group (1 <= e8 <= 248) and rounds x / 2^(e8 - 127) to
 * nearest, ties to even: each number is off by at most half a step, max|x|/127 at
 * most (numbers beyond 127 * 2^121 = 3.38e38 are held to it).  A group holding an infinity or a NaN gets e8 = 255 and reads back as NaN.
 * Reading is exact in fp32 and in bf16.
 *
 *   state  : (rows, n) dtype (fp32 or bf16), read by _write, written by _read.
 *   slots  : (rows) int32 on the device: row r is kept in slot slots[r]; NULL means
 *            slot r (then n_slots >= rows is required).  A slot that is negative or
 *            not below n_slots: _write leaves the row out, _read gives zeros (a
 *            request without a cached state starts from zero).  _read may name a
 *            slot for several rows; a slot written by two rows of one call is left
 *            unspecified.
 *   codes  : (n_slots, n) int8.   exps : (n_slots, ceil(n / 32)) uint8.
 *
 * Sizes: rows, n, n_slots >= 1; rows * n < 2^46, and fewer than 2^24 workgroups of 1024
 * consecutive numbers of a row (4096 for vector accesses and rows * n of 2^23 or more), so that
 * a launch has fewer than 2^32 threads.  Alignment: element size
 * (16 bytes and n % 4 == 0 select vector accesses).  No workspace.
 */
#ifndef MAMBA_STATE_CACHE_H_
#define MAMBA_STATE_CACHE_H_

#include "mamba_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

int mamba_state_cache_write(const void* state, const int32_t* slots, int8_t* codes, uint8_t* exps,
                            int64_t rows, int64_t n, int64_t n_slots, mamba_dtype_t dtype, hipStream_t stream);

int mamba_state_cache_read(const int8_t* codes, const uint8_t* exps, const int32_t* slots, void* state,
                           int64_t rows, int64_t n, int64_t n_slots, mamba_dtype_t dtype, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA_STATE_CACHE_H_ */
