/*
 * peagle_w4.h -- C ABI of products with 4-bit weights on one GB300 (sm_103a):
 * a few rows times a matrix whose entries are 4-bit codes with a scale for
 * each group of inputs, for the projections and the LM head of a quantised
 * drafter.  Beside pe_linear and pe_linear_static (16-bit weights).
 *
 * Entry (n, j) of a matrix [n, k] is (code - 8) * scale[n][j / group], codes
 * 0 .. 15, scales bf16 (the P-EAGLE pages have no counterpart: their drafter
 * has 16-bit weights).
 *
 * Conventions are those of peagle.h: caller-owned device memory,
 * asynchronous on `stream`, host-checkable errors returned before anything is
 * launched, no C++ exception across the ABI, every tensor on the current
 * device.  No handle, no workspace, no device error: calls may overlap as
 * long as no buffer that one writes is used by the other.
 */
#ifndef PEAGLE_W4_H_
#define PEAGLE_W4_H_

#include <stdint.h>

#include "peagle.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of a packed matrix [n, k] (the layout is the library's own); 0 on a
 * bad argument.  group: 32, 64 or 128 inputs a scale; the last group of a row
 * may be shorter. */
int64_t pe_w4_bytes(int32_t n, int32_t k, int32_t group);

/* Lay out codes and scales once, as pe_w4_linear reads them.
 * codes [n, (k + 1) / 2] bytes, input 2 j in the low half of byte j and input
 * 2 j + 1 in the high half (the spare half of an odd k is not used); scales
 * [n, ceil(k / group)] bf16.  packed: pe_w4_bytes bytes, 16-byte aligned, not
 * overlapping the inputs.
 * PE_ERR_INVALID_ARGUMENT: n or k < 1, a group other than 32, 64 and 128, a
 * null or misaligned pointer.  PE_ERR_UNSUPPORTED: k past 2^17 (one
 * row of x in fp32 has to fit into the shared memory of eight SMs), n past 2^24. */
pe_status pe_w4_pack(const uint8_t* codes, const void* scales, int32_t n, int32_t k,
                     int32_t group, void* packed, void* stream);

/* Round a matrix [n, k] of `dtype` (pe_dtype), rows w_stride elements apart,
 * to 4 bits and lay it out.  Each group's scale is the largest |w| of the
 * group over 7, rounded to bf16; a code is the nearest whole number of scales
 * (ties to even), at most 7 and at least -8.  A group of zeros has the scale
 * 0.  Entries are expected to be finite.  Refusals as pe_w4_pack's, and a
 * stride shorter than a row. */
pe_status pe_w4_quantize(const void* w, int32_t dtype, int64_t w_stride, int32_t n, int32_t k,
                         int32_t group, void* packed, void* stream);

/* y[r, i] = sum_j x[r, j] * (code[i, j] - 8) * scale[i, j / group], r < rows.
 * x [rows, k] of x_dtype and y [rows, n] of y_dtype (pe_dtype): bf16 -> bf16,
 * bf16 -> fp32 or fp32 -> fp32; rows x_stride and y_stride elements apart, y
 * not overlapping x.  Products are exact, sums and scales are in fp32, in an
 * order that depends on the sizes and the device only; y is rounded once.
 * x is held to 2^-38 of the largest element of its row: exactly down to 2^-30 of
 * that in bf16 and to 2^-14 in fp32, whose smaller elements have fewer bits than
 * their 24 (at 2^-24 of the largest 14).  A row with an infinite or NaN
 * element gives infinities and NaN, the other rows are as they would be.
 * Scales are any finite bf16 numbers.  Where a sum leaves fp32's range on the
 * way (never below scales of 2^92), that result is summed again in 64 bits, by
 * one thread: right, but slow where there are many.
 * Made for a few rows: up to 32 cost one pass over the weights, each further
 * 32 another (fewer where 32 rows of x do not fit into the shared memory of
 * eight SMs).
 * PE_ERR_INVALID_ARGUMENT: rows < 1, sizes as pe_w4_pack, another
 * combination of types, a stride shorter than a row, a null pointer, packed
 * not 16-byte aligned, x or y not aligned to its elements. */
pe_status pe_w4_linear(const void* packed, int32_t n, int32_t k, int32_t group, int32_t rows,
                       int32_t x_dtype, const void* x, int64_t x_stride, int32_t y_dtype, void* y,
                       int64_t y_stride, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PEAGLE_W4_H_ */
