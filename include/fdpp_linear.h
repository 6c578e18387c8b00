/*
 * fdpp_linear.h -- C ABI of libfdpp's 8-bit linear layers on GB300 (sm_103a): the RMS norm that comes
 * before a linear layer, with the residual's addition and an output in 8 bits, and the linear layer
 * itself on operands in 8 bits with block scales.
 *
 *     fdpp_rms_norm      x + residual     -> normed rows, in e4m3 with scales (or in x's type); the sum
 *     fdpp_scaled_gemm   e4m3 x, e4m3 w   -> y = x W^T, for any number of rows
 *
 * 8-bit operands are e4m3 (4 exponent bits, 3 of mantissa, largest value 448), each with one fp32 scale
 * for FDPP_SCALE_BLOCK consecutive channels: a value stands for e4m3 x scale. Activations have a scale for
 * every row and block of channels, weights one for every block of rows and block of channels. (The norm is the only call
 * here that makes such operands; where no norm precedes a layer they are the caller's.)
 *
 * Conventions: as in fdpp.h (caller-owned DEVICE buffers, stream-ordered calls without a host
 * synchronisation, synchronous argument errors with fdpp_last_error()). Offsets are 64-bit.
 */
#ifndef FDPP_LINEAR_H
#define FDPP_LINEAR_H

#include <stddef.h>
#include <stdint.h>

#include "fdpp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A type of these calls besides fdpp_dtype's. */
#define FDPP_E4M3 2
/* Channels (and weight rows) that share a scale. */
#define FDPP_SCALE_BLOCK 128
/* Most channels of a row that fdpp_rms_norm takes (a row stays in one CTA's registers). */
#define FDPP_NORM_MAX_DIM 32768

/* ---- RMS norm ------------------------------------------------------------------------------- */

typedef struct fdpp_norm_params {
    int num_tokens;          /* T >= 0 rows */
    int dim;                 /* channels of a row: a multiple of 8, at most FDPP_NORM_MAX_DIM */
    int dtype;               /* fdpp_dtype of x, residual, weight and sum_out */
    int out_dtype;           /* dtype, or FDPP_E4M3 */
    long long x_stride, residual_stride, out_stride, sum_stride;
                             /* elements from one row to the next: >= dim, and multiples of 16 bytes (an e4m3
                                output's: of 8; fdpp_scaled_gemm takes multiples of 16) */
    long long scale_stride;  /* floats from one row's scales to the next, >= ceil(dim / 128) (E4M3) */
    float eps;               /* >= 0, finite */
    float weight_offset;     /* added to every weight (1 where weights are stored as w - 1) */
} fdpp_norm_params;

/* For every row: r = x + residual, y = r / sqrt(mean(r^2) + eps) (weight + weight_offset), in fp32 (r
 * before it is rounded; the squares are summed in fp32: where their sum reaches 2^128, as with |r| = 2^64 / sqrt(dim)
 * throughout, it is infinite and y 0. Small r keep their accuracy with any eps; a row of zeros with eps 0 is 0 / 0, NaN);
 * sum_out = r and out = y, each rounded once. With out_dtype FDPP_E4M3, for every
 * block of 128 channels (the last may be shorter)
 *     scale = max(max |y| / 448, 2^-126),   out = y (1 / scale) rounded to nearest even,
 * where a NaN among a block's values makes its scale and all its values NaN.
 *   x            DEVICE [T][dim], 16-byte aligned, as residual, out and sum_out.
 *   residual     DEVICE [T][dim], or NULL (r = x).
 *   weight       DEVICE [dim], 16-byte aligned, or NULL (all 1; weight_offset is not added).
 *   out          DEVICE [T][dim] of out_dtype. May be x where the types and strides are the same.
 *   scales       DEVICE float [T][ceil(dim / 128)], 4-byte aligned (E4M3); otherwise NULL.
 *   sum_out      DEVICE [T][dim], or NULL. May be residual or x where the strides are the same.
 * Otherwise the buffers do not overlap. With T = 0 they may be NULL. */
fdpp_status fdpp_rms_norm(const void* x, const void* residual, const void* weight, const fdpp_norm_params* p,
                          void* out, float* scales, void* sum_out, fdpp_stream stream);

/* ---- linear layer --------------------------------------------------------------------------- */

typedef struct fdpp_scaled_gemm_params {
    int M, N, K;             /* M >= 0, N >= 1, K >= 16 and a multiple of 16 */
    int out_dtype;           /* fdpp_dtype of y */
    long long x_stride, w_stride;   /* bytes from one row to the next: >= K, multiples of 16 */
    long long y_stride;      /* elements from one row of y to the next, >= N */
    long long x_scale_stride;       /* floats from one row's scales to the next, >= ceil(K / 128) */
    int split_k;             /* ranges of K that an output tile is made of, added up in order: 0 chooses, otherwise
                                1 .. min(ceil(K / 128), 8); not followed where, with M > 64, tiles of 256 x 256 by
                                pairs of CTAs fill the GPU by themselves */
} fdpp_scaled_gemm_params;

/* Bytes of workspace (the sticky error word). 0 if the parameters are invalid. */
size_t fdpp_scaled_gemm_workspace_size(const fdpp_scaled_gemm_params* p);

/* y[m][n] = sum_b x_scales[m][b] w_scales[n / 128][b] sum_{k in block b} x[m][k] w[n][k]: each block's
 * products are summed by the tensor cores in fp32, then scaled and added in fp32; y is rounded once.
 * The two scales' product is taken in fp32, of any two scales whose product is finite or one of which is 0. Below 2^-126 it
 * has fewer bits, which is less than 2^-125 of y for each block; an infinite one makes the block's part infinite, or NaN.
 *   x          DEVICE e4m3 [M][K], 16-byte aligned.
 *   x_scales   DEVICE float [M][ceil(K / 128)], 4-byte aligned.
 *   w          DEVICE e4m3 [N][K] (a linear layer's weight as stored), 16-byte aligned. As in
 *              fdpp_flat_gemm, a call may start reading w while the kernel before it on the stream
 *              finishes: w must not be written by that kernel (a layer's weights are not).
 *   w_scales   DEVICE float [ceil(N / 128)][ceil(K / 128)], 4-byte aligned.
 *   workspace  DEVICE, 256-byte aligned, >= 256 bytes, zeroed before its first use (it collects the
 *              calls' error bits; read them with fdpp_read_error of fdpp_cache.h).
 *   y          DEVICE [M][N] of out_dtype, aligned to its elements (stores are wider where y and its rows
 *              are 16-byte aligned). With M = 0 it, x and x_scales may be NULL. */
fdpp_status fdpp_scaled_gemm(const void* x, const float* x_scales, const void* w, const float* w_scales,
                             const fdpp_scaled_gemm_params* p, void* workspace, size_t workspace_bytes, void* y,
                             fdpp_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* FDPP_LINEAR_H */
