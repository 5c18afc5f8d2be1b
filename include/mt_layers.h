/*
 * mt_layers — the operators of a transformer's feed-forward block around the
 * products of mt_sgemm.h, for one NVIDIA GB300 (sm_103a).  Same library
 * (libmtsgemm.so), same rules: device pointers owned by the caller, calls
 * return before the work finishes (stream-ordered, no implicit
 * synchronisation), every entry point returns an mt_status and launches
 * nothing on an argument error, no state is kept between calls, all entry
 * points are thread-safe, and there is no CPU fallback.  Scratch a call
 * needs comes from the current device's stream-ordered pool and goes back
 * to it on the same stream.
 *
 * Matrices are row-major with a row pitch in elements (at least the row's
 * length); rows may be strided, columns are contiguous.  Types are mt_dtype
 * codes.  "16-bit" is MT_DTYPE_F16 or MT_DTYPE_BF16.  All sums, statistics
 * and activations are computed in fp32 and rounded once, to nearest even,
 * when a result is stored.
 */
#ifndef MT_LAYERS_H
#define MT_LAYERS_H

#include "mt_sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* An unused fp8 scale is never smaller than this (2^-126): a row of zeros
 * gets it, and its 8-bit values are zeros. */
#define MT_SCALE_MIN 1.17549435082228751e-38f
/* Largest finite e4m3 value. */
#define MT_E4M3_MAX 448.0f

/*
 * Root-mean-square norm with the residual's addition:
 *
 *     h[i][k] = x[i][k] + residual[i][k]            (residual NULL: x)
 *     r[i]    = 1 / sqrt(mean_k h[i][k]^2 + eps)
 *     y[i][k] = h[i][k] * r[i] * weight[k]          (weight NULL: ones)
 *
 * h is summed in fp32 and enters the norm unrounded.  Written: h in x's type
 * (h NULL: not written), r to `rstd` (rows floats; NULL: not written; the
 * gradient reads it), and y either in x's type (out_dtype == dtype) or in 8
 * bits with one scale per row (out_dtype == MT_DTYPE_E4M3):
 *
 *     scale[i] = max(max_k |y[i][k]| / 448, 2^-126)
 *     y8[i][k] = e4m3(y[i][k] / scale[i])           (nearest even)
 *
 * A NaN in a row makes the whole row, its r and its scale NaN; an infinite
 * element makes r 0 and its own y NaN (and, in 8 bits, the whole row and its
 * scale NaN).
 */
typedef struct {
    int64_t rows, d;
    const void *x;
    int64_t ldx;
    const void *residual;
    int64_t ldr;
    const void *weight;
    void *h;
    int64_t ldh;
    void *y;
    int64_t ldy;
    float *scale;         /* rows floats; out_dtype MT_DTYPE_E4M3 only, else NULL */
    float *rstd;
    float eps;            /* finite, >= 0 */
    int32_t dtype;        /* x, residual, h: MT_DTYPE_F16, _BF16 or _F32 */
    int32_t out_dtype;    /* y: dtype or MT_DTYPE_E4M3 */
    int32_t weight_dtype; /* dtype or MT_DTYPE_F32 */
} mt_rms_norm_args;

/*
 * rows == 0 does nothing; d == 0 writes r (and scale) of empty rows.  h may
 * be x or residual itself, and y may be x itself (same pointer and pitch);
 * any other overlap of an output with an input or another output is
 * MT_ERR_ALIAS.  Pointers must be aligned to their element.  Other errors:
 * MT_ERR_INVALID_ARG (NULL args, negative or too large size, pitch shorter
 * than a row, missing pointer, unknown type combination, eps negative or
 * not finite), MT_ERR_NO_DEVICE, MT_ERR_LAUNCH.
 */
MT_API mt_status mt_rms_norm(const mt_rms_norm_args *args, cudaStream_t stream);

/*
 * The gradient of mt_rms_norm: with xhat = h * rstd and g = dy * weight,
 *
 *     dx[i][k]   = rstd[i] * (g[i][k] - xhat[i][k] * mean_k(g[i] * xhat[i])) + dh[i][k]
 *     dweight[k] = sum_i dy[i][k] * xhat[i][k]
 *
 * dy is the gradient of y (of the 8-bit y as if it were not rounded), dh the
 * gradient that reaches h directly (the residual stream; NULL: none).  dx is
 * the gradient of x and of the residual alike.  h and rstd are the forward
 * call's (h: x itself where there was no residual).  dweight: d floats, each
 * a sum over the rows in a fixed order (the same call gives the same bits);
 * NULL: not computed.
 */
typedef struct {
    int64_t rows, d;
    const void *dy;
    int64_t lddy;
    const void *h;
    int64_t ldh;
    const void *weight;   /* NULL: ones */
    const float *rstd;
    const void *dh;
    int64_t lddh;
    void *dx;
    int64_t lddx;
    float *dweight;
    int32_t dtype;        /* dy, h, dh, dx: MT_DTYPE_F16, _BF16 or _F32 */
    int32_t weight_dtype; /* dtype or MT_DTYPE_F32 */
} mt_rms_norm_backward_args;

/* dx may be dy or dh itself (same pointer and pitch); any other overlap of an
 * output is MT_ERR_ALIAS.  rows == 0 writes zeros to dweight.  Other errors
 * as mt_rms_norm, and MT_ERR_CUDA when scratch cannot be allocated. */
MT_API mt_status mt_rms_norm_backward(const mt_rms_norm_backward_args *args,
                                      cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MT_LAYERS_H */
