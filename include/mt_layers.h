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
 * length); rows may be strided, columns are contiguous.  Matrices overlap when
 * they share an element: columns side by side in rows of one pitch in bytes do
 * not; of other pitches the whole spans count.  Types are mt_dtype codes.
 * "16-bit" is MT_DTYPE_F16 or MT_DTYPE_BF16.  All sums, statistics and
 * activations are computed in fp32 and rounded once, to nearest even, when a
 * result is stored.
 */
#ifndef MT_LAYERS_H
#define MT_LAYERS_H

#include "mt_sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* No fp8 scale is smaller than this (2^-126): a row of zeros gets it, and its
 * 8-bit values are zeros. */
#define MT_SCALE_MIN 1.17549435082228751e-38f
/* Largest finite e4m3 value. */
#define MT_E4M3_MAX 448.0f

/*
 * Root-mean-square norm with the residual's addition:
 *
 *     h[i][k] = x[i][k] + residual[i][k]            (residual NULL: x)
 *     r[i]    = 1 / sqrt(mean_k h[i][k]^2 + eps)    (0 for 1 / 0)
 *     y[i][k] = h[i][k] * r[i] * weight[k]          (weight NULL: ones)
 *
 * A row whose mean square is 0 with eps 0 gets r = 0: its y is zeros, and the
 * gradient below leaves it dh alone.  h is summed in fp32 and enters the norm
 * unrounded.  Written: h in x's type (h NULL: not written), r to `rstd` (rows
 * floats; NULL: not written; the gradient reads it), and y either in x's type
 * (out_dtype == dtype) or in 8 bits with one scale per row (out_dtype ==
 * MT_DTYPE_E4M3):
 *
 *     scale[i] = max(max_k |y[i][k]| / 448, 2^-126)
 *     y8[i][k] = e4m3(y[i][k] / scale[i])           (nearest even)
 *
 * with the maximum as max_k |h * weight| * r and the quotient as y * (1 /
 * scale), all in fp32: within 4 ulp before its rounding, so a value that near
 * the middle between two e4m3 values may become either (h * weight has to fit
 * fp32, as y has).
 *
 * A NaN in a row makes the whole row, its r and its scale NaN; a mean square
 * past fp32's range (values past 1.8e19) makes r and a finite y 0; an infinite
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
 * MT_ERR_INVALID_ARG (NULL args, a negative size, d past 2^31 - 512, rows past
 * 2^31 - 1, pitch shorter than a row, missing pointer, unknown type
 * combination, eps negative or not finite), MT_ERR_NO_DEVICE, MT_ERR_LAUNCH.
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
    int32_t fault_inject; /* test hook, 0 = off: 1 = the copies that rows starting
                             on 16 bytes arrive by are not issued, so the waits
                             on them run out, dx and dweight hold nothing of
                             use and mt_check_device_status returns
                             MT_ERR_TIMEOUT */
    int32_t reserved;     /* 0 */
} mt_rms_norm_backward_args;

/* dx may be dy or dh itself (same pointer and pitch); any other overlap of an
 * output is MT_ERR_ALIAS.  rows == 0 writes zeros to dweight.  Other errors
 * as mt_rms_norm, and MT_ERR_CUDA when scratch cannot be allocated. */
MT_API mt_status mt_rms_norm_backward(const mt_rms_norm_backward_args *args,
                                      cudaStream_t stream);

/* Activations of mt_linear, in fp32: identity, max(z, 0) (a NaN stays one),
 * z * Phi(z) with the normal distribution's Phi, its tanh form
 * z / 2 * (1 + tanh(sqrt(2/pi) * (z + 0.044715 z^3))), z / (1 + exp(-z)).
 * Evaluated to 2^-20 of the result where Y is fp32 (the tanh form's argument,
 * -2 u say, adds 5 |u| 2^-24 of it), to 2^-15 of it before its rounding where
 * Y is 16-bit; there, what is below 2^-110 may be zero. */
typedef enum {
    MT_ACT_NONE = 0,
    MT_ACT_RELU = 1,
    MT_ACT_GELU = 2,
    MT_ACT_GELU_TANH = 3,
    MT_ACT_SILU = 4
} mt_activation;

/*
 * The product with bias, activation and residual in its epilogue:
 *
 *     z[i][j] = (scale_a[i] * scale_b[j] *) sum_k A[i][k] * B[k][j]  + bias[j]
 *     Y[i][j] = act(z[i][j]) + residual[i][j]
 *
 * A is M x K, B is K x N (B[k*ldb + j]) or, with trans_b, stored N x K
 * (B[j*ldb + k]); bias, residual and Z may be NULL.  Z receives z (the
 * pre-activation, which the gradient of an activation needs).  A and B hold
 * 16-bit values (both the same type, no scales), or e4m3 values with fp32
 * scales for every row of A and every column of B (trans_b only: both
 * operands K-contiguous, as mt_rms_norm writes its 8-bit rows).  Products
 * and sums are fp32 on the tensor cores; Y, Z and residual have out_dtype.
 */
typedef struct {
    int64_t M, N, K;
    const void *A;
    int64_t lda;
    const void *B;
    int64_t ldb;
    void *Y;
    int64_t ldy;
    void *Z;
    int64_t ldz;
    const void *residual;
    int64_t ldr;
    const float *bias;     /* N floats */
    const float *scale_a;  /* M floats; e4m3 only */
    const float *scale_b;  /* N floats; e4m3 only */
    int32_t trans_b;       /* 0 or 1 */
    int32_t dtype;         /* A, B: MT_DTYPE_F16, _BF16 or _E4M3 */
    int32_t out_dtype;     /* Y, Z, residual: dtype or MT_DTYPE_F32; for e4m3
                              inputs MT_DTYPE_F16, _BF16 or _F32 */
    int32_t activation;    /* mt_activation */
    int32_t fault_inject;  /* test hook, 0 = off: 1 = the copy threads issue
                              nothing, so the waits on their data run out, Y is
                              left unwritten and mt_check_device_status returns
                              MT_ERR_TIMEOUT */
    int32_t reserved;      /* 0 */
} mt_linear_args;

/*
 * M or N == 0 does nothing; K == 0 gives act(bias) + residual.  residual may
 * be Y itself (same pointer and pitch); any other overlap of Y or Z with an
 * operand or with each other is MT_ERR_ALIAS.  TMA reads A and B in place
 * when their base is 16-byte aligned and their row pitch a multiple of 16
 * bytes; otherwise the call first copies them into padded scratch.  Nothing
 * depends on the alignment of the other operands.  Errors as mt_rms_norm,
 * MT_ERR_UNSUPPORTED for more than 2^31 - 1 tiles, and MT_ERR_CUDA when the
 * driver's tensor-map encoder cannot be found or scratch cannot be
 * allocated.
 */
MT_API mt_status mt_linear(const mt_linear_args *args, cudaStream_t stream);

/*
 * The launch mt_linear would make for these arguments on a GPU with `sms`
 * SMs, without launching anything (pointers are inspected for alignment
 * only and may be NULL).  bm: rows of Y per tile, bn: columns; split_k:
 * CTAs that share a tile's K; vec_ab: 1 when A and B are read in place;
 * workspace_bytes: the scratch for their copies.  Fields that describe other
 * kernels are 0.
 */
MT_API mt_status mt_linear_plan(const mt_linear_args *args, int sms, mt_plan *out);

/*
 * The gradient of mt_linear with 16-bit inputs: with dz = dY * act'(Z), in
 * fp32 and rounded to dtype for the two products,
 *
 *     dA       = dz * B^T                    M x K, dtype
 *     dB       = A^T * dz, stored as B is    K x N (N x K with trans_b), db_dtype
 *     dbias[j] = sum_i dz[i][j]              N floats, of the unrounded dz, in
 *                                            a fixed order (same bits each time)
 *
 * The residual's gradient is dY itself.  Z is the forward call's
 * pre-activation (not read for MT_ACT_NONE).  dA, dB and dbias may each be
 * NULL: not computed; B is read for dA only, A for dB only.
 */
typedef struct {
    int64_t M, N, K;
    const void *dY;
    int64_t lddy;
    const void *Z;
    int64_t ldz;
    const void *A;
    int64_t lda;
    const void *B;
    int64_t ldb;
    void *dA;
    int64_t ldda;
    void *dB;
    int64_t lddb;
    float *dbias;
    int32_t trans_b;    /* 0 or 1 */
    int32_t dtype;      /* dY, Z, A, B, dA: MT_DTYPE_F16 or MT_DTYPE_BF16 */
    int32_t db_dtype;   /* dB: dtype or MT_DTYPE_F32 */
    int32_t activation; /* mt_activation */
} mt_linear_backward_args;

/* An empty sum gives zeros (M == 0: dB and dbias; N == 0: dA).  Outputs
 * overlap nothing (MT_ERR_ALIAS).  Scratch: dz, unless the activation is the
 * identity and TMA reads dY in place, column sums for dbias, and copies of
 * operands TMA cannot read in place.  Other errors as mt_linear. */
MT_API mt_status mt_linear_backward(const mt_linear_backward_args *args, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MT_LAYERS_H */
