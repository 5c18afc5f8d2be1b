/*
 * mt_model — what joins a transformer's blocks into a residual stream in
 * training, and what ends the model, for one NVIDIA GB300 (sm_103a): layer
 * norm and dropout with the residual's addition, and the softmax cross entropy
 * of a product with the vocabulary's weight, with their gradients.  Same
 * library (libmtsgemm.so) and rules as mt_layers.h: device pointers owned by
 * the caller, stream-ordered, every entry point returns an mt_status and
 * launches nothing on an argument error, no state kept between calls,
 * thread-safe, no CPU fallback; matrices row-major with a row pitch in
 * elements; sums and statistics in fp32, rounded once, to nearest even, when a
 * result is stored.
 */
#ifndef MT_MODEL_H
#define MT_MODEL_H

#include "mt_layers.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Dropout's random words.  The word of column j of row i of a call is word
 * j % 4 of Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random
 * numbers: as easy as 1, 2, 3", 2011) with
 *
 *     key     = the lower and upper 32 bits of *seed
 *     counter = (j / 4, i, the lower and upper 32 bits of sequence)
 *
 * and with D(v) = v / (1 - p) where the word is at least floor(p * 2^32), else
 * 0 (whatever v is; 1 / (1 - p) is rounded to fp32).  A mask depends on seed,
 * sequence, row and column alone, so the gradient recomputes it and it is
 * never stored.  seed is read from device memory when the kernel runs: a
 * captured graph whose seed advances drops other elements at each replay.
 * sequence tells the calls of one seed apart (a layer's number, say).
 */

/*
 * Layer norm with dropout and the residual's addition:
 *
 *     h[i][k] = D(x[i][k]) + residual[i][k]         (residual NULL: D(x))
 *     m[i]    = mean_k h[i][k]
 *     r[i]    = 1 / sqrt(mean_k (h[i][k] - m[i])^2 + eps)   (0 for 1 / 0)
 *     y[i][k] = (h[i][k] - m[i]) * r[i] * weight[k] + bias[k]
 *
 * weight NULL: ones; bias NULL: zeros.  h enters the norm unrounded.  Written:
 * h in x's type (NULL: not written), m and r to `mean` and `rstd` (rows floats;
 * NULL: not written; the gradient reads both) and y.  The variance is that of
 * the differences from the mean, so a common offset costs it nothing.  A NaN in a
 * row makes its m, r and y NaN, an infinity r and y (and m infinite or NaN); a
 * variance past fp32's range (differences past 1.8e19) makes r 0 and y the bias.
 * Differences below 1e-19 have subnormal squares: with eps (nearly) 0 r loses digits.
 */
typedef struct {
    int64_t rows, d;
    const void *x;
    int64_t ldx;
    const void *residual;
    int64_t ldr;
    const void *weight;
    const void *bias;
    void *h;
    int64_t ldh;
    void *y;
    int64_t ldy;
    float *mean;
    float *rstd;
    const int64_t *seed;  /* one value in device memory; read for dropout > 0 */
    uint64_t sequence;
    double dropout;       /* p: 0 <= p < 1 (0: none) */
    float eps;            /* finite, >= 0 */
    int32_t dtype;        /* x, residual, h, y: MT_DTYPE_F16, _BF16 or _F32 */
    int32_t weight_dtype; /* weight and bias: dtype or MT_DTYPE_F32 */
    int32_t reserved;     /* 0 */
} mt_layer_norm_args;

/*
 * rows == 0 does nothing; d == 0 writes the statistics of empty rows (m 0, r
 * from eps).  h may be x or residual itself, and y may be x itself (same
 * pointer and pitch); any other overlap of an output is MT_ERR_ALIAS.
 * Pointers must be aligned to their element.  Other errors as mt_rms_norm, and
 * MT_ERR_INVALID_ARG for a dropout outside [0, 1) or without a seed.
 */
MT_API mt_status mt_layer_norm(const mt_layer_norm_args *args, cudaStream_t stream);

/*
 * The gradient of mt_layer_norm: with xhat = (h - mean) * rstd, g = dy * weight,
 *
 *     dresidual[i][k] = rstd[i] * (g[i][k] - mean_k(g[i]) - xhat[i][k] * mean_k(g[i] * xhat[i]))
 *                       + dh[i][k]
 *     dx[i][k]        = D(dresidual[i][k]), of the unrounded dresidual
 *     dweight[k]      = sum_i dy[i][k] * xhat[i][k]
 *     dbias[k]        = sum_i dy[i][k]
 *
 * dh is the gradient that reaches h directly (the residual stream; NULL: none).
 * Without dropout dx is dresidual too and dresidual has to be NULL; with it
 * dresidual NULL is not written.  dweight, dbias: d floats, each a sum over the
 * rows in a fixed order (the same call gives the same bits); NULL: not computed.
 */
typedef struct {
    int64_t rows, d;
    const void *dy;
    int64_t lddy;
    const void *h;
    int64_t ldh;
    const void *weight;   /* NULL: ones */
    const float *mean;
    const float *rstd;
    const void *dh;
    int64_t lddh;
    void *dx;
    int64_t lddx;
    void *dresidual;
    int64_t lddres;
    float *dweight;
    float *dbias;
    const int64_t *seed;  /* seed, sequence, dropout: the forward call's */
    uint64_t sequence;
    double dropout;
    int32_t dtype;        /* dy, h, dh, dx, dresidual: MT_DTYPE_F16, _BF16 or _F32 */
    int32_t weight_dtype; /* dtype or MT_DTYPE_F32 */
    int32_t fault_inject; /* test hook, as mt_rms_norm_backward's */
    int32_t reserved;     /* 0 */
} mt_layer_norm_backward_args;

/* dx may be dy or dh itself, and dresidual too (same pointer and pitch, not
 * both the same one); any other overlap of an output is MT_ERR_ALIAS.  rows == 0
 * writes zeros to dweight and dbias.  Other errors as mt_layer_norm, and
 * MT_ERR_CUDA when scratch cannot be allocated. */
MT_API mt_status mt_layer_norm_backward(const mt_layer_norm_backward_args *args,
                                        cudaStream_t stream);

/*
 * Dropout with the residual's addition: y = D(x) + residual (NULL: D(x)), in
 * fp32 and rounded once.  Its gradient with respect to x is the same call on
 * the gradient of y without a residual; with respect to the residual it is the
 * gradient of y itself.
 */
typedef struct {
    int64_t rows, d;
    const void *x;
    int64_t ldx;
    const void *residual;
    int64_t ldr;
    void *y;
    int64_t ldy;
    const int64_t *seed;  /* one value in device memory */
    uint64_t sequence;
    double p;             /* 0 <= p < 1 */
    int32_t dtype;        /* MT_DTYPE_F16, _BF16 or _F32 */
    int32_t reserved;     /* 0 */
} mt_dropout_args;

/* Nothing to do for rows or d == 0.  y may be x or residual itself (same
 * pointer and pitch); any other overlap is MT_ERR_ALIAS.  Other errors as
 * mt_layer_norm. */
MT_API mt_status mt_dropout(const mt_dropout_args *args, cudaStream_t stream);

/*
 * Softmax cross entropy of a product with the vocabulary's weight.  With the
 * logits z = A * op(B) (T x V, products and sums in fp32, never in memory):
 *
 *     lse[i]  = log sum_v exp(z[i][v])
 *     loss[i] = lse[i] - (1 - s) * z[i][target[i]] - s * mean_v z[i][v] + c * lse[i]^2
 *
 * s = label_smoothing, c = z_loss.  A is T x K, B is K x V, or V x K with
 * trans_b.  A row whose target is ignore_index has loss 0 (its lse is
 * computed); a target outside [0, V) that is not ignore_index makes the row's
 * loss NaN.  A logit that is NaN or +infinity makes its row's lse NaN.  The
 * products' sums are the tensor cores', which truncate as they accumulate: within
 * 5e-5 of the sum of absolute values, as mt_linear's (lse to some 1e-6 for 4096
 * values of K).
 */
typedef struct {
    int64_t T, K, V;
    const void *A;
    int64_t lda;
    const void *B;
    int64_t ldb;
    const int64_t *target;  /* T values */
    float *loss;            /* T floats */
    float *lse;             /* T floats */
    int64_t ignore_index;
    float label_smoothing;  /* 0 <= s <= 1 */
    float z_loss;           /* finite, >= 0 */
    int32_t trans_b;        /* 0 or 1 */
    int32_t dtype;          /* A, B: MT_DTYPE_F16 or MT_DTYPE_BF16 */
    int32_t fault_inject;   /* test hook, as mt_linear's: loss and lse then hold
                               nothing of use */
    int32_t reserved;       /* 0 */
} mt_linear_cross_entropy_args;

/*
 * T == 0 does nothing; V == 0 with rows is MT_ERR_INVALID_ARG; K == 0 gives the
 * loss of zero logits.  Outputs overlap nothing (MT_ERR_ALIAS).  Scratch: a float a token,
 * two floats (three with smoothing) for every token and 128 columns of the vocabulary
 * (32 for few tokens), and copies of operands TMA cannot read in place (see
 * mt_linear).
 * Other errors as mt_linear.
 */
MT_API mt_status mt_linear_cross_entropy(const mt_linear_cross_entropy_args *args,
                                         cudaStream_t stream);

/*
 * The gradient of mt_linear_cross_entropy.  With p = exp(z - lse), z computed
 * again,
 *
 *     D[i][v] = dloss[i] * (p[i][v] * (1 + 2 c lse[i]) - s / V - (1 - s) [v == target[i]])
 *     dA = D * op(B)^T                     T x K, dtype
 *     dB = A^T * D, stored as B is         K x V (V x K with trans_b), db_dtype
 *
 * D is rounded to dtype for the two products, whatever db_dtype is, and held for one
 * piece of the vocabulary at a time (up to 1 GiB, but at least 256 columns).  In fp16,
 * and in bf16 for (T + 256) K V of 2^36 and more, it is held times a scale that makes the
 * largest |dloss| (1 - s) of the call a power of two, so that a dloss that all tokens
 * have is not rounded with D, and brings the largest |dloss| (1 + 2 c |lse|) to 2^13 or
 * more, so that fp16 keeps all bits of values down to 2^-27 of it (p is at most 1 with
 * the forward call's lse; with another D may overflow).  Smaller bf16 calls round dloss
 * with D, alike for every token that has it: by up to 2^-8, a power of two not at all.  A
 * row whose target is ignore_index has a D of zeros whatever its logits, dloss and lse
 * are; its row of A still enters dB's sums, times zero, and has to be finite.  Any other
 * target outside [0, V) makes the row's D NaN.  dA or dB may be NULL: not computed.
 * The gradient is that of loss: nothing reaches A or B through lse on its own.
 */
typedef struct {
    int64_t T, K, V;
    const float *dloss;     /* T floats */
    const void *A;
    int64_t lda;
    const void *B;
    int64_t ldb;
    const int64_t *target;
    const float *lse;       /* the forward call's */
    void *dA;
    int64_t ldda;
    void *dB;
    int64_t lddb;
    int64_t ignore_index;
    float label_smoothing;
    float z_loss;
    int32_t trans_b;
    int32_t dtype;          /* A, B, dA: MT_DTYPE_F16 or MT_DTYPE_BF16 */
    int32_t db_dtype;       /* dB: dtype or MT_DTYPE_F32 */
    int32_t reserved;       /* 0 */
} mt_linear_cross_entropy_backward_args;

/* T == 0 writes zeros to dB.  Outputs overlap nothing (MT_ERR_ALIAS).  Results do
 * not depend on which of dA and dB are asked for, and are the same bits each time.
 * Scratch: a piece of D; for several pieces of the vocabulary or a long one dA's sums in
 * fp32, up to sms / 2 times (slices), T rounded up to whole 256 rows; where D is scaled
 * 32 bytes a token and two vectors of max(T, K, the piece's columns) floats; and copies of
 * operands TMA cannot read in place.  Other errors as mt_linear_cross_entropy. */
MT_API mt_status mt_linear_cross_entropy_backward(
    const mt_linear_cross_entropy_backward_args *args, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MT_MODEL_H */
