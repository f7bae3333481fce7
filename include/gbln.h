/*
 * gbln.h - fused residual add + LayerNorm for GB300 (sm_103a), its backward pass,
 * and dropout, alone and in front of the add: C ABI.
 *
 * The operation (lpqz.cn CUDA tutorial, sections 5.1-5.2): for each row of a
 * [rows, cols] matrix, h = x + residual, then
 *     mean = sum(h) / cols,  var = sum((h - mean)^2) / cols,
 *     y = (h - mean) / sqrt(var + eps) * gamma + beta,
 * all in one kernel that reads x and residual once and writes y (and h) once;
 * the statistics are merged in registers (per-thread chunks, combined with
 * the parallel form of Welford's update through warp shuffles and shared
 * memory), never written between passes.  The page builds it as the second
 * fused operator after attention, to show that a low-arithmetic-intensity
 * operator is set by the bytes it moves: the kernel is HBM-bound.
 *
 * Layout.  Row r of x starts at x + r * x_stride (elements), the same for
 * residual, y and h; columns are contiguous.  gamma and beta are float32
 * [cols].  mean and rstd (= 1 / sqrt(var + eps)) are float32 [rows].
 *
 * Constraints.  1 <= cols <= 16384; rows >= 0; strides >= cols; every pointer
 * aligned to its element size.  Rows move as 16-byte vectors when every
 * pointer is 16-byte aligned and every stride a multiple of 16 bytes, element
 * by element otherwise.  residual, h, gamma, beta, mean and rstd may be NULL:
 * no residual (h = x), h not stored, gamma = 1, beta = 0, statistics not stored.
 *
 * Ownership and errors are as for gbattn.h: the caller owns every buffer; the
 * library allocates nothing; argument errors return before any work is queued
 * (attn_last_error() says why); the call only queues work on `stream`.
 */
#ifndef GBLN_H
#define GBLN_H

#include <stddef.h>
#include <stdint.h>

#include "gbattn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int64_t rows, cols;
  int64_t x_stride, r_stride, y_stride, h_stride; /* elements between consecutive rows */
  float eps;
  attn_dtype_t dtype; /* element type of x, residual, y, h (ATTN_BF16 or ATTN_F32) */
} ln_params_t;

/*
 * y = LayerNorm(x + residual) * gamma + beta, per row, with h = x + residual
 * (rounded to dtype) optionally stored.  Arithmetic in float32.  Returns
 * ATTN_OK once the work is queued.
 */
attn_status_t ln_residual_fwd(const ln_params_t* p, const void* x, const void* residual, const float* gamma,
                              const float* beta, void* y, void* h, float* mean, float* rstd, void* stream);

/*
 * Dropout.  The mask is never stored: it follows from a seed, an offset and an
 * element's place, so that the backward pass makes the same one.  Element (row,
 * col) has 16 bits: with the counter (col / 8, row, offset low 32, offset high 32) and
 * the key (seed low 32, seed high 32), Philox4x32 with 7 rounds (Salmon, Moraes,
 * Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011) gives four words;
 * bits 16 (col % 8) .. 16 (col % 8) + 15 of them, words and bits lowest first.  With
 * t = floor(65536 p + 1/2), an element whose 16 bits are below t is dropped: it becomes 0,
 * whatever it held (NaN and infinities too).  Another is multiplied by 65536 / (65536 - t),
 * so that the mean is that of the rate really used, t / 65536.
 *
 * seed and offset are modulo 2^64 the sums of the two members and, if rng is not
 * NULL, of the pair {seed, offset} in device memory that the kernel reads when it
 * runs: a captured graph drops anew when that pair is changed between replays.  The
 * backward pass needs the values of the forward pass.
 * The same sums give the same mask, so every dropout of every step needs sums of its own.  With
 * member offsets 0 .. n - 1 in a step's dropouts, the pair's offset has to grow by n at least from
 * step to step (2^32 is simple): growing by 1, dropout k of a step has the mask of dropout k - 1 of the next.
 */
typedef struct {
  double p;            /* probability of being dropped, 0 <= p <= 1 */
  uint64_t seed, offset;
  const uint64_t* rng; /* device, 2 numbers, 8-byte aligned, or NULL */
} ln_dropout_t;

/*
 * y = D(x) over [rows, cols] (x_stride, y_stride; the other strides and eps are not
 * looked at), and, on a gradient, dropout's backward pass.  y may be x itself (with
 * y_stride == x_stride); other rows that share an element are refused.  rows and cols
 * below 2^32.  d must not be NULL.  D is taken in float32 and rounded once.  16-byte
 * vectors as above.
 */
attn_status_t ln_dropout(const ln_params_t* p, const ln_dropout_t* d, const void* x, void* y, void* stream);

/*
 * ln_residual_fwd with h = D(x) + residual: D(x) is not rounded before the sum.
 * d may be NULL (no dropout: the same call as ln_residual_fwd); with dropout rows below 2^32.
 */
attn_status_t ln_dropout_residual_fwd(const ln_params_t* p, const ln_dropout_t* d, const void* x, const void* residual,
                                      const float* gamma, const float* beta, void* y, void* h, float* mean,
                                      float* rstd, void* stream);

typedef struct {
  int64_t rows, cols;
  int64_t dy_stride, dh_stride, h_stride, dx_stride, dr_stride; /* elements between consecutive rows */
  attn_dtype_t dtype; /* element type of dy, dh, h, dx, dr (ATTN_BF16 or ATTN_F32) */
} ln_bwd_params_t;

/*
 * The backward pass of ln_dropout_residual_fwd, from the stored h, mean and rstd.  With
 * xh = (h - mean) rstd and g = dy gamma, per row
 *     dr = dh + rstd (g - sum(g) / cols - xh sum(g xh) / cols),   dx = D(dr),
 * and over the rows dgamma = sum(dy xh), dbeta = sum(dy).  dy is the gradient at y,
 * dh the one that arrives at h by another way (NULL: none); dr is the residual's
 * gradient and dx that of x (D(dr) of the unrounded dr).  Without dropout (d NULL or t
 * = 0) the two are equal and either may be NULL; so may either with dropout.  gamma
 * NULL: 1.  dgamma and dbeta, float32 [cols], may be NULL each; where rows is 0 they are
 * set to 0.  Arithmetic and sums in float32; a row's columns and a column's rows are added in an
 * order that sizes and alignment decide (the results are bit-identical from run to run).  A dy, h,
 * mean or rstd that is not finite reaches its row and the columns' sums; a dh its own element.
 *
 * Constraints as for ln_residual_fwd; outputs and workspace must not overlap inputs or one another
 * (refused), except that dx or dr may be dy or dh itself, with the same stride, and without dropout dr itself dx.  workspace:
 * device scratch, 256-byte aligned, >= ln_residual_bwd_workspace_size(p) bytes (SIZE_MAX
 * if the parameters are invalid), not needed if dgamma and dbeta are NULL; calls that
 * may overlap need one each.
 */
size_t ln_residual_bwd_workspace_size(const ln_bwd_params_t* p);
attn_status_t ln_residual_bwd(const ln_bwd_params_t* p, const ln_dropout_t* d, const void* dy, const void* dh,
                              const void* h, const float* mean, const float* rstd, const float* gamma, void* dx,
                              void* dr, float* dgamma, float* dbeta, void* workspace, size_t workspace_bytes,
                              void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GBLN_H */
