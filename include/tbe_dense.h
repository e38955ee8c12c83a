/*
 * tbe_dense.h -- the dense side of a training step around the table-batched embedding: layer norm
 * over each table's columns of the pooled output (forward and backward), the global norm of many
 * gradients, and one AdamW update of many tensors.
 *
 * Layer norm stands on either side of the embedding: tbe_forward writes the pooled rows it
 * reads, and its dx is the grad_out that tbe_backward_update takes.  The gradient norm leaves its
 * clip coefficient on the device, where the AdamW update reads it, so a step needs no host
 * synchronisation.
 *
 * Conventions are those of tbe.h: device memory is the caller's; every call is asynchronous on
 * `stream`, allocates nothing and copies nothing to the host; return values report what the host
 * can see.  Host descriptions (structs, widths, tensor lists) are read before the call returns
 * and not kept.  All sums and statistics are held in fp32, or wider where stated.
 */
#ifndef TBE_DENSE_H
#define TBE_DENSE_H

#include <stddef.h>
#include <stdint.h>

#include "tbe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------------------------
 * Layer norm
 *
 * A row holds `segments` segments side by side; each is normalised on its own.  One segment is
 * the ordinary layer norm; the pooled output [B, sum D] with one segment per table normalises
 * every table's embedding.  For segment s of row r, with n = widths[s]:
 *   mean = sum x / n,  rstd = 1 / sqrt(sum (x - mean)^2 / n + eps),
 *   y = (x - mean) * rstd * weight + bias
 * and backward, with xhat = (x - mean) * rstd and h = dy * weight:
 *   dx = rstd * (h - sum h / n - xhat * sum (h * xhat) / n),
 *   dweight = sum over rows of dy * xhat,  dbias = sum over rows of dy.
 * A segment of one column, or of equal values (the pooled row of an empty bag), has xhat = 0,
 * exactly: mean is then the value itself (for magnitudes from 2^-50 on; below, to 2^-18 of it).
 * eps counts as 2^-126 at least: with eps = 0 and no spread, rstd is 2^63.  A row's sums, and its
 * mean times rstd, have to stay within fp32.
 * Limits: 4096 segments, 2^30 columns, fewer than 2^39 elements (TBE_ERR_UNSUPPORTED beyond).
 * ------------------------------------------------------------------------------------------ */
typedef struct {
  int64_t rows;                /* >= 0 */
  int32_t segments;            /* 1 .. 4096 */
  const int32_t* widths;       /* host [segments], each >= 1 */
  /* DEVICE [segments + 1], first column of each segment (tbe_tables.D_offsets of the pooled
   * output); may be NULL when all widths are equal.  It has to agree with widths. */
  const int32_t* col_offsets;
  int64_t x_stride;            /* elements between rows of x; at least sum widths, as the others */
  int64_t y_stride;            /* ... of y (forward) and dy (backward) */
  int64_t dx_stride;           /* ... of dx (backward only) */
  tbe_dtype xdtype;            /* type of x and dx */
  tbe_dtype ydtype;            /* type of y and dy: equal to xdtype, or one of the two TBE_F32 */
  tbe_dtype wdtype;            /* type of weight, bias, dweight and dbias */
  float eps;                   /* >= 0 and finite */
} tbe_norm_problem;

/* weight and bias [sum widths], each may be NULL (1 and 0).  mean and rstd: fp32 [rows, segments],
 * both or neither (inference).  y may be x itself (same type and stride); no other overlap.
 * Buffers are aligned to their element; 16-byte alignment of the buffers and strides, and widths
 * that are multiples of 4 (8 where both types are 16-bit) take the vectorised kernels. */
tbe_status tbe_layer_norm_forward(const tbe_norm_problem* prob, const void* x, const void* weight,
                                  const void* bias, void* y, float* mean, float* rstd, void* stream);

/* mean and rstd as the forward left them.  dweight and dbias [sum widths] are overwritten, each may
 * be NULL, and dx may be NULL.  dx may be x or dy itself (same type and stride); no other overlap.
 * rows == 0 gives zero dweight and dbias.  The sums over rows have a fixed order on a given GPU:
 * the same inputs give the same bits.  ws: tbe_layer_norm_backward_workspace_size() bytes,
 * 16-byte aligned. */
size_t tbe_layer_norm_backward_workspace_size(const tbe_norm_problem* prob);
tbe_status tbe_layer_norm_backward(const tbe_norm_problem* prob, const void* dy, const void* x,
                                   const float* mean, const float* rstd, const void* weight, void* dx,
                                   void* dweight, void* dbias, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------------------------
 * Many tensors at once
 * ------------------------------------------------------------------------------------------ */
/* How AdamW's two states are held. F32: fp32.  Q8: one byte an element and one fp32 scale (the
 * largest magnitude) for each block of TBE_Q8_BLOCK consecutive elements of a tensor, the last one
 * ragged.  With b bits of magnitude (the first moment: a sign bit, then 7; the second: 8) and k the
 * place of a code's leading one, code c >= 1 stands for (7 c + 7 - 6 * 2^k) * 2^(2 k - 3 b) times
 * the scale, and 0 for 0: each leading zero is a power of 8, the bits below the leading one
 * divide its interval evenly, the largest code is the scale itself.  (After the dynamic
 * exponents of Dettmers et al., "8-bit Optimizers via Block-wise Quantization", 2022; base 8
 * makes every value exact in binary.)  A magnitude takes the nearest code, except next to 0: of
 * the first moment it takes code 0 up to 0.5625 of code 1's value (the middle of 8^-7 and 8^-6 times the
 * scale), and a positive second moment takes at least code 1: rounded to zero it would leave the
 * first moment divided by eps alone.  A block without a magnitude of 2^-120 or more is held as zeros,
 * its scale too. */
typedef enum { TBE_STATE_F32 = 0, TBE_STATE_Q8 = 1 } tbe_state_type;
#define TBE_Q8_BLOCK 256

typedef struct {
  void* param;             /* pdtype [numel] */
  const void* grad;        /* gdtype [numel] */
  float* master;           /* fp32 [numel] of 16-bit params, for all tensors or for none (NULL): then
                              param itself is read */
  void* exp_avg;           /* first moment: fp32 or uint8 [numel] */
  void* exp_avg_sq;        /* second moment */
  float* exp_avg_scale;    /* TBE_STATE_Q8: fp32 [ceil(numel / TBE_Q8_BLOCK)]; else not read */
  float* exp_avg_sq_scale;
  int64_t numel;           /* 0 .. 2^40 */
  float lr_scale;          /* the tensor's learning rate is lr * lr_scale */
  float weight_decay;
} tbe_dense_tensor;

typedef struct {
  int32_t count;                     /* tensors, >= 0 */
  const tbe_dense_tensor* tensors;   /* host [count] */
  tbe_dtype pdtype;
  tbe_dtype gdtype;
  tbe_state_type states;
  double beta1, beta2;               /* in [0, 1) */
  float eps;                         /* >= 0 and finite */
} tbe_adamw_problem;

/* The norm of all gradients together and the coefficient that clips it to max_norm:
 *   out[0] = sqrt(sum of squares),  out[1] = min(1, max_norm / (out[0] + 1e-6))
 * with out fp32 [2] on the device.  Squares are summed in fp32 by thread (at most 130 of them) and in fp64
 * from there on, in a fixed order; a non-finite gradient, or a square beyond fp32, gives a non-finite norm, and squares below
 * 2^-150 count as 0.  grads:
 * host [count] device pointers, numels: host [count].  max_norm >= 0 (infinity: no clipping).
 * ws: tbe_grad_norm_workspace_size() bytes, 16-byte aligned, that the caller has zeroed once and no
 * other call uses at the same time; the call leaves it zeroed where that matters. */
size_t tbe_grad_norm_workspace_size(void);
tbe_status tbe_grad_norm(int32_t count, const void* const* grads, const int64_t* numels, tbe_dtype dtype,
                         float max_norm, float* out, void* ws, size_t ws_bytes, void* stream);

/* One AdamW step of every tensor, in place, with g = grad * clip[1] and t = *step + 1:
 *   m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2,
 *   p = p (1 - lr wd) - lr (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps)
 * in fp32, where v under the root counts as 2^-126 at least (its root as 2^-63, which matters beside a smaller
 * eps); p is the master where there is one (param then gets its rounding), else param.  step:
 * device int64, the updates done so far, which the call increments.  clip: NULL (coefficient 1), or
 * the out of tbe_grad_norm: where its norm is not finite the call changes nothing, step
 * included.  In Q8, the update uses the moments before they are rounded to their codes; a
 * non-finite gradient makes its block's states non-finite.  Tensors do not overlap.  ws:
 * tbe_adamw_workspace_size() bytes, zeroed once by the caller, as for tbe_grad_norm. */
size_t tbe_adamw_workspace_size(void);
tbe_status tbe_adamw_update(const tbe_adamw_problem* prob, float lr, const float* clip, int64_t* step, void* ws,
                            size_t ws_bytes, void* stream);

/* What the 8-bit states stand for, as fp32: exp_avg_values[i] and exp_avg_sq_values[i] are device
 * fp32 [numel of tensor i] (the host arrays of pointers, or single ones, may be NULL).
 * TBE_ERR_INVALID_ARG for TBE_STATE_F32. */
tbe_status tbe_adamw_state_values(const tbe_adamw_problem* prob, float* const* exp_avg_values,
                                  float* const* exp_avg_sq_values, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TBE_DENSE_H */
