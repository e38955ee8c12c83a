/*
 * tbe_tokens.h -- one table's rows as a model's two ends: the lookup of a row for each token (or item) with
 * its gradient as a tensor, and the softmax cross entropy over the table's rows with its gradient.
 *
 * tbe_forward pools bags and tbe_backward_update updates tables in place; here each id has an output row of its
 * own, and the gradient is left as a tensor, for AdamW (tbe_dense.h), for clipping, and for a table that the loss
 * and the lookup share: tbe_softmax_loss_backward writes dweight, tbe_lookup_backward adds to it.
 *
 * Conventions are those of tbe.h: device memory is the caller's; every call is asynchronous on `stream`, allocates
 * nothing and copies nothing to the host; return values report what the host can see.  Structs are read before
 * the call returns and not kept.  Sums and softmax statistics are held in fp32.  The same inputs give the same
 * bits on a given GPU.  Two calls that use the same workspace must not overlap in time.
 * d_stats: NULL, or int64 [TBE_NUM_STATS] on the device: ids past the table are counted in TBE_STAT_UNREPAIRED (targets by
 * the forward alone), a bounded device-side wait that gave up (its results are then not valid) in
 * TBE_STAT_WAIT_TIMEOUT.
 */
#ifndef TBE_TOKENS_H
#define TBE_TOKENS_H

#include <stddef.h>
#include <stdint.h>

#include "tbe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------------------------
 * Lookup
 *
 * out[i] = scale * table[ids[i]],  and zeros where ids[i] is not a row of the table (padding: any negative id);
 * grad[v] = (accumulate ? grad[v] : 0) + scale * sum of dout[i] over the tokens i with ids[i] = v, in the tokens'
 * order, chunk by chunk, rounded once to grad's type.  Rows without a token become zeros, or stay untouched when
 * accumulating.
 * Limits: 1 <= rows < 2^31, 1 <= dim <= 65536, tokens <= 2^31 - 2^16, tokens * dim <= 2^40;
 * TBE_ERR_UNSUPPORTED beyond.
 * ------------------------------------------------------------------------------------------ */
typedef struct {
  int64_t tokens;              /* >= 0 */
  int64_t rows;                /* of the table */
  int32_t dim;                 /* elements of a row */
  int64_t table_stride;        /* elements between rows of table (forward) and grad (backward); >= dim */
  int64_t out_stride;          /* elements between rows of out (forward) and dout (backward); >= dim */
  tbe_dtype tdtype;            /* type of table and grad */
  tbe_dtype odtype;            /* type of out and dout: equal to tdtype, or one of the two TBE_F32 */
  tbe_itype itype;             /* type of ids */
  float scale;                 /* finite */
} tbe_lookup_problem;

/* Buffers are aligned to their element; 16-byte alignment of buffers and strides takes vector accesses. */
tbe_status tbe_lookup_forward(const tbe_lookup_problem* prob, const void* table, const void* ids, void* out,
                              int64_t* d_stats, void* stream);

/* ws: tbe_lookup_backward_workspace_size() bytes (0: a problem that is refused), 256-byte aligned; it serves every call of
 * at most as many tokens. */
size_t tbe_lookup_backward_workspace_size(const tbe_lookup_problem* prob);
tbe_status tbe_lookup_backward(const tbe_lookup_problem* prob, const void* dout, const void* ids, void* grad,
                               int32_t accumulate, void* ws, size_t ws_bytes, int64_t* d_stats, void* stream);

/* ------------------------------------------------------------------------------------------
 * Softmax cross entropy over the rows of a table
 *
 * With z[i][v] = scale * (hidden[i] . weight[v]):
 *   lse[i] = log sum_v exp z[i][v],  loss[i] = lse[i] - z[i][targets[i]],
 *   mean = { sum of loss / count, 1 / count },  count: the tokens whose target is a row of the table.
 * A token whose target is no row (padding: any negative one) has loss and lse 0 and no part in the gradients (its row of
 * dhidden is zeros), even if its hidden row holds infinities or NaN, and costs next to nothing in the backward and, of 1024
 * tokens or more, in the forward; mean is {0, 0} where none counts.  Backward, with the coefficient
 * c[i] = dloss[i] * mean[1] (1 for each that is NULL) of the tokens that count and 0 of the others,
 *   dz[i][v] = c[i] * (exp(z[i][v] - lse[i]) - [v = targets[i]]),
 *   dhidden = scale * dz weight,  dweight = scale * dz^T hidden.
 * The logits are never kept: the forward holds them a tile at a time, the backward takes a piece of the table's rows
 * at a time, of which dz is held in 16 bits (type dtype, scaled by a factor that the largest |c[i]| gives).  In fp16 a
 * token of a smaller |c[i]| has a power of two of its own: its probabilities from 1 / (8 rows) on keep all bits that
 * the type has where |c[i]| >= 2^-34 rows / (its hidden row's largest element) of the largest; what is smaller than
 * that product loses its last bits first.  bf16 has fp32's range.  Products are of 16-bit operands, summed in fp32 by
 * the tensor cores, which need not round to nearest; exponentials are 2^x good to 2 units in the last place, of
 * logits that take scale * log2(e) as one factor.  lse and loss are so within some 2^-20 of the logits' size (3e-7 to
 * 6e-7 of their norm with 1024 and 2048 columns), and the loss of a token that is all but certain may be as much
 * below 0; small gradients lose a sixth of their own rounding in bf16 and a third in fp16 to dz's 16 bits.
 * Limits: 1 <= rows < 2^31 - 2^16, 1 <= dim <= 65536, tokens <= 2^24, tokens * rows <= 2^45; dtype TBE_F16 or
 * TBE_BF16; TBE_ERR_UNSUPPORTED beyond.  weight: 16-byte aligned where its stride is a multiple of 8; the other
 * buffers, and weight otherwise, are aligned to their element.
 * ------------------------------------------------------------------------------------------ */
typedef struct {
  int64_t tokens;              /* >= 0 */
  int64_t rows;                /* of weight: the classes */
  int32_t dim;
  int64_t hidden_stride;       /* elements between rows, at least dim, as the others */
  int64_t weight_stride;
  int64_t dhidden_stride;      /* backward only */
  int64_t dweight_stride;      /* backward only */
  tbe_dtype dtype;             /* of hidden, weight, dhidden and dweight */
  tbe_itype itype;             /* of targets */
  float scale;                 /* > 0 and finite */
} tbe_softmax_problem;

/* loss, lse: fp32 [tokens]; mean: fp32 [2].  ws: the size that the query gives (0: a problem that is refused),
 * 256-byte aligned; it serves every call of at most as many tokens, and any hidden_stride, with the same table.  It holds
 * 8 bytes for each token and 128 rows of the table, up to 256 MB of them or 16 bytes a token, some 30 bytes a token
 * more, a copy of hidden, and one of a table whose weight_stride is no multiple of 8. */
size_t tbe_softmax_loss_workspace_size(const tbe_softmax_problem* prob);
tbe_status tbe_softmax_loss_forward(const tbe_softmax_problem* prob, const void* hidden, const void* weight,
                                    const void* targets, float* loss, float* lse, float* mean, void* ws, size_t ws_bytes,
                                    int64_t* d_stats, void* stream);

/* lse as the forward left it.  The workspace holds dz of a piece of the table (up to 512 MB, or 512 bytes a token where
 * that is more), fp32 sums (dhidden's size, and up to 100 MB) and copies of hidden and of a weight that needs one.
 * dhidden [tokens, dim] and dweight [rows, dim] are overwritten; they overlap nothing. */
size_t tbe_softmax_loss_backward_workspace_size(const tbe_softmax_problem* prob);
tbe_status tbe_softmax_loss_backward(const tbe_softmax_problem* prob, const void* hidden, const void* weight,
                                     const void* targets, const float* lse, const float* dloss, const float* mean,
                                     void* dhidden, void* dweight, void* ws, size_t ws_bytes, int64_t* d_stats,
                                     void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TBE_TOKENS_H */
