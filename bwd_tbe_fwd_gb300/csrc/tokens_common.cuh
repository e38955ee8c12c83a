// tokens_common.cuh -- what the units behind tbe_tokens.h share: the validated problems and the launchers.
#pragma once

#include "dense_common.cuh"
#include "tbe_tokens.h"

namespace tbe {

constexpr int kMaxDim = 65536;
constexpr int64_t kMaxLossTokens = int64_t(1) << 24;

inline int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
inline int64_t ceil_div(int64_t v, int64_t m) { return (v + m - 1) / m; }

// ------------------------------------------------------------------------------------------
// Softmax cross entropy
// ------------------------------------------------------------------------------------------
struct LossArgs {
  int64_t tokens, rows, hidden_stride, weight_stride, dhidden_stride, dweight_stride;
  int dim, dtype, itype;
  float scale;
  bool copy_hidden, copy_weight;   // rows that TMA cannot address are copied to aligned ones first
  unsigned long long* stats;
};

// Workspace of the forward: parts of the rows' softmax statistics, copies; bytes from its start.
struct LossForwardLayout {
  int64_t parts_rows;              // leading dimension of the parts: tokens, rounded up
  int64_t piece;                   // rows of the table at a time
  int parts;                       // of a piece; behind them, where there are several, one for the pieces before
  size_t part, logit, ticket, live, place, target, row, hidden, weight, total;
};
struct LossBackwardLayout {
  int64_t dim_pad;                 // row of the fp32 sums of dhidden
  int64_t piece;                   // rows of the table at a time
  int64_t dz_rows;                 // of a block of 64 columns of dz
  int splits;                      // parts of the long sums of dhidden
  int out_splits;                  // parts of the sums of dweight
  bool direct;                     // it is written as it is: one piece, one split
  size_t meta, live, place, target, row, coef, down, lse2, hidden, hidden_low, weight, dz, sums, out_sums, total;
};
LossForwardLayout loss_forward_layout(const LossArgs& a);
LossBackwardLayout loss_backward_layout(const LossArgs& a, const DeviceInfo& dev);

tbe_status launch_loss_forward(const LossArgs& a, const LossForwardLayout& l, const void* hidden, const void* weight,
                               const void* targets, float* loss, float* lse, float* mean, char* ws, const DeviceInfo& dev,
                               cudaStream_t s);
tbe_status launch_loss_backward(const LossArgs& a, const LossBackwardLayout& l, const void* hidden, const void* weight,
                                const void* targets, const float* lse, const float* dloss, const float* mean, void* dhidden,
                                void* dweight, char* ws, const DeviceInfo& dev, cudaStream_t s);

// ------------------------------------------------------------------------------------------
// Lookup
// ------------------------------------------------------------------------------------------
struct LookupArgs {
  int64_t tokens, rows, table_stride, out_stride;
  int dim, ttype, otype, itype;
  float scale;
  unsigned long long* stats;
};
size_t lookup_backward_bytes(const LookupArgs& a, const DeviceInfo& dev);
tbe_status launch_lookup_forward(const LookupArgs& a, const void* table, const void* ids, void* out, const DeviceInfo& dev,
                                 cudaStream_t s);
tbe_status launch_lookup_backward(const LookupArgs& a, const void* dout, const void* ids, void* grad, bool accumulate, char* ws,
                                  const DeviceInfo& dev, cudaStream_t s);

}  // namespace tbe
