// tokens_api.cu -- the C interface of tbe_tokens.h: argument validation and workspaces.
#include <cmath>

#include "tokens_common.cuh"

namespace tbe {
namespace {

tbe_status make_lookup(const tbe_lookup_problem* p, int64_t* stats, LookupArgs* a) {
  if (p == nullptr || p->tokens < 0 || p->rows < 1 || p->dim < 1) return TBE_ERR_INVALID_ARG;
  if (p->tokens > kMaxIndices || p->rows >= (int64_t(1) << 31) || p->dim > kMaxDim) return TBE_ERR_UNSUPPORTED;
  if (p->tokens > (int64_t(1) << 40) / p->dim) return TBE_ERR_UNSUPPORTED;
  if (!dtype_ok(p->tdtype) || !dtype_ok(p->odtype) || (p->itype != TBE_I32 && p->itype != TBE_I64)) return TBE_ERR_UNSUPPORTED;
  if (p->tdtype != p->odtype && p->tdtype != TBE_F32 && p->odtype != TBE_F32) return TBE_ERR_UNSUPPORTED;
  if (!std::isfinite(p->scale) || p->table_stride < p->dim || p->out_stride < p->dim) return TBE_ERR_INVALID_ARG;
  if (p->table_stride > INT64_MAX / 8 / p->rows || (p->tokens > 0 && p->out_stride > INT64_MAX / 8 / p->tokens))
    return TBE_ERR_UNSUPPORTED;
  if (!is_aligned(stats, 8)) return TBE_ERR_INVALID_ARG;
  a->tokens = p->tokens;
  a->rows = p->rows;
  a->table_stride = p->table_stride;
  a->out_stride = p->out_stride;
  a->dim = p->dim;
  a->ttype = p->tdtype;
  a->otype = p->odtype;
  a->itype = p->itype;
  a->scale = p->scale;
  a->stats = reinterpret_cast<unsigned long long*>(stats);
  return TBE_OK;
}

bool buffer_ok(const void* p, size_t align) { return p != nullptr && is_aligned(p, align); }
size_t itype_bytes(int itype) { return itype == TBE_I32 ? 4 : 8; }

tbe_status make_loss(const tbe_softmax_problem* p, int64_t* stats, bool backward, LossArgs* a) {
  if (p == nullptr || p->tokens < 0 || p->rows < 1 || p->dim < 1) return TBE_ERR_INVALID_ARG;
  if (p->tokens > kMaxLossTokens || p->rows >= kMaxIndices || p->dim > kMaxDim) return TBE_ERR_UNSUPPORTED;
  if (p->tokens > (int64_t(1) << 45) / p->rows) return TBE_ERR_UNSUPPORTED;  // tiles of 256 x 256: below 2^30
  if ((p->dtype != TBE_F16 && p->dtype != TBE_BF16) || (p->itype != TBE_I32 && p->itype != TBE_I64)) return TBE_ERR_UNSUPPORTED;
  if (!(p->scale > 0) || std::isinf(p->scale)) return TBE_ERR_INVALID_ARG;
  if (p->hidden_stride < p->dim || p->weight_stride < p->dim) return TBE_ERR_INVALID_ARG;
  if (backward && (p->dhidden_stride < p->dim || p->dweight_stride < p->dim)) return TBE_ERR_INVALID_ARG;
  // a tensor map's strides are below 2^40 bytes
  const int64_t most = int64_t(1) << 38;
  if (p->hidden_stride > most || p->weight_stride > most) return TBE_ERR_UNSUPPORTED;
  if (backward && (p->dhidden_stride > most || p->dweight_stride > most)) return TBE_ERR_UNSUPPORTED;
  if (!is_aligned(stats, 8)) return TBE_ERR_INVALID_ARG;
  a->tokens = p->tokens;
  a->rows = p->rows;
  a->hidden_stride = p->hidden_stride;
  a->weight_stride = p->weight_stride;
  a->dhidden_stride = p->dhidden_stride;
  a->dweight_stride = p->dweight_stride;
  a->dim = p->dim;
  a->dtype = p->dtype;
  a->itype = p->itype;
  a->scale = p->scale;
  a->copy_hidden = p->hidden_stride % 8 != 0;
  a->copy_weight = p->weight_stride % 8 != 0;
  a->stats = reinterpret_cast<unsigned long long*>(stats);
  return TBE_OK;
}

tbe_status check_workspace(const void* ws, size_t bytes, size_t need) {
  if (need == 0) return TBE_ERR_CUDA;
  if (ws == nullptr || bytes < need) return TBE_ERR_WORKSPACE;
  return is_aligned(ws, 256) ? TBE_OK : TBE_ERR_INVALID_ARG;
}

}  // namespace
}  // namespace tbe

using namespace tbe;

extern "C" {

tbe_status tbe_lookup_forward(const tbe_lookup_problem* prob, const void* table, const void* ids, void* out, int64_t* d_stats,
                              void* stream) {
  LookupArgs a;
  tbe_status st = make_lookup(prob, d_stats, &a);
  if (st != TBE_OK) return st;
  if (a.tokens == 0) return TBE_OK;
  if (!buffer_ok(table, dtype_bytes(a.ttype)) || !buffer_ok(out, dtype_bytes(a.otype)) || !buffer_ok(ids, itype_bytes(a.itype)))
    return TBE_ERR_INVALID_ARG;
  DeviceInfo dev;
  if ((st = device_info(&dev)) != TBE_OK) return st;
  return launch_lookup_forward(a, table, ids, out, dev, static_cast<cudaStream_t>(stream));
}

size_t tbe_lookup_backward_workspace_size(const tbe_lookup_problem* prob) {
  LookupArgs a;
  DeviceInfo dev;
  if (make_lookup(prob, nullptr, &a) != TBE_OK || device_info(&dev) != TBE_OK) return 0;
  return lookup_backward_bytes(a, dev);
}

tbe_status tbe_lookup_backward(const tbe_lookup_problem* prob, const void* dout, const void* ids, void* grad, int32_t accumulate,
                               void* ws, size_t ws_bytes, int64_t* d_stats, void* stream) {
  LookupArgs a;
  tbe_status st = make_lookup(prob, d_stats, &a);
  if (st != TBE_OK) return st;
  if (!buffer_ok(grad, dtype_bytes(a.ttype))) return TBE_ERR_INVALID_ARG;
  if (a.tokens > 0 && (!buffer_ok(dout, dtype_bytes(a.otype)) || !buffer_ok(ids, itype_bytes(a.itype)))) return TBE_ERR_INVALID_ARG;
  DeviceInfo dev;
  if ((st = device_info(&dev)) != TBE_OK) return st;
  if ((st = check_workspace(ws, ws_bytes, lookup_backward_bytes(a, dev))) != TBE_OK) return st;
  return launch_lookup_backward(a, dout, ids, grad, accumulate != 0, static_cast<char*>(ws), dev, static_cast<cudaStream_t>(stream));
}

size_t tbe_softmax_loss_workspace_size(const tbe_softmax_problem* prob) {
  LossArgs a;
  if (make_loss(prob, nullptr, false, &a) != TBE_OK) return 0;
  return loss_forward_layout(a).total;
}

tbe_status tbe_softmax_loss_forward(const tbe_softmax_problem* prob, const void* hidden, const void* weight, const void* targets,
                                    float* loss, float* lse, float* mean, void* ws, size_t ws_bytes, int64_t* d_stats,
                                    void* stream) {
  LossArgs a;
  tbe_status st = make_loss(prob, d_stats, false, &a);
  if (st != TBE_OK) return st;
  if (!buffer_ok(mean, 4)) return TBE_ERR_INVALID_ARG;
  if (!is_aligned(hidden, 16)) a.copy_hidden = true;
  if (a.tokens > 0 && (!buffer_ok(hidden, 2) || !buffer_ok(weight, a.copy_weight ? 2 : 16) ||
                       !buffer_ok(targets, itype_bytes(a.itype)) || !buffer_ok(loss, 4) || !buffer_ok(lse, 4)))
    return TBE_ERR_INVALID_ARG;
  const LossForwardLayout l = loss_forward_layout(a);
  if ((st = check_workspace(ws, ws_bytes, l.total)) != TBE_OK) return st;
  DeviceInfo dev;
  if ((st = device_info(&dev)) != TBE_OK) return st;
  return launch_loss_forward(a, l, hidden, weight, targets, loss, lse, mean, static_cast<char*>(ws), dev,
                             static_cast<cudaStream_t>(stream));
}

size_t tbe_softmax_loss_backward_workspace_size(const tbe_softmax_problem* prob) {
  LossArgs a;
  DeviceInfo dev;
  if (make_loss(prob, nullptr, true, &a) != TBE_OK || device_info(&dev) != TBE_OK) return 0;
  return loss_backward_layout(a, dev).total;
}

tbe_status tbe_softmax_loss_backward(const tbe_softmax_problem* prob, const void* hidden, const void* weight, const void* targets,
                                     const float* lse, const float* dloss, const float* mean, void* dhidden, void* dweight,
                                     void* ws, size_t ws_bytes, int64_t* d_stats, void* stream) {
  LossArgs a;
  tbe_status st = make_loss(prob, d_stats, true, &a);
  if (st != TBE_OK) return st;
  if (!buffer_ok(dweight, 2) || !is_aligned(dloss, 4) || !is_aligned(mean, 4)) return TBE_ERR_INVALID_ARG;
  if (a.tokens > 0 && (!buffer_ok(hidden, 2) || !buffer_ok(weight, a.copy_weight ? 2 : 16) ||
                       !buffer_ok(targets, itype_bytes(a.itype)) || !buffer_ok(lse, 4) || !buffer_ok(dhidden, 2)))
    return TBE_ERR_INVALID_ARG;
  DeviceInfo dev;
  if ((st = device_info(&dev)) != TBE_OK) return st;
  const LossBackwardLayout l = loss_backward_layout(a, dev);
  if ((st = check_workspace(ws, ws_bytes, l.total)) != TBE_OK) return st;
  return launch_loss_backward(a, l, hidden, weight, targets, lse, dloss, mean, dhidden, dweight, static_cast<char*>(ws), dev,
                              static_cast<cudaStream_t>(stream));
}

}  // extern "C"
