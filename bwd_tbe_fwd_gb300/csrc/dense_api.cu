// dense_api.cu -- the layer norm's C interface (tbe_dense.h): argument validation and the choice of
// vector width.
#include <cfloat>
#include <cmath>

#include "dense_common.cuh"

namespace tbe {
namespace {

constexpr int64_t kMaxCols = int64_t(1) << 30;
constexpr int64_t kMaxElems = (int64_t(1) << 39) - 1;

tbe_status make_norm(const tbe_norm_problem* p, NormArgs* a) {
  if (p == nullptr || p->rows < 0 || p->segments < 1 || p->widths == nullptr) return TBE_ERR_INVALID_ARG;
  if (p->segments > kMaxTables) return TBE_ERR_UNSUPPORTED;
  if (!dtype_ok(p->xdtype) || !dtype_ok(p->ydtype) || !dtype_ok(p->wdtype)) return TBE_ERR_UNSUPPORTED;
  if (p->xdtype != p->ydtype && p->xdtype != TBE_F32 && p->ydtype != TBE_F32) return TBE_ERR_UNSUPPORTED;
  if (!(p->eps >= 0) || std::isinf(p->eps)) return TBE_ERR_INVALID_ARG;
  int64_t cols = 0, widest = 0;
  bool equal = true;
  for (int s = 0; s < p->segments; ++s) {
    const int64_t w = p->widths[s];
    if (w < 1) return TBE_ERR_INVALID_ARG;
    cols += w;
    widest = w > widest ? w : widest;
    equal = equal && w == p->widths[0];
  }
  if (cols > kMaxCols || p->rows > kMaxElems / cols) return TBE_ERR_UNSUPPORTED;
  if (!equal && (p->col_offsets == nullptr || !is_aligned(p->col_offsets, 4))) return TBE_ERR_INVALID_ARG;
  a->rows = p->rows;
  a->x_stride = p->x_stride;
  a->y_stride = p->y_stride;
  a->dx_stride = p->dx_stride;
  a->col_offsets = equal ? nullptr : p->col_offsets;
  a->segments = p->segments;
  a->width = static_cast<int>(widest);
  a->cols = static_cast<int>(cols);
  a->wtype = p->wdtype;
  a->eps = p->eps > FLT_MIN ? p->eps : FLT_MIN;  // 2^-126: a segment without spread has an rstd all the same
  return TBE_OK;
}

// Elements of a vector access that every row, segment and buffer allows: 8 (both types 16-bit), 4 or 1.
int vector_width(const tbe_norm_problem& p, const void* x, const void* y, const void* dx) {
  const int xb = dtype_bytes(p.xdtype), yb = dtype_bytes(p.ydtype);
  for (int vec = xb == 2 && yb == 2 ? 8 : 4; vec > 1; vec /= 2) {
    if (vec == 2) break;
    bool ok = p.x_stride % vec == 0 && p.y_stride % vec == 0 && (dx == nullptr || p.dx_stride % vec == 0) &&
              is_aligned(x, vec * xb) && is_aligned(y, vec * yb) && is_aligned(dx, vec * xb);
    for (int s = 0; ok && s < p.segments; ++s) ok = p.widths[s] % vec == 0;
    if (ok) return vec;
  }
  return 1;
}

bool strided_ok(const void* p, int64_t stride, const NormArgs& a, int bytes) {
  return p != nullptr && stride >= a.cols && is_aligned(p, bytes);
}

}  // namespace
}  // namespace tbe

using namespace tbe;

extern "C" {

tbe_status tbe_layer_norm_forward(const tbe_norm_problem* prob, const void* x, const void* weight, const void* bias, void* y,
                                  float* mean, float* rstd, void* stream) {
  NormArgs a;
  tbe_status st = make_norm(prob, &a);
  if (st != TBE_OK) return st;
  if ((mean == nullptr) != (rstd == nullptr) || !is_aligned(mean, 4) || !is_aligned(rstd, 4)) return TBE_ERR_INVALID_ARG;
  const int wb = dtype_bytes(prob->wdtype);
  if (!is_aligned(weight, wb) || !is_aligned(bias, wb)) return TBE_ERR_INVALID_ARG;
  if (a.rows == 0) return TBE_OK;
  if (!strided_ok(x, a.x_stride, a, dtype_bytes(prob->xdtype)) || !strided_ok(y, a.y_stride, a, dtype_bytes(prob->ydtype)))
    return TBE_ERR_INVALID_ARG;
  if (x == y && (prob->xdtype != prob->ydtype || a.x_stride != a.y_stride)) return TBE_ERR_INVALID_ARG;
  DeviceInfo dev;
  if ((st = device_info(&dev)) != TBE_OK) return st;
  return launch_norm_forward(a, prob->xdtype, prob->ydtype, vector_width(*prob, x, y, nullptr), x, weight, bias, y, mean,
                             rstd, dev, static_cast<cudaStream_t>(stream));
}

size_t tbe_layer_norm_backward_workspace_size(const tbe_norm_problem* prob) {
  NormArgs a;
  DeviceInfo dev;
  if (make_norm(prob, &a) != TBE_OK || device_info(&dev) != TBE_OK) return 0;
  const int slots = norm_backward_slots(a, dev);
  return slots > 1 ? 2 * sizeof(float) * static_cast<size_t>(slots) * a.cols : 16;
}

tbe_status tbe_layer_norm_backward(const tbe_norm_problem* prob, const void* dy, const void* x, const float* mean,
                                   const float* rstd, const void* weight, void* dx, void* dweight, void* dbias, void* ws,
                                   size_t ws_bytes, void* stream) {
  NormArgs a;
  tbe_status st = make_norm(prob, &a);
  if (st != TBE_OK) return st;
  const int wb = dtype_bytes(prob->wdtype), xb = dtype_bytes(prob->xdtype);
  if (!is_aligned(weight, wb) || !is_aligned(dweight, wb) || !is_aligned(dbias, wb)) return TBE_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.rows == 0) {  // sums over no rows
    if (dweight != nullptr && (st = cuda_status(cudaMemsetAsync(dweight, 0, static_cast<size_t>(a.cols) * wb, s))) != TBE_OK)
      return st;
    if (dbias != nullptr) return cuda_status(cudaMemsetAsync(dbias, 0, static_cast<size_t>(a.cols) * wb, s));
    return TBE_OK;
  }
  if (!strided_ok(x, a.x_stride, a, xb) || !strided_ok(dy, a.y_stride, a, dtype_bytes(prob->ydtype)) ||
      (dx != nullptr && !strided_ok(dx, a.dx_stride, a, xb)))
    return TBE_ERR_INVALID_ARG;
  if (mean == nullptr || rstd == nullptr || !is_aligned(mean, 4) || !is_aligned(rstd, 4)) return TBE_ERR_INVALID_ARG;
  if (dx != nullptr && dx == x && a.dx_stride != a.x_stride) return TBE_ERR_INVALID_ARG;
  if (dx != nullptr && dx == dy && (prob->xdtype != prob->ydtype || a.dx_stride != a.y_stride)) return TBE_ERR_INVALID_ARG;
  if (dx == nullptr && dweight == nullptr && dbias == nullptr) return TBE_OK;
  const size_t need = tbe_layer_norm_backward_workspace_size(prob);
  if (need == 0) return TBE_ERR_CUDA;
  if ((dweight != nullptr || dbias != nullptr) && need > 16) {
    if (ws == nullptr || ws_bytes < need) return TBE_ERR_WORKSPACE;
    if (!is_aligned(ws, 16)) return TBE_ERR_INVALID_ARG;
  }
  DeviceInfo dev;
  if ((st = device_info(&dev)) != TBE_OK) return st;
  return launch_norm_backward(a, prob->xdtype, prob->ydtype, vector_width(*prob, x, dy, dx), dy, x, mean, rstd, weight, dx,
                              dweight, dbias, static_cast<float*>(ws), dev, s);
}

}  // extern "C"
