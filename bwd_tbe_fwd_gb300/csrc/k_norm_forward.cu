// k_norm_forward.cu -- layer norm over the segments of a row (tbe_layer_norm_forward).
//
// Every element is read once and written once; the bound is DRAM.  The mean and the sum of squared
// deviations are taken in that order over the row held in registers, so no cancellation of
// E[x^2] - mean^2 and no second read.
#include "dense_common.cuh"

namespace tbe {
namespace {

constexpr int kRowThreads = 256;
// Widest segment that a warp keeps in its registers.
template <int V> constexpr int kRowMax = V == 1 ? 256 : 128 * V;

// L lanes to a row, J vectors of V elements to a lane, U rows at a time: U * J loads in flight.
template <typename X, typename Y, int V, int L, int J, int U>
__device__ __forceinline__ void rows_body(const NormArgs& a, int seg, int col0, int width, int64_t row0, int64_t row1,
                                          const X* x, const void* weight, const void* bias, Y* y, float* mean,
                                          float* rstd) {
  constexpr int kGroups = kRowThreads / L;
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  bool in[J];
  float w[J][V], b[J][V];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = (j * L + lane) * V;
    in[j] = c < width;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      w[j][i] = in[j] && weight != nullptr ? load_any(weight, a.wtype, col0 + c + i) : 1.f;
      b[j][i] = in[j] && bias != nullptr ? load_any(bias, a.wtype, col0 + c + i) : 0.f;
    }
  }
  const float inv_n = 1.f / static_cast<float>(width);
  for (int64_t base = row0; base < row1; base += kGroups * U) {
    Pack<X, V> v[U][J];
    float mu[U], rs[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = base + u * kGroups + group;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        v[u][j].zero();
        if (r < row1 && in[j]) v[u][j].load(x + r * a.x_stride + col0 + (j * L + lane) * V);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) s += v[u][j].get(i);
      mu[u] = lanes_sum<L>(s) * inv_n;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float d = v[u][j].get(i) - mu[u];
          if (in[j]) s = fmaf(d, d, s);
        }
      rs[u] = __frsqrt_rn(fmaf(lanes_sum<L>(s), inv_n, a.eps));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = base + u * kGroups + group;
      if (r >= row1) continue;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (!in[j]) continue;
        float f[V];
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = fmaf((v[u][j].get(i) - mu[u]) * rs[u], w[j][i], b[j][i]);
        Pack<Y, V> o;
        o.set(f);
        o.store(y + r * a.y_stride + col0 + (j * L + lane) * V);
      }
      if (mean != nullptr && lane == 0) {
        mean[r * a.segments + seg] = mu[u];
        rstd[r * a.segments + seg] = rs[u];
      }
    }
  }
}

// A CTA takes one segment of rows_tile rows; neighbouring CTAs take neighbouring segments of the
// same rows, so what is in flight at one time is a band of whole rows.  The lanes to a row follow
// the segment's own width: the tables of one launch may be of different widths.
template <typename X, typename Y, int V>
__global__ void __launch_bounds__(kRowThreads)
    norm_rows_kernel(const __grid_constant__ NormArgs a, int64_t rows_tile, const X* x, const void* weight,
                     const void* bias, Y* y, float* mean, float* rstd) {
  const int seg = blockIdx.x % a.segments;
  const int64_t row0 = (blockIdx.x / a.segments) * rows_tile;
  const int64_t row1 = min(row0 + rows_tile, a.rows);
  int col0, width;
  segment_span<V>(a, seg, &col0, &width);
#define TBE_BODY(L, J, U) \
  rows_body<X, Y, V, L, J, U>(a, seg, col0, width, row0, row1, x, weight, bias, y, mean, rstd)
  if (V > 1 && width <= 8 * V) TBE_BODY(8, 1, 4);
  else if (V > 1 && width <= 16 * V) TBE_BODY(16, 1, 4);
  else if (width <= 32 * V) TBE_BODY(32, 1, 4);
  else if (width <= 64 * V) TBE_BODY(32, 2, 2);
  else if (V > 1 || width <= 128 * V) TBE_BODY(32, 4, 1);
  else TBE_BODY(32, 8, 1);
#undef TBE_BODY
}

// One CTA to a row (segment) of up to blockDim.x * J * V elements.
template <typename X, typename Y, int V, int J, int T>
__global__ void __launch_bounds__(T)
    norm_wide_kernel(const __grid_constant__ NormArgs a, int64_t row_slots, const X* x, const void* weight,
                     const void* bias, Y* y, float* mean, float* rstd) {
  __shared__ float part[2][32];
  const int seg = blockIdx.x % a.segments;
  int col0, width;
  segment_span<V>(a, seg, &col0, &width);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto block_sum = [&](float s, float* buf) {
    s = lanes_sum<32>(s);
    if (lane == 0) buf[warp] = s;
    __syncthreads();
    return lanes_sum<32>(lane < T / 32 ? buf[lane] : 0.f);
  };
  bool in[J];
  float w[J][V], b[J][V];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = (j * T + threadIdx.x) * V;
    in[j] = c < width;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      w[j][i] = in[j] && weight != nullptr ? load_any(weight, a.wtype, col0 + c + i) : 1.f;
      b[j][i] = in[j] && bias != nullptr ? load_any(bias, a.wtype, col0 + c + i) : 0.f;
    }
  }
  const float inv_n = 1.f / static_cast<float>(width);
  for (int64_t r = blockIdx.x / a.segments; r < a.rows; r += row_slots) {
    Pack<X, V> v[J];
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      v[j].zero();
      if (in[j]) v[j].load(x + r * a.x_stride + col0 + (j * T + threadIdx.x) * V);
    }
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) s += v[j].get(i);
    const float mu = block_sum(s, part[0]) * inv_n;
    s = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float d = v[j].get(i) - mu;
        if (in[j]) s = fmaf(d, d, s);
      }
    // the barrier inside also keeps the next row's first sums behind this row's reads of part[0]
    const float rs = __frsqrt_rn(fmaf(block_sum(s, part[1]), inv_n, a.eps));
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if (!in[j]) continue;
      float f[V];
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = fmaf((v[j].get(i) - mu) * rs, w[j][i], b[j][i]);
      Pack<Y, V> o;
      o.set(f);
      o.store(y + r * a.y_stride + col0 + (j * T + threadIdx.x) * V);
    }
    if (mean != nullptr && threadIdx.x == 0) {
      mean[r * a.segments + seg] = mu;
      rstd[r * a.segments + seg] = rs;
    }
  }
}

// Rows wider than the registers of a CTA: three passes over the row, the second and third from the
// caches.
template <typename X, typename Y, int V>
__global__ void __launch_bounds__(1024)
    norm_long_kernel(const __grid_constant__ NormArgs a, int64_t row_slots, const X* x, const void* weight,
                     const void* bias, Y* y, float* mean, float* rstd) {
  __shared__ float part[2][32];
  const int seg = blockIdx.x % a.segments;
  int col0, width;
  segment_span<V>(a, seg, &col0, &width);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto block_sum = [&](float s, float* buf) {
    s = lanes_sum<32>(s);
    if (lane == 0) buf[warp] = s;
    __syncthreads();
    return lanes_sum<32>(buf[lane]);
  };
  const float inv_n = 1.f / static_cast<float>(width);
  for (int64_t r = blockIdx.x / a.segments; r < a.rows; r += row_slots) {
    const X* xr = x + r * a.x_stride + col0;
    float s = 0.f;
#pragma unroll 4
    for (int c = threadIdx.x * V; c < width; c += 1024 * V) {
      Pack<X, V> v;
      v.load(xr + c);
#pragma unroll
      for (int i = 0; i < V; ++i) s += v.get(i);
    }
    const float mu = block_sum(s, part[0]) * inv_n;
    s = 0.f;
#pragma unroll 4
    for (int c = threadIdx.x * V; c < width; c += 1024 * V) {
      Pack<X, V> v;
      v.load(xr + c);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float d = v.get(i) - mu;
        s = fmaf(d, d, s);
      }
    }
    const float rs = __frsqrt_rn(fmaf(block_sum(s, part[1]), inv_n, a.eps));
    for (int c = threadIdx.x * V; c < width; c += 1024 * V) {
      Pack<X, V> v;
      v.load(xr + c);
      float f[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float w = weight != nullptr ? load_any(weight, a.wtype, col0 + c + i) : 1.f;
        const float b = bias != nullptr ? load_any(bias, a.wtype, col0 + c + i) : 0.f;
        f[i] = fmaf((v.get(i) - mu) * rs, w, b);
      }
      Pack<Y, V> o;
      o.set(f);
      o.store(y + r * a.y_stride + col0 + c);
    }
    if (mean != nullptr && threadIdx.x == 0) {
      mean[r * a.segments + seg] = mu;
      rstd[r * a.segments + seg] = rs;
    }
  }
}

template <typename X, typename Y, int V>
tbe_status launch(const NormArgs& a, const void* x, const void* weight, const void* bias, void* y, float* mean,
                  float* rstd, const DeviceInfo& dev, cudaStream_t s) {
  const X* xp = static_cast<const X*>(x);
  Y* yp = static_cast<Y*>(y);
  if (a.width <= kRowMax<V>) {
    // about 16 CTAs to an SM, and no fewer rows to a CTA than its warps
    const int64_t want = a.rows * a.segments / (static_cast<int64_t>(dev.sms) * 16);
    int64_t tile = want < 8 ? 8 : want > 256 ? 256 : want / 8 * 8;
    int64_t tiles = (a.rows + tile - 1) / tile;
    while (tiles * a.segments > INT32_MAX) {
      tile *= 2;
      tiles = (a.rows + tile - 1) / tile;
    }
    const unsigned grid = static_cast<unsigned>(tiles * a.segments);
    norm_rows_kernel<X, Y, V><<<grid, kRowThreads, 0, s>>>(a, tile, xp, weight, bias, yp, mean, rstd);
  } else {
    constexpr int J = 16 / V;
    auto wide = [&](auto kernel, int threads) {
      const int per_seg = persistent_grid(kernel, threads, 0, dev, INT32_MAX) / a.segments;
      const int64_t slots = per_seg < 1 ? 1 : per_seg < a.rows ? per_seg : a.rows;
      kernel<<<static_cast<unsigned>(slots * a.segments), threads, 0, s>>>(a, slots, xp, weight, bias, yp, mean, rstd);
    };
    if (a.width <= 64 * 16) wide(norm_wide_kernel<X, Y, V, J, 64>, 64);
    else if (a.width <= 128 * 16) wide(norm_wide_kernel<X, Y, V, J, 128>, 128);
    else if (a.width <= 256 * 16) wide(norm_wide_kernel<X, Y, V, J, 256>, 256);
    else if (a.width <= 512 * 16) wide(norm_wide_kernel<X, Y, V, J, 512>, 512);
    else if (a.width <= 1024 * 16) wide(norm_wide_kernel<X, Y, V, J, 1024>, 1024);
    else wide(norm_long_kernel<X, Y, V>, 1024);
  }
  note_launch();
  return cuda_status(cudaGetLastError());
}

}  // namespace

tbe_status launch_norm_forward(const NormArgs& a, int xtype, int ytype, int vec, const void* x, const void* weight,
                               const void* bias, void* y, float* mean, float* rstd, const DeviceInfo& dev,
                               cudaStream_t s) {
  return with_type(xtype, [&](auto xt) {
    return with_type(ytype, [&](auto yt) {
      using X = typename decltype(xt)::type;
      using Y = typename decltype(yt)::type;
      if constexpr (sizeof(X) == 2 && sizeof(Y) == 2 && !std::is_same<X, Y>::value) {
        return TBE_ERR_UNSUPPORTED;
      } else {
        if constexpr (sizeof(X) == 2 && sizeof(Y) == 2)
          if (vec >= 8) return launch<X, Y, 8>(a, x, weight, bias, y, mean, rstd, dev, s);
        if (vec >= 4) return launch<X, Y, 4>(a, x, weight, bias, y, mean, rstd, dev, s);
        return launch<X, Y, 1>(a, x, weight, bias, y, mean, rstd, dev, s);
      }
    });
  });
}

}  // namespace tbe
