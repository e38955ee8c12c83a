// k_norm_backward.cu -- gradients of the layer norm (tbe_layer_norm_backward): dx by row, dweight
// and dbias by sums over all rows.
//
// One pass reads x and dy once, writes dx and keeps each column's sums of dy * xhat and dy in registers
// over the rows that a CTA takes (its slot); the slots' sums meet in a second kernel, in a fixed
// order.  The bound is DRAM; the partial rows add 16 bytes a column and slot to it.
#include "dense_common.cuh"

namespace tbe {
namespace {

constexpr int kRowThreads = 256;
// Widest segment that a warp keeps in its registers (x, dy, the weight and the two sums of each column).
template <int V> constexpr int kRowMax = V == 1 ? 128 : V == 4 ? 512 : 512;
constexpr int kWideElems = 16;                    // elements of a row to a thread of a wide row
constexpr int kWideMax = 512 * kWideElems;        // wider rows take two kernels

// Where the sums of a slot go: to its row of the partial sums, or, with a single slot, out.
struct SumsOut {
  float* partial;        // [2][slots][cols], or NULL: one slot
  int64_t slots;
  void* dweight;
  void* dbias;
  __device__ __forceinline__ void put(const NormArgs& a, int64_t slot, int c, float dw, float db) const {
    if (partial != nullptr) {
      partial[slot * a.cols + c] = dw;
      partial[(slots + slot) * a.cols + c] = db;
    } else {
      if (dweight != nullptr) store_any(dweight, a.wtype, c, dw);
      if (dbias != nullptr) store_any(dbias, a.wtype, c, db);
    }
  }
};

struct RowIn {
  const void* dy;
  const void* x;
  const float* mean;
  const float* rstd;
  const void* weight;
  void* dx;
};

// L lanes to a row, J vectors of V elements to a lane, U rows at a time.
template <typename X, typename Y, int V, int L, int J, int U>
__device__ __forceinline__ void rows_body(const NormArgs& a, int seg, int col0, int width, int64_t row0, int64_t row1,
                                          const RowIn& in, const SumsOut& out, int64_t slot, float* smem) {
  constexpr int kGroups = kRowThreads / L;
  const X* x = static_cast<const X*>(in.x);
  const Y* dy = static_cast<const Y*>(in.dy);
  X* dx = static_cast<X*>(in.dx);
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  bool has[J];
  float w[J][V], dw[J][V], db[J][V];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = (j * L + lane) * V;
    has[j] = c < width;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      w[j][i] = has[j] && in.weight != nullptr ? load_any(in.weight, a.wtype, col0 + c + i) : 1.f;
      dw[j][i] = db[j][i] = 0.f;
    }
  }
  const float inv_n = 1.f / static_cast<float>(width);
  for (int64_t base = row0; base < row1; base += kGroups * U) {
    Pack<X, V> vx[U][J];
    Pack<Y, V> vy[U][J];
    float mu[U], rs[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = base + u * kGroups + group;
      mu[u] = rs[u] = 0.f;
      if (r < row1) {
        mu[u] = in.mean[r * a.segments + seg];
        rs[u] = in.rstd[r * a.segments + seg];
      }
#pragma unroll
      for (int j = 0; j < J; ++j) {
        vx[u][j].zero();
        vy[u][j].zero();
        if (r < row1 && has[j]) {
          vx[u][j].load(x + r * a.x_stride + col0 + (j * L + lane) * V);
          vy[u][j].load(dy + r * a.y_stride + col0 + (j * L + lane) * V);
        }
      }
    }
    float c1[U], c2[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      c1[u] = c2[u] = 0.f;
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float d = vy[u][j].get(i), xh = (vx[u][j].get(i) - mu[u]) * rs[u], h = d * w[j][i];
          c1[u] += h;
          c2[u] = fmaf(h, xh, c2[u]);
          dw[j][i] = fmaf(d, xh, dw[j][i]);
          db[j][i] += d;
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      c1[u] = lanes_sum<L>(c1[u]) * inv_n;
      c2[u] = lanes_sum<L>(c2[u]) * inv_n;
    }
    if (dx != nullptr) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t r = base + u * kGroups + group;
        if (r >= row1) continue;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if (!has[j]) continue;
          float f[V];
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float xh = (vx[u][j].get(i) - mu[u]) * rs[u];
            f[i] = rs[u] * (fmaf(vy[u][j].get(i), w[j][i], -c1[u]) - xh * c2[u]);
          }
          Pack<X, V> o;
          o.set(f);
          o.store(dx + r * a.dx_stride + col0 + (j * L + lane) * V);
        }
      }
    }
  }
  if (out.partial == nullptr && out.dweight == nullptr && out.dbias == nullptr) return;
  // the groups of a warp, then the warps (kGroups / kSub rows of sums), one after the other
  constexpr int kSub = 32 / L, kWarps = kRowThreads / 32, kSpan = L * J * V;
  const int warp = threadIdx.x / 32;
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int o = 16; o >= L; o >>= 1) {
        dw[j][i] += __shfl_xor_sync(kFull, dw[j][i], o);
        db[j][i] += __shfl_xor_sync(kFull, db[j][i], o);
      }
  (void)kSub;
  float* sw = smem;
  float* sb = smem + kWarps * kSpan;
  if ((threadIdx.x & 31) < L) {
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = (j * L + lane) * V + i;
        sw[warp * kSpan + c] = dw[j][i];
        sb[warp * kSpan + c] = db[j][i];
      }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < width; c += kRowThreads) {
    float tw = 0.f, tb = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      tw += sw[k * kSpan + c];
      tb += sb[k * kSpan + c];
    }
    out.put(a, slot, col0 + c, tw, tb);
  }
}

// A CTA takes one segment of a slot's rows, with lanes to a row by the segment's own width.
template <typename X, typename Y, int V>
__global__ void __launch_bounds__(kRowThreads)
    norm_backward_rows_kernel(const __grid_constant__ NormArgs a, const __grid_constant__ RowIn in,
                              const __grid_constant__ SumsOut out) {
  constexpr int kMaxJ = kRowMax<V> / (32 * V);
  __shared__ float smem[2 * (kRowThreads / 32) * 32 * kMaxJ * V];
  const int seg = blockIdx.x % a.segments;
  const int64_t slot = blockIdx.x / a.segments;
  const int64_t per = (a.rows + out.slots - 1) / out.slots;
  const int64_t row0 = min(slot * per, a.rows), row1 = min(row0 + per, a.rows);
  int col0, width;
  segment_span<V>(a, seg, &col0, &width);
#define TBE_BODY(L, J, U) rows_body<X, Y, V, L, J, U>(a, seg, col0, width, row0, row1, in, out, slot, smem)
  if (V > 1 && width <= 8 * V) TBE_BODY(8, 1, 4);
  else if (V > 1 && width <= 16 * V) TBE_BODY(16, 1, 4);
  else if (width <= 32 * V) TBE_BODY(32, 1, 4);
  else if (kMaxJ == 2 || width <= 64 * V) TBE_BODY(32, 2, 2);
  else if constexpr (kMaxJ > 2) TBE_BODY(32, 4, 1);
#undef TBE_BODY
}

// One CTA to a row (segment) of up to T * J * V columns, over the rows of its slot; each thread owns
// its columns' sums.
template <typename X, typename Y, int V, int T>
__global__ void __launch_bounds__(T)
    norm_backward_wide_kernel(const __grid_constant__ NormArgs a, const __grid_constant__ RowIn in,
                              const __grid_constant__ SumsOut out) {
  constexpr int J = kWideElems / V;
  __shared__ float2 part[2][T / 32];
  const X* x = static_cast<const X*>(in.x);
  const Y* dy = static_cast<const Y*>(in.dy);
  X* dx = static_cast<X*>(in.dx);
  const int seg = blockIdx.x % a.segments;
  const int64_t slot = blockIdx.x / a.segments;
  int col0, width;
  segment_span<V>(a, seg, &col0, &width);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  bool has[J];
  float w[J][V], dw[J][V], db[J][V];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = (j * T + threadIdx.x) * V;
    has[j] = c < width;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      w[j][i] = has[j] && in.weight != nullptr ? load_any(in.weight, a.wtype, col0 + c + i) : 1.f;
      dw[j][i] = db[j][i] = 0.f;
    }
  }
  const float inv_n = 1.f / static_cast<float>(width);
  Pack<X, V> vx[J];
  Pack<Y, V> vy[J];
  float mu = 0.f, rs = 0.f;
  auto fetch = [&](int64_t r) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      vx[j].zero();
      vy[j].zero();
      if (r < a.rows && has[j]) {
        vx[j].load(x + r * a.x_stride + col0 + (j * T + threadIdx.x) * V);
        vy[j].load(dy + r * a.y_stride + col0 + (j * T + threadIdx.x) * V);
      }
    }
    if (r < a.rows) {
      mu = in.mean[r * a.segments + seg];
      rs = in.rstd[r * a.segments + seg];
    }
  };
  int buf = 0;
  for (int64_t r = slot; r < a.rows; r += out.slots, buf ^= 1) {
    fetch(r);
    float c1 = 0.f, c2 = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float d = vy[j].get(i), xh = (vx[j].get(i) - mu) * rs, h = d * w[j][i];
        c1 += h;
        c2 = fmaf(h, xh, c2);
        if (has[j]) dw[j][i] = fmaf(d, xh, dw[j][i]);
        db[j][i] += d;
      }
    c1 = lanes_sum<32>(c1);
    c2 = lanes_sum<32>(c2);
    if (lane == 0) part[buf][warp] = make_float2(c1, c2);
    __syncthreads();  // the next row writes the other buffer
    const float2 p = lane < T / 32 ? part[buf][lane] : make_float2(0.f, 0.f);
    c1 = lanes_sum<32>(p.x) * inv_n;
    c2 = lanes_sum<32>(p.y) * inv_n;
    if (dx != nullptr) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (!has[j]) continue;
        float f[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float xh = (vx[j].get(i) - mu) * rs;
          f[i] = rs * (fmaf(vy[j].get(i), w[j][i], -c1) - xh * c2);
        }
        Pack<X, V> o;
        o.set(f);
        o.store(dx + r * a.dx_stride + col0 + (j * T + threadIdx.x) * V);
      }
    }
  }
  if (out.partial == nullptr && out.dweight == nullptr && out.dbias == nullptr) return;
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (has[j]) out.put(a, slot, col0 + (j * T + threadIdx.x) * V + i, dw[j][i], db[j][i]);
}

// Rows wider than a CTA's registers.  First the columns' sums: a thread to a column, down the rows of
// a slot (dx may overwrite x or dy afterwards).
template <typename X, typename Y>
__global__ void __launch_bounds__(256)
    norm_backward_columns_kernel(const __grid_constant__ NormArgs a, const __grid_constant__ RowIn in,
                                 const __grid_constant__ SumsOut out) {
  const X* x = static_cast<const X*>(in.x);
  const Y* dy = static_cast<const Y*>(in.dy);
  int col0, width;
  segment_span<1>(a, blockIdx.y, &col0, &width);
  const int tiles = (a.width + 255) / 256;
  const int c = static_cast<int>(blockIdx.x % tiles) * 256 + threadIdx.x;
  const int64_t slot = blockIdx.x / tiles;
  if (c >= width) return;
  const int64_t per = (a.rows + out.slots - 1) / out.slots;
  const int64_t row0 = min(slot * per, a.rows), row1 = min(row0 + per, a.rows);
  float dw = 0.f, db = 0.f;
#pragma unroll 8
  for (int64_t r = row0; r < row1; ++r) {
    Pack<X, 1> vx;
    Pack<Y, 1> vy;
    vx.load(x + r * a.x_stride + col0 + c);
    vy.load(dy + r * a.y_stride + col0 + c);
    const float d = vy.get(0);
    dw = fmaf(d, (vx.get(0) - in.mean[r * a.segments + blockIdx.y]) * in.rstd[r * a.segments + blockIdx.y], dw);
    db += d;
  }
  out.put(a, slot, col0 + c, dw, db);
}

// Then dx, in two passes over each row.
template <typename X, typename Y, int V>
__global__ void __launch_bounds__(1024)
    norm_backward_long_kernel(const __grid_constant__ NormArgs a, const __grid_constant__ RowIn in, int64_t row_slots) {
  __shared__ float2 part[2][32];
  const X* x = static_cast<const X*>(in.x);
  const Y* dy = static_cast<const Y*>(in.dy);
  X* dx = static_cast<X*>(in.dx);
  const int seg = blockIdx.x % a.segments;
  int col0, width;
  segment_span<V>(a, seg, &col0, &width);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float inv_n = 1.f / static_cast<float>(width);
  int buf = 0;
  for (int64_t r = blockIdx.x / a.segments; r < a.rows; r += row_slots, buf ^= 1) {
    const float mu = in.mean[r * a.segments + seg], rs = in.rstd[r * a.segments + seg];
    const X* xr = x + r * a.x_stride + col0;
    const Y* yr = dy + r * a.y_stride + col0;
    X* dr = dx + r * a.dx_stride + col0;
    float c1 = 0.f, c2 = 0.f;
#pragma unroll 2
    for (int c = threadIdx.x * V; c < width; c += 1024 * V) {
      Pack<X, V> vx;
      Pack<Y, V> vy;
      vx.load(xr + c);
      vy.load(yr + c);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float h = vy.get(i) * (in.weight != nullptr ? load_any(in.weight, a.wtype, col0 + c + i) : 1.f);
        c1 += h;
        c2 = fmaf(h, (vx.get(i) - mu) * rs, c2);
      }
    }
    c1 = lanes_sum<32>(c1);
    c2 = lanes_sum<32>(c2);
    if (lane == 0) part[buf][warp] = make_float2(c1, c2);
    __syncthreads();
    const float2 p = part[buf][lane];
    c1 = lanes_sum<32>(p.x) * inv_n;
    c2 = lanes_sum<32>(p.y) * inv_n;
    for (int c = threadIdx.x * V; c < width; c += 1024 * V) {
      Pack<X, V> vx;
      Pack<Y, V> vy;
      vx.load(xr + c);
      vy.load(yr + c);
      float f[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float w = in.weight != nullptr ? load_any(in.weight, a.wtype, col0 + c + i) : 1.f;
        f[i] = rs * (fmaf(vy.get(i), w, -c1) - (vx.get(i) - mu) * rs * c2);
      }
      Pack<X, V> o;
      o.set(f);
      o.store(dr + c);
    }
  }
}

// The slots' sums of 32 columns: 32 warps each take every 32nd slot, then their sums are added in order.
__global__ void __launch_bounds__(1024)
    norm_sum_slots_kernel(const float* partial, int64_t slots, int cols, int wtype, void* dweight, void* dbias) {
  __shared__ float sums[2][32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float dw = 0.f, db = 0.f;
  if (c < cols) {
#pragma unroll 4
    for (int64_t s = warp; s < slots; s += 32) {
      dw += partial[s * cols + c];
      db += partial[(slots + s) * cols + c];
    }
  }
  sums[0][warp][lane] = dw;
  sums[1][warp][lane] = db;
  __syncthreads();
  if (warp < 2) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) t += sums[warp][k][lane];
    void* out = warp == 0 ? dweight : dbias;
    if (c < cols && out != nullptr) store_any(out, wtype, c, t);
  }
}

template <typename X, typename Y, int V>
tbe_status launch(const NormArgs& a, const RowIn& in, SumsOut out, const DeviceInfo& dev, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(out.slots * a.segments);
  if (a.width <= kRowMax<V>) {
    norm_backward_rows_kernel<X, Y, V><<<grid, kRowThreads, 0, s>>>(a, in, out);
  } else if (a.width <= 64 * kWideElems) {
    norm_backward_wide_kernel<X, Y, V, 64><<<grid, 64, 0, s>>>(a, in, out);
  } else if (a.width <= 128 * kWideElems) {
    norm_backward_wide_kernel<X, Y, V, 128><<<grid, 128, 0, s>>>(a, in, out);
  } else if (a.width <= 256 * kWideElems) {
    norm_backward_wide_kernel<X, Y, V, 256><<<grid, 256, 0, s>>>(a, in, out);
  } else if (a.width <= kWideMax) {
    norm_backward_wide_kernel<X, Y, V, 512><<<grid, 512, 0, s>>>(a, in, out);
  } else {
    if (out.dweight != nullptr || out.dbias != nullptr) {
      const int64_t tiles = (a.width + 255) / 256;
      norm_backward_columns_kernel<X, Y>
          <<<dim3(static_cast<unsigned>(tiles * out.slots), a.segments), 256, 0, s>>>(a, in, out);
      note_launch();
    }
    if (in.dx != nullptr) {
      const int per_seg = persistent_grid(norm_backward_long_kernel<X, Y, V>, 1024, 0, dev, INT32_MAX) / a.segments;
      const int64_t row_slots = per_seg < 1 ? 1 : per_seg < a.rows ? per_seg : a.rows;
      norm_backward_long_kernel<X, Y, V>
          <<<static_cast<unsigned>(row_slots * a.segments), 1024, 0, s>>>(a, in, row_slots);
      note_launch();
    }
    return cuda_status(cudaGetLastError());
  }
  note_launch();
  return cuda_status(cudaGetLastError());
}

}  // namespace

int norm_backward_slots(const NormArgs& a, const DeviceInfo& dev) {
  // rows by warps: about 16 CTAs to an SM, no fewer than 32 rows to a slot; rows by CTAs: two to four to an SM;
  // wider still: enough that 256-column tiles fill the SMs four times
  int64_t want, least;
  if (a.width <= 512) {
    want = static_cast<int64_t>(dev.sms) * 16 / a.segments;
    least = 32;
  } else if (a.width <= kWideMax) {
    want = static_cast<int64_t>(dev.sms) * (a.width <= 2048 ? 4 : 2) / a.segments;
    least = 4;
  } else {
    want = static_cast<int64_t>(dev.sms) * 4 / (static_cast<int64_t>(a.segments) * ((a.width + 255) / 256));
    least = 16;
  }
  const int64_t most = (a.rows + least - 1) / least;
  if (want > most) want = most;
  return static_cast<int>(want < 1 ? 1 : want);
}

tbe_status launch_norm_backward(const NormArgs& a, int xtype, int ytype, int vec, const void* dy, const void* x,
                                const float* mean, const float* rstd, const void* weight, void* dx, void* dweight,
                                void* dbias, float* partial, const DeviceInfo& dev, cudaStream_t s) {
  const RowIn in{dy, x, mean, rstd, weight, dx};
  SumsOut out{nullptr, norm_backward_slots(a, dev), dweight, dbias};
  const bool sums = dweight != nullptr || dbias != nullptr;
  if (sums && out.slots > 1) out.partial = partial;
  const tbe_status st = with_type(xtype, [&](auto xt) {
    return with_type(ytype, [&](auto yt) {
      using X = typename decltype(xt)::type;
      using Y = typename decltype(yt)::type;
      if constexpr (sizeof(X) == 2 && sizeof(Y) == 2 && !std::is_same<X, Y>::value) {
        return TBE_ERR_UNSUPPORTED;
      } else {
        if constexpr (sizeof(X) == 2 && sizeof(Y) == 2)
          if (vec >= 8) return launch<X, Y, 8>(a, in, out, dev, s);
        if (vec >= 4) return launch<X, Y, 4>(a, in, out, dev, s);
        return launch<X, Y, 1>(a, in, out, dev, s);
      }
    });
  });
  if (st != TBE_OK || out.partial == nullptr) return st;
  norm_sum_slots_kernel<<<(a.cols + 31) / 32, 1024, 0, s>>>(partial, out.slots, a.cols, a.wtype, dweight, dbias);
  note_launch();
  return cuda_status(cudaGetLastError());
}

}  // namespace tbe
