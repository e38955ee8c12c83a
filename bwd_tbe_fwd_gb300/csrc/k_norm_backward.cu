// k_norm_backward.cu -- gradients of the layer norm (tbe_layer_norm_backward): dx by row, dweight
// and dbias by sums over all rows.
//
// One pass reads x and dy once, writes dx and keeps each column's sums of dy * xhat and dy in registers
// over the rows that a CTA takes (its slot); the slots' sums meet in a second kernel, in a fixed
// order.  The bound is DRAM; the partial rows add 16 bytes a column and slot to it.
//
// Measured on a GB300 (copy rate 6.78 TB/s): 8192 rows of 26 tables of 128, fp32 with bf16 dy, 43.9 us and 2.9 us for the slots'
// sums, 6.2 TB/s while the rows last; 16384 rows of 4096 bf16 69 + 4 us, 5.8 TB/s: there the latency of a row's two sums
// shows, as the columns' sums (32 registers a thread, with x, dy and the weight 117) leave 16 warps to an SM.  Reading
// the row a second time from shared memory for a third CTA an SM was slower (90 us), as were 2, 4 or 6 stages (75 to 76
// before the statistics came by shuffle).
#include "norm_rows.cuh"

namespace tbe {
namespace {

// Where the sums of a slot go: to its row of the partial sums, or, with a single slot, out.
struct SumsOut {
  float* partial;        // [2][slots][cols], or NULL: one slot
  int64_t slots;
  void* dweight;
  void* dbias;
  __device__ __forceinline__ bool wanted() const { return partial != nullptr || dweight != nullptr || dbias != nullptr; }
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

template <typename X, typename Y, int V, int L, int T>
__device__ __forceinline__ void backward_rows(const NormArgs& a, const RowIn& g, const SumsOut& out, int64_t slot, int seg,
                                              int col0, int width, const RowWalk& walk, char* smem) {
  constexpr int J = kPer / V;
  __shared__ float2 part[2][T / 32];
  const int lane = threadIdx.x % L;
  bool in[J];
#pragma unroll
  for (int j = 0; j < J; ++j) in[j] = (j * L + lane) * V < width;
  RowReader<X, V, L, T> x(g.x, a.x_stride, col0, width, walk.first, walk.step, smem);
  RowReader<Y, V, L, T> dy(g.dy, a.y_stride, col0, width, walk.first, walk.step, smem + kStages * stage_bytes<X, V>(T));
  for (int k = 0; k < kStages - 1; ++k) {
    x.copy(k, k < walk.mine, in);
    dy.copy(k, k < walk.mine, in);
    async_commit();
  }
  F2 w[kPer / 2], dw[kPer / 2], db[kPer / 2];
  read_weights<V, L>(g.weight, a.wtype, in[0] ? col0 + lane * V : col0, in, 1.f, w);
#pragma unroll
  for (int i = 0; i < kPer / 2; ++i) dw[i] = db[i] = F2(0.f);
  const float inv_n = 1.f / static_cast<float>(width);
  // The rows' statistics.  Wide rows of 16-bit types: 32 rows to a load (a lane each), a batch ahead, and a row's by shuffle
  // (16384 x 4096: 69 us, 74 by the other way).  Others: each row's, a row ahead (16384 x 4096 fp32 with bf16 dy: 106 us, 124
  // by shuffles; rows shared by parts of warps: the same).
  constexpr bool kBatches = V == 8 && L > 32;
  constexpr int B = kBatches ? 32 : 1;
  const int64_t stat_step = walk.step * a.segments, stat0 = walk.first * a.segments + seg;
  const int my_row = kBatches ? threadIdx.x % B : 0;
  auto stats = [&](int k0) {
    const bool have = k0 + my_row < walk.mine;
    const int64_t at = stat0 + (k0 + my_row) * stat_step;
    return make_float2(have ? g.mean[at] : 0.f, have ? g.rstd[at] : 0.f);
  };
  float2 batch = stats(0), batch_ahead = kBatches ? stats(B) : make_float2(0.f, 0.f);
  int stage = 0;
  X* dx = static_cast<X*>(g.dx) + walk.first * a.dx_stride + col0 + lane * V;
  const int64_t dx_step = walk.step * a.dx_stride;
  for (int k = 0; k < walk.count; ++k, dx += dx_step) {
    const bool more = k + kStages - 1 < walk.mine;
    x.reuse();
    x.copy(stage == 0 ? kStages - 1 : stage - 1, more, in);
    dy.copy(stage == 0 ? kStages - 1 : stage - 1, more, in);
    async_commit();
    async_wait<kStages - 1>();
    x.share();
    const bool valid = k < walk.mine;
    F2 xh[kPer / 2], h[kPer / 2];
    x.read(stage, valid, in, xh);
    dy.read(stage, valid, in, h);
    stage = stage == kStages - 1 ? 0 : stage + 1;
    float mu = batch.x, q = batch.y;  // 0 past the rows
    if constexpr (kBatches) {
      mu = __shfl_sync(kFull, mu, k % B);
      q = __shfl_sync(kFull, q, k % B);
      if (k % B == B - 1) {
        batch = batch_ahead;
        batch_ahead = stats(k + 1 + B);
      }
    } else {
      batch = stats(k + 1);
    }
    const F2 shift(-mu), scale(q);
    F2 s1(0.f), s2(0.f);
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) {
      xh[i] = (xh[i] + shift) * scale;  // outside the row times dy = 0
      dw[i] = fma2(h[i], xh[i], dw[i]);
      db[i] = db[i] + h[i];
      h[i] = h[i] * w[i];
      s1 = s1 + h[i];
      s2 = fma2(h[i], xh[i], s2);
    }
    if (g.dx == nullptr) {
      x.share();
      continue;
    }
    // the next row's sums go to the other buffer: one barrier a row
    const float2 c = row_sum2<L, T>(make_float2(s1.lo() + s1.hi(), s2.lo() + s2.hi()), part[k & 1]);
    if (!valid) continue;
    const F2 c1(-c.x * inv_n * q), c2(-c.y * inv_n * q);
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) h[i] = fma2(xh[i], c2, fma2(h[i], scale, c1));
    write_row<X, V, L>(dx, in, h);
  }
  if (!out.wanted()) return;
  auto value = [](const F2 (&f)[kPer / 2], int i) { return i & 1 ? f[i / 2].hi() : f[i / 2].lo(); };
  if constexpr (L > 32) {  // each thread owns its columns
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (in[j]) out.put(a, slot, col0 + (j * L + lane) * V + i, value(dw, j * V + i), value(db, j * V + i));
  } else {  // the T / L groups of the CTA hold the same columns: [groups][kPer * L] sums in shared memory, added in order
    async_wait<0>();
    __syncthreads();  // every thread is done with the stages
    float* sums = reinterpret_cast<float*>(smem);
    constexpr int kSpan = kPer * L;
    bool all[J];
#pragma unroll
    for (int j = 0; j < J; ++j) all[j] = true;
    write_row<float, V, L>(sums + threadIdx.x / L * kSpan + lane * V, all, dw);
    write_row<float, V, L>(sums + T * kPer + threadIdx.x / L * kSpan + lane * V, all, db);
    __syncthreads();
    for (int c = threadIdx.x; c < width; c += T) {
      float tw = 0.f, tb = 0.f;
#pragma unroll 8
      for (int k = 0; k < T / L; ++k) {
        tw += sums[k * kSpan + c];
        tb += sums[T * kPer + k * kSpan + c];
      }
      out.put(a, slot, col0 + c, tw, tb);
    }
  }
}

// Shared memory of a CTA: the stages, and then, where groups share columns, their sums.
template <typename X, typename Y, int V>
constexpr int backward_smem(int T, bool groups) {
  const int stages = kStages * (stage_bytes<X, V>(T) + stage_bytes<Y, V>(T));
  const int sums = groups ? 2 * T * kPer * static_cast<int>(sizeof(float)) : 0;
  return stages > sums ? stages : sums;
}

// A CTA takes one segment of a slot's rows, with lanes to a row by the segment's own width.
template <typename X, typename Y, int V>
__global__ void __launch_bounds__(kGroupThreads, 4)
    norm_backward_rows_kernel(const __grid_constant__ NormArgs a, const __grid_constant__ RowIn g,
                              const __grid_constant__ SumsOut out) {
  extern __shared__ __align__(16) char smem[];
  constexpr int T = kGroupThreads;
  const int seg = blockIdx.x % a.segments;
  const int64_t slot = blockIdx.x / a.segments;
  const int64_t per = (a.rows + out.slots - 1) / out.slots;
  const int64_t row0 = min(slot * per, a.rows), row1 = min(row0 + per, a.rows);
  int col0, width;
  segment_span<V>(a, seg, &col0, &width);
  auto go = [&](auto lanes) {
    constexpr int L = decltype(lanes)::value;
    const RowWalk walk(row0 + threadIdx.x / L, T / L, row0, row1);
    backward_rows<X, Y, V, L, T>(a, g, out, slot, seg, col0, width, walk, smem);
  };
  if (width <= row_capacity(4)) go(std::integral_constant<int, 4>());
  else if (width <= row_capacity(8)) go(std::integral_constant<int, 8>());
  else if (width <= row_capacity(16)) go(std::integral_constant<int, 16>());
  else go(std::integral_constant<int, 32>());
}

// A CTA of T threads to a row, over every slots-th row.
template <typename X, typename Y, int V, int T>
__global__ void __launch_bounds__(T, 512 / T)
    norm_backward_wide_kernel(const __grid_constant__ NormArgs a, const __grid_constant__ RowIn g,
                              const __grid_constant__ SumsOut out) {
  extern __shared__ __align__(16) char smem[];
  const int seg = blockIdx.x % a.segments;
  const int64_t slot = blockIdx.x / a.segments;
  int col0, width;
  segment_span<V>(a, seg, &col0, &width);
  const RowWalk walk(slot, out.slots, slot, a.rows);
  backward_rows<X, Y, V, T, T>(a, g, out, slot, seg, col0, width, walk, smem);
}

// Rows wider than a CTA's registers.  First the columns' sums: a thread to V columns, down the rows of a slot (dx may
// overwrite x or dy afterwards).
constexpr int kColumnThreads = 128;

template <typename X, typename Y, int V>
__global__ void __launch_bounds__(kColumnThreads)
    norm_backward_columns_kernel(const __grid_constant__ NormArgs a, const __grid_constant__ RowIn in,
                                 const __grid_constant__ SumsOut out) {
  int col0, width;
  segment_span<V>(a, blockIdx.y, &col0, &width);
  const int tiles = (a.width + kColumnThreads * V - 1) / (kColumnThreads * V);
  const int c = (static_cast<int>(blockIdx.x % tiles) * kColumnThreads + threadIdx.x) * V;
  const int64_t slot = blockIdx.x / tiles;
  if (c >= width) return;
  const int64_t per = (a.rows + out.slots - 1) / out.slots;
  const int64_t row0 = min(slot * per, a.rows), row1 = min(row0 + per, a.rows);
  const X* x = static_cast<const X*>(in.x) + row0 * a.x_stride + col0 + c;
  const Y* dy = static_cast<const Y*>(in.dy) + row0 * a.y_stride + col0 + c;
  const float* mean = in.mean + row0 * a.segments + blockIdx.y;
  const float* rstd = in.rstd + row0 * a.segments + blockIdx.y;
  float dw[V], db[V];
#pragma unroll
  for (int i = 0; i < V; ++i) dw[i] = db[i] = 0.f;
#pragma unroll 4
  for (int64_t r = row0; r < row1; ++r) {
    Pack<X, V> vx;
    Pack<Y, V> vy;
    vx.load(x);
    vy.load(dy);
    const float mu = *mean, rs = *rstd;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float d = vy.get(i);
      dw[i] = fmaf(d, (vx.get(i) - mu) * rs, dw[i]);
      db[i] += d;
    }
    x += a.x_stride;
    dy += a.y_stride;
    mean += a.segments;
    rstd += a.segments;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) out.put(a, slot, col0 + c + i, dw[i], db[i]);
}

// Then dx, in two passes over each row.
constexpr int kLongThreads = 512;

template <typename X, typename Y, int V>
__global__ void __launch_bounds__(kLongThreads)
    norm_backward_long_kernel(const __grid_constant__ NormArgs a, const __grid_constant__ RowIn in, int64_t row_slots) {
  __shared__ float2 part[2][kLongThreads / 32];
  const X* x = static_cast<const X*>(in.x);
  const Y* dy = static_cast<const Y*>(in.dy);
  X* dx = static_cast<X*>(in.dx);
  const int seg = blockIdx.x % a.segments;
  int col0, width;
  segment_span<V>(a, seg, &col0, &width);
  const float inv_n = 1.f / static_cast<float>(width);
  int buf = 0;
  for (int64_t r = blockIdx.x / a.segments; r < a.rows; r += row_slots, buf ^= 1) {
    const float mu = in.mean[r * a.segments + seg], rs = in.rstd[r * a.segments + seg];
    const X* xr = x + r * a.x_stride + col0;
    const Y* yr = dy + r * a.y_stride + col0;
    X* dr = dx + r * a.dx_stride + col0;
    float c1 = 0.f, c2 = 0.f;
#pragma unroll 2
    for (int c = threadIdx.x * V; c < width; c += kLongThreads * V) {
      Pack<X, V> vx;
      Pack<Y, V> vy;
      vx.load(xr + c);
      vy.load(yr + c);
      float w[V];
      load_weights<V>(in.weight, a.wtype, col0 + c, 1.f, w);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float h = vy.get(i) * w[i];
        c1 += h;
        c2 = fmaf(h, (vx.get(i) - mu) * rs, c2);
      }
    }
    const float2 sums = row_sum2<kLongThreads, kLongThreads>(make_float2(c1, c2), part[buf]);
    c1 = sums.x * inv_n;
    c2 = sums.y * inv_n;
#pragma unroll 2
    for (int c = threadIdx.x * V; c < width; c += kLongThreads * V) {
      Pack<X, V> vx;
      Pack<Y, V> vy;
      vx.load(xr + c);
      vy.load(yr + c);
      float w[V], f[V];
      load_weights<V>(in.weight, a.wtype, col0 + c, 1.f, w);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = rs * (fmaf(vy.get(i), w[i], -c1) - (vx.get(i) - mu) * rs * c2);
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
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while the kernel before it ends
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float dw = 0.f, db = 0.f;
  if (c < cols) {
#pragma unroll 8
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

constexpr int kWideMax = row_capacity(512);  // wider rows take two kernels

template <typename X, typename Y, int V>
tbe_status launch(const NormArgs& a, const RowIn& in, SumsOut out, const DeviceInfo& dev, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(out.slots * a.segments);
  cudaError_t bad = cudaSuccess;
  auto go = [&](auto kernel, int threads, bool groups) {
    const int smem = backward_smem<X, Y, V>(threads, groups);
    if (smem > kPlainSmem) bad = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (bad == cudaSuccess) kernel<<<grid, threads, smem, s>>>(a, in, out);
  };
  if (a.width <= row_capacity(32)) {
    go(norm_backward_rows_kernel<X, Y, V>, kGroupThreads, true);
  } else if (a.width <= row_capacity(64)) {
    go(norm_backward_wide_kernel<X, Y, V, 64>, 64, false);
  } else if (a.width <= row_capacity(128)) {
    go(norm_backward_wide_kernel<X, Y, V, 128>, 128, false);
  } else if (a.width <= row_capacity(256)) {
    go(norm_backward_wide_kernel<X, Y, V, 256>, 256, false);
  } else if (a.width <= kWideMax) {
    go(norm_backward_wide_kernel<X, Y, V, 512>, 512, false);
  } else {
    if (out.dweight != nullptr || out.dbias != nullptr) {
      const int64_t tiles = (a.width + kColumnThreads * V - 1) / (kColumnThreads * V);
      norm_backward_columns_kernel<X, Y, V>
          <<<dim3(static_cast<unsigned>(tiles * out.slots), a.segments), kColumnThreads, 0, s>>>(a, in, out);
      note_launch();
    }
    if (in.dx != nullptr) {
      const int per_seg = persistent_grid(norm_backward_long_kernel<X, Y, V>, kLongThreads, 0, dev, INT32_MAX) / a.segments;
      const int64_t row_slots = per_seg < 1 ? 1 : per_seg < a.rows ? per_seg : a.rows;
      norm_backward_long_kernel<X, Y, V>
          <<<static_cast<unsigned>(row_slots * a.segments), kLongThreads, 0, s>>>(a, in, row_slots);
      note_launch();
    }
    return cuda_status(cudaGetLastError());
  }
  if (bad != cudaSuccess) return cuda_status(bad);
  note_launch();
  return cuda_status(cudaGetLastError());
}

}  // namespace

int norm_backward_slots(const NormArgs& a, const DeviceInfo& dev) {
  // By parts of warps: two waves of four CTAs to an SM, no fewer than 32 rows to a slot.  By CTAs: one wave of 512
  // threads to an SM.  Wider still: enough that tiles of 1024 columns fill the SMs sixteen times.
  int64_t want, least;
  if (a.width <= row_capacity(32)) {
    want = static_cast<int64_t>(dev.sms) * 8 / a.segments;
    least = 32;
  } else if (a.width <= kWideMax) {
    int threads = 64;
    while (row_capacity(threads) < a.width) threads *= 2;
    want = static_cast<int64_t>(dev.sms) * (512 / threads) / a.segments;
    least = 1;
  } else {
    want = static_cast<int64_t>(dev.sms) * 16 / (static_cast<int64_t>(a.segments) * ((a.width + 1023) / 1024));
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
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t config = {};
  config.gridDim = dim3((a.cols + 31) / 32);
  config.blockDim = dim3(1024);
  config.stream = s;
  config.attrs = &early;
  config.numAttrs = 1;
  note_launch();
  return cuda_status(cudaLaunchKernelEx(&config, norm_sum_slots_kernel, static_cast<const float*>(partial), out.slots, a.cols,
                                        a.wtype, dweight, dbias));
}

}  // namespace tbe
