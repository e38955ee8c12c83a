// k_norm_forward.cu -- layer norm over the segments of a row (tbe_layer_norm_forward).
//
// Every element is read once and written once; the bound is DRAM.  The mean and the sum of squared
// deviations are taken one after the other over the row held in registers: no cancellation of
// E[x^2] - mean^2 and no second read.  Rows of equal values come out without deviations at all: the sums of 16-bit
// ones are exact, and where the rounding of an fp32 row's sum may be all of its deviations the mean is corrected (is_flat).
//
// Measured on a GB300 (copy rate 6.78 TB/s): 16384 rows of 64 tables of 32 to 256 columns, fp32 -> bf16, 121 us, 6.3 TB/s;
// 67M elements in rows of 512 fp32 83 us, 6.5 TB/s, of 4096 bf16 45 us, 6.0 TB/s; fp16 rows of 1001, which allow no
// vector, 62 us, 4.3 TB/s (60% of the issue slots, 28% of the warps; 76 while each element was asked for).
#include "norm_rows.cuh"

namespace tbe {
namespace {

struct ForwardArgs {
  const void* x;
  const void* weight;
  const void* bias;
  void* y;
  float* mean;
  float* rstd;
};

// True where the sum of up to `most` vectors of equal values is exact in any order: the value's 8 or 11 bits of
// significand and those that count the vectors are no more than fp32's 24.
template <typename X>
constexpr bool exact_sums(int most) {
  return std::is_same<X, __nv_bfloat16>::value ? most <= 1 << 16 : std::is_same<X, __half>::value ? most <= 1 << 13 : false;
}

// The one form whose sums need a bit more, 2^14 equal values of 11 bits: it keeps what the last addition leaves out.
template <typename X, int V, int L>
constexpr bool kApart = std::is_same<X, __half>::value && V == 1 && L == 1024;
template <int T>
__device__ __forceinline__ float2 row_sum_in_two(float v, float* part) {
  static_assert(T == 1024, "a part to a lane");
  v = lanes_sum<32>(v);
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
  __syncthreads();
  v = part[threadIdx.x % 32];
#pragma unroll
  for (int o = 16; o > 1; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  const float u = __shfl_xor_sync(kFull, v, 1), s = v + u, u_in = s - v;
  return make_float2(s, isinf(s) ? 0.f : (v - (s - u_in)) + (u - u_in));
}

// A row is flat where its deviations are no larger than what the rounding of its sum may put the mean off by, `slack` of it:
// its mean is then corrected by the deviations' own.  In a row of equal values these are exact and alike, and after the
// correction exactly zero.  (Where there are none the mean is exact.  Below 2^-50 their squares may leave fp32.)
__device__ __forceinline__ bool is_flat(float mu, float var, float slack) {
  const float most = mu * slack;
  return var > 0.f && var <= most * most;
}
constexpr float kSlack = 0x1p-18f;  // twice the roundings (some 20) of a sum by threads of 16 elements

// A flat row again, row r of segment blockIdx.x % segments, from its stage; all threads that share sums call it, `flat` for
// those of such rows.  Rare, so in few registers: a vector at a time, and what can be is made anew from opaque indexes, so that
// nothing is computed ahead of the loop over rows and kept through it.
template <typename X, typename Y, int V, int L, int T>
__device__ __forceinline__ void forward_flat_row(const NormArgs& a, const ForwardArgs& g, char* smem, float (&part)[2][T / 32],
                                                 int stage, int64_t r, float mu, bool flat) {
  int lane, seg, col0, width;
  asm volatile("mov.u32 %0, %%tid.x;" : "=r"(lane));
  asm volatile("mov.u32 %0, %%ctaid.x;" : "=r"(seg));
  lane %= L;
  seg %= a.segments;
  segment_span<V>(a, seg, &col0, &width);
  const float inv_n = 1.f / static_cast<float>(width);
  const X* x = static_cast<const X*>(g.x) + r * a.x_stride + col0;
  Y* y = static_cast<Y*>(g.y) + r * a.y_stride + col0;
  auto over = [&](auto&& f) {
#pragma unroll 1
    for (int j = 0; j < kPer / V; ++j) {
      const int c = (j * L + lane) * V;
      if (!flat || c >= width) continue;
      Pack<X, V> v;
      RowReader<X, V, L, T>::read_one(smem, stage, x, j, lane, v);
      f(c, v);
    }
  };
  float s = 0.f;
  over([&](int, const Pack<X, V>& v) {
#pragma unroll
    for (int i = 0; i < V; ++i) s += v.get(i) - mu;
  });
  mu += row_sum<L, T>(s, part[0]) * inv_n;
  s = 0.f;
  over([&](int, const Pack<X, V>& v) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float d = v.get(i) - mu;
      s = fmaf(d, d, s);
    }
  });
  const float rs = __frsqrt_rn(fmaf(row_sum<L, T>(s, part[1]), inv_n, a.eps));
  over([&](int c, const Pack<X, V>& v) {
    float w[V], b[V], f[V];
    load_weights<V>(g.weight, a.wtype, col0 + c, 1.f, w);
    load_weights<V>(g.bias, a.wtype, col0 + c, 0.f, b);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = fmaf((v.get(i) - mu) * rs, w[i], b[i]);
    Pack<Y, V> o;
    o.set(f);
    o.store(y + c);
  });
  if (flat && g.mean != nullptr && lane == 0) {
    g.mean[r * a.segments + seg] = mu;
    g.rstd[r * a.segments + seg] = rs;
  }
  RowReader<X, V, L, T>::share();  // the stage is filled again next, by any of the threads that share it
}

template <typename X, typename Y, int V, int L, int T>
__device__ __forceinline__ void forward_rows(const NormArgs& a, const ForwardArgs& g, int seg, int col0, int width,
                                             const RowWalk& walk, char* smem) {
  constexpr int J = kPer / V;
  __shared__ float part[2][T / 32];
  const int lane = threadIdx.x % L;
  bool in[J];
#pragma unroll
  for (int j = 0; j < J; ++j) in[j] = (j * L + lane) * V < width;
  RowReader<X, V, L, T> x(g.x, a.x_stride, col0, width, walk.first, walk.step, smem);
  for (int k = 0; k < kStages - 1; ++k) {
    x.copy(k, k < walk.mine, in);
    async_commit();
  }
  F2 w[kPer / 2], b[kPer / 2];
  const int first_col = in[0] ? col0 + lane * V : col0;
  read_weights<V, L>(g.weight, a.wtype, first_col, in, 1.f, w);
  read_weights<V, L>(g.bias, a.wtype, first_col, in, 0.f, b);
  F2 part_of[V == 1 ? kPer / 2 : 1];  // V = 1: -1 for the row's elements, 0 past its end
  if constexpr (V == 1) {
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) part_of[i] = F2(in[2 * i] ? -1.f : 0.f, in[2 * i + 1] ? -1.f : 0.f);
  }
  constexpr bool kExact = exact_sums<X>(row_capacity(L) / V) || kApart<X, V, L>;
  // kExact: 1 / width in two parts, so that the mean of an exact sum is exact.  Both are positive: an infinite sum stays so.
  const float n = static_cast<float>(width), inv_n = kExact ? __frcp_rd(n) : 1.f / n;
  const float inv_n_rest = fmaxf(fmaf(inv_n, -n, 1.f) * inv_n, 0x1p-100f);
  int stage = 0;
  const int64_t r = walk.first;
  Y* y = static_cast<Y*>(g.y) + r * a.y_stride + col0 + lane * V;
  const int64_t y_step = walk.step * a.y_stride, stat_step = walk.step * a.segments;
  int64_t stat = r * a.segments + seg;
  for (int k = 0; k < walk.count; ++k, y += y_step, stat += stat_step) {
    x.reuse();
    x.copy(stage == 0 ? kStages - 1 : stage - 1, k + kStages - 1 < walk.mine, in);
    async_commit();
    async_wait<kStages - 1>();
    x.share();
    const bool valid = k < walk.mine;
    F2 f[kPer / 2];
    x.read(stage, valid, in, f);
    F2 s(0.f);
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) s = s + f[i];
    float mu;
    if constexpr (kApart<X, V, L>) {
      const float2 sum = row_sum_in_two<T>(s.lo() + s.hi(), part[0]);
      mu = fmaf(sum.x, inv_n, fmaf(sum.x, inv_n_rest, sum.y * inv_n));
    } else {
      const float sum = row_sum<L, T>(s.lo() + s.hi(), part[0]);
      mu = kExact ? fmaf(sum, inv_n, sum * inv_n_rest) : sum * inv_n;
    }
    s = F2(0.f);
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) {
      if constexpr (V == 1) {
        f[i] = fma2(part_of[i], F2(mu), f[i]);
        s = fma2(f[i], f[i], s);
      } else {
        f[i] = f[i] + F2(-mu);
        if (in[2 * i / V]) s = fma2(f[i], f[i], s);
      }
    }
    const float q = row_sum<L, T>(s.lo() + s.hi(), part[1]);
    const bool flat = !kExact && is_flat(mu, q * inv_n, kSlack);
    if (valid && !flat) {
      const float rs = __frsqrt_rn(fmaf(q, inv_n, a.eps));
#pragma unroll
      for (int i = 0; i < kPer / 2; ++i) f[i] = fma2(f[i] * F2(rs), w[i], b[i]);
      write_row<Y, V, L>(y, in, f);
      if (g.mean != nullptr && lane == 0) {
        g.mean[stat] = mu;
        g.rstd[stat] = rs;
      }
    }
    if constexpr (!kExact)
      if (L > 32 ? flat : __any_sync(kFull, flat))
        forward_flat_row<X, Y, V, L, T>(a, g, smem, part, stage, walk.first + k * walk.step, mu, flat);
    stage = stage == kStages - 1 ? 0 : stage + 1;
  }
}

// A CTA takes one segment of `tile` rows; neighbouring CTAs take neighbouring segments of the same rows, so what is
// in flight at one time is a band of whole rows.  The lanes to a row follow the segment's own width: the tables of one
// launch may be of different widths.  Without vectors one CTA less to an SM, for the registers of the row's mask and of the
// look for flat rows (67M fp32 in rows of 37: 123 us, 132 with 6).
template <typename X, typename Y, int V>
__global__ void __launch_bounds__(kGroupThreads, V == 1 ? 5 : 6)
    norm_rows_kernel(const __grid_constant__ NormArgs a, const __grid_constant__ ForwardArgs g, int64_t tile) {
  extern __shared__ __align__(16) char smem[];
  constexpr int T = kGroupThreads;
  const int seg = blockIdx.x % a.segments;
  const int64_t row0 = (blockIdx.x / a.segments) * tile, row1 = min(row0 + tile, a.rows);
  int col0, width;
  segment_span<V>(a, seg, &col0, &width);
  auto go = [&](auto lanes) {
    constexpr int L = decltype(lanes)::value;
    const RowWalk walk(row0 + threadIdx.x / L, T / L, row0, row1);
    forward_rows<X, Y, V, L, T>(a, g, seg, col0, width, walk, smem);
  };
  if (width <= row_capacity(4)) go(std::integral_constant<int, 4>());
  else if (width <= row_capacity(8)) go(std::integral_constant<int, 8>());
  else if (width <= row_capacity(16)) go(std::integral_constant<int, 16>());
  else go(std::integral_constant<int, 32>());
}

// A CTA of T threads to a row, over every slots-th row.  (Without vectors, 640 threads to an SM: 67M fp16 in rows of 1001 62 us, 66
// with 768; fp32 in rows of 3001 103, 123.)
template <typename X, typename Y, int V, int T>
__global__ void __launch_bounds__(T, T <= 256 ? (V == 1 ? 640 : 768) / T : 1)
    norm_wide_kernel(const __grid_constant__ NormArgs a, const __grid_constant__ ForwardArgs g, int64_t slots) {
  extern __shared__ __align__(16) char smem[];
  const int seg = blockIdx.x % a.segments;
  const int64_t slot = blockIdx.x / a.segments;
  int col0, width;
  segment_span<V>(a, seg, &col0, &width);
  const RowWalk walk(slot, slots, slot, a.rows);
  forward_rows<X, Y, V, T, T>(a, g, seg, col0, width, walk, smem);
}

// A flat row wider than the registers of a CTA, anew: each of three corrections leaves as small a part of the mean's rounding
// as that is of the mean.  Rare.
template <typename X, typename Y, int V>
__device__ __forceinline__ void norm_long_flat_row(const NormArgs& a, const ForwardArgs& g, int64_t r, float mu, float (&part)[2][32]) {
  int seg, col0, width;
  asm volatile("mov.u32 %0, %%ctaid.x;" : "=r"(seg));  // opaque, as in forward_flat_row
  seg %= a.segments;
  segment_span<V>(a, seg, &col0, &width);
  const float inv_n = 1.f / static_cast<float>(width);
  const X* x = static_cast<const X*>(g.x) + r * a.x_stride + col0;
  Y* y = static_cast<Y*>(g.y) + r * a.y_stride + col0;
  auto over = [&](auto&& f) {
#pragma unroll 1
    for (int c = threadIdx.x * V; c < width; c += 1024 * V) {
      Pack<X, V> v;
      v.load(x + c);
      f(c, v);
    }
  };
#pragma unroll 1
  for (int k = 0; k < 3; ++k) {
    float s = 0.f;
    over([&](int, const Pack<X, V>& v) {
#pragma unroll
      for (int i = 0; i < V; ++i) s += v.get(i) - mu;
    });
    mu += row_sum<1024, 1024>(s, part[k & 1]) * inv_n;
  }
  float q = 0.f;
  over([&](int, const Pack<X, V>& v) {
#pragma unroll
    for (int i = 0; i < V; ++i) q = fmaf(v.get(i) - mu, v.get(i) - mu, q);
  });
  const float rs = __frsqrt_rn(fmaf(row_sum<1024, 1024>(q, part[1]), inv_n, a.eps));
  over([&](int c, const Pack<X, V>& v) {
    float w[V], b[V], f[V];
    load_weights<V>(g.weight, a.wtype, col0 + c, 1.f, w);
    load_weights<V>(g.bias, a.wtype, col0 + c, 0.f, b);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = fmaf((v.get(i) - mu) * rs, w[i], b[i]);
    Pack<Y, V> o;
    o.set(f);
    o.store(y + c);
  });
  if (g.mean != nullptr && threadIdx.x == 0) {
    g.mean[r * a.segments + seg] = mu;
    g.rstd[r * a.segments + seg] = rs;
  }
}

// Rows wider than the registers of a CTA: three passes over the row, the second and third from the caches.  (Without vectors two
// CTAs to an SM: 67M fp16 in rows of 20001 142 us, 216 with one and its loads unrolled twice as far.)
template <typename X, typename Y, int V>
__global__ void __launch_bounds__(1024, V == 1 ? 2 : 1)
    norm_long_kernel(const __grid_constant__ NormArgs a, const __grid_constant__ ForwardArgs g, int64_t slots) {
  __shared__ float part[2][32];
  const int seg = blockIdx.x % a.segments;
  int col0, width;
  segment_span<V>(a, seg, &col0, &width);
  const float inv_n = 1.f / static_cast<float>(width);
  for (int64_t r = blockIdx.x / a.segments; r < a.rows; r += slots) {
    const X* x = static_cast<const X*>(g.x) + r * a.x_stride + col0;
    Y* y = static_cast<Y*>(g.y) + r * a.y_stride + col0;
    float s = 0.f;
#pragma unroll 4
    for (int c = threadIdx.x * V; c < width; c += 1024 * V) {
      Pack<X, V> v;
      v.load(x + c);
#pragma unroll
      for (int i = 0; i < V; ++i) s += v.get(i);
    }
    const float mu = row_sum<1024, 1024>(s, part[0]) * inv_n;
    s = 0.f;
#pragma unroll 4
    for (int c = threadIdx.x * V; c < width; c += 1024 * V) {
      Pack<X, V> v;
      v.load(x + c);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float d = v.get(i) - mu;
        s = fmaf(d, d, s);
      }
    }
    const float q = row_sum<1024, 1024>(s, part[1]);
    // the sum by threads of width / 1024 elements has as many more roundings
    if (is_flat(mu, q * inv_n, fmaf(static_cast<float>(width), 0x1p-33f, kSlack))) {
      norm_long_flat_row<X, Y, V>(a, g, r, mu, part);
      continue;
    }
    const float rs = __frsqrt_rn(fmaf(q, inv_n, a.eps));
    for (int c = threadIdx.x * V; c < width; c += 1024 * V) {
      Pack<X, V> v;
      v.load(x + c);
      float w[V], b[V], f[V];
      load_weights<V>(g.weight, a.wtype, col0 + c, 1.f, w);
      load_weights<V>(g.bias, a.wtype, col0 + c, 0.f, b);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = fmaf((v.get(i) - mu) * rs, w[i], b[i]);
      Pack<Y, V> o;
      o.set(f);
      o.store(y + c);
    }
    if (g.mean != nullptr && threadIdx.x == 0) {
      g.mean[r * a.segments + seg] = mu;
      g.rstd[r * a.segments + seg] = rs;
    }
  }
}

template <typename X, typename Y, int V>
tbe_status launch(const NormArgs& a, const ForwardArgs& g, const DeviceInfo& dev, cudaStream_t s) {
  if (a.width <= row_capacity(32)) {
    constexpr int T = kGroupThreads;
    constexpr int smem = kStages * stage_bytes<X, V>(T);
    // about 24 CTAs to an SM (4 waves), and no fewer rows to a CTA than one pass of its threads over the widest rows
    const int64_t want = a.rows * a.segments / (static_cast<int64_t>(dev.sms) * 24);
    int64_t tile = want < 16 ? 16 : want > 512 ? 512 : want / 16 * 16;
    while ((a.rows + tile - 1) / tile * a.segments > INT32_MAX) tile *= 2;
    const unsigned grid = static_cast<unsigned>((a.rows + tile - 1) / tile * a.segments);
    norm_rows_kernel<X, Y, V><<<grid, T, smem, s>>>(a, g, tile);
  } else {
    // 1024 threads to a row have 64 registers each: without vectors, and where flat rows are looked for, too few (67M fp32
    // in rows of 12001 175 us; by three passes 162)
    constexpr int kWidest = V == 1 && std::is_same<X, float>::value ? 512 : 1024;
    cudaError_t bad = cudaSuccess;
    auto wide = [&](auto kernel, int threads, int smem) {
      if (smem > kPlainSmem) bad = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (bad != cudaSuccess) return;
      const int per_seg = persistent_grid(kernel, threads, smem, dev, INT32_MAX) / a.segments;
      const int64_t slots = per_seg < 1 ? 1 : per_seg < a.rows ? per_seg : a.rows;
      kernel<<<static_cast<unsigned>(slots * a.segments), threads, smem, s>>>(a, g, slots);
    };
    if (a.width <= row_capacity(64)) wide(norm_wide_kernel<X, Y, V, 64>, 64, kStages * stage_bytes<X, V>(64));
    else if (a.width <= row_capacity(128)) wide(norm_wide_kernel<X, Y, V, 128>, 128, kStages * stage_bytes<X, V>(128));
    else if (a.width <= row_capacity(256)) wide(norm_wide_kernel<X, Y, V, 256>, 256, kStages * stage_bytes<X, V>(256));
    else if (a.width <= row_capacity(512)) wide(norm_wide_kernel<X, Y, V, 512>, 512, kStages * stage_bytes<X, V>(512));
    else if (kWidest == 1024 && a.width <= row_capacity(1024))
      wide(norm_wide_kernel<X, Y, V, kWidest>, kWidest, kStages * stage_bytes<X, V>(kWidest));
    else wide(norm_long_kernel<X, Y, V>, 1024, 0);
    if (bad != cudaSuccess) return cuda_status(bad);
  }
  note_launch();
  return cuda_status(cudaGetLastError());
}

}  // namespace

tbe_status launch_norm_forward(const NormArgs& a, int xtype, int ytype, int vec, const void* x, const void* weight,
                               const void* bias, void* y, float* mean, float* rstd, const DeviceInfo& dev,
                               cudaStream_t s) {
  const ForwardArgs g{x, weight, bias, y, mean, rstd};
  return with_type(xtype, [&](auto xt) {
    return with_type(ytype, [&](auto yt) {
      using X = typename decltype(xt)::type;
      using Y = typename decltype(yt)::type;
      if constexpr (sizeof(X) == 2 && sizeof(Y) == 2 && !std::is_same<X, Y>::value) {
        return TBE_ERR_UNSUPPORTED;
      } else {
        if constexpr (sizeof(X) == 2 && sizeof(Y) == 2)
          if (vec >= 8) return launch<X, Y, 8>(a, g, dev, s);
        if (vec >= 4) return launch<X, Y, 4>(a, g, dev, s);
        return launch<X, Y, 1>(a, g, dev, s);
      }
    });
  });
}

}  // namespace tbe
