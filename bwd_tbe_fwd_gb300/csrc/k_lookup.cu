// k_lookup.cu -- rows of a table by token, and the table's gradient by sorted tokens (tbe_tokens.h).
#include "tokens_common.cuh"

namespace tbe {
namespace {

__device__ __forceinline__ int64_t load_id(const void* ids, int itype, int64_t i) {
  return itype == TBE_I32 ? ld_int<int32_t>(ids, i) : ld_int<int64_t>(ids, i);
}

// ------------------------------------------------------------------------------------------
// Forward
// ------------------------------------------------------------------------------------------
constexpr int kFwdThreads = 256;

struct ForwardArgs {
  const void* table;
  const void* ids;
  void* out;
  int64_t tokens, rows, table_stride, out_stride;
  int dim, groups, itype;    // groups: of V elements in a row
  float scale;
  unsigned long long* stats;
};

// A thread takes V elements of U tokens at a time, U rows in flight.
template <typename TT, typename OT, int V>
__global__ void __launch_bounds__(kFwdThreads) lookup_forward_kernel(const __grid_constant__ ForwardArgs a) {
  constexpr int U = 4;
  const int64_t total = a.tokens * a.groups, step = static_cast<int64_t>(gridDim.x) * kFwdThreads;
  for (int64_t x0 = static_cast<int64_t>(blockIdx.x) * kFwdThreads + threadIdx.x; x0 < total; x0 += U * step) {
    Pack<TT, V> row[U];
    int64_t tok[U];
    int col[U];
    bool in[U], live[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t x = x0 + u * step;
      in[u] = x < total;
      tok[u] = in[u] ? x / a.groups : 0;
      col[u] = static_cast<int>(x - tok[u] * a.groups) * V;
      const int64_t id = in[u] ? load_id(a.ids, a.itype, tok[u]) : -1;
      live[u] = id >= 0 && id < a.rows;
      if (in[u] && id >= a.rows && col[u] == 0) stat_add(a.stats, TBE_STAT_UNREPAIRED, 1);
      row[u].zero();
      if (live[u]) {
        const TT* p = static_cast<const TT*>(a.table) + id * a.table_stride + col[u];
        if (V == 1 || col[u] + V <= a.dim) row[u].load(p);
        else row[u].load_some(p, a.dim - col[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!in[u]) continue;
      float f[V];
#pragma unroll
      for (int k = 0; k < V; ++k) f[k] = live[u] ? row[u].get(k) * a.scale : 0.0f;
      Pack<OT, V> o;
      o.set(f);
      OT* p = static_cast<OT*>(a.out) + tok[u] * a.out_stride + col[u];
      if (V == 1 || col[u] + V <= a.dim) o.store(p);
      else o.store_some(p, a.dim - col[u]);
    }
  }
}

// ------------------------------------------------------------------------------------------
// Backward
// ------------------------------------------------------------------------------------------
constexpr int kChunk = 32;        // sorted tokens of a warp
constexpr int kSumThreads = 128;

struct KeyArgs {
  const void* ids;
  int64_t tokens, rows;
  int itype;
  uint32_t* keys;
  uint32_t* vals;
  uint32_t* counters;
  unsigned long long* stats;
};

__global__ void __launch_bounds__(256) lookup_keys_kernel(const __grid_constant__ KeyArgs a) {
  if (blockIdx.x == 0 && threadIdx.x == 0) a.counters[TBE_CNT_N] = static_cast<uint32_t>(a.tokens);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < a.tokens; i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t id = load_id(a.ids, a.itype, i);
    if (id >= a.rows) stat_add(a.stats, TBE_STAT_UNREPAIRED, 1);
    a.keys[i] = id >= 0 && id < a.rows ? static_cast<uint32_t>(id) : static_cast<uint32_t>(a.rows);  // padding last
    a.vals[i] = static_cast<uint32_t>(i);
  }
}

struct SumArgs {
  const uint32_t* keys;      // sorted
  const uint32_t* vals;
  const void* dout;
  void* grad;
  float* partial;            // [chunks][2][dim_pad]: what a chunk has of the run before it, and of the run after it
  int64_t tokens, rows, table_stride, out_stride, dim_pad, chunks;
  int dim, slabs;
  float scale;
  int accumulate;
};

template <typename TT, int V>
__device__ __forceinline__ void write_row(const SumArgs& a, uint32_t key, int col, float (&f)[V]) {
  TT* p = static_cast<TT*>(a.grad) + key * a.table_stride + col;
  const int n = a.dim - col;
  if (n <= 0) return;
#pragma unroll
  for (int k = 0; k < V; ++k) f[k] *= a.scale;
  Pack<TT, V> g;
  if (a.accumulate) {
    if (n >= V) g.load(p);
    else g.load_some(p, n);
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] += g.get(k);
  }
  g.set(f);
  if (n >= V) g.store(p);
  else g.store_some(p, n);
}

// A warp adds up 32 V columns of a chunk of sorted tokens.  Runs that begin and end in the chunk are written, what
// belongs to runs that reach over its ends is left for the join.
template <typename TT, typename OT, int V>
__global__ void __launch_bounds__(kSumThreads) lookup_sum_kernel(const __grid_constant__ SumArgs a) {
  constexpr int U = 8;
  const int lane = lane_id();
  const int64_t item = (static_cast<int64_t>(blockIdx.x) * kSumThreads + threadIdx.x) / kWarp;
  const int64_t chunk = item / a.slabs;
  if (chunk >= a.chunks) return;
  const int col = (static_cast<int>(item - chunk * a.slabs) * kWarp + lane) * V;
  const int64_t p0 = chunk * kChunk;
  const int n = static_cast<int>(a.tokens - p0 < kChunk ? a.tokens - p0 : kChunk);
  const uint32_t none = static_cast<uint32_t>(a.rows);
  const uint32_t my_key = lane < n ? a.keys[p0 + lane] : none, my_val = lane < n ? a.vals[p0 + lane] : 0;
  const uint32_t before = p0 > 0 ? a.keys[p0 - 1] : none, after = p0 + n < a.tokens ? a.keys[p0 + n] : none;
  const uint32_t first = __shfl_sync(kFull, my_key, 0);
  float sum[V] = {};
  uint32_t run = first;
  bool head = first == before;   // the run began in an earlier chunk
  const OT* dout = static_cast<const OT*>(a.dout);
  float* partial = a.partial + chunk * 2 * a.dim_pad + col;
  for (int i0 = 0; i0 < n && run != none; i0 += U) {
    Pack<OT, V> d[U];
    uint32_t key[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      key[u] = __shfl_sync(kFull, my_key, i0 + u);
      const uint32_t val = __shfl_sync(kFull, my_val, i0 + u);
      d[u].zero();
      if (key[u] != none && col < a.dim) {
        const OT* p = dout + val * a.out_stride + col;
        if (V == 1 || col + V <= a.dim) d[u].load(p);
        else d[u].load_some(p, a.dim - col);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (key[u] != run) {
        if (head) {
#pragma unroll
          for (int k = 0; k < V; ++k) partial[k] = sum[k];
        } else if (run != none) {
          write_row<TT, V>(a, run, col, sum);
        }
#pragma unroll
        for (int k = 0; k < V; ++k) sum[k] = 0.0f;
        run = key[u];
        head = false;
      }
#pragma unroll
      for (int k = 0; k < V; ++k) sum[k] += d[u].get(k);
    }
  }
  if (run == none) return;
  if (head) {
#pragma unroll
    for (int k = 0; k < V; ++k) partial[k] = sum[k];
  } else if (run == after) {
#pragma unroll
    for (int k = 0; k < V; ++k) partial[a.dim_pad + k] = sum[k];
  } else {
    write_row<TT, V>(a, run, col, sum);
  }
}

// The runs that reach over the end of the chunk in which they begin: a block to such a chunk and 32 V columns, the chunks that the
// run goes on through shared out to the warps in order.
template <typename TT, int V>
__global__ void __launch_bounds__(256) lookup_join_kernel(const __grid_constant__ SumArgs a) {
  constexpr int kWarps = 8;
  __shared__ float s_sum[kWarps][kWarp * V];
  const int64_t chunk = blockIdx.x / a.slabs;
  const int slab = static_cast<int>(blockIdx.x - chunk * a.slabs), lane = lane_id(), w = threadIdx.x / kWarp;
  const int64_t p0 = chunk * kChunk, p1 = p0 + kChunk;
  if (p1 >= a.tokens) return;
  const uint32_t run = a.keys[p1 - 1];
  if (run >= a.rows || a.keys[p1] != run || (p0 > 0 && a.keys[p0 - 1] == run)) return;
  int64_t lo = chunk + 1, hi = a.chunks;   // the last chunk that begins with the run
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) / 2;
    if (a.keys[mid * kChunk] == run) lo = mid;
    else hi = mid;
  }
  const int64_t count = lo - chunk;
  const int col = (slab * kWarp + lane) * V;
  float sum[V] = {};
  for (int64_t c = chunk + 1 + count * w / kWarps; c < chunk + 1 + count * (w + 1) / kWarps; ++c) {
    const float* p = a.partial + c * 2 * a.dim_pad + col;
#pragma unroll
    for (int k = 0; k < V; ++k) sum[k] += p[k];
  }
#pragma unroll
  for (int k = 0; k < V; ++k) s_sum[w][lane * V + k] = sum[k];
  __syncthreads();
  if (w != 0) return;
#pragma unroll
  for (int k = 0; k < V; ++k) sum[k] = a.partial[(chunk * 2 + 1) * a.dim_pad + col + k];
  for (int q = 0; q < kWarps; ++q)
#pragma unroll
    for (int k = 0; k < V; ++k) sum[k] += s_sum[q][lane * V + k];
  write_row<TT, V>(a, run, col, sum);
}

// ------------------------------------------------------------------------------------------
// Host
// ------------------------------------------------------------------------------------------
// Elements to a vector access that every row and buffer allows: 8, 4 or 1.
int row_vector(const LookupArgs& a, const void* table, const void* out) {
  const int tb = dtype_bytes(a.ttype), ob = dtype_bytes(a.otype);
  for (int vec : {8, 4}) {
    const int ta = vec * tb < 16 ? vec * tb : 16, oa = vec * ob < 16 ? vec * ob : 16;
    if (a.dim % vec == 0 && a.table_stride * tb % ta == 0 && a.out_stride * ob % oa == 0 && is_aligned(table, ta) && is_aligned(out, oa))
      return vec;
  }
  return 1;
}

// Calls f with the types of table and out (equal, or one of them fp32) and the vector width.
template <typename F>
tbe_status with_types(const LookupArgs& a, int vec, F&& f) {
  return with_type(a.ttype, [&](auto t) {
    using TT = typename decltype(t)::type;
    auto widths = [&](auto o) {
      if (vec == 8) return f(t, o, std::integral_constant<int, 8>());
      if (vec == 4) return f(t, o, std::integral_constant<int, 4>());
      return f(t, o, std::integral_constant<int, 1>());
    };
    if (a.otype == a.ttype) return widths(t);
    if constexpr (std::is_same<TT, float>::value) {
      if (a.otype == TBE_F16) return widths(TypeTag<__half>());
      return widths(TypeTag<__nv_bfloat16>());
    } else {
      return widths(TypeTag<float>());
    }
  });
}

struct BackwardLayout {
  BwdLayout sort;
  int64_t chunks, dim_pad;
  size_t counters, keys[2], vals[2], counts, totals, partial, total;
};

BackwardLayout backward_layout(const LookupArgs& a, const DeviceInfo& dev) {
  BackwardLayout l{};
  size_t at = 0;
  auto take = [&](int64_t bytes) {
    const size_t here = at;
    at += static_cast<size_t>(round_up(bytes, 256));
    return here;
  };
  int bits = 1;
  while (bits < 31 && (int64_t(1) << bits) <= a.rows) ++bits;  // keys 0 .. rows
  l.sort.passes = (bits + kMaxRadixBits - 1) / kMaxRadixBits;
  for (int p = 0, left = bits; p < l.sort.passes; ++p) {
    const int b = (left + l.sort.passes - p - 1) / (l.sort.passes - p);
    l.sort.pass_bits[p] = b < 8 ? 8 : b;
    left -= b;
  }
  int64_t grid = dev.sms * 2;
  if (grid > ceil_div(a.tokens, kSortTile)) grid = ceil_div(a.tokens, kSortTile);
  l.sort.sort_grid = grid < 1 ? 1 : static_cast<int>(grid);
  l.sort.final_buf = l.sort.passes & 1;
  l.chunks = ceil_div(a.tokens, kChunk);
  l.dim_pad = round_up(a.dim, 256);
  l.counters = take(TBE_NUM_COUNTERS * 4);
  for (int k = 0; k < 2; ++k) l.keys[k] = take(a.tokens * 4), l.vals[k] = take(a.tokens * 4);
  l.counts = take((int64_t(4) << kMaxRadixBits) * l.sort.sort_grid);
  l.totals = take(int64_t(4) << kMaxRadixBits);
  l.partial = take(l.chunks > 1 ? l.chunks * 2 * l.dim_pad * 4 : 0);
  l.total = at;
  return l;
}

}  // namespace

size_t lookup_backward_bytes(const LookupArgs& a, const DeviceInfo& dev) { return backward_layout(a, dev).total; }

tbe_status launch_lookup_forward(const LookupArgs& a, const void* table, const void* ids, void* out, const DeviceInfo& dev,
                                 cudaStream_t s) {
  const int vec = row_vector(a, table, out);
  ForwardArgs f{table, ids, out, a.tokens, a.rows, a.table_stride, a.out_stride, a.dim, static_cast<int>(ceil_div(a.dim, vec)), a.itype,
                a.scale, a.stats};
  int64_t blocks = ceil_div(a.tokens * f.groups, kFwdThreads);
  if (blocks > dev.sms * 16) blocks = dev.sms * 16;
  return with_types(a, vec, [&](auto t, auto o, auto v) {
    lookup_forward_kernel<typename decltype(t)::type, typename decltype(o)::type, decltype(v)::value>
        <<<static_cast<unsigned>(blocks), kFwdThreads, 0, s>>>(f);
    note_launch();
    return cuda_status(cudaGetLastError());
  });
}

tbe_status launch_lookup_backward(const LookupArgs& a, const void* dout, const void* ids, void* grad, bool accumulate, char* ws,
                                  const DeviceInfo& dev, cudaStream_t s) {
  const BackwardLayout l = backward_layout(a, dev);
  if (!accumulate) {
    const size_t row = static_cast<size_t>(a.dim) * dtype_bytes(a.ttype), pitch = static_cast<size_t>(a.table_stride) * dtype_bytes(a.ttype);
    const tbe_status st = cuda_status(row == pitch ? cudaMemsetAsync(grad, 0, row * a.rows, s)
                                                   : cudaMemset2DAsync(grad, pitch, 0, row, a.rows, s));
    if (st != TBE_OK) return st;
  }
  if (a.tokens == 0) return TBE_OK;
  BwdCtx c{};
  c.counters = reinterpret_cast<uint32_t*>(ws + l.counters);
  for (int k = 0; k < 2; ++k) {
    c.keys[k] = reinterpret_cast<uint32_t*>(ws + l.keys[k]);
    c.vals[k] = reinterpret_cast<uint32_t*>(ws + l.vals[k]);
  }
  c.sort_counts = reinterpret_cast<uint32_t*>(ws + l.counts);
  c.sort_totals = reinterpret_cast<uint32_t*>(ws + l.totals);
  c.stats = a.stats;
  const KeyArgs ka{ids, a.tokens, a.rows, a.itype, c.keys[0], c.vals[0], c.counters, a.stats};
  int64_t blocks = ceil_div(a.tokens, 256);
  if (blocks > dev.sms * 8) blocks = dev.sms * 8;
  lookup_keys_kernel<<<static_cast<unsigned>(blocks), 256, 0, s>>>(ka);
  note_launch();
  tbe_status st = cuda_status(cudaGetLastError());
  if (st == TBE_OK) st = cuda_status(launch_sort(Problem(), c, l.sort, s));
  if (st != TBE_OK) return st;
  const int vec = row_vector(a, grad, dout);
  SumArgs f{c.keys[l.sort.final_buf], c.vals[l.sort.final_buf], dout, grad, reinterpret_cast<float*>(ws + l.partial), a.tokens, a.rows,
            a.table_stride, a.out_stride, l.dim_pad, l.chunks, a.dim, static_cast<int>(ceil_div(a.dim, vec * kWarp)), a.scale, accumulate};
  return with_types(a, vec, [&](auto t, auto o, auto v) {
    using TT = typename decltype(t)::type;
    using OT = typename decltype(o)::type;
    constexpr int V = decltype(v)::value;
    lookup_sum_kernel<TT, OT, V><<<static_cast<unsigned>(ceil_div(l.chunks * f.slabs, kSumThreads / kWarp)), kSumThreads, 0, s>>>(f);
    note_launch();
    if (l.chunks > 1) {
      lookup_join_kernel<TT, V><<<static_cast<unsigned>((l.chunks - 1) * f.slabs), 256, 0, s>>>(f);
      note_launch();
    }
    return cuda_status(cudaGetLastError());
  });
}

}  // namespace tbe
