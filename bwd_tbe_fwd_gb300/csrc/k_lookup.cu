// k_lookup.cu -- rows of a table by token, and the table's gradient by sorted tokens (tbe_tokens.h).
#include "cluster.cuh"
#include "lookup_plan.cuh"
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
  int groups, itype;         // groups: of V elements in a row
  float scale;
  unsigned long long* stats;
};

// A pack to memory: 32 bytes in one access (row_vector grants 8 fp32 elements only where they are aligned to that).
template <typename T, int V>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, V>& v) {
  if constexpr (Pack<T, V>::kBytes == 32) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v.w[0]), "r"(v.w[1]), "r"(v.w[2]), "r"(v.w[3]),
                 "r"(v.w[4]), "r"(v.w[5]), "r"(v.w[6]), "r"(v.w[7])
                 : "memory");
  } else {
    v.store(p);
  }
}

// x / groups, in 32 bits where that is enough (a 64-bit division takes some 40 instructions).
__device__ __forceinline__ int64_t split(int64_t x, int groups) {
  return x >> 32 == 0 ? static_cast<int64_t>(static_cast<uint32_t>(x) / static_cast<uint32_t>(groups)) : x / groups;
}

// A thread takes V elements of U tokens at a time, U rows in flight.  (131072 rows of 128 fp16 to fp32, 2 at a time: 18.4 us; 4: 20.4,
// 8: 22.6; 82 MB, at the copy rate 12.1.)
template <typename TT, typename OT, int V>
__global__ void __launch_bounds__(kFwdThreads) lookup_forward_kernel(const __grid_constant__ ForwardArgs a) {
  constexpr int U = 2;
  const int64_t total = a.tokens * a.groups, step = static_cast<int64_t>(gridDim.x) * kFwdThreads;
  unsigned bad = 0;  // counted at the end: an atomic between the loads would hold them apart
  for (int64_t x0 = static_cast<int64_t>(blockIdx.x) * kFwdThreads + threadIdx.x; x0 < total; x0 += U * step) {
    Pack<TT, V> row[U];
    int64_t tok[U], id[U];
    int col[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t x = x0 + u * step;
      tok[u] = x < total ? split(x, a.groups) : 0;
      col[u] = static_cast<int>(x - tok[u] * a.groups) * V;
      id[u] = x < total ? load_id(a.ids, a.itype, tok[u]) : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      bad += id[u] >= a.rows && col[u] == 0;
      row[u].zero();
      if (id[u] >= 0 && id[u] < a.rows) row[u].load(static_cast<const TT*>(a.table) + id[u] * a.table_stride + col[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (x0 + u * step >= total) break;
      const bool live = id[u] >= 0 && id[u] < a.rows;
      float f[V];
#pragma unroll
      for (int k = 0; k < V; ++k) f[k] = live ? row[u].get(k) * a.scale : 0.0f;
      Pack<OT, V> o;
      o.set(f);
      store_pack(static_cast<OT*>(a.out) + tok[u] * a.out_stride + col[u], o);
    }
  }
  stat_add(a.stats, TBE_STAT_UNREPAIRED, bad);
}

// Rows of 64 elements or more that allow no vector of 16 bytes: a warp to a token, so that its id is read and its row found once.  (us a
// call by the kernel above and so: 27884 rows of 1597 fp32 to bf16 134 and 28; 50000 rows of fp16 of 129 22.8 and 14.5, of 65 14.3
// and 12.7, of 33 12.6 and 12.7.)
template <typename TT, typename OT, int V>
__global__ void __launch_bounds__(kFwdThreads) lookup_rows_kernel(const __grid_constant__ ForwardArgs a) {
  constexpr int U = 4;
  const int lane = lane_id();
  unsigned bad = 0;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kFwdThreads / kWarp);
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * kFwdThreads + threadIdx.x) / kWarp; i < a.tokens; i += warps) {
    const int64_t id = load_id(a.ids, a.itype, i);
    const bool live = id >= 0 && id < a.rows;
    bad += id >= a.rows && lane == 0;
    const TT* src = static_cast<const TT*>(a.table) + (live ? id : 0) * a.table_stride;
    OT* dst = static_cast<OT*>(a.out) + i * a.out_stride;
    for (int g0 = lane; g0 < a.groups; g0 += kWarp * U) {
      Pack<TT, V> row[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        row[u].zero();
        if (live && g0 + u * kWarp < a.groups) row[u].load(src + (g0 + u * kWarp) * V);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (g0 + u * kWarp >= a.groups) break;
        float f[V];
#pragma unroll
        for (int k = 0; k < V; ++k) f[k] = live ? row[u].get(k) * a.scale : 0.0f;
        Pack<OT, V> o;
        o.set(f);
        o.store(dst + (g0 + u * kWarp) * V);
      }
    }
  }
  stat_add(a.stats, TBE_STAT_UNREPAIRED, bad);
}

// ------------------------------------------------------------------------------------------
// Backward: sort
// ------------------------------------------------------------------------------------------
struct KeyArgs {
  const void* ids;
  int64_t tokens, rows;
  int itype;
  uint32_t* keys;
  uint32_t* vals;
  uint32_t* counters;
  unsigned long long* stats;
};

// An id as a sort key; what is no row of the table sorts last.
__device__ __forceinline__ uint32_t sort_key(int64_t id, int64_t rows) {
  return id >= 0 && id < rows ? static_cast<uint32_t>(id) : static_cast<uint32_t>(rows);
}

__global__ void __launch_bounds__(256) lookup_keys_kernel(const __grid_constant__ KeyArgs a) {
  if (blockIdx.x == 0 && threadIdx.x == 0) a.counters[TBE_CNT_N] = static_cast<uint32_t>(a.tokens);
  unsigned bad = 0;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < a.tokens; i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t id = load_id(a.ids, a.itype, i);
    bad += id >= a.rows;
    a.keys[i] = sort_key(id, a.rows);
    a.vals[i] = static_cast<uint32_t>(i);
  }
  stat_add(a.stats, TBE_STAT_UNREPAIRED, bad);
}

constexpr int kClusterWarps = kClusterThreads / kWarp;

struct ClusterSortArgs {
  KeyArgs k;                 // keys, vals: the sorted ones
  int passes, bits[kMaxRadixPasses];
  // the rest of the grid sets the gradient to zero meanwhile
  void* grad;
  int64_t rows, row_bytes, pitch;   // pitch == row_bytes: one range of rows * row_bytes
  int elem;                         // bytes of an element, which grad is aligned to
};

// `bytes` zeros from p on, by `n` threads of which this is number t.
__device__ __forceinline__ void zero_range(char* p, int64_t bytes, int elem, int64_t t, int64_t n) {
  const int64_t head = min(bytes, static_cast<int64_t>(-reinterpret_cast<uintptr_t>(p) & 15));
  const int64_t body = (bytes - head) / 16, tail = bytes - head - body * 16;
  if (t < (head + tail) / elem) {  // at most 14 bytes at either end, element by element
    const int64_t at = t * elem < head ? t * elem : bytes - tail + (t * elem - head);
    if (elem == 4) *reinterpret_cast<uint32_t*>(p + at) = 0;
    else *reinterpret_cast<uint16_t*>(p + at) = 0;
  }
  uint4* v = reinterpret_cast<uint4*>(p + head);
  for (int64_t i = t; i < body; i += n) v[i] = make_uint4(0, 0, 0, 0);
}

// The same by CTAs of which this is number t of n, for a long range: bulk copies of zeros in shared memory.  (264 MB beside
// the sort: plain 16- and 32-byte stores of 1024 threads an SM take 62 us.)
constexpr int kZeroPiece = 32768;
__device__ __forceinline__ void zero_long_range(char* p, int64_t bytes, int elem, int t, int n, uint8_t* s_zero) {
  const int64_t head = min(bytes, static_cast<int64_t>(-reinterpret_cast<uintptr_t>(p) & 15));
  const int64_t body = (bytes - head) / 16 * 16, tail = bytes - head - body;
  if (t == 0) {
    zero_range(p, head, elem, threadIdx.x, blockDim.x);
    zero_range(p + head + body, tail, elem, threadIdx.x, blockDim.x);
  }
  for (int i = threadIdx.x; i < kZeroPiece / 16; i += blockDim.x) reinterpret_cast<uint4*>(s_zero)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int64_t at = static_cast<int64_t>(t) * kZeroPiece; at < body; at += static_cast<int64_t>(n) * kZeroPiece) {
    const uint32_t some = static_cast<uint32_t>(min(body - at, static_cast<int64_t>(kZeroPiece)));
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(p + head + at), "r"(smem_u32(s_zero)), "r"(some)
                 : "memory");
  }
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// The sum of v over the threads before this one; s_wsum: a word for each warp, not in use elsewhere between two barriers.
__device__ __forceinline__ uint32_t block_before(uint32_t v, uint32_t* s_wsum) {
  const int lane = lane_id(), w = threadIdx.x / kWarp;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < kWarp; o <<= 1) {
    const uint32_t y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  if (lane == kWarp - 1) s_wsum[w] = x;
  __syncthreads();
  uint32_t y = s_wsum[lane];
#pragma unroll
  for (int o = 1; o < kWarp; o <<= 1) {
    const uint32_t z = __shfl_up_sync(kFull, y, o);
    if (lane >= o) y += z;
  }
  y = __shfl_sync(kFull, y, w > 0 ? w - 1 : 0);
  return x - v + (w > 0 ? y : 0);
}

// So few tokens that a thread to each counts those that come before it.  (us a call, by digits and so: 32 tokens 10.3 and 8.7, 256 tokens
// 12.3 and 10.5, 500 tokens 12.6 and 16.6.)
constexpr int kRankTokens = 256;
__device__ __forceinline__ void rank_few(const KeyArgs& a, uint32_t* s_key) {
  const int t = threadIdx.x, n = static_cast<int>(a.tokens);
  uint32_t key = 0xffffffffu;
  if (t < kRankTokens) {
    if (t < n) {
      const int64_t id = load_id(a.ids, a.itype, t);
      key = sort_key(id, a.rows);
      stat_add(a.stats, TBE_STAT_UNREPAIRED, id >= a.rows);
    }
    s_key[t] = key;
  }
  __syncthreads();
  if (t >= n) return;
  uint32_t at = 0;
  for (int j = 0; j < n; j += 4) {
    const uint4 k = *reinterpret_cast<const uint4*>(s_key + j);
    at += (k.x < key || (k.x == key && j < t)) + (k.y < key || (k.y == key && j + 1 < t)) + (k.z < key || (k.z == key && j + 2 < t)) +
          (k.w < key || (k.w == key && j + 3 < t));
  }
  a.keys[at] = key;
  a.vals[at] = static_cast<uint32_t>(t);
}

// Stable radix sort of (id, token) by one cluster, up to 131072 of them: the items stay in its shared memory, each CTA
// holding a contiguous 1024 IPT of the current order.  A pass ranks a CTA's items by ballots and counters of its
// warps' own, joins the CTAs' digit counts through distributed shared memory, and sends each item to its place in whichever CTA
// holds it.  One launch for what takes two to four passes of three launches through memory, and the other clusters of
// the grid write the gradient's zeros at the same time.  (16384 tokens of 131072 rows: 14 us, 32768: 16; the latency of two passes
// of eight barriers each.)
template <int IPT>
__global__ void __launch_bounds__(kClusterThreads, 1) lookup_sort_kernel(const __grid_constant__ ClusterSortArgs a) {
  extern __shared__ __align__(16) uint8_t s_raw[];
  __shared__ uint32_t s_wsum[2][kClusterWarps];
  const uint32_t ctas = cluster_size(), cta = cluster_rank();
  may_follow();
  if (blockIdx.x >= ctas) {
    const int64_t n = static_cast<int64_t>(gridDim.x - ctas) * kClusterThreads;
    const int64_t t = static_cast<int64_t>(blockIdx.x - ctas) * kClusterThreads + threadIdx.x;
    char* p = static_cast<char*>(a.grad);
    if (a.pitch == a.row_bytes) {
      zero_long_range(p, a.rows * a.row_bytes, a.elem, blockIdx.x - ctas, gridDim.x - ctas, s_raw);
    } else {
      for (int64_t r = t / kWarp; r < a.rows; r += n / kWarp) zero_range(p + r * a.pitch, a.row_bytes, a.elem, t % kWarp, kWarp);
    }
    return;
  }
  if (IPT == 1 && a.k.tokens <= kRankTokens) {
    rank_few(a.k, reinterpret_cast<uint32_t*>(s_raw));
    return;
  }
  constexpr int kPer = kClusterThreads * IPT;
  uint2* s_item = reinterpret_cast<uint2*>(s_raw);
  uint2* s_turn = s_item + kPer;                                       // the CTA's items in the order of their digits
  uint32_t* s_count = reinterpret_cast<uint32_t*>(s_turn + kPer);
  uint32_t* s_base = s_count + kMaxRadix;                              // where a digit's items go, less where they lie in s_turn
  uint16_t* s_hist = reinterpret_cast<uint16_t*>(s_base + kMaxRadix);  // [warps][digits]
  const int lane = lane_id(), w = threadIdx.x / kWarp;
  const unsigned lt = lanemask_lt();
  const int64_t left = a.k.tokens - static_cast<int64_t>(cta) * kPer;
  const int here = static_cast<int>(left < 0 ? 0 : left < kPer ? left : kPer);
  uint32_t key[IPT], val[IPT], rank[IPT];
  int shift = 0;
  unsigned bad = 0;
  for (int pass = 0; pass < a.passes; ++pass) {
    const int rb = a.bits[pass], R = 1 << rb;
#pragma unroll
    for (int i = 0; i < IPT; ++i) {
      const int e = (w * IPT + i) * kWarp + lane;
      key[i] = 0, val[i] = 0;
      if (e < here) {
        if (pass == 0) {
          val[i] = cta * kPer + e;
          const int64_t id = load_id(a.k.ids, a.k.itype, val[i]);
          bad += id >= a.k.rows;
          key[i] = sort_key(id, a.k.rows);
        } else {
          const uint2 kv = s_item[e];
          key[i] = kv.x, val[i] = kv.y;
        }
      }
    }
    for (int j = threadIdx.x; j < kClusterWarps * R / 2; j += kClusterThreads) reinterpret_cast<uint32_t*>(s_hist)[j] = 0;
    __syncthreads();
    uint16_t* hist = s_hist + w * R;
#pragma unroll
    for (int i = 0; i < IPT; ++i) {
      const bool live = (w * IPT + i) * kWarp + lane < here;
      const uint32_t d = (key[i] >> shift) & (R - 1);
      unsigned peers = __ballot_sync(kFull, live);
      for (int b = 0; b < rb; ++b) {
        const unsigned set = __ballot_sync(kFull, (d >> b) & 1u);
        peers &= (d >> b) & 1u ? set : ~set;
      }
      const int leader = live ? __ffs(peers) - 1 : lane;
      uint32_t before = 0;
      if (live && lane == leader) {
        before = hist[d];
        hist[d] = static_cast<uint16_t>(before + __popc(peers));
      }
      before = __shfl_sync(kFull, before, leader);
      rank[i] = before + __popc(peers & lt);
      __syncwarp();
    }
    __syncthreads();
    const int d = threadIdx.x;
    uint32_t count = 0;
    if (d < R) {
#pragma unroll
      for (int q = 0; q < kClusterWarps; ++q) count += s_hist[q * R + d];
      s_count[d] = count;
    }
    cluster_arrive();  // the counts are there, and this CTA's items in registers
    const uint32_t local = block_before(count, s_wsum[0]);
    if (d < R) {  // where each warp's items of the digit lie in s_turn
      uint32_t at = local;
#pragma unroll
      for (int q0 = 0; q0 < kClusterWarps; q0 += 8) {
        uint32_t c[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) c[q] = s_hist[(q0 + q) * R + d];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          s_hist[(q0 + q) * R + d] = static_cast<uint16_t>(at);
          at += c[q];
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < IPT; ++i)
      if ((w * IPT + i) * kWarp + lane < here) s_turn[hist[(key[i] >> shift) & (R - 1)] + rank[i]] = make_uint2(key[i], val[i]);
    cluster_wait();
    uint32_t total = 0, earlier = 0;
    if (d < R) {
#pragma unroll 1
      for (uint32_t c0 = 0; c0 < ctas; c0 += 8) {
        uint32_t n[8];
#pragma unroll
        for (uint32_t c = 0; c < 8; ++c) {  // all of them in flight
          n[c] = 0;
          if (c0 + c < ctas)
            asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(n[c]) : "r"(cluster_address(smem_u32(s_count + d), c0 + c)) : "memory");
        }
#pragma unroll
        for (uint32_t c = 0; c < 8; ++c) {
          total += n[c];
          if (c0 + c < cta) earlier += n[c];
        }
      }
    }
    const uint32_t before = block_before(total, s_wsum[1]);
    if (d < R) s_base[d] = before + earlier - local;
    __syncthreads();
    const bool last = pass + 1 == a.passes;
#pragma unroll
    for (int i = 0; i < IPT; ++i) {  // neighbours of one digit go to neighbouring places
      const int e = i * kClusterThreads + threadIdx.x;
      if (e >= here) break;
      const uint2 kv = s_turn[e];
      const uint32_t at = s_base[(kv.x >> shift) & (R - 1)] + e;
      if (last) {
        a.k.keys[at] = kv.x;
        a.k.vals[at] = kv.y;
      } else {
        const uint32_t to = cluster_address(smem_u32(s_item + at % kPer), at / kPer);
        asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(to), "r"(kv.x), "r"(kv.y) : "memory");
      }
    }
    cluster_sync();  // the items are in place, and nobody reads this CTA's counts any more
    shift += rb;
  }
  stat_add(a.k.stats, TBE_STAT_UNREPAIRED, bad);
}

constexpr size_t cluster_sort_smem(int ipt) {
  return size_t(kClusterThreads) * ipt * 16 + 2 * kMaxRadix * 4 + size_t(kClusterWarps) * 2 * kMaxRadix;
}
static_assert(cluster_sort_smem(1) >= kZeroPiece && cluster_sort_smem(kMaxPerThread) <= 227 * 1024 - 256, "");

// ------------------------------------------------------------------------------------------
// Backward: sums
// ------------------------------------------------------------------------------------------
constexpr int kSumWarps = 8;
constexpr int kSumThreads = kSumWarps * kWarp;

struct SumArgs {
  const uint32_t* keys;      // sorted
  const uint32_t* vals;
  const void* dout;
  void* grad;
  float* partial;            // [chunks][2][dim_pad]: what a chunk has of the run before it, and of the run after it
  int64_t tokens, rows, table_stride, out_stride, dim_pad, chunks;
  int dim, slabs;
  float scale;
};

template <bool ACC, typename TT, int V>
__device__ __forceinline__ void write_row(const SumArgs& a, uint32_t key, int col, float (&f)[V], const Pack<TT, V>& old) {
  const int n = a.dim - col;
  if (n <= 0) return;
  TT* p = static_cast<TT*>(a.grad) + key * a.table_stride + col;
#pragma unroll
  for (int k = 0; k < V; ++k) f[k] *= a.scale;
  if (ACC) {
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] += old.get(k);
  }
  Pack<TT, V> g;
  g.set(f);
  store_pack(p, g);
}

// The row's elements that a sum is added to, where it is (zeros otherwise).  Rows are a multiple of V wide.
template <bool ACC, typename TT, int V>
__device__ __forceinline__ Pack<TT, V> old_row(const SumArgs& a, uint32_t key, int col, bool wanted) {
  Pack<TT, V> g;
  g.zero();
  if (ACC && wanted && col < a.dim) g.load(static_cast<const TT*>(a.grad) + key * a.table_stride + col);
  return g;
}

// A CTA adds up 32 V columns of 8 T sorted tokens, a warp T of them, 8 rows in flight.  A warp writes the runs that
// begin and end among its tokens; what it has of runs that reach over its first or last token meets in shared memory, and what
// the CTA has of runs that reach over its own is left for the join.  A run's additions keep the tokens' order, warp by
// warp and chunk by chunk.  (65536 x 1024 bf16: 31 us for 184 MB, 87% of the copy rate; 16384: 14 us.)
template <typename TT, typename OT, int V, bool ACC, int T>
__global__ void __launch_bounds__(kSumThreads) lookup_sum_kernel(const __grid_constant__ SumArgs a) {
  constexpr int U = 8;
  __shared__ float s_part[kSumWarps][2][kWarp * V];  // a warp's part of the run before it, of the run after it
  __shared__ uint32_t s_first[kSumWarps], s_last[kSumWarps];
  const int lane = lane_id(), w = threadIdx.x / kWarp;
  const int64_t chunk = blockIdx.x / a.slabs;
  const int col = (static_cast<int>(blockIdx.x - chunk * a.slabs) * kWarp + lane) * V;
  const int64_t p0 = (chunk * kSumWarps + w) * T;
  may_follow();
  wait_before();
  const int n = static_cast<int>(clamp64(a.tokens - p0, 0, T));
  const uint32_t none = static_cast<uint32_t>(a.rows);
  const uint32_t my_key = lane < n ? a.keys[p0 + lane] : none, my_val = lane < n ? a.vals[p0 + lane] : 0;
  const uint32_t before = n > 0 && p0 > 0 ? a.keys[p0 - 1] : none, after = n > 0 && p0 + n < a.tokens ? a.keys[p0 + n] : none;
  uint32_t next_key = __shfl_down_sync(kFull, my_key, 1);
  if (lane == T - 1) next_key = after;
  const unsigned ends = __ballot_sync(kFull, my_key != next_key && my_key != none);   // the tokens that end a run
  const int live = __popc(__ballot_sync(kFull, my_key != none));                      // padding sorts last
  const uint32_t first = __shfl_sync(kFull, my_key, 0), last = __shfl_sync(kFull, my_key, T - 1);
  float sum[V] = {};
  bool head = first == before && first != none;   // the current run began in an earlier warp
  const OT* dout = static_cast<const OT*>(a.dout);
  const int in_col = col < a.dim ? col : 0;
  for (int i0 = 0; i0 < live; i0 += U) {
    Pack<OT, V> d[U];
    Pack<TT, V> old[U];
    // Tokens past the live ones read the last live one's row, and columns past the row its first: no branch holds the
    // loads apart.
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = min(i0 + u, live - 1);
      d[u].load(dout + static_cast<int64_t>(__shfl_sync(kFull, my_val, i)) * a.out_stride + in_col);
      if (ACC) old[u].load(static_cast<const TT*>(a.grad) + static_cast<int64_t>(__shfl_sync(kFull, my_key, i)) * a.table_stride + in_col);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int k = 0; k < V; ++k) sum[k] += d[u].get(k);  // (past the live ones to a sum that nobody reads)
      if (!(ends >> (i0 + u) & 1)) continue;
      if (head) {
#pragma unroll
        for (int k = 0; k < V; ++k) s_part[w][0][k * kWarp + lane] = sum[k];
      } else {
        write_row<ACC, TT, V>(a, __shfl_sync(kFull, my_key, i0 + u), col, sum, old[u]);
      }
      head = false;
#pragma unroll
      for (int k = 0; k < V; ++k) sum[k] = 0.0f;
    }
  }
  const bool open = n > 0 && last != none && last == after;  // the last run goes on (a warp whose tokens run out has none)
  if (open) {
#pragma unroll
    for (int k = 0; k < V; ++k) s_part[w][head ? 0 : 1][k * kWarp + lane] = sum[k];
  }
  // s_first: the run that a warp's tokens begin with, if it began before them; s_last: the one they leave open
  if (lane == 0) {
    s_first[w] = first == before ? first : none;
    s_last[w] = open ? last : none;
  }
  __syncthreads();
  // The warp in which a run begins (or the CTA's first one, of a run that began before the CTA) adds up the parts.
  const bool begins = open && !head;
  const bool carried = w == 0 && s_first[0] != none;
  for (int turn = 0; turn < 2; ++turn) {
    if (turn == 0 ? !carried : !begins) continue;
    const uint32_t run = turn == 0 ? first : last;
    int q = w;   // the last warp whose part belongs to the run
#pragma unroll
    for (int k = 0; k < V; ++k) sum[k] = s_part[w][turn][k * kWarp + lane];
    while (s_last[q] == run && q + 1 < kSumWarps && s_first[q + 1] == run) {
      ++q;
#pragma unroll
      for (int k = 0; k < V; ++k) sum[k] += s_part[q][0][k * kWarp + lane];
    }
    const bool goes_on = s_last[q] == run;   // over the CTA's last token
    if (turn == 0 || goes_on) {
      float* p = a.partial + (chunk * 2 + turn) * a.dim_pad + col;
#pragma unroll
      for (int k = 0; k < V; ++k) p[k] = sum[k];
    } else {
      write_row<ACC, TT, V>(a, run, col, sum, old_row<ACC, TT, V>(a, run, col, true));
    }
  }
}

// The runs that reach over the end of the chunk in which they begin: a CTA to such a chunk and 32 V columns, the chunks that the
// run goes on through shared out to the warps in order.
template <typename TT, int V, bool ACC, int T>
__global__ void __launch_bounds__(kSumThreads) lookup_join_kernel(const __grid_constant__ SumArgs a) {
  __shared__ float s_sum[kSumWarps][kWarp * V];
  const int64_t chunk = blockIdx.x / a.slabs;
  const int slab = static_cast<int>(blockIdx.x - chunk * a.slabs), lane = lane_id(), w = threadIdx.x / kWarp;
  constexpr int kChunk = kSumWarps * T;
  wait_before();
  const int64_t p0 = chunk * kChunk, p1 = p0 + kChunk, p2 = p1 + kChunk;
  if (p1 >= a.tokens) return;
  const uint32_t none = static_cast<uint32_t>(a.rows);   // loaded at once, not as each is asked for
  const uint32_t run = a.keys[p1 - 1], next = a.keys[p1], before = p0 > 0 ? a.keys[p0 - 1] : none, later = p2 < a.tokens ? a.keys[p2] : none;
  if (run == none || next != run || before == run) return;
  const int col = (slab * kWarp + lane) * V;
  float begun[V];
  Pack<TT, V> old;
  if (w == 0) {
#pragma unroll
    for (int k = 0; k < V; ++k) begun[k] = a.partial[(chunk * 2 + 1) * a.dim_pad + col + k];
    old = old_row<ACC, TT, V>(a, run, col, true);
  }
  int64_t lo = chunk + 1, hi = later == run ? a.chunks : lo + 1;   // the last chunk that begins with the run, 32 places looked at at once
  while (hi - lo > 1) {
    const int64_t step = (hi - lo + kWarp - 1) / kWarp, at = lo + lane * step;
    const int hits = __popc(__ballot_sync(kFull, at < hi && a.keys[at * kChunk] == run));
    lo += (hits - 1) * step;
    hi = min(hi, lo + step);
  }
  const int64_t count = lo - chunk, end = chunk + 1 + count * (w + 1) / kSumWarps;
  float sum[V] = {};
#pragma unroll 4
  for (int64_t c = chunk + 1 + count * w / kSumWarps; c < end; ++c) {
    const float* p = a.partial + c * 2 * a.dim_pad + col;
#pragma unroll
    for (int k = 0; k < V; ++k) sum[k] += p[k];
  }
#pragma unroll
  for (int k = 0; k < V; ++k) s_sum[w][k * kWarp + lane] = sum[k];
  __syncthreads();
  if (w != 0) return;
#pragma unroll
  for (int k = 0; k < V; ++k) sum[k] = begun[k];
  for (int q = 0; q < kSumWarps; ++q)
#pragma unroll
    for (int k = 0; k < V; ++k) sum[k] += s_sum[q][k * kWarp + lane];
  write_row<ACC, TT, V>(a, run, col, sum, old);
}

// ------------------------------------------------------------------------------------------
// Host
// ------------------------------------------------------------------------------------------
// Whether every row and buffer allows accesses of vec elements.
bool whole_vectors(const LookupArgs& a, const void* table, const void* out, int vec) {
  const int tb = dtype_bytes(a.ttype), ob = dtype_bytes(a.otype);
  return a.dim % vec == 0 && a.table_stride % vec == 0 && a.out_stride % vec == 0 && is_aligned(table, vec * tb) && is_aligned(out, vec * ob);
}

// Elements to a vector access: 8, 4 or 1.
int row_vector(const LookupArgs& a, const void* table, const void* out) {
  return whole_vectors(a, table, out, 8) ? 8 : whole_vectors(a, table, out, 4) ? 4 : 1;
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
  int64_t dim_pad;
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
  l.dim_pad = round_up(a.dim, 256);
  l.counters = take(TBE_NUM_COUNTERS * 4);
  for (int k = 0; k < 2; ++k) l.keys[k] = take(a.tokens * 4), l.vals[k] = take(a.tokens * 4);
  l.counts = take((int64_t(4) << kMaxRadixBits) * l.sort.sort_grid);
  l.totals = take(int64_t(4) << kMaxRadixBits);
  // chunks of 8 warps' tokens: 8 of them to a warp for up to sms / 2 chunks of 32, 32 beyond
  const int64_t most = static_cast<int64_t>(dev.sms) * 16 * kSumWarps;
  const int64_t few = ceil_div(a.tokens < most ? a.tokens : most, 8 * kSumWarps);
  const int64_t chunks = few > ceil_div(a.tokens, 32 * kSumWarps) ? few : ceil_div(a.tokens, 32 * kSumWarps);
  l.partial = take(chunks * 2 * l.dim_pad * 4);
  l.total = at;
  return l;
}

// Sorted tokens of a warp: 32, or 8 where that leaves half of the SMs without a CTA (32 tokens of 64 columns: 9 us by 32, 5 by 8;
// 16384 of 1024: 14 us by 32, 18 by 8).
int tokens_per_warp(const LookupArgs& a, int slabs, const DeviceInfo& dev) {
  return ceil_div(a.tokens, 32 * kSumWarps) * slabs * 2 < dev.sms ? 8 : 32;
}

// How many clusters of `ctas` that sort run at once (a cluster lies within one of the GPU's processing clusters: 15 of 8 CTAs on 152
// SMs); asked once for each device, and again after a question that failed.
template <int IPT>
int clusters_at_once(int ctas, const DeviceInfo& dev) {
  static std::atomic<int> known[64][5];   // by device and the logarithm of the size: one more than the number, 0: not known
  int log = 0;
  while (1 << log < ctas) ++log;
  std::atomic<int>* slot = dev.id < 64 ? &known[dev.id][log] : nullptr;
  if (slot != nullptr && slot->load(std::memory_order_relaxed) > 0) return slot->load(std::memory_order_relaxed) - 1;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {static_cast<unsigned>(ctas), 1, 1};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kClusterThreads);
  cfg.dynamicSmemBytes = cluster_sort_smem(IPT);
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  static std::atomic<uint64_t> allowed{0};
  int n = 0;
  if (allow_smem(lookup_sort_kernel<IPT>, cluster_sort_smem(IPT), allowed, true) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, lookup_sort_kernel<IPT>, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    return 0;
  }
  if (slot != nullptr) slot->store(n + 1, std::memory_order_relaxed);
  return n;
}

// Calls f with the number of tokens to a thread.
template <typename F>
auto with_per_thread(int per_thread, F&& f) {
  if (per_thread <= 1) return f(std::integral_constant<int, 1>());
  if (per_thread <= 2) return f(std::integral_constant<int, 2>());
  if (per_thread <= 4) return f(std::integral_constant<int, 4>());
  return f(std::integral_constant<int, kMaxPerThread>());
}

// One cluster sorts; where there is a gradient to set to zero, others do that, as many as run beside it (each takes an equal share).
tbe_status launch_cluster_sort(const LookupArgs& a, const SortPlan& plan, const KeyArgs& k, void* grad, int64_t row_bytes, int64_t pitch,
                               cudaStream_t s) {
  ClusterSortArgs c{k, 0, {}, grad, a.rows, row_bytes, pitch, dtype_bytes(a.ttype)};
  int bits = 1;
  while (bits < 31 && (int64_t(1) << bits) <= a.rows) ++bits;  // keys 0 .. rows
  c.passes = (bits + kMaxRadixBits - 1) / kMaxRadixBits;
  for (int p = 0, left = bits; p < c.passes; ++p) {
    c.bits[p] = (left + c.passes - p - 1) / (c.passes - p);
    left -= c.bits[p];
  }
  int64_t others = 0;
  if (grad != nullptr) {
    others = ceil_div(ceil_div(a.rows * row_bytes, 2 * kZeroPiece), plan.ctas);
    if (others > plan.clusters - 1) others = plan.clusters - 1;
    if (others < 1) others = 1;
  }
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {static_cast<unsigned>(plan.ctas), 1, 1};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(plan.ctas * (1 + others)));
  cfg.blockDim = dim3(kClusterThreads);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return with_per_thread(plan.per_thread, [&](auto ipt) {
    constexpr int IPT = decltype(ipt)::value;
    cfg.dynamicSmemBytes = cluster_sort_smem(IPT);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, lookup_sort_kernel<IPT>, c);
    note_launch();
    return cuda_status(e);
  });
}

}  // namespace

size_t lookup_backward_bytes(const LookupArgs& a, const DeviceInfo& dev) { return backward_layout(a, dev).total; }

tbe_status launch_lookup_forward(const LookupArgs& a, const void* table, const void* ids, void* out, const DeviceInfo& dev,
                                 cudaStream_t s) {
  int vec = row_vector(a, table, out);
  const bool by_row = vec == 1 && a.dim >= 2 * kWarp;
  if (by_row && whole_vectors(a, table, out, 2)) vec = 2;
  const ForwardArgs f{table, ids, out, a.tokens, a.rows, a.table_stride, a.out_stride, a.dim / vec, a.itype, a.scale, a.stats};
  int64_t blocks = by_row ? ceil_div(a.tokens, kFwdThreads / kWarp) : ceil_div(a.tokens * f.groups, kFwdThreads);
  if (blocks > dev.sms * 16) blocks = dev.sms * 16;
  return with_types(a, by_row ? 1 : vec, [&](auto t, auto o, auto v) {
    using TT = typename decltype(t)::type;
    using OT = typename decltype(o)::type;
    auto* kernel = lookup_forward_kernel<TT, OT, decltype(v)::value>;
    if (by_row) kernel = vec == 2 ? lookup_rows_kernel<TT, OT, 2> : lookup_rows_kernel<TT, OT, 1>;
    kernel<<<static_cast<unsigned>(blocks), kFwdThreads, 0, s>>>(f);
    note_launch();
    return cuda_status(cudaGetLastError());
  });
}

tbe_status launch_lookup_backward(const LookupArgs& a, const void* dout, const void* ids, void* grad, bool accumulate, char* ws,
                                  const DeviceInfo& dev, cudaStream_t s) {
  const BackwardLayout l = backward_layout(a, dev);
  const int64_t elem = dtype_bytes(a.ttype), row = a.dim * elem, pitch = a.table_stride * elem;
  SortPlan plan{0, 0, 0};
  if (a.tokens > 0) {
    const bool long_zeros = !accumulate && zeros_are_long(a.tokens, a.rows * row);
    plan = plan_sort(a.tokens, long_zeros, [&](int ctas, int per_thread) {
      return with_per_thread(per_thread, [&](auto ipt) { return clusters_at_once<decltype(ipt)::value>(ctas, dev); });
    });
  }
  const bool in_cluster = plan.ctas > 0;
  if (!accumulate && !in_cluster) {
    const tbe_status st = cuda_status(row == pitch ? cudaMemsetAsync(grad, 0, row * a.rows, s)
                                                   : cudaMemset2DAsync(grad, pitch, 0, row, a.rows, s));
    if (st != TBE_OK) return st;
  }
  if (a.tokens == 0) return TBE_OK;
  const int final_buf = in_cluster ? 0 : l.sort.final_buf;
  uint32_t* keys[2] = {reinterpret_cast<uint32_t*>(ws + l.keys[0]), reinterpret_cast<uint32_t*>(ws + l.keys[1])};
  uint32_t* vals[2] = {reinterpret_cast<uint32_t*>(ws + l.vals[0]), reinterpret_cast<uint32_t*>(ws + l.vals[1])};
  const KeyArgs ka{ids, a.tokens, a.rows, a.itype, keys[0], vals[0], reinterpret_cast<uint32_t*>(ws + l.counters), a.stats};
  tbe_status st;
  if (in_cluster) {
    st = launch_cluster_sort(a, plan, ka, accumulate ? nullptr : grad, row, pitch, s);
  } else {
    int64_t blocks = ceil_div(a.tokens, 256);
    if (blocks > dev.sms * 8) blocks = dev.sms * 8;
    lookup_keys_kernel<<<static_cast<unsigned>(blocks), 256, 0, s>>>(ka);
    note_launch();
    st = cuda_status(cudaGetLastError());
    if (st != TBE_OK) return st;
    BwdCtx c{};
    c.counters = ka.counters;
    for (int k = 0; k < 2; ++k) c.keys[k] = keys[k], c.vals[k] = vals[k];
    c.sort_counts = reinterpret_cast<uint32_t*>(ws + l.counts);
    c.sort_totals = reinterpret_cast<uint32_t*>(ws + l.totals);
    c.stats = a.stats;
    st = cuda_status(launch_sort(Problem(), c, l.sort, s));
  }
  if (st != TBE_OK) return st;
  const int vec = row_vector(a, grad, dout);
  const int slabs = static_cast<int>(ceil_div(a.dim, vec * kWarp));
  const int per_warp = tokens_per_warp(a, slabs, dev);
  const int64_t chunks = ceil_div(a.tokens, per_warp * kSumWarps);
  const SumArgs f{keys[final_buf], vals[final_buf], dout, grad, reinterpret_cast<float*>(ws + l.partial), a.tokens, a.rows,
                  a.table_stride, a.out_stride, l.dim_pad, chunks, a.dim, slabs, a.scale};
  return with_types(a, vec, [&](auto t, auto o, auto v) {
    using TT = typename decltype(t)::type;
    using OT = typename decltype(o)::type;
    constexpr int V = decltype(v)::value;
    auto run = [&](auto acc, auto per) {
      constexpr bool ACC = decltype(acc)::value;
      constexpr int T = decltype(per)::value;
      cudaError_t e = launch_after(lookup_sum_kernel<TT, OT, V, ACC, T>, static_cast<unsigned>(chunks * slabs), kSumThreads, 0, s, f);
      if (e == cudaSuccess && chunks > 1)
        e = launch_after(lookup_join_kernel<TT, V, ACC, T>, static_cast<unsigned>((chunks - 1) * slabs), kSumThreads, 0, s, f);
      return cuda_status(e);
    };
    using Few = std::integral_constant<int, 8>;
    using Many = std::integral_constant<int, 32>;
    if (accumulate) return per_warp == 8 ? run(std::true_type(), Few()) : run(std::true_type(), Many());
    return per_warp == 8 ? run(std::false_type(), Few()) : run(std::false_type(), Many());
  });
}

}  // namespace tbe
