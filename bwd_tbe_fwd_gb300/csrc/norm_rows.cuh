// norm_rows.cuh -- how the layer norm's kernels walk over rows.
//
// L threads share a row (a segment of one), 16 elements to a thread: 4 to 32 lanes of a warp, or a whole
// CTA.  16 elements keep a row, its weights and the backward's two sums in registers, and leave few
// shuffles to an element (with 4 elements to a thread, half of the instructions were shuffles and
// addresses: 27 an element forward, 39 backward, against 10 and 16 now; 8192 x 26 x 128 backward took 67 us instead
// of 47).  Rows to come are copied into shared memory asynchronously, kStages - 1 ahead, each thread's elements to
// its own place: loads stay in flight over the reductions without registers to hold them.
#pragma once

#include "dense_common.cuh"

namespace tbe {

constexpr int kPer = 16;    // elements of a row to a thread
constexpr int kStages = 3;
constexpr int kGroupThreads = 128;  // threads of a CTA whose rows belong to parts of warps

// Dynamic shared memory that a launch may take without asking: 48 KB, less what the kernels declare.
constexpr int kPlainSmem = 47 * 1024;

// Widest row that L threads share.
constexpr int row_capacity(int L) { return kPer * L; }

// Bytes of one stage of type E for T threads; of rows without vectors (V = 1), 32 more for each row.
template <typename E, int V>
constexpr int stage_bytes(int T) {
  return T * kPer * static_cast<int>(sizeof(E)) + (V > 1 ? 0 : 32 * (T <= kGroupThreads ? T / 4 : 1));
}

// One matrix's rows as a thread sees them: V > 1, each thread copies its own elements.
template <typename E, int V, int L, int T>
struct RowReader {
  static constexpr int J = kPer / V;
  static constexpr int kChunk = V * static_cast<int>(sizeof(E)) >= 16 ? 16 : V * static_cast<int>(sizeof(E));
  static constexpr int kChunks = V * static_cast<int>(sizeof(E)) / kChunk;
  const E* next;       // the thread's first element in the next row to copy
  int64_t step;        // from one of the thread's rows to the next
  uint32_t place;      // shared memory: the thread's first chunk of stage 0

  __device__ __forceinline__ RowReader(const void* p, int64_t stride, int col, int, int64_t first_row, int64_t row_step, char* smem)
      : next(static_cast<const E*>(p) + first_row * stride + col + threadIdx.x % L * V), step(row_step * stride),
        place(smem_u32(smem) + threadIdx.x * kChunk) {}

  // Begins the copy of the next row into a stage; `valid`: the row exists.
  __device__ __forceinline__ void copy(int stage, bool valid, const bool (&in)[J]) {
    if (valid) {
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (in[j]) {
#pragma unroll
          for (int k = 0; k < kChunks; ++k)
            async_copy<kChunk>(place + stage * stage_bytes<E, V>(T) + (j * kChunks + k) * T * kChunk,
                               reinterpret_cast<const char*>(next + j * L * V) + k * kChunk);
        }
    }
    next += step;
  }

  // The thread's elements of the row in a stage (zero outside it), in pairs: those of vector 0, of vector 1, ...
  __device__ __forceinline__ void read(int stage, bool valid, const bool (&in)[J], F2 (&f)[kPer / 2]) const {
    Pack<E, V> v[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      v[j].zero();
      if (valid && in[j]) {
#pragma unroll
        for (int k = 0; k < kChunks; ++k)
          shared_words<kChunk>(place + stage * stage_bytes<E, V>(T) + (j * kChunks + k) * T * kChunk, &v[j].w[(kChunk / 4) * k]);
      }
    }
#pragma unroll
    for (int k = 0; k < kPer / 2; ++k)
      f[k] = F2(v[2 * k / V].get(2 * k % V), v[(2 * k + 1) / V].get((2 * k + 1) % V));
  }

  // Vector j of a row in a stage, which starts at `row` in memory; the vector lies in the row.
  static __device__ __forceinline__ void read_one(char* smem, int stage, const E*, int j, int, Pack<E, V>& v) {
#pragma unroll
    for (int k = 0; k < kChunks; ++k)
      shared_words<kChunk>(smem_u32(smem) + threadIdx.x * kChunk + stage * stage_bytes<E, V>(T) + (j * kChunks + k) * T * kChunk,
                           &v.w[(kChunk / 4) * k]);
  }

  static __device__ __forceinline__ void share() {}
  static __device__ __forceinline__ void reuse() {}
};

// V = 1: rows that start anywhere.  The 16-byte pieces that a row lies in are copied by the threads that share
// it, whichever element they hold; a piece's bytes past the row's end are not read but filled with zeros, and so is the
// rest of the row's region, so that every thread reads 16 elements without asking which of them exist (the
// questions were a third of the instructions).  Bytes before a row's start belong to rows before it (or to the gap between
// them); a piece that begins before the matrix is loaded element by element.
template <typename E, int L, int T>
struct RowReader<E, 1, L, T> {
  static constexpr int J = kPer;
  static constexpr int kRegion = kPer * L * static_cast<int>(sizeof(E)) + 32;  // of a row in a stage
  const char* base;    // the segment's first byte in row 0
  const char* start;   // ... in the next row to copy
  int64_t step;        // bytes from one of the thread's rows to the next
  int bytes;           // of the segment
  uint32_t place;      // shared memory: the row's region of stage 0

  __device__ __forceinline__ RowReader(const void* p, int64_t stride, int col, int width, int64_t first_row, int64_t row_step,
                                       char* smem)
      : base(reinterpret_cast<const char*>(static_cast<const E*>(p) + col)),
        start(base + first_row * stride * static_cast<int64_t>(sizeof(E))), step(row_step * stride * static_cast<int64_t>(sizeof(E))),
        bytes(width * static_cast<int>(sizeof(E))), place(smem_u32(smem) + threadIdx.x / L * kRegion) {
    for (int s = 0; s < kStages; ++s)
      for (int at = threadIdx.x % L * 16; at < kRegion; at += L * 16)
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(place + s * stage_bytes<E, 1>(T) + at), "r"(0) : "memory");
    share();
  }

  static __device__ __forceinline__ void put(uint32_t at, const char* from, bool have) {
    if constexpr (sizeof(E) == 2) {
      const uint16_t v = have ? *reinterpret_cast<const uint16_t*>(from) : 0;
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"(v) : "memory");
    } else {
      const uint32_t v = have ? *reinterpret_cast<const uint32_t*>(from) : 0;
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
    }
  }

  __device__ __forceinline__ void copy(int stage, bool valid, const bool (&)[J]) {
    if (valid) {
      const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(start) % 16);
      const uint32_t dst = place + stage * stage_bytes<E, 1>(T);
      // as many pieces as any start may need: those that this one does not are zeros
      for (int at = threadIdx.x % L * 16; at < bytes + 15; at += L * 16) {
        if (at == 0 && start - skew < base) {
          for (int k = 0; k < 16 - skew; k += static_cast<int>(sizeof(E))) put(dst + skew + k, start + k, k < bytes);
        } else {
          const int n = max(min(16, skew + bytes - at), 0);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + at), "l"(n > 0 ? start - skew + at : start - skew),
                       "r"(n) : "memory");
        }
      }
    }
    start += step;
  }

  __device__ __forceinline__ void read(int stage, bool valid, const bool (&)[J], F2 (&f)[kPer / 2]) const {
    // the row in the stage is kStages rows behind the next one to copy
    const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(start - kStages * step) % 16);
    const uint32_t src = place + stage * stage_bytes<E, 1>(T) + skew + threadIdx.x % L * static_cast<int>(sizeof(E));
    Pack<E, 1> v[J];
    if (valid) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if constexpr (sizeof(E) == 2) {
          uint16_t h;
          asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(src + j * L * 2) : "memory");
          v[j].w[0] = h;
        } else {
          shared_words<4>(src + j * L * 4, v[j].w);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < J; ++j) v[j].zero();
    }
#pragma unroll
    for (int k = 0; k < kPer / 2; ++k) f[k] = F2(v[2 * k].get(0), v[2 * k + 1].get(0));
  }

  static __device__ __forceinline__ void read_one(char* smem, int stage, const E* row, int j, int lane, Pack<E, 1>& v) {
    const uint32_t src = smem_u32(smem) + threadIdx.x / L * kRegion + stage * stage_bytes<E, 1>(T) +
                         static_cast<int>(reinterpret_cast<uintptr_t>(row) % 16) + (j * L + lane) * static_cast<int>(sizeof(E));
    if constexpr (sizeof(E) == 2) {
      uint16_t h;
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(src) : "memory");
      v.w[0] = h;
    } else {
      shared_words<4>(src, v.w);
    }
  }

  // Before other threads' copies are read.
  static __device__ __forceinline__ void share() {
    if constexpr (L <= 32) __syncwarp();
    else __syncthreads();
  }
  // Before a stage that other threads have read is filled again (a CTA's row sum has a barrier since).
  static __device__ __forceinline__ void reuse() {
    if constexpr (L <= 32) __syncwarp();
  }
};

// The weights of a thread's elements, in pairs as RowReader::read's.
template <int V, int L>
__device__ __forceinline__ void read_weights(const void* p, int type, int col, const bool (&in)[kPer / V], float none,
                                             F2 (&f)[kPer / 2]) {
  float w[kPer / V][V];
#pragma unroll
  for (int j = 0; j < kPer / V; ++j) load_weights<V>(p, type, in[j] ? col + j * L * V : col, none, w[j]);
#pragma unroll
  for (int k = 0; k < kPer / 2; ++k) f[k] = F2(w[2 * k / V][2 * k % V], w[(2 * k + 1) / V][(2 * k + 1) % V]);
}

// Stores a thread's elements, rounded.
template <typename E, int V, int L>
__device__ __forceinline__ void write_row(E* p, const bool (&in)[kPer / V], const F2 (&f)[kPer / 2]) {
  float s[kPer];
#pragma unroll
  for (int k = 0; k < kPer / 2; ++k) f[k].get(s[2 * k], s[2 * k + 1]);
#pragma unroll
  for (int j = 0; j < kPer / V; ++j)
    if (in[j]) {
      float part[V];
#pragma unroll
      for (int i = 0; i < V; ++i) part[i] = s[j * V + i];
      Pack<E, V> o;
      o.set(part);
      o.store(p + j * L * V);
    }
}

// The rows of a thread: `first`, then every `step`th, `mine` of them; the CTA's threads all go round `count` times.  (A
// matrix of fewer than 2^39 elements has no more rows to a thread than 31 bits count.)
struct RowWalk {
  int64_t first, step;
  int count, mine;
  __device__ __forceinline__ RowWalk(int64_t first_, int64_t step_, int64_t begin, int64_t end)
      : first(first_), step(step_), count(static_cast<int>((end - begin + step_ - 1) / step_)),
        mine(first_ < end ? static_cast<int>((end - first_ + step_ - 1) / step_) : 0) {}
};

// Sum over the L threads that share a row.  `part`: shared memory of T / 32 floats that no other sum uses until
// all threads have passed another barrier.
template <int L, int T>
__device__ __forceinline__ float row_sum(float v, float* part) {
  if constexpr (L <= 32) {
    return lanes_sum<L>(v);
  } else {
    v = lanes_sum<32>(v);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    return lanes_sum<T / 32>(part[threadIdx.x % (T / 32)]);
  }
}

// Two sums at once, x by one half of the lanes and y by the other: half the shuffles.  `part`: T / 32 pairs.
template <int L>
__device__ __forceinline__ float lanes_sum_halves(float x, float y) {
  const bool upper = threadIdx.x % L >= L / 2;
  const float mine = upper ? y : x, other = upper ? x : y;
  return lanes_sum<L / 2>(mine + __shfl_xor_sync(kFull, other, L / 2));
}
template <int L, int T>
__device__ __forceinline__ float2 row_sum2(float2 v, float2* part) {
  constexpr int N = L <= 32 ? L : 32;
  float s = lanes_sum_halves<N>(v.x, v.y);
  if constexpr (L > 32) {
    constexpr int W = T / 32;
    const int lane = threadIdx.x % 32;
    if (lane % 16 == 0) reinterpret_cast<float*>(part)[threadIdx.x / 32 * 2 + lane / 16] = s;
    __syncthreads();
    static_assert(W <= 16, "a part of each sum to half a warp's lanes");
    s = lanes_sum<W>(reinterpret_cast<const float*>(part)[lane % W * 2 + lane / 16]);
  }
  const float t = __shfl_xor_sync(kFull, s, N / 2);
  const bool upper = threadIdx.x % N >= N / 2;
  return upper ? make_float2(t, s) : make_float2(s, t);
}

}  // namespace tbe
