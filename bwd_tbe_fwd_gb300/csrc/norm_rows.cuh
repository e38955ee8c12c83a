// norm_rows.cuh -- how the layer norm's kernels walk over rows.
//
// L threads share a row (a segment of one), 16 elements to a thread: 4 to 32 lanes of a warp, or a whole
// CTA.  16 elements keep a row, its weights and the backward's two sums in registers, and leave few
// shuffles to an element (with 4 elements to a thread, half of the instructions were shuffles and
// addresses, and the kernels were bound by issue).  Rows to come are copied into shared memory
// asynchronously, kStages - 1 ahead, each thread's elements to its own place: loads stay in flight over the
// reductions without registers to hold them.  Elements that allow no vector (V = 1) are loaded directly.
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

// Bytes of one stage of type E for T threads.
template <typename E, int V>
constexpr int stage_bytes(int T) { return V == 1 ? 0 : T * kPer * static_cast<int>(sizeof(E)); }

// One matrix's rows as a thread sees them.
template <typename E, int V, int L, int T>
struct RowReader {
  static constexpr int J = kPer / V;
  static constexpr int kChunk = V * static_cast<int>(sizeof(E)) >= 16 ? 16 : V * static_cast<int>(sizeof(E));
  static constexpr int kChunks = V == 1 ? 1 : V * static_cast<int>(sizeof(E)) / kChunk;
  const E* next;       // the thread's first element in the next row to copy (V = 1: to read)
  int64_t step;        // from one of the thread's rows to the next
  uint32_t place;      // shared memory: the thread's first chunk of stage 0

  __device__ __forceinline__ RowReader(const void* p, int64_t stride, int col, int64_t first_row, int64_t row_step, char* smem)
      : next(static_cast<const E*>(p) + first_row * stride + col), step(row_step * stride),
        place(smem_u32(smem) + threadIdx.x * kChunk) {}

  // Begins the copy of the next row into a stage; `valid`: the row exists.
  __device__ __forceinline__ void copy(int stage, bool valid, const bool (&in)[J]) {
    if constexpr (V > 1) {
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
  }

  // The thread's elements of the row in a stage (zero outside it), in pairs: those of vector 0, of vector 1, ...
  __device__ __forceinline__ void read(int stage, bool valid, const bool (&in)[J], F2 (&f)[kPer / 2]) {
    Pack<E, V> v[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      v[j].zero();
      if (valid && in[j]) {
        if constexpr (V == 1) {
          v[j].load(next + j * L);
        } else {
#pragma unroll
          for (int k = 0; k < kChunks; ++k) {
            const uint32_t at = place + stage * stage_bytes<E, V>(T) + (j * kChunks + k) * T * kChunk;
            shared_words<kChunk>(at, &v[j].w[(kChunk / 4) * k]);
          }
        }
      }
    }
    if constexpr (V == 1) next += step;
#pragma unroll
    for (int k = 0; k < kPer / 2; ++k)
      f[k] = F2(v[2 * k / V].get(2 * k % V), v[(2 * k + 1) / V].get((2 * k + 1) % V));
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

// The rows of a thread: `first`, then every `step`th below `end`, `count` of them for every thread of the CTA.
struct RowWalk {
  int64_t first, step, end;
  int64_t count;
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
    return lanes_sum<32>(threadIdx.x % 32 < T / 32 ? part[threadIdx.x % 32] : 0.f);
  }
}

}  // namespace tbe
