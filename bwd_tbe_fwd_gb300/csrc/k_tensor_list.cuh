// k_tensor_list.cuh -- how the kernels over many tensors (gradient norm, AdamW) find their work.
//
// A launch carries the descriptions of its tensors as a kernel parameter (the constant bank): no
// table to upload, none to go stale when gradients move, and a captured graph holds its own copy.  A
// tensor is cut into chunks; the first chunk of each tensor is searched for by binary search.
#pragma once

#include "dense_common.cuh"

namespace tbe {

// Two sizes of parameter block, so that a call with few tensors does not pass 30 KB.
constexpr int kSmallList = 40;

template <typename Entry, int CAP>
struct TensorList {
  int count;
  uint32_t chunk_elems;
  uint32_t first[CAP + 1];  // first chunk of each tensor; first[count] = all
  Entry e[CAP];
};

// The tensor of a chunk: the last t with first[t] <= chunk (tensors without elements have no chunk).
template <typename List>
__device__ __forceinline__ int tensor_of_chunk(const List& l, uint32_t chunk) {
  int lo = 0, hi = l.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (l.first[mid] <= chunk) lo = mid;
    else hi = mid;
  }
  return lo;
}

// True in every thread of the CTA that arrives last; resets the ticket for the next launch.  What
// thread 0 wrote before, and what any thread has read, is ordered before the last CTA's accesses.
__device__ __forceinline__ bool last_cta(uint32_t* ticket) {
  __shared__ bool last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(ticket, 1u) == gridDim.x - 1;
    if (last) *ticket = 0;
    __threadfence();
  }
  __syncthreads();
  return last;
}

}  // namespace tbe
