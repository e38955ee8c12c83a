// dense_common.cuh -- what the kernels of the dense side (tbe_dense.h) share: vectors of V elements
// of a storage type, type dispatch on the host, and small reductions.
#pragma once

#include "tbe_dense.h"
#include "tbe_internal.cuh"

namespace tbe {

constexpr unsigned kFull = 0xffffffffu;

// V consecutive elements of storage type T as they lie in memory (a multiple of 4 bytes, or one
// element), so that a row waiting in registers takes no more of them than its bytes.
template <typename T, int V>
struct Pack {
  static constexpr int kBytes = V * static_cast<int>(sizeof(T));
  static constexpr int kWords = kBytes < 4 ? 1 : kBytes / 4;
  uint32_t w[kWords];

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }

  // p is aligned to kBytes, or to 16 where that is less
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kBytes == 2) {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    } else if constexpr (kBytes == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (kBytes == 8) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    } else {
      static_assert(kBytes % 16 == 0, "");
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
    }
  }

  // The first n elements one by one, zeros after them.
  __device__ __forceinline__ void load_some(const T* p, int n) {
    zero();
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) {
        if constexpr (sizeof(T) == 4) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
        else w[i / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[i]) << (16 * (i % 2));
      }
  }
  __device__ __forceinline__ void store_some(T* p, int n) const {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) {
        if constexpr (sizeof(T) == 4) reinterpret_cast<uint32_t*>(p)[i] = w[i];
        else reinterpret_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i % 2)));
      }
  }

  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kBytes == 2) {
      *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w[0]);
    } else if constexpr (kBytes == 4) {
      *reinterpret_cast<uint32_t*>(p) = w[0];
    } else if constexpr (kBytes == 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i)
        reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
  }

  __device__ __forceinline__ float get(int i) const {
    if constexpr (std::is_same<T, float>::value) {
      return __uint_as_float(w[i]);
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
      return __uint_as_float((i & 1) ? (w[i >> 1] & 0xffff0000u) : (w[i >> 1] << 16));
    } else {
      return __half2float(__ushort_as_half(static_cast<unsigned short>((i & 1) ? w[i >> 1] >> 16 : w[i >> 1])));
    }
  }

  // Round to nearest even.
  __device__ __forceinline__ void set(const float (&f)[V]) {
    if constexpr (std::is_same<T, float>::value) {
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] = __float_as_uint(f[i]);
    } else if constexpr (V == 1) {
      if constexpr (std::is_same<T, __nv_bfloat16>::value) w[0] = __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
      else w[0] = __half_as_ushort(__float2half_rn(f[0]));
    } else {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
          __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
          w[i] = *reinterpret_cast<uint32_t*>(&h);
        } else {
          __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
          w[i] = *reinterpret_cast<uint32_t*>(&h);
        }
      }
    }
  }
};

// Two fp32 values in a register pair: one instruction for both.
struct F2 {
  uint64_t b;
  __device__ __forceinline__ F2() {}
  __device__ __forceinline__ F2(float lo, float hi) { asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(lo), "f"(hi)); }
  __device__ __forceinline__ explicit F2(float both) : F2(both, both) {}
  __device__ __forceinline__ void get(float& lo, float& hi) const {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(b));
  }
  __device__ __forceinline__ float lo() const { float x, y; get(x, y); return x; }
  __device__ __forceinline__ float hi() const { float x, y; get(x, y); return y; }
};
__device__ __forceinline__ F2 operator*(F2 x, F2 y) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.b) : "l"(x.b), "l"(y.b));
  return r;
}
__device__ __forceinline__ F2 operator+(F2 x, F2 y) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.b) : "l"(x.b), "l"(y.b));
  return r;
}
// x y + z, rounded once.  A product that has to be rounded before it is added to something is fma2(x, y, -0) with a zero
// that the compiler does not know: ptxas contracts mul.rn.f32x2 and add.rn.f32x2 into one operation.
__device__ __forceinline__ F2 fma2(F2 x, F2 y, F2 z) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.b) : "l"(x.b), "l"(y.b), "l"(z.b));
  return r;
}

// One element of a buffer whose type is only known at run time (weights, read once for many rows).
__device__ __forceinline__ float load_any(const void* p, int type, int64_t i) {
  if (type == TBE_F32) return static_cast<const float*>(p)[i];
  if (type == TBE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void store_any(void* p, int type, int64_t i, float v) {
  if (type == TBE_F32) static_cast<float*>(p)[i] = v;
  else if (type == TBE_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p)[i] = __float2half_rn(v);
}

// V weights from column c on (1 or 0 where there are none), with vector loads where the buffer allows.
template <int V>
__device__ __forceinline__ void load_weights(const void* p, int type, int64_t c, float none, float (&f)[V]) {
  if (p == nullptr) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = none;
  } else if (V > 1 && type == TBE_F32 && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
    Pack<float, V> v;
    v.load(static_cast<const float*>(p) + c);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = v.get(i);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = load_any(p, type, c + i);
  }
}

// Asynchronous copy of one thread's BYTES (4, 8 or 16) into its own place in shared memory; the thread
// that copied them is the only one to read them, after async_wait, so no barrier is needed.
template <int BYTES>
__device__ __forceinline__ void async_copy(uint32_t dst, const void* src) {
  if constexpr (BYTES < 16) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
  } else {
    static_assert(BYTES == 16, "");
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  }
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

// What async_copy put there: BYTES / 4 words.
template <int BYTES>
__device__ __forceinline__ void shared_words(uint32_t src, uint32_t* w) {
  if constexpr (BYTES == 4) {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(src) : "memory");
  } else if constexpr (BYTES == 8) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(src) : "memory");
  } else {
    static_assert(BYTES == 16, "");
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(src) : "memory");
  }
}

// Sum over the L lanes (a power of two, aligned) that a thread is one of.
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

template <typename T> struct TypeTag { using type = T; };

// Calls f with the type tag of a tbe_dtype.
template <typename F>
auto with_type(int dtype, F&& f) {
  if (dtype == TBE_F32) return f(TypeTag<float>());
  if (dtype == TBE_F16) return f(TypeTag<__half>());
  return f(TypeTag<__nv_bfloat16>());
}

inline int dtype_bytes(int dtype) { return dtype == TBE_F32 ? 4 : 2; }
inline bool dtype_ok(int dtype) { return dtype == TBE_F32 || dtype == TBE_F16 || dtype == TBE_BF16; }
inline bool is_aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// ------------------------------------------------------------------------------------------
// Layer norm
// ------------------------------------------------------------------------------------------
// The validated problem, and what the kernels get of it.
struct NormArgs {
  int64_t rows, x_stride, y_stride, dx_stride;
  const int32_t* col_offsets;   // device, or NULL: segment s starts at s * width
  int segments, width, cols;    // width: the widest segment; cols: their sum
  int wtype;
  float eps;
};

tbe_status launch_norm_forward(const NormArgs& a, int xtype, int ytype, int vec, const void* x, const void* weight,
                               const void* bias, void* y, float* mean, float* rstd, const DeviceInfo& dev,
                               cudaStream_t s);
// Row slots of the backward's sums over rows: each leaves one partial row of dweight and dbias.
int norm_backward_slots(const NormArgs& a, const DeviceInfo& dev);
tbe_status launch_norm_backward(const NormArgs& a, int xtype, int ytype, int vec, const void* dy, const void* x,
                                const float* mean, const float* rstd, const void* weight, void* dx, void* dweight,
                                void* dbias, float* partial, const DeviceInfo& dev, cudaStream_t s);

// Columns [c0, c1) of a row of `cols`, as first column and width (at most `widest`), clamped so that whatever c0 and c1
// are the columns lie in the row and start and end at multiples of V.  The first column has V columns of the row from it on
// even where the width is 0: a thread without a column of its own reads the weights there.
template <int V>
__host__ __device__ __forceinline__ void clamp_span(int c0, int c1, int cols, int widest, int* col, int* width) {
  c0 = c0 < 0 ? 0 : c0 > cols - V ? cols - V : c0;
  c1 = c1 < c0 ? c0 : c1 > cols ? cols : c1;
  c0 -= c0 % V;
  const int w = c1 - c0 < widest ? c1 - c0 : widest;
  *col = c0;
  *width = w - w % V;
}

// First column and width of segment s; col_offsets that disagree with the host's widths give wrong sums but no access outside
// a row or the weights and none that is misaligned.
template <int V>
__device__ __forceinline__ void segment_span(const NormArgs& a, int s, int* col, int* width) {
  if (a.col_offsets == nullptr) {
    *col = s * a.width;
    *width = a.width;
    return;
  }
  clamp_span<V>(__ldg(a.col_offsets + s), __ldg(a.col_offsets + s + 1), a.cols, a.width, col, width);
}

}  // namespace tbe
