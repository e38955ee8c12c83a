// k_adamw.cu -- one AdamW step of many tensors (tbe_adamw_update), the values of its 8-bit states
// (tbe_adamw_state_values) and the global norm of many gradients (tbe_grad_norm).
//
// Each element is read and written once.  A thread takes 8 consecutive elements: 16 bytes of a 16-bit type, 32
// of fp32, 8 of codes; a warp then takes one block of the 8-bit states, whose scale needs one reduction over the
// warp and no shared memory.
//
// Measured on a GB300 (copy rate 6.78 TB/s): 32-bit states are bound by DRAM (227M bf16 parameters with masters,
// 28 bytes an element: 923 us, 6.87 TB/s), so is the norm (227M bf16: 71 us, 6.4 TB/s) and, with a write
// for every quarter byte read, the states' values (113M of each moment: 178 us, 6.4 TB/s).  The 8-bit step (113M bf16: 248 us, 4.6
// TB/s) has 60 instructions an element for 10 bytes of traffic, of which decoding takes 15, the step 15, scaling and encoding 20; two
// thirds of the issue slots are taken, and the largest stall is the wait for a block's loads.
#include <algorithm>
#include <cmath>

#include "k_tensor_list.cuh"

namespace tbe {
namespace {

constexpr int kThreads = 256;
constexpr int kVec = 8;
constexpr int kStep = kThreads * kVec;     // elements of a CTA's pass over its chunk
constexpr int kScalar = 0xff;              // AdamEntry.head: the tensor's buffers share no vector alignment
static_assert(TBE_Q8_BLOCK == 32 * kVec, "a warp takes one block");

struct AdamEntry {
  void* p;
  const void* g;
  float* master;
  void* m;
  void* v;
  float* ms;
  float* vs;
  int64_t n;
  float lr_scale, decay;
  int32_t head;   // elements before the first aligned vector, or kScalar (8-bit states: 0 or kScalar)
  int32_t pad;
};

struct AdamScalars {
  float beta1, beta2, one_minus_beta1, one_minus_beta2, log_beta1, log_beta2, eps, lr, minus_zero;
  const float* clip;
  int64_t* step;
  uint32_t* ticket;
  int advance;    // the call's last launch increments the step
};

template <int CAP> using AdamList = TensorList<AdamEntry, CAP>;
constexpr int kLargeAdam = 360;
static_assert(sizeof(AdamList<kLargeAdam>) + sizeof(AdamScalars) <= 32764, "kernel parameters");

// What a step multiplies by.
struct AdamFactors {
  float coef, beta1, beta2, omb1, omb2, step_size, inv_sqrt_bc2, eps, lr;  // step_size: lr / (1 - beta1^t)
  float minus_zero;
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The products and sums of the moments are rounded one by one (no fused multiply-add): the moments
// are then the same in any program that evaluates the formulas in fp32, and so are their 8-bit codes.
// The root and the reciprocal are the hardware's (within 2^-22 together, far inside p's rounding),
// in the forms without subnormals, one instruction each: a root counts as at least 2^-63, which matters only where
// eps is smaller still.
__device__ __forceinline__ void adam_moments(const AdamFactors& f, F2 grad, F2& m, F2& v) {
  const F2 none(f.minus_zero);
  const F2 g = grad * F2(f.coef);
  m = fma2(m, F2(f.beta1), none) + fma2(g, F2(f.omb1), none);
  v = fma2(v, F2(f.beta2), none) + fma2(g * g, F2(f.omb2), none);
}

// What a tensor's learning rate and decay make of the factors (negative, as they are added).
struct AdamRates {
  F2 step, decay;
  __device__ __forceinline__ AdamRates(const AdamFactors& f, float lr_scale, float weight_decay)
      : step(-f.step_size * lr_scale), decay(-f.lr * lr_scale * weight_decay) {}
};

__device__ __forceinline__ F2 adam_param(const AdamFactors& f, const AdamRates& rates, F2 p, F2 m, F2 v) {
  float v0, v1, r0, r1, i0, i1;
  v.get(v0, v1);
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(max_nan(v0, 0x1p-126f)));
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(max_nan(v1, 0x1p-126f)));
  fma2(F2(r0, r1), F2(f.inv_sqrt_bc2), F2(f.eps)).get(r0, r1);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(i0) : "f"(r0));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(i1) : "f"(r1));
  return fma2(rates.step, m * F2(i0, i1), fma2(rates.decay, p, p));
}

// 1 - beta^t, without the cancellation of small t.
__device__ __forceinline__ float bias_correction(float log_beta, int64_t t) {
  return -expm1f(static_cast<float>(t) * log_beta);
}

// A CTA's start: one thread reads the step and the clip coefficient and makes the factors (while the others' first loads
// are in flight), then takes a ticket; the last one to take one knows that every CTA has read the step, and advances it.
struct AdamStart {
  float coef, step_size, inv_sqrt_bc2;
  bool go;  // false: the gradients' norm says that the step is to be left out
  uint32_t place;
  int64_t t;
};

// Before the CTA's barrier, thread 0 only.
__device__ __forceinline__ void adam_begin(const AdamScalars& s, AdamStart& start) {
  float norm = 0.f, coef = 1.f;
  const int64_t t = *s.step + 1;
  if (s.clip != nullptr) {
    norm = s.clip[0];
    coef = s.clip[1];
  }
  start.coef = coef;
  start.step_size = s.lr / bias_correction(s.log_beta1, t);
  start.inv_sqrt_bc2 = __frsqrt_rn(bias_correction(s.log_beta2, t));
  start.go = isfinite(norm);
  start.t = t;
}

__device__ __forceinline__ AdamFactors adam_factors(const AdamScalars& s, const AdamStart& start) {
  AdamFactors f;
  f.coef = start.coef;
  f.beta1 = s.beta1, f.beta2 = s.beta2, f.omb1 = s.one_minus_beta1, f.omb2 = s.one_minus_beta2;
  f.step_size = start.step_size;
  f.inv_sqrt_bc2 = start.inv_sqrt_bc2;
  f.eps = s.eps;
  f.lr = s.lr;
  f.minus_zero = s.minus_zero;
  return f;
}

// After the barrier, thread 0 only: its place among the CTAs; and, at the kernel's end, what the last one does.
__device__ __forceinline__ void adam_arrive(const AdamScalars& s, AdamStart& start) {
  __threadfence();
  start.place = atomicAdd(s.ticket, 1u);
}
__device__ __forceinline__ void adam_end(const AdamScalars& s, const AdamStart& start) {
  if (start.place == gridDim.x - 1) {
    __threadfence();
    *s.ticket = 0;
    if (s.advance) *s.step = start.t;
  }
}

// 8 elements at p (aligned), or the first `n` of them one by one.
template <typename T>
__device__ __forceinline__ Pack<T, kVec> load8(const T* p, int n, bool vec) {
  Pack<T, kVec> v;
  if (vec && n >= kVec) v.load(p);
  else v.load_some(p, n);
  return v;
}
template <typename T>
__device__ __forceinline__ void unpack8(const Pack<T, kVec>& v, F2 (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = F2(v.get(2 * i), v.get(2 * i + 1));
}
template <typename T>
__device__ __forceinline__ void store8(T* p, int n, bool vec, const F2 (&f)[4]) {
  Pack<T, kVec> v;
  float s[kVec];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i].get(s[2 * i], s[2 * i + 1]);
  v.set(s);
  if (vec && n >= kVec) v.store(p);
  else v.store_some(p, n);
}

// ------------------------------------------------------------------------------------------
// 32-bit states
// ------------------------------------------------------------------------------------------
// 8 elements of a tensor from `at` on, the first n of them in it.
template <typename P, typename G, bool MASTER>
struct AdamPart {
  using Held = typename std::conditional<MASTER, float, P>::type;
  Pack<G, kVec> g;
  Pack<Held, kVec> p;
  Pack<float, kVec> m, v;

  __device__ __forceinline__ void load(const AdamEntry& e, int64_t at, int n, bool vec) {
    g = load8(static_cast<const G*>(e.g) + at, n, vec);
    m = load8(static_cast<const float*>(e.m) + at, n, vec);
    v = load8(static_cast<const float*>(e.v) + at, n, vec);
    p = load8((MASTER ? reinterpret_cast<const Held*>(e.master) : static_cast<const Held*>(e.p)) + at, n, vec);
  }
  __device__ __forceinline__ void step(const AdamEntry& e, const AdamFactors& f, int64_t at, int n, bool vec) const {
    F2 pf[4], gf[4], mf[4], vf[4];
    unpack8(g, gf);
    unpack8(m, mf);
    unpack8(v, vf);
    unpack8(p, pf);
    const AdamRates rates(f, e.lr_scale, e.decay);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      adam_moments(f, gf[i], mf[i], vf[i]);
      pf[i] = adam_param(f, rates, pf[i], mf[i], vf[i]);
    }
    if constexpr (MASTER) store8(e.master + at, n, vec, pf);
    store8(static_cast<P*>(e.p) + at, n, vec, pf);
    store8(static_cast<float*>(e.m) + at, n, vec, mf);
    store8(static_cast<float*>(e.v) + at, n, vec, vf);
  }
};

constexpr int kResident = 3;  // CTAs to an SM (227M bf16 parameters with masters: 923 us; 2: 935, 4: 942)

// A CTA takes a chunk; its first loads are in flight while thread 0 makes the factors (297K fp32 parameters: 4.1 us,
// 4.8 with the factors first and the ticket last).
template <typename P, typename G, bool MASTER, int CAP>
__global__ void __launch_bounds__(kThreads, kResident)
    adamw_kernel(const __grid_constant__ AdamList<CAP> list, const __grid_constant__ AdamScalars s) {
  __shared__ AdamStart start;
  const bool any = blockIdx.x < list.first[list.count];  // a list without elements has one CTA, for the step alone
  const int t = any ? tensor_of_chunk(list, blockIdx.x) : 0;
  const AdamEntry& e = list.e[t];
  const bool vec = any && e.head != kScalar;
  const int64_t begin = any ? static_cast<int64_t>(blockIdx.x - list.first[t]) * list.chunk_elems : 0;
  const int64_t end = any ? min(begin + list.chunk_elems, e.n) : 0;
  // aligned: vectors start `head` elements in; else a thread takes single elements
  const int64_t stop = vec ? min(end + e.head, e.n) : end;
  const int stride = vec ? kStep : kThreads;
  int64_t at = begin + (vec ? e.head + threadIdx.x * kVec : threadIdx.x);
  auto count = [&] { return vec ? static_cast<int>(min(static_cast<int64_t>(kVec), stop - at)) : 1; };
  AdamPart<P, G, MASTER> part;
  if (at < stop) part.load(e, at, count(), vec);
  if (threadIdx.x == 0) adam_begin(s, start);
  __syncthreads();
  if (!start.go) return;  // in every CTA alike
  if (threadIdx.x == 0) adam_arrive(s, start);
  const AdamFactors f = adam_factors(s, start);
  while (at < stop) {
    part.step(e, f, at, count(), vec);
    at += stride;
    if (at < stop) part.load(e, at, count(), vec);
  }
  if (vec && begin == 0 && threadIdx.x == 0 && e.head > 0) {  // the elements before the first vector
    const int n = static_cast<int>(min(static_cast<int64_t>(e.head), e.n));
    part.load(e, 0, n, false);
    part.step(e, f, 0, n, false);
  }
  if (threadIdx.x == 0) adam_end(s, start);
}

// ------------------------------------------------------------------------------------------
// 8-bit states
// ------------------------------------------------------------------------------------------
// Scales below this (whose reciprocals would leave fp32) count as zero.
constexpr float kQ8Least = 0x1p-120f;

// The code of a magnitude r in [0, 1] is the nearest integer to slope * r + offset: with z the code's leading zeros (r
// lies between 8^-(z+1) and 8^-z) and low its leading one, the line of that interval is
// ((8^(z+1) r - 1) / 7) low + low - 1.  z follows from r's exponent; slope and offset come from a table by it, in
// shared memory (12 instructions an element less than computing them; few exponents occur in a block, and equal
// ones are one access).
struct Q8Lines {
  float2 m[256];  // 7 bits of magnitude
  float2 v[256];  // 8 bits
};

__device__ __forceinline__ float2 q8_line(int bits, int e) {
  const int z = max(min(((126 - e) * 0x5556) >> 16, bits - 1), 0);  // (126 - e) / 3
  const float low = __uint_as_float(static_cast<uint32_t>(127 + bits - 1 - z) << 23);
  const float slope = __uint_as_float(__float_as_uint(1.f / 7.f) + (static_cast<uint32_t>(bits + 2 + 2 * z) << 23));
  return make_float2(slope, __fadd_rn(__fmul_rn(low, 6.f / 7.f), -1.f));
}

__device__ __forceinline__ void q8_fill(Q8Lines& t) {
  static_assert(kThreads == 256, "a thread to an exponent");
  t.m[threadIdx.x] = q8_line(7, threadIdx.x);
  t.v[threadIdx.x] = q8_line(8, threadIdx.x);
}

// The values of two codes (the low 8 bits of each half of `pair`), in units of the scale: with c the
// code, low its leading one, (7 c + 7 - 6 low) low^2 2^(-3 BITS); every step is exact in fp16.
template <int BITS>
__device__ __forceinline__ __half2 q8_decode2(uint32_t pair) {
  const uint32_t magic = pair | 0x64006400u;  // 1024 + c
  const __half2 c = __hadd2(*reinterpret_cast<const __half2*>(&magic), __float2half2_rn(-1024.f));
  uint32_t low_bits = *reinterpret_cast<const uint32_t*>(&c) & 0x7c007c00u;
  const __half2 low = *reinterpret_cast<const __half2*>(&low_bits);
  // BITS = 8: q = 7 c + 7 - 6 low, times (low 2^-12)^2; BITS = 7: q / 2, times (low 2^-10)^2
  constexpr float k = BITS == 8 ? 1.f : 0.5f;
  const __half2 q = __hfma2(low, __float2half2_rn(-6.f * k), __hfma2(c, __float2half2_rn(7.f * k), __float2half2_rn(7.f * k)));
  const __half2 lows = __hmul2(low, __float2half2_rn(BITS == 8 ? 0x1p-12f : 0x1p-10f));
  return __hmul2(__hmul2(q, lows), lows);
}

// 8 codes in two words -> fp32; SIGNED: the top bit is the sign.
template <bool SIGNED>
__device__ __forceinline__ void q8_values(uint2 codes, float scale, F2 (&f)[4]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t w = h ? codes.y : codes.x;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t pair = __byte_perm(w, 0, k ? 0x4342 : 0x4140);  // two codes, each in a half
      __half2 d = q8_decode2<SIGNED ? 7 : 8>(SIGNED ? pair & 0x007f007fu : pair);
      if (SIGNED) {
        uint32_t b = *reinterpret_cast<uint32_t*>(&d) | ((pair & 0x00800080u) << 8);
        d = *reinterpret_cast<__half2*>(&b);
      }
      const float2 v = __half22float2(d);
      f[2 * h + k] = F2(v.x, v.y) * F2(scale);
    }
  }
}

// The first n codes at p, one by one.
__device__ __forceinline__ uint2 load_codes(const uint8_t* p, int n) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < kVec; ++i)
    if (i < n) w[i / 4] |= static_cast<uint32_t>(p[i]) << (8 * (i % 4));
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store_codes(uint8_t* p, int n, uint2 c) {
#pragma unroll
  for (int i = 0; i < kVec; ++i)
    if (i < n) p[i] = static_cast<uint8_t>((i < 4 ? c.x : c.y) >> (8 * (i % 4)));
}

// Codes of a warp's block, 8 values to a lane, and its scale.  A block with a NaN or an infinity gets it as its
// scale.  Magnitudes are compared across the warp as integers, which orders them and puts NaN on top.
template <bool SIGNED>
__device__ __forceinline__ uint2 q8_block(const float2 (&lines)[256], const F2 (&f)[4], float* scale) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max_nan(max_nan(top, fabsf(f[i].lo())), fabsf(f[i].hi()));
  float a = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(top)));
  if (a < kQ8Least) a = 0.f;
  const float inv = a > 0.f ? __frcp_rn(a) : 0.f;
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const F2 x = f[2 * h + i / 2];
      const float r = __fmul_rn(fabsf(i & 1 ? x.hi() : x.lo()), inv);
      const float2 line = lines[__float_as_uint(r) >> 23];
      // adding 1.5 * 2^23 rounds to the nearest integer, which is then the low byte
      c[i] = __float_as_uint(__fadd_rn(__fadd_rn(__fmul_rn(r, line.x), line.y), 12582912.f));
    }
    w[h] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
    if (SIGNED) {
      uint32_t s[4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        s[2 * k] = __float_as_uint(f[2 * h + k].lo());
        s[2 * k + 1] = __float_as_uint(f[2 * h + k].hi());
      }
      w[h] |= __byte_perm(__byte_perm(s[0], s[1], 0x0073), __byte_perm(s[2], s[3], 0x0073), 0x5410) & 0x80808080u;
    }
  }
  if (!SIGNED) {
    // a positive second moment gets code 1 at least; bytes of zero are rare
    auto has_zero = [](uint32_t v) { return (v - 0x01010101u) & ~v & 0x80808080u; };
    if (has_zero(w[0]) | has_zero(w[1])) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const float x = i & 1 ? f[i / 2].hi() : f[i / 2].lo();
        if (!(w[i / 4] >> (8 * (i % 4)) & 0xffu) && x > 0.f && inv > 0.f) w[i / 4] |= 1u << (8 * (i % 4));
      }
    }
  }
  *scale = a;
  return make_uint2(w[0], w[1]);
}

// One block, a lane's 8 elements (`n` within the tensor): `get` and `put` read and write its parts, each as late and as
// early as the registers want it.
template <typename P, typename G, bool MASTER, typename Get, typename Put>
__device__ __forceinline__ void q8_step(const AdamFactors& f, const AdamRates& rates, const Q8Lines& lines, int n,
                                        const Get& get, const Put& put) {
  F2 m[4], v[4], x[4];
  q8_values<true>(get.m(), get.ms(), m);
  q8_values<false>(get.v(), get.vs(), v);
  unpack8(get.g(), x);
#pragma unroll
  for (int i = 0; i < 4; ++i) adam_moments(f, x[i], m[i], v[i]);
  unpack8(get.p(), x);
  float s[kVec];
#pragma unroll
  for (int i = 0; i < 4; ++i) adam_param(f, rates, x[i], m[i], v[i]).get(s[2 * i], s[2 * i + 1]);
  if constexpr (MASTER) {
    Pack<float, kVec> full;
    full.set(s);
    put.master(full);
  }
  Pack<P, kVec> p;
  p.set(s);
  put.p(p);
  if (n < kVec) {  // past the tensor's end: no part of the block's scale
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (2 * i >= n) m[i] = v[i] = F2(0.f);
      else if (2 * i + 1 >= n) m[i] = F2(m[i].lo(), 0.f), v[i] = F2(v[i].lo(), 0.f);
    }
  }
  float scale;
  put.m(q8_block<true>(lines.m, m, &scale));
  put.ms(scale);
  put.v(q8_block<false>(lines.v, v, &scale));
  put.vs(scale);
}

// Where a lane's part of a block is.
template <typename P, typename G, bool MASTER>
struct Q8Place {
  using Held = typename std::conditional<MASTER, float, P>::type;
  static constexpr int kNext = kStep / TBE_Q8_BLOCK;  // blocks of a pass
  uint8_t* m_;
  uint8_t* v_;
  const G* g_;
  P* p_;
  Held* held_;
  float* ms_;
  float* vs_;
  bool writer;

  __device__ __forceinline__ Q8Place(const AdamEntry& e, uint64_t block) : writer(threadIdx.x % 32 == 0) {
    const uint64_t at = block * TBE_Q8_BLOCK + threadIdx.x % 32 * kVec;
    m_ = static_cast<uint8_t*>(e.m) + at;
    v_ = static_cast<uint8_t*>(e.v) + at;
    g_ = static_cast<const G*>(e.g) + at;
    p_ = static_cast<P*>(e.p) + at;
    held_ = MASTER ? reinterpret_cast<Held*>(e.master) + at : reinterpret_cast<Held*>(p_);
    ms_ = e.ms + block;
    vs_ = e.vs + block;
  }
  __device__ __forceinline__ void advance() {
    m_ += kStep, v_ += kStep, g_ += kStep, p_ += kStep, held_ += kStep, ms_ += kNext, vs_ += kNext;
  }
  // Asks for a later block's data, `ahead` passes on.
  __device__ __forceinline__ void prefetch(int ahead) const {
    auto ask = [](const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); };
    ask(m_ + ahead * kStep);
    ask(v_ + ahead * kStep);
    ask(g_ + ahead * kStep);
    ask(held_ + ahead * kStep);
  }
};

// A whole block's part, all loads issued at once.
template <typename Place, typename G>
struct Q8Whole {
  uint2 m_, v_;
  Pack<G, kVec> g_;
  Pack<typename Place::Held, kVec> p_;
  float ms_, vs_;
  __device__ __forceinline__ explicit Q8Whole(const Place& o)
      : m_(*reinterpret_cast<const uint2*>(o.m_)), v_(*reinterpret_cast<const uint2*>(o.v_)), ms_(*o.ms_), vs_(*o.vs_) {
    g_.load(o.g_);
    p_.load(o.held_);
  }
  __device__ __forceinline__ uint2 m() const { return m_; }
  __device__ __forceinline__ uint2 v() const { return v_; }
  __device__ __forceinline__ float ms() const { return ms_; }
  __device__ __forceinline__ float vs() const { return vs_; }
  __device__ __forceinline__ const Pack<G, kVec>& g() const { return g_; }
  __device__ __forceinline__ const Pack<typename Place::Held, kVec>& p() const { return p_; }
};

template <typename Place, typename P>
struct Q8PutWhole {
  const Place& o;
  __device__ __forceinline__ void m(uint2 c) const { *reinterpret_cast<uint2*>(o.m_) = c; }
  __device__ __forceinline__ void v(uint2 c) const { *reinterpret_cast<uint2*>(o.v_) = c; }
  __device__ __forceinline__ void ms(float x) const { if (o.writer) *o.ms_ = x; }
  __device__ __forceinline__ void vs(float x) const { if (o.writer) *o.vs_ = x; }
  __device__ __forceinline__ void p(const Pack<P, kVec>& x) const { x.store(o.p_); }
  __device__ __forceinline__ void master(const Pack<float, kVec>& x) const { x.store(reinterpret_cast<float*>(o.held_)); }
};

// The first n elements, one by one.
template <typename Place, typename P, typename G>
struct Q8Ragged {
  const Place& o;
  int n;
  __device__ __forceinline__ uint2 m() const { return load_codes(o.m_, n); }
  __device__ __forceinline__ uint2 v() const { return load_codes(o.v_, n); }
  __device__ __forceinline__ float ms() const { return *o.ms_; }
  __device__ __forceinline__ float vs() const { return *o.vs_; }
  __device__ __forceinline__ Pack<G, kVec> g() const { Pack<G, kVec> x; x.load_some(o.g_, n); return x; }
  __device__ __forceinline__ Pack<typename Place::Held, kVec> p() const {
    Pack<typename Place::Held, kVec> x;
    x.load_some(o.held_, n);
    return x;
  }
  __device__ __forceinline__ void m(uint2 c) const { store_codes(o.m_, n, c); }
  __device__ __forceinline__ void v(uint2 c) const { store_codes(o.v_, n, c); }
  __device__ __forceinline__ void ms(float x) const { if (o.writer) *o.ms_ = x; }
  __device__ __forceinline__ void vs(float x) const { if (o.writer) *o.vs_ = x; }
  __device__ __forceinline__ void p(const Pack<P, kVec>& x) const { x.store_some(o.p_, n); }
  __device__ __forceinline__ void master(const Pack<float, kVec>& x) const { x.store_some(reinterpret_cast<float*>(o.held_), n); }
};

// A CTA takes a contiguous share of the chunks (of one pass, a block to a warp), so that the table and the factors
// are made once for it (every gridDim-th chunk instead: 312 us, for 113M bf16 parameters, against 250).  Whole blocks of a
// tensor go by running pointers, the next one asked for in L2 while this one's codes are computed (without that 295;
// loaded into registers instead 280, into shared memory 294: their waits or traffic meet the table's); what is ragged or
// not aligned is loaded element by element.
constexpr int kQ8Ahead = 1;     // passes (2: 266 us)
// CTAs to an SM, as bf16 without masters wants it: 3 274 us, 4 263, 5 248, in spite of 30 words that each thread reloads a pass.
// Others, 4 and 5: bf16 with masters 341 and 334; fp32 320 and 331; bf16 with fp32 gradients and masters (50 words) 355 and 389.
constexpr int kQ8Resident = 5;

template <typename P, typename G, bool MASTER, int CAP>
__global__ void __launch_bounds__(kThreads, kQ8Resident)
    adamw_q8_kernel(const __grid_constant__ AdamList<CAP> list, const __grid_constant__ AdamScalars s) {
  __shared__ Q8Lines lines;
  __shared__ AdamStart start;
  if (threadIdx.x == 0) adam_begin(s, start);
  q8_fill(lines);
  __syncthreads();
  if (!start.go) return;  // in every CTA alike
  if (threadIdx.x == 0) adam_arrive(s, start);
  const AdamFactors f = adam_factors(s, start);
  using Place = Q8Place<P, G, MASTER>;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint64_t chunks = list.first[list.count];
  uint32_t chunk = static_cast<uint32_t>(chunks * blockIdx.x / gridDim.x);
  const uint32_t end = static_cast<uint32_t>(chunks * (blockIdx.x + 1) / gridDim.x);
  for (int t = chunk < end ? tensor_of_chunk(list, chunk) : 0; chunk < end; ++t) {
    const uint32_t stop = min(end, list.first[t + 1]);
    if (stop <= chunk) continue;  // a tensor without elements
    const AdamEntry& e = list.e[t];
    const AdamRates rates(f, e.lr_scale, e.decay);
    const uint64_t block = static_cast<uint64_t>(chunk - list.first[t]) * Place::kNext + warp;
    // this warp's blocks of the share: whole ones, then perhaps a ragged one
    const uint64_t whole = static_cast<uint64_t>(e.n) / TBE_Q8_BLOCK;
    const int count = static_cast<int>(stop - chunk);
    int fast = 0;
    if (e.head != kScalar && block < whole)
      fast = static_cast<int>(min(static_cast<uint64_t>(count), (whole - block + Place::kNext - 1) / Place::kNext));
    chunk = stop;
    Place at(e, block);
    for (int k = 0; k < fast; ++k, at.advance()) {
      const Q8Whole<Place, G> in(at);
      if (k + kQ8Ahead < fast) at.prefetch(kQ8Ahead);
      q8_step<P, G, MASTER>(f, rates, lines, kVec, in, Q8PutWhole<Place, P>{at});
    }
    for (int k = fast; k < count; ++k, at.advance()) {
      const int64_t left = e.n - static_cast<int64_t>(block + static_cast<uint64_t>(k) * Place::kNext) * TBE_Q8_BLOCK;
      if (left <= 0) break;
      const int n = max(min(static_cast<int>(min(left, int64_t(TBE_Q8_BLOCK))) - lane * kVec, kVec), 0);
      const Q8Ragged<Place, P, G> ragged{at, n};
      q8_step<P, G, MASTER>(f, rates, lines, n, ragged, ragged);
    }
  }
  if (threadIdx.x == 0) adam_end(s, start);
}

// ------------------------------------------------------------------------------------------
// Values of the 8-bit states
// ------------------------------------------------------------------------------------------
struct ValuesEntry {
  const void* m;
  const void* v;
  const float* ms;
  const float* vs;
  float* m_out;
  float* v_out;
  int64_t n;
  int32_t vec;
  int32_t pad;
};
constexpr int kLargeValues = 480;

template <int CAP>
__global__ void __launch_bounds__(kThreads) q8_values_kernel(const __grid_constant__ TensorList<ValuesEntry, CAP> list) {
  const int t = tensor_of_chunk(list, blockIdx.x);
  const ValuesEntry& e = list.e[t];
  const int64_t begin = static_cast<int64_t>(blockIdx.x - list.first[t]) * list.chunk_elems;
  const int64_t end = min(begin + list.chunk_elems, e.n);
  for (int64_t at = begin + threadIdx.x * kVec; at < end; at += kStep) {
    const int n = static_cast<int>(min(end - at, static_cast<int64_t>(kVec)));
    auto one = [&](auto sign, const void* codes, const float* scale, float* out) {
      if (out == nullptr) return;
      const uint8_t* c = static_cast<const uint8_t*>(codes) + at;
      const bool vec = e.vec && n == kVec;
      F2 f[4];
      q8_values<decltype(sign)::value>(vec ? *reinterpret_cast<const uint2*>(c) : load_codes(c, n), scale[at / TBE_Q8_BLOCK], f);
      store8(out + at, n, vec, f);
    };
    one(std::true_type(), e.m, e.ms, e.m_out);
    one(std::false_type(), e.v, e.vs, e.v_out);
  }
}

// ------------------------------------------------------------------------------------------
// Gradient norm
// ------------------------------------------------------------------------------------------
struct NormEntry {
  const void* g;
  int64_t n;
};
constexpr int kLargeNorm = 1500;
static_assert(sizeof(TensorList<NormEntry, kLargeNorm>) + 64 <= 32764, "kernel parameters");

constexpr int kNormMaxGrid = 4096;
// CTAs to an SM: 2.4M bf16 gradients 8.5 us, 10.0 with 8; 9.4M 13.1, 14.1; 38M 16.8, 17.8; 227M 71, 70.4.  At a few million
// elements the fp64 pipe is the busiest part (41% of the SMs' active cycles): every thread adds in fp64 once a chunk and in the
// CTA's sum.
constexpr int kNormResident = 4;
struct NormWs {
  uint32_t ticket;
  uint32_t pad;
  double earlier;                 // the squares of the call's earlier launches
  double partial[kNormMaxGrid];   // of this launch's CTAs
};

template <typename G, int CAP>
__global__ void __launch_bounds__(kThreads, kNormResident)
    grad_norm_kernel(const __grid_constant__ TensorList<NormEntry, CAP> list, NormWs* ws, int first, int last,
                     float max_norm, float* out) {
  double sum = 0.0;
  for (uint32_t chunk = blockIdx.x; chunk < list.first[list.count]; chunk += gridDim.x) {
    const int t = tensor_of_chunk(list, chunk);
    const G* g = static_cast<const G*>(list.e[t].g);
    const int64_t n = list.e[t].n, begin = static_cast<int64_t>(chunk - list.first[t]) * list.chunk_elems;
    const int64_t end = min(begin + list.chunk_elems, n);
    // elements before the first 16-byte boundary, whole vectors, the rest
    const int64_t head = min(static_cast<int64_t>((16 - reinterpret_cast<uintptr_t>(g + begin) % 16) % 16 / sizeof(G)), end - begin);
    float q = 0.f;
    if (threadIdx.x < head) {
      Pack<G, 1> v;
      v.load(g + begin + threadIdx.x);
      q = v.get(0) * v.get(0);
    }
    constexpr int N = 16 / sizeof(G);
    const int64_t vectors = (end - begin - head) / N;
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < vectors; i += kThreads) {
      Pack<G, N> v;
      v.load(g + begin + head + i * N);
#pragma unroll
      for (int k = 0; k < N; ++k) q = fmaf(v.get(k), v.get(k), q);
    }
    const int64_t tail = begin + head + vectors * N + threadIdx.x;
    if (tail < end) {
      Pack<G, 1> v;
      v.load(g + tail);
      q = fmaf(v.get(0), v.get(0), q);
    }
    sum += static_cast<double>(q);
  }
  __shared__ double part[kThreads / 32];
  auto block_sum = [&](double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    double total = 0.0;
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) total += part[k];
    return total;
  };
  sum = block_sum(sum);
  if (threadIdx.x == 0) ws->partial[blockIdx.x] = sum;
  if (!last_cta(&ws->ticket)) return;
  sum = 0.0;
  for (unsigned i = threadIdx.x; i < gridDim.x; i += kThreads) sum += __ldcg(&ws->partial[i]);
  sum = block_sum(sum);
  if (threadIdx.x != 0) return;
  if (!first) sum += ws->earlier;
  if (!last) {
    ws->earlier = sum;
    return;
  }
  const float norm = static_cast<float>(sqrt(sum));
  out[0] = norm;
  const float coef = __fdiv_rn(max_norm, norm + 1e-6f);
  out[1] = coef > 1.f ? 1.f : coef;
}

// ------------------------------------------------------------------------------------------
// Host
// ------------------------------------------------------------------------------------------
// Elements of a chunk: up to `most` passes of a CTA (a power of two), fewer while that leaves less than 16 chunks to an SM.
// AdamW with 32-bit states takes 4 (at 227M, 1 took a ninth longer), the norm 16 (with eight CTAs an SM 70 us; 4: 74), the values 1 (178 us; 4: 200,
// 16: 228: two streams in and two out like a narrow band).
uint32_t chunk_elems(int64_t total, const DeviceInfo& dev, int most) {
  int passes = 1;
  while (passes < most && total / (2 * passes * kStep) >= 16 * static_cast<int64_t>(dev.sms)) passes *= 2;
  return static_cast<uint32_t>(passes * kStep);
}

// Splits the tensors into launches of at most the list's capacity and at most 2^31 - 1 chunks; fill(i, entry)
// describes tensor i, go(list, first, last) launches.
template <typename Entry, int LARGE, typename Numel, typename Fill, typename Go>
tbe_status for_lists(int count, uint32_t chunk, Numel&& numel, Fill&& fill, Go&& go) {
  int at = 0;
  bool first = true;
  do {
    auto part = [&](auto& list, int cap) {
      list.chunk_elems = chunk;
      int k = 0;
      int64_t chunks = 0;
      while (k < cap && at < count) {
        const int64_t more = (numel(at) + chunk - 1) / chunk;
        if (chunks + more > INT32_MAX) break;
        list.first[k] = static_cast<uint32_t>(chunks);
        fill(at, &list.e[k]);
        chunks += more;
        ++k;
        ++at;
      }
      list.count = k;
      list.first[k] = static_cast<uint32_t>(chunks);
      const tbe_status st = go(list, first, at >= count);
      first = false;
      return st;
    };
    tbe_status st;
    if (count - at <= kSmallList) {
      TensorList<Entry, kSmallList> list;
      st = part(list, kSmallList);
    } else {
      TensorList<Entry, LARGE> list;
      st = part(list, LARGE);
    }
    if (st != TBE_OK) return st;
  } while (at < count);
  return TBE_OK;
}

constexpr int64_t kMaxNumel = int64_t(1) << 40;  // one tensor's chunks fit a launch

// Elements before the first at which every buffer is aligned for vectors of 8, or kScalar.
int vector_head(const tbe_dense_tensor& d, int pdtype, int gdtype) {
  auto congruent = [](const void* p, int size, int head) {
    return (reinterpret_cast<uintptr_t>(p) + static_cast<uintptr_t>(head) * size) % 16 == 0;
  };
  for (int head = 0; head < kVec; ++head) {
    if (congruent(d.param, dtype_bytes(pdtype), head) && congruent(d.grad, dtype_bytes(gdtype), head) &&
        congruent(d.exp_avg, 4, head) && congruent(d.exp_avg_sq, 4, head) && congruent(d.master, 4, d.master ? head : 0))
      return head;
  }
  return kScalar;
}

tbe_status check_adamw(const tbe_adamw_problem* p, bool values_only) {
  if (p == nullptr || p->count < 0 || (p->count > 0 && p->tensors == nullptr)) return TBE_ERR_INVALID_ARG;
  if (!dtype_ok(p->pdtype) || !dtype_ok(p->gdtype)) return TBE_ERR_UNSUPPORTED;
  if (p->states != TBE_STATE_F32 && p->states != TBE_STATE_Q8) return TBE_ERR_INVALID_ARG;
  if (!(p->beta1 >= 0 && p->beta1 < 1 && p->beta2 >= 0 && p->beta2 < 1)) return TBE_ERR_INVALID_ARG;
  if (!(p->eps >= 0) || std::isinf(p->eps)) return TBE_ERR_INVALID_ARG;
  const bool q8 = p->states == TBE_STATE_Q8;
  bool master = false, plain = false;
  for (int i = 0; i < p->count; ++i) {
    const tbe_dense_tensor& d = p->tensors[i];
    if (d.numel < 0) return TBE_ERR_INVALID_ARG;
    if (d.numel > kMaxNumel) return TBE_ERR_UNSUPPORTED;
    if (d.numel == 0) continue;
    if (d.exp_avg == nullptr || d.exp_avg_sq == nullptr) return TBE_ERR_INVALID_ARG;
    if (q8 && (d.exp_avg_scale == nullptr || d.exp_avg_sq_scale == nullptr || !is_aligned(d.exp_avg_scale, 4) ||
               !is_aligned(d.exp_avg_sq_scale, 4)))
      return TBE_ERR_INVALID_ARG;
    if (values_only) continue;
    if (d.param == nullptr || d.grad == nullptr || !is_aligned(d.param, dtype_bytes(p->pdtype)) ||
        !is_aligned(d.grad, dtype_bytes(p->gdtype)) || !is_aligned(d.master, 4))
      return TBE_ERR_INVALID_ARG;
    if (!q8 && (!is_aligned(d.exp_avg, 4) || !is_aligned(d.exp_avg_sq, 4))) return TBE_ERR_INVALID_ARG;
    if (!std::isfinite(d.lr_scale) || !std::isfinite(d.weight_decay)) return TBE_ERR_INVALID_ARG;
    (d.master != nullptr ? master : plain) = true;
  }
  if (master && (plain || p->pdtype == TBE_F32)) return TBE_ERR_UNSUPPORTED;  // all tensors or none, 16-bit params
  return TBE_OK;
}

template <typename P, typename G, bool MASTER>
tbe_status launch_adamw(const tbe_adamw_problem& prob, AdamScalars sc, const DeviceInfo& dev, cudaStream_t s) {
  int64_t total = 0;
  for (int i = 0; i < prob.count; ++i) total += prob.tensors[i].numel;
  const bool q8 = prob.states == TBE_STATE_Q8;
  return for_lists<AdamEntry, kLargeAdam>(
      prob.count, q8 ? kStep : chunk_elems(total, dev, 4), [&](int i) { return prob.tensors[i].numel; },
      [&](int i, AdamEntry* e) {
        const tbe_dense_tensor& d = prob.tensors[i];
        int head = d.numel == 0 ? 0 : kScalar;
        if (d.numel > 0 && q8) {
          if (is_aligned(d.param, 16) && is_aligned(d.grad, 16) && is_aligned(d.master, 16) && is_aligned(d.exp_avg, 8) &&
              is_aligned(d.exp_avg_sq, 8))
            head = 0;
        } else if (d.numel > 0) {
          head = vector_head(d, prob.pdtype, prob.gdtype);
        }
        *e = AdamEntry{d.param,         d.grad,  d.master,   d.exp_avg,      d.exp_avg_sq, d.exp_avg_scale,
                       d.exp_avg_sq_scale, d.numel, d.lr_scale, d.weight_decay, head,         0};
      },
      [&](auto& list, bool, bool last) {
        constexpr int CAP = static_cast<int>(sizeof(list.e) / sizeof(list.e[0]));
        const uint32_t chunks = list.first[list.count];
        sc.advance = last;
        const unsigned grid = chunks > 0 ? chunks : 1;
        if (q8) {
          const unsigned resident = std::min(grid, static_cast<unsigned>(dev.sms * kQ8Resident));
          adamw_q8_kernel<P, G, MASTER, CAP><<<resident, kThreads, 0, s>>>(list, sc);
        }
        if (!q8) adamw_kernel<P, G, MASTER, CAP><<<grid, kThreads, 0, s>>>(list, sc);
        note_launch();
        return cuda_status(cudaGetLastError());
      });
}

}  // namespace
}  // namespace tbe

using namespace tbe;

extern "C" {

size_t tbe_grad_norm_workspace_size(void) { return sizeof(NormWs); }

tbe_status tbe_grad_norm(int32_t count, const void* const* grads, const int64_t* numels, tbe_dtype dtype, float max_norm,
                         float* out, void* ws, size_t ws_bytes, void* stream) {
  if (count < 0 || (count > 0 && (grads == nullptr || numels == nullptr)) || out == nullptr || !is_aligned(out, 4))
    return TBE_ERR_INVALID_ARG;
  if (!dtype_ok(dtype)) return TBE_ERR_UNSUPPORTED;
  if (!(max_norm >= 0)) return TBE_ERR_INVALID_ARG;
  int64_t total = 0;
  for (int i = 0; i < count; ++i) {
    if (numels[i] < 0) return TBE_ERR_INVALID_ARG;
    if (numels[i] > kMaxNumel) return TBE_ERR_UNSUPPORTED;
    if (numels[i] > 0 && (grads[i] == nullptr || !is_aligned(grads[i], dtype_bytes(dtype)))) return TBE_ERR_INVALID_ARG;
    total += numels[i];
  }
  if (ws == nullptr || ws_bytes < sizeof(NormWs)) return TBE_ERR_WORKSPACE;
  if (!is_aligned(ws, 16)) return TBE_ERR_INVALID_ARG;
  DeviceInfo dev;
  const tbe_status st = device_info(&dev);
  if (st != TBE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return with_type(dtype, [&](auto tag) {
    using G = typename decltype(tag)::type;
    return for_lists<NormEntry, kLargeNorm>(
        count, chunk_elems(total, dev, 16), [&](int i) { return numels[i]; },
        [&](int i, NormEntry* e) { *e = NormEntry{grads[i], numels[i]}; },
        [&](auto& list, bool first, bool last) {
          constexpr int CAP = static_cast<int>(sizeof(list.e) / sizeof(list.e[0]));
          const int64_t chunks = list.first[list.count];
          const int64_t most = std::min<int64_t>(kNormMaxGrid, static_cast<int64_t>(dev.sms) * kNormResident);
          const unsigned grid = static_cast<unsigned>(std::max<int64_t>(1, std::min(chunks, most)));
          grad_norm_kernel<G, CAP><<<grid, kThreads, 0, s>>>(list, static_cast<NormWs*>(ws), first, last, max_norm, out);
          note_launch();
          return cuda_status(cudaGetLastError());
        });
  });
}

size_t tbe_adamw_workspace_size(void) { return 16; }

tbe_status tbe_adamw_update(const tbe_adamw_problem* prob, float lr, const float* clip, int64_t* step, void* ws,
                            size_t ws_bytes, void* stream) {
  tbe_status st = check_adamw(prob, false);
  if (st != TBE_OK) return st;
  if (!std::isfinite(lr) || step == nullptr || !is_aligned(step, 8) || !is_aligned(clip, 4)) return TBE_ERR_INVALID_ARG;
  if (ws == nullptr || ws_bytes < tbe_adamw_workspace_size()) return TBE_ERR_WORKSPACE;
  if (!is_aligned(ws, 16)) return TBE_ERR_INVALID_ARG;
  DeviceInfo dev;
  if ((st = device_info(&dev)) != TBE_OK) return st;
  AdamScalars sc;
  sc.beta1 = static_cast<float>(prob->beta1);
  sc.beta2 = static_cast<float>(prob->beta2);
  sc.one_minus_beta1 = static_cast<float>(1.0 - prob->beta1);
  sc.one_minus_beta2 = static_cast<float>(1.0 - prob->beta2);
  sc.log_beta1 = static_cast<float>(std::log(prob->beta1));  // beta = 0: -infinity, whose correction is 1
  sc.log_beta2 = static_cast<float>(std::log(prob->beta2));
  sc.eps = prob->eps;
  sc.lr = lr;
  sc.minus_zero = -0.f;
  sc.clip = clip;
  sc.step = step;
  sc.ticket = static_cast<uint32_t*>(ws);
  sc.advance = 0;
  bool master = false;
  for (int i = 0; i < prob->count; ++i) master = master || (prob->tensors[i].numel > 0 && prob->tensors[i].master != nullptr);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return with_type(prob->pdtype, [&](auto pt) {
    return with_type(prob->gdtype, [&](auto gt) {
      using P = typename decltype(pt)::type;
      using G = typename decltype(gt)::type;
      if constexpr (sizeof(P) == 2)
        if (master) return launch_adamw<P, G, true>(*prob, sc, dev, s);
      return launch_adamw<P, G, false>(*prob, sc, dev, s);
    });
  });
}

tbe_status tbe_adamw_state_values(const tbe_adamw_problem* prob, float* const* exp_avg_values,
                                  float* const* exp_avg_sq_values, void* stream) {
  tbe_status st = check_adamw(prob, true);
  if (st != TBE_OK) return st;
  if (prob->states != TBE_STATE_Q8) return TBE_ERR_INVALID_ARG;
  int64_t total = 0;
  for (int i = 0; i < prob->count; ++i) {
    if (prob->tensors[i].numel == 0) continue;
    total += prob->tensors[i].numel;
    if (exp_avg_values != nullptr && !is_aligned(exp_avg_values[i], 4)) return TBE_ERR_INVALID_ARG;
    if (exp_avg_sq_values != nullptr && !is_aligned(exp_avg_sq_values[i], 4)) return TBE_ERR_INVALID_ARG;
  }
  DeviceInfo dev;
  if ((st = device_info(&dev)) != TBE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return for_lists<ValuesEntry, kLargeValues>(
      prob->count, kStep, [&](int i) { return prob->tensors[i].numel; },
      [&](int i, ValuesEntry* e) {
        const tbe_dense_tensor& d = prob->tensors[i];
        float* m = exp_avg_values != nullptr ? exp_avg_values[i] : nullptr;
        float* v = exp_avg_sq_values != nullptr ? exp_avg_sq_values[i] : nullptr;
        const bool vec = is_aligned(d.exp_avg, 8) && is_aligned(d.exp_avg_sq, 8) && is_aligned(m, 16) && is_aligned(v, 16);
        *e = ValuesEntry{d.exp_avg, d.exp_avg_sq, d.exp_avg_scale, d.exp_avg_sq_scale, m, v, d.numel, vec, 0};
      },
      [&](auto& list, bool, bool) {
        constexpr int CAP = static_cast<int>(sizeof(list.e) / sizeof(list.e[0]));
        const uint32_t chunks = list.first[list.count];
        if (chunks == 0) return TBE_OK;
        q8_values_kernel<CAP><<<chunks, kThreads, 0, s>>>(list);
        note_launch();
        return cuda_status(cudaGetLastError());
      });
}

}  // extern "C"
