// k_softmax.cu -- softmax cross entropy over a table's rows without keeping the logits (tbe_tokens.h).
//
// Forward: z = scale * hidden weight^T a 256 x 256 tile at a time on the tensor cores (pair_mma.cuh); the epilogue reduces
// a tile's row to its maximum and sum of exponentials (in powers of 2), and picks the target's logit when its column
// comes by; a second kernel joins a row's parts (of a piece of the table's rows at a time where there are many).  Backward: for a
// piece of the table's rows at a time, the logits again, whose epilogue makes dz = c (p - onehot) in 16 bits, then
// dhidden += dz weight (summed over the pieces in fp32) and dweight = dz^T hidden, which is complete for the piece's rows.
#include <cfloat>

#include "pair_mma.cuh"
#include "tokens_common.cuh"

namespace tbe {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));  // 2 ulp; below 2^-126 it is 0
  return y;
}

// A token's target as a row of the table, or -1.
__device__ __forceinline__ int load_target(const void* targets, int itype, int64_t i, int64_t rows) {
  const int64_t t = itype == TBE_I32 ? ld_int<int32_t>(targets, i) : ld_int<int64_t>(targets, i);
  return t >= 0 && t < rows ? static_cast<int>(t) : -1;
}

// Rows of the selected tokens with those that fill up the last block of k, which are zeros.
__device__ __forceinline__ int filled(int live) { return (max(live, 1) + kPairK - 1) / kPairK * kPairK; }

// 32 bytes at p, which is aligned to them.
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// ------------------------------------------------------------------------------------------
// Epilogues
// ------------------------------------------------------------------------------------------
struct NoRow {
  template <typename A>
  __device__ __forceinline__ void load(const A&, const PairItem&, int) {}
};
struct NoState {};

// Goes through the N columns from `tmem` on, 32 at a time, the next ones requested while f(j, columns) works on the j-th.
template <int N, typename R, typename F>
__device__ __forceinline__ void each_columns(uint32_t tmem, R&& release, F&& f) {
  pair::Columns c[2];
  c[0].request(tmem);
#pragma unroll
  for (int j = 0; j < N / 32; ++j) {
    c[j & 1].landed();
    if (j + 1 < N / 32) c[(j + 1) & 1].request(tmem + (j + 1) * 32);
    else release();
    f(j, c[j & 1]);
  }
}

// A warp's 32 rows of 64 16-bit elements by way of shared memory, so that a store has whole 128-byte lines of 4 rows instead of a
// sector of each of 32: a thread puts 32 elements of its row (the `half`-th) there, and all of them store together; the
// pieces of 16 bytes are exchanged within a row by its number, so that no 8 rows meet in the same banks.
template <typename T>
__device__ __forceinline__ void stage_half(uint32_t staging, int lane, int half, const Pack<T, 16> (&p)[2]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t at = staging + lane * 128 + (((half * 4 + q) ^ (lane & 7)) << 4);
    const uint32_t* w = p[q / 2].w + q % 2 * 4;
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
  }
}
// f(row, c, piece): the 8 elements from column 8 c on of the warp's row `row`.
template <typename F>
__device__ __forceinline__ void unstage(uint32_t staging, int lane, F&& f) {
  __syncwarp();
  uint4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = i * 4 + lane / 8;
    shared_words<16>(staging + row * 128 + (((lane & 7) ^ (row & 7)) << 4), reinterpret_cast<uint32_t*>(&v[i]));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) f(i * 4 + lane / 8, lane & 7, v[i]);
  __syncwarp();
}

// A row's part of the softmax over half a tile's columns: {maximum of z in powers of 2, sum of 2^(z - maximum)}.  The maximum is the
// running one of 32 columns at a time, so that they need no second reading.  (8192 x 131072 x 1024 bf16, 98% of the tokens: the
// product takes 1229 us with it, 1754 TFLOP/s; the tensor cores bound it, the epilogue runs under the next tile's products.)
struct StatsJob {
  struct Args {
    const void* targets;
    const int* selected;   // NULL, or the targets of the tokens that count, one after the other
    const int* live;       // ... and how many they are
    float2* part;          // [parts][parts_rows]
    float* target_logit;   // [tokens]
    uint32_t* ticket;      // set to 0 for the kernel that joins the parts
    int64_t parts_rows, rows;
    int64_t first, end;    // the piece's rows of the table
    int tokens, itype;
    int carry;             // one tile of rows: a thread's parts are joined from tile to tile, one for each pair (or single CTA)
    int width;             // columns of a tile
    float scale, scale2;   // scale2 = scale * log2(e)
  };
  struct Row {
    int target;
    __device__ __forceinline__ void load(const Args& a, const PairItem& it, int row) {
      const int i = it.m * kPairM + row;
      target = -1;
      if (a.selected != nullptr) {
        if (i < *a.live) target = a.selected[i];
      } else if (i < a.tokens) {
        target = load_target(a.targets, a.itype, i, a.rows);
      }
    }
  };
  struct State {
    float top = -INFINITY, sum = 0.0f;
  };
  template <typename R>
  static __device__ __forceinline__ void tile(const Args& a, const Row& r, State& s, const PairItem& it, int row, int half, uint32_t tmem,
                                              uint32_t, R&& release) {
    const int i = it.m * kPairM + row;
    const int64_t col0 = a.first + static_cast<int64_t>(it.n) * a.width + half * 128;
    if (it.m == 0 && it.n == 0 && row == 0 && half == 0) *a.ticket = 0;
    const int most = min(128, a.width - half * 128);         // columns of this half, which may have none
    const int live = static_cast<int>(a.end - col0 < most ? a.end - col0 : most);
    const int64_t tl = r.target < 0 || r.target - col0 >= live ? -1 : r.target - col0;  // the target's column of this half
    float top = s.top, sum = s.sum;
    each_columns<128>(tmem, release, [&](int j, pair::Columns& c) {
      if (live < j * 32 + 32) {
#pragma unroll
        for (int k = 0; k < 32; ++k)
          if (j * 32 + k >= live) c.r[k] = 0xff800000u;  // past the table: no part in the softmax
      }
      float most = c.get(0);
#pragma unroll
      for (int k = 1; k < 32; ++k) most = fmaxf(most, c.get(k));
      const float next = fmaxf(top, most * a.scale2);
      const float ref = next == -INFINITY ? 0.0f : next;  // nothing but -inf so far: no inf - inf
      const F2 by(a.scale2), less(-ref);
      F2 s0(0.0f), s1(0.0f);
#pragma unroll
      for (int k = 0; k < 32; k += 4) {
        const F2 x = fma2(F2(c.get(k), c.get(k + 1)), by, less), y = fma2(F2(c.get(k + 2), c.get(k + 3)), by, less);
        s0 = s0 + F2(exp2_fast(x.lo()), exp2_fast(x.hi()));
        s1 = s1 + F2(exp2_fast(y.lo()), exp2_fast(y.hi()));
      }
      s0 = s0 + s1;
      sum = sum * exp2_fast(top - ref) + (s0.lo() + s0.hi());
      top = next;
      const int tj = tl >= j * 32 && tl < j * 32 + 32 ? static_cast<int>(tl) - j * 32 : -1;
      if (__any_sync(kFull, tj >= 0)) {
        float z = 0.0f;
#pragma unroll
        for (int k = 0; k < 32; ++k) z = tj == k ? c.get(k) : z;
        if (tj >= 0) a.target_logit[i] = z * a.scale;
      }
    });
    if (a.carry) s.top = top, s.sum = sum;
    else if (i < a.tokens) a.part[static_cast<int64_t>(it.n * 2 + half) * a.parts_rows + i] = make_float2(top, sum);
  }
  static __device__ __forceinline__ void finish(const Args& a, const State& s, int pair, int row, int half) {
    if (a.carry && row < a.tokens) a.part[static_cast<int64_t>(pair * 2 + half) * a.parts_rows + row] = make_float2(s.top, s.sum);
  }
};

// dz = c (p - onehot), times the factor that keeps it in 16 bits, for the selected tokens; zeros in the rows that fill up the
// last block of k.
template <typename T>
struct GradJob {
  struct Args {
    const float* meta;     // {factor, ...}
    const int* live;       // how many tokens are selected
    const float* coef;     // of the selected tokens
    const float* lse2;     // lse in powers of 2
    const int* target;     // -1 in the rows that fill up
    T* dz;                 // [blocks of 64 columns][dz_rows][64]
    int64_t dz_rows;
    int first, here;       // first row of the piece, rows of the table from there on
    float scale2;
  };
  struct Row {
    int target, rows;        // rows: of the warp's 32, how many there are
    float coef, lse2, factor;
    __device__ __forceinline__ void load(const Args& a, const PairItem& it, int row) {
      const int i = it.m * kPairM + row;
      target = -1, coef = 0.0f, lse2 = 0.0f;
      factor = a.meta[0];
      rows = filled(*a.live) - i + lane_id();
      if (i < filled(*a.live)) target = a.target[i], coef = a.coef[i], lse2 = a.lse2[i];
    }
  };
  using State = NoState;
  template <typename R>
  static __device__ __forceinline__ void tile(const Args& a, const Row& r, State&, const PairItem& it, int row, int half, uint32_t tmem,
                                              uint32_t staging, R&& release) {
    const int i = it.m * kPairM + row, lane = lane_id();
    const int col0 = it.n * 256 + half * 128, t = r.target;
    const int tl = t < 0 ? -1 : t - a.first - col0;
    const F2 g(r.coef * r.factor), by(a.scale2), less(-r.lse2);
    T* first = a.dz + (col0 / 64 * a.dz_rows + i - lane) * 64;   // the warp's first row
    each_columns<128>(tmem, release, [&](int j, pair::Columns& c) {
      const int tj = tl >= j * 32 && tl < j * 32 + 32 ? tl - j * 32 : -1;
      float v[32];
#pragma unroll
      for (int k = 0; k < 32; k += 2) {
        const F2 x = fma2(F2(c.get(k), c.get(k + 1)), by, less);
        v[k] = exp2_fast(x.lo()), v[k + 1] = exp2_fast(x.hi());
      }
      if (__any_sync(kFull, tj >= 0)) {
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] -= tj == k ? 1.0f : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < 32; k += 2) (F2(v[k], v[k + 1]) * g).get(v[k], v[k + 1]);
      if (__any_sync(kFull, t < 0) || col0 + j * 32 + 32 > a.here) {  // the last tiles: zeros, whatever the logits are
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = t < 0 || col0 + j * 32 + k >= a.here ? 0.0f : v[k];
      }
      Pack<T, 16> p[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float f[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) f[k] = v[q * 16 + k];
        p[q].set(f);
      }
      stage_half<T>(staging, lane, j & 1, p);
      if (j & 1) {
        T* dst = first + j / 2 * a.dz_rows * 64;
        unstage(staging, lane, [&](int x, int c, const uint4& piece) {
          if (x < r.rows) *reinterpret_cast<uint4*>(dst + x * 64 + c * 8) = piece;
        });
      }
    });
  }
  static __device__ __forceinline__ void finish(const Args&, const State&, int, int, int) {}
};

constexpr int kStageRow = 34;  // elements from one row to the next of rows that begin anywhere: 17 words, no bank twice

// A gradient's rows: the product times alpha, rounded.  (With dhidden's sums, 4864 x 19456 x 1024 bf16: 220 us, 1762 TFLOP/s, the tensor
// pipe active in 79% of the cycles.)
template <typename T>
struct OutJob {
  struct Args {
    const float* meta;     // {.., alpha}
    T* out;
    int64_t stride, first, rows;   // first row of the product in `out`, rows of out
    const int* place;      // NULL, or the row of out for each row of the product, of which there are *live
    const int* live;
    const float* down;     // NULL, or another factor for each row of the product
    int cols, width;       // width: of a tile
    int vec;               // rows allow 16-byte stores
  };
  struct Row {
    float alpha;
    int out;               // row of out, or -1
    __device__ __forceinline__ void load(const Args& a, const PairItem& it, int row) {
      alpha = a.meta[1];
      const int64_t i = a.first + static_cast<int64_t>(it.m) * kPairM + row;
      out = -1;
      if (a.place != nullptr) {
        if (i < *a.live) out = a.place[i];
        if (out >= 0 && a.down != nullptr) alpha *= a.down[i];
      } else if (i < a.rows) {
        out = static_cast<int>(i);
      }
    }
  };
  using State = NoState;
  template <typename R>
  static __device__ __forceinline__ void tile(const Args& a, const Row& r, State&, const PairItem& it, int row, int half, uint32_t tmem,
                                              uint32_t staging, R&& release) {
    const int col0 = it.n * a.width + half * 128, lane = lane_id();
    const int here = min(a.cols - col0, a.width - half * 128);   // columns of this half; the same for the whole warp
    each_columns<128>(tmem, release, [&](int j, pair::Columns& c) {
      const int left = here - j * 32;
      if (left <= 0) return;
      Pack<T, 16> p[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float f[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) f[k] = c.get(q * 16 + k) * r.alpha;
        p[q].set(f);
      }
      if (a.vec) {
        stage_half<T>(staging, lane, j & 1, p);
        if ((j & 1) || left <= 32) {
          T* dst = a.out + col0 + j / 2 * 64;
          const int cols = here - j / 2 * 64;
          unstage(staging, lane, [&](int x, int c, const uint4& piece) {
            const int to = __shfl_sync(kFull, r.out, x);
            if (to < 0 || c * 8 >= cols) return;
            if (c * 8 + 8 <= cols) *reinterpret_cast<uint4*>(dst + to * a.stride + c * 8) = piece;
            else reinterpret_cast<const Pack<T, 8>&>(piece).store_some(dst + to * a.stride + c * 8, cols - c * 8);
          });
        }
        return;
      }
      // Rows that begin anywhere: 32 elements of a row to a store.
      const uint32_t words = staging + lane * (kStageRow * 2), column = staging + lane * 2;
#pragma unroll
      for (int k = 0; k < 16; ++k) asm volatile("st.shared.u32 [%0], %1;" ::"r"(words + k * 4), "r"(p[k / 8].w[k % 8]) : "memory");
      __syncwarp();
      uint16_t v[32];
#pragma unroll
      for (int x = 0; x < 32; ++x) asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v[x]) : "r"(column + x * (kStageRow * 2)) : "memory");
      uint16_t* dst = reinterpret_cast<uint16_t*>(a.out) + col0 + j * 32 + lane;
#pragma unroll
      for (int x = 0; x < 32; ++x) {
        const int to = __shfl_sync(kFull, r.out, x);
        if (to >= 0 && lane < left) dst[to * a.stride] = v[x];
      }
      __syncwarp();
    });
  }
  static __device__ __forceinline__ void finish(const Args&, const State&, int, int, int) {}
};

// Sums in fp32, [split][rows][stride]: stored by the first piece, added to by the others (each by one thread, so that the order is
// the pieces').
struct SumJob {
  struct Args {
    float* sums;
    int64_t stride;        // a multiple of 8
    int rows, add, width;
  };
  using Row = NoRow;
  using State = NoState;
  template <typename R>
  static __device__ __forceinline__ void tile(const Args& a, const Row&, State&, const PairItem& it, int row, int half, uint32_t tmem, uint32_t,
                                              R&& release) {
    const int i = it.m * kPairM + row;
    const int col0 = it.n * a.width + half * 128;
    float* dst = a.sums + (static_cast<int64_t>(it.split) * a.rows + i) * a.stride + col0;
    each_columns<128>(tmem, release, [&](int j, pair::Columns& c) {
      if (half * 128 + j * 32 >= a.width) return;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (i >= a.rows || col0 + j * 32 + q * 8 >= a.stride) continue;
        if (a.add) {
#pragma unroll
          for (int x = 0; x < 2; ++x)
            asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(dst + j * 32 + q * 8 + x * 4), "f"(c.get(q * 8 + x * 4)),
                         "f"(c.get(q * 8 + x * 4 + 1)), "f"(c.get(q * 8 + x * 4 + 2)), "f"(c.get(q * 8 + x * 4 + 3))
                         : "memory");
        } else {
          uint32_t v[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = c.r[q * 8 + k];
          store32(dst + j * 32 + q * 8, v);
        }
      }
    });
  }
  static __device__ __forceinline__ void finish(const Args&, const State&, int, int, int) {}
};

// ------------------------------------------------------------------------------------------
// Before and after the products
// ------------------------------------------------------------------------------------------
// Rows copied to where TMA can address them (and, of hidden, those of the selected tokens one after the other, with zeros in the
// rows that fill up the last block of k), and zeros in the rows of dhidden of the tokens that are not selected.
struct CopyArgs {
  const int* live;      // with place and row: of loss_select_kernel; NULL for all tokens
  const int* place;
  const int* row;
  const uint16_t* hidden;
  const uint16_t* weight;
  uint16_t* hidden_copy;   // [.][dim_pad]
  uint16_t* weight_copy;   // NULL: none
  uint16_t* dhidden;       // NULL: none
  int64_t tokens, rows, hidden_stride, weight_stride, dhidden_stride;
  int dim, dim_pad;
  int at_once;             // the CTA that selects gathers the rows too
  // fp16 with a coefficient for each token; NULL otherwise
  const float* meta;       // {.., .., largest coefficient}
  float* coef;             // of the selected tokens: times 2^e
  float* down;             // 2^-e
  uint16_t* hidden_low;    // hidden_copy with each row times 2^-e
  int rows_log;            // ceil(log2(rows))
};

// 8 elements of a row from column c on, zeros past its end.
__device__ __forceinline__ uint4 row_piece(const uint16_t* src, int c, int dim, bool vec) {
  if (vec) return *reinterpret_cast<const uint4*>(src + c);
  uint32_t h[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) h[k] = c + k < dim ? src[c + k] : 0;
  return make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
}

// 8 elements to a thread, two at a time; from(r): the row of src that is row r of dst, or -1 for zeros.
template <typename F>
__device__ __forceinline__ void copy_rows(uint16_t* dst, const uint16_t* src, int64_t rows, int64_t stride, int dim, int dim_pad,
                                          int64_t t, int64_t n, F&& from) {
  const int groups = dim_pad / 8;
  const bool vec = reinterpret_cast<uintptr_t>(src) % 16 == 0 && dim % 8 == 0 && stride % 8 == 0;
  const int64_t total = rows * groups;
  for (int64_t x0 = t; x0 < total; x0 += 2 * n) {
    uint4 v[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t x = x0 + u * n;
      v[u] = make_uint4(0, 0, 0, 0);
      if (x >= total) continue;
      const int64_t r = total >> 32 == 0 ? static_cast<uint32_t>(x) / static_cast<uint32_t>(groups) : x / groups;
      const int64_t f = from(r);
      if (f >= 0) v[u] = row_piece(src + f * stride, static_cast<int>(x - r * groups) * 8, dim, vec);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (x0 + u * n < total) *reinterpret_cast<uint4*>(dst + (x0 + u * n) * 8) = v[u];
  }
}

// dz = c (p - onehot) has one factor for all tokens, which takes the largest |c| to 2^13, so that of a token whose c is 2^-k of it
// fp16 keeps all bits of probabilities down to 2^(k - 27) alone and nothing below 2^(k - 38): with 131072 classes a token of 10^-4
// would keep one or two levels of its p, and one of 10^-6 the term of its target only.  So tokens of a small c have a power of
// two of their own, 2^e: dz is that much larger, dhidden's row is divided by it again, and dweight's product takes hidden's row
// divided by it.  e = k + log2(rows) - 24 keeps all bits of p from 1 / (8 rows) on, is no more than k (dz stays below 2^14),
// and no more than takes the row's largest element to 2^-10: hidden's smaller ones lose what lies below 2^-25, 2^-15 of the
// largest.  A warp to a row.  (bf16 has fp32's range; e = 0 where all coefficients are alike, as a mean's.  1777 x 50021 x 301: 172.9
// us a gradient with it, 171.6 without; 200 x 1000 x 64 26.9 and 24.8.)
constexpr int kTopBits = 24, kLowestRow = -10, kMostUp = 25;
__device__ __forceinline__ void scale_rows(const CopyArgs& a, int live, float size, int64_t t, int64_t n) {
  const int lane = lane_id(), groups = a.dim_pad / 8;
  const bool vec = reinterpret_cast<uintptr_t>(a.hidden) % 16 == 0 && a.dim % 8 == 0 && a.hidden_stride % 8 == 0;
  for (int64_t r = t / kWarp; r < filled(live); r += n / kWarp) {
    uint16_t* dst = a.hidden_low + r * a.dim_pad;
    if (r >= live) {
      for (int g = lane; g < groups; g += kWarp) *reinterpret_cast<uint4*>(dst + g * 8) = make_uint4(0, 0, 0, 0);
      continue;
    }
    const uint16_t* src = a.hidden + a.place[r] * a.hidden_stride;
    const float c = a.coef[r];
    int e = 0;
    if (c != 0.0f && fabsf(c) <= size) {  // and finite: size is
      const int k = ilogbf(size) - ilogbf(c);
      e = min(k, k + a.rows_log - kTopBits);
    }
    if (e > 0) {
      float top = 0.0f;
      for (int i = lane; i < a.dim; i += kWarp) top = fmaxf(top, fabsf(__half2float(__ushort_as_half(src[i]))));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
      if (top > 0.0f && top < INFINITY) e = min(e, ilogbf(top) - kLowestRow);
      e = max(min(e, kMostUp), 0);
    } else {
      e = 0;
    }
    const float low = ldexpf(1.0f, -e);
    for (int g = lane; g < groups; g += kWarp) {
      uint4 v = row_piece(src, g * 8, a.dim, vec);
      if (e > 0) {
        Pack<__half, 8>& p = reinterpret_cast<Pack<__half, 8>&>(v);
        float f[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = p.get(k) * low;
        p.set(f);
      }
      *reinterpret_cast<uint4*>(dst + g * 8) = v;
    }
    __syncwarp();  // all lanes have read coef
    if (lane == 0) a.coef[r] = c * ldexpf(1.0f, e), a.down[r] = low;
  }
}

// The selected tokens' rows by n threads of which this is number t; place and row are written.  size: the largest coefficient.
__device__ __forceinline__ void gather_rows(const CopyArgs& a, int live, float size, int64_t t, int64_t n) {
  if (a.hidden_low != nullptr) scale_rows(a, live, size, t, n);
  copy_rows(a.hidden_copy, a.hidden, filled(live), a.hidden_stride, a.dim, a.dim_pad, t, n,
            [&](int64_t r) { return r < live ? static_cast<int64_t>(a.place[r]) : int64_t(-1); });
  if (a.dhidden == nullptr || live == a.tokens) return;
  for (int64_t i = t / kWarp; i < a.tokens; i += n / kWarp)
    if (a.row[i] < 0)
      for (int c = static_cast<int>(t % kWarp); c < a.dim; c += kWarp) a.dhidden[i * a.dhidden_stride + c] = 0;
}

// The tokens whose target is a row of the table, in their order, and what the products need of them: the others take no part in
// any product, so that a batch with a third of padding costs a third less, and what their hidden rows hold is not looked at.
struct SelectArgs {
  const void* targets;
  int64_t tokens, rows;
  int itype;
  int* live;         // how many
  int* place;        // [selected] the token
  int* target;       // [selected] its target; -1 in the rows that fill up the last block of k
  int* row;          // [tokens] where a token is among the selected, or -1
  // backward
  const float* lse;
  const float* dloss;
  const float* mean;
  float scale;
  float* meta;       // {factor of dz, scale over it, the coefficient that the factor is made for}
  float* coef;       // [selected]
  float* lse2;       // [selected] lse in powers of 2
  unsigned long long* stats;
};

__device__ __forceinline__ float coefficient(const SelectArgs& a, int64_t i, float mean) {
  return (a.dloss != nullptr ? a.dloss[i] : 1.0f) * mean;
}

constexpr int kSelectThreads = 1024;
constexpr int kCopyThreads = 256;

// One CTA, 4 tokens to a thread at a time, as the order of the tokens has to be kept and a scan over CTAs would take another launch (4864
// tokens: 13 us from cold caches, latency all of it); the others, where there are any, copy the table meanwhile.
template <bool BACKWARD>
__global__ void __launch_bounds__(kSelectThreads) loss_select_kernel(const __grid_constant__ SelectArgs a, const __grid_constant__ CopyArgs c) {
  constexpr int kEach = 4, kWarps = kSelectThreads / kWarp;
  __shared__ int s_count[kWarps];
  __shared__ float s_top[kWarps];
  const int lane = lane_id(), w = threadIdx.x / kWarp;
  may_follow();
  if (blockIdx.x > 0) {
    copy_rows(c.weight_copy, c.weight, c.rows, c.weight_stride, c.dim, c.dim_pad,
              static_cast<int64_t>(blockIdx.x - 1) * kSelectThreads + threadIdx.x, static_cast<int64_t>(gridDim.x - 1) * kSelectThreads,
              [](int64_t r) { return r; });
    return;
  }
  const float mean = BACKWARD && a.mean != nullptr ? a.mean[1] : 1.0f;
  int base = 0;
  float top = 0.0f;
  for (int64_t i0 = 0; i0 < a.tokens; i0 += kSelectThreads * kEach) {
    const int64_t i = i0 + threadIdx.x * kEach;
    int t[kEach], mine = 0;
#pragma unroll
    for (int k = 0; k < kEach; ++k) t[k] = i + k < a.tokens ? load_target(a.targets, a.itype, i + k, a.rows) : -1;
#pragma unroll
    for (int k = 0; k < kEach; ++k) mine += t[k] >= 0;
    int before = mine;
#pragma unroll
    for (int o = 1; o < kWarp; o <<= 1) {
      const int y = __shfl_up_sync(kFull, before, o);
      if (lane >= o) before += y;
    }
    if (lane == kWarp - 1) s_count[w] = before;
    __syncthreads();
    int sum = s_count[lane];
#pragma unroll
    for (int o = 1; o < kWarp; o <<= 1) {
      const int y = __shfl_up_sync(kFull, sum, o);
      if (lane >= o) sum += y;
    }
    const int all = __shfl_sync(kFull, sum, kWarps - 1), warps = __shfl_sync(kFull, sum, w > 0 ? w - 1 : 0);
    int j = base + before - mine + (w > 0 ? warps : 0);
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      if (i + k < a.tokens) a.row[i + k] = t[k] >= 0 ? j : -1;
      if (t[k] < 0) continue;
      a.place[j] = static_cast<int>(i + k);
      a.target[j] = t[k];
      if (BACKWARD) {
        const float c = coefficient(a, i + k, mean), size = fabsf(c);
        a.coef[j] = c;
        a.lse2[j] = a.lse[i + k] * kLog2e;
        if (size <= FLT_MAX) top = fmaxf(top, size);
      }
      ++j;
    }
    base += all;
    __syncthreads();
  }
  for (int j = base + threadIdx.x; j < filled(base); j += kSelectThreads) {
    a.target[j] = -1;
    if (BACKWARD) a.coef[j] = 0.0f, a.lse2[j] = 0.0f;
  }
  if (threadIdx.x == 0) *a.live = base;
  float size = 0.0f;
  if constexpr (BACKWARD) {
    // The largest finite coefficient takes dz to 2^13: |p - onehot| is at most 1, fp16 ends at 2^16, and what is 2^-27 of the
    // largest is still a normal number there (for tokens of far smaller coefficients see scale_rows).  Not a power of two: the
    // terms of the targets, 1 - p of their coefficient, are what most of the gradients is, and where all coefficients are the same (a mean's) they would all be rounded the same way.
    // So scaled they are 2^13 (1 - p).  (8192 x 131072 x 1024 bf16, 2-norm against 64 bits: 0.0029 by a power of two, 0.0017
    // so, which is the rounding of the gradients themselves.)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    if (lane == 0) s_top[w] = top;
    __syncthreads();
    top = s_top[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    size = top > 0.0f ? fmaxf(top, 0x1p-100f) : 8192.0f;
    if (threadIdx.x == 0) {
      a.meta[0] = 8192.0f / size;
      a.meta[1] = a.scale * (size / 8192.0f);
      a.meta[2] = size;
    }
  }
  if (c.at_once) {
    __syncthreads();
    gather_rows(c, base, size, threadIdx.x, kSelectThreads);
  }
}

__global__ void __launch_bounds__(kCopyThreads) loss_copy_kernel(const __grid_constant__ CopyArgs a) {
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x, n = static_cast<int64_t>(gridDim.x) * kCopyThreads;
  may_follow();
  wait_before();
  if (a.weight_copy != nullptr)
    copy_rows(a.weight_copy, a.weight, a.rows, a.weight_stride, a.dim, a.dim_pad, t, n, [](int64_t r) { return r; });
  if (a.live != nullptr) gather_rows(a, *a.live, a.meta != nullptr ? a.meta[2] : 0.0f, t, n);
  else copy_rows(a.hidden_copy, a.hidden, a.tokens, a.hidden_stride, a.dim, a.dim_pad, t, n, [](int64_t r) { return r; });
}

// Joins the parts of 32 tokens' rows, a lane to a token, the parts dealt out to the warps.
constexpr int kJoinThreads = 1024;

struct PartArgs {
  float2* part;            // [..][rows]: a token's parts, and behind them (number `before`) those of earlier pieces, joined
  int64_t rows;
  int parts, before;       // before: -1 for the first piece
};

// {maximum, sum of exponentials} of token j of this lane, in the first warp's threads; all of the block's call it.
__device__ __forceinline__ float2 join_parts(const PartArgs& a, int64_t j, bool counts) {
  constexpr int kWarps = kJoinThreads / kWarp;
  __shared__ float2 s_part[kWarps][kWarp + 1];
  const int lane = lane_id(), w = threadIdx.x / kWarp;
  float top = -INFINITY, sum = 0.0f;
  auto add = [&](const float2& v) {
    const float next = fmaxf(top, v.x), ref = next == -INFINITY ? 0.0f : next;
    sum = sum * exp2_fast(top - ref) + v.y * exp2_fast(v.x - ref);
    top = next;
  };
  if (counts) {
#pragma unroll 8
    for (int p = w; p < a.parts; p += kWarps) add(a.part[p * a.rows + j]);
    if (a.before >= 0 && w == 0) add(a.part[a.before * a.rows + j]);
  }
  s_part[w][lane] = make_float2(top, sum);
  __syncthreads();
  if (w != 0) return make_float2(0.0f, 0.0f);
  top = -INFINITY;
#pragma unroll
  for (int k = 0; k < kWarps; ++k) top = fmaxf(top, s_part[k][lane].x);
  const float ref = top == -INFINITY ? 0.0f : top;
  float s4[4] = {};
#pragma unroll
  for (int k = 0; k < kWarps; ++k) s4[k % 4] += s_part[k][lane].y * exp2_fast(s_part[k][lane].x - ref);
  return make_float2(top, (s4[0] + s4[1]) + (s4[2] + s4[3]));
}

// Between two pieces of the table: a token's parts to the one behind them.
__global__ void __launch_bounds__(kJoinThreads) loss_fold_kernel(const __grid_constant__ PartArgs a, const int* live, int64_t tokens, int to) {
  wait_before();
  const int64_t j = static_cast<int64_t>(blockIdx.x) * kWarp + lane_id();
  const bool counts = j < (live != nullptr ? *live : tokens);
  const float2 v = join_parts(a, j, counts);
  if (threadIdx.x < kWarp && counts) a.part[to * a.rows + j] = v;
}

// A token's loss from all of its parts; the last block adds up the losses.  (8192 tokens of 1024 parts: 22 us, 67 MB; 16 of 304: 7,
// latency.)
struct BlockSum {
  double loss;
  long long count;
};

struct JoinArgs {
  PartArgs parts;
  const float* target_logit;
  const void* targets;
  const int* row;          // NULL, or where a token is among the selected
  float* loss;
  float* lse;
  float* mean;
  BlockSum* sums;
  uint32_t* ticket;
  int64_t tokens, rows;
  int itype;
  unsigned long long* stats;
};

__device__ __forceinline__ void write_mean(float* mean, double d, long long n) {
  mean[0] = n > 0 ? static_cast<float>(d / static_cast<double>(n)) : 0.0f;
  mean[1] = n > 0 ? static_cast<float>(1.0 / static_cast<double>(n)) : 0.0f;
}

__global__ void __launch_bounds__(kJoinThreads) loss_join_kernel(const __grid_constant__ JoinArgs a) {
  constexpr int kWarps = kJoinThreads / kWarp;
  __shared__ double s_loss[kWarps];
  __shared__ long long s_count[kWarps];
  __shared__ bool s_last;
  const int lane = lane_id(), w = threadIdx.x / kWarp;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kWarp + lane;
  wait_before();
  const int64_t raw = i >= a.tokens ? -1 : a.itype == TBE_I32 ? ld_int<int32_t>(a.targets, i) : ld_int<int64_t>(a.targets, i);
  const bool counts = raw >= 0 && raw < a.rows;
  const int64_t j = !counts ? 0 : a.row != nullptr ? a.row[i] : i;
  const float logit = w == 0 && counts ? a.target_logit[j] : 0.0f;
  const float2 all = join_parts(a.parts, j, counts);
  if (w == 0) {
    const float lse = counts ? ((all.x == -INFINITY ? 0.0f : all.x) + log2f(all.y)) * kLn2 : 0.0f;
    const float loss = counts ? lse - logit : 0.0f;
    if (i < a.tokens) a.lse[i] = lse, a.loss[i] = loss;
    const unsigned bad = __ballot_sync(kFull, raw >= a.rows);
    const unsigned live = __ballot_sync(kFull, counts);
    double d = loss;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(kFull, d, o);
    if (lane == 0) {
      stat_add(a.stats, TBE_STAT_UNREPAIRED, __popc(bad));
      s_last = false;
      if (gridDim.x == 1) {
        write_mean(a.mean, d, __popc(live));
      } else {
        a.sums[blockIdx.x] = BlockSum{d, __popc(live)};
        __threadfence();
        s_last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
        __threadfence();
      }
    }
  }
  __syncthreads();
  if (!s_last) return;
  double d = 0.0;
  long long n = 0;
  for (unsigned b = threadIdx.x; b < gridDim.x; b += kJoinThreads) d += __ldcg(&a.sums[b].loss), n += __ldcg(&a.sums[b].count);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(kFull, d, o), n += __shfl_xor_sync(kFull, n, o);
  if (lane == 0) s_loss[w] = d, s_count[w] = n;
  __syncthreads();
  if (w != 0) return;
  d = s_loss[lane], n = s_count[lane];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(kFull, d, o), n += __shfl_xor_sync(kFull, n, o);
  if (lane == 0) write_mean(a.mean, d, n);
}

// A gradient's rows = alpha * the sums of all splits: dhidden's to the selected tokens' rows, dweight's as they are.  (8192 x 1024: 10 us,
// 50 MB.)
template <typename T>
struct FinishArgs {
  const float* sums;
  const float* meta;
  const int* live;         // NULL: all rows
  const int* live_k;       // NULL, or the length of the sums, of whose blocks there may be fewer than splits
  const int* place;
  const float* down;       // NULL, or another factor for each selected row
  T* out;
  int64_t rows, sums_stride, stride;
  int splits, cols, vec;
};

template <typename T>
__global__ void __launch_bounds__(256) loss_finish_kernel(const __grid_constant__ FinishArgs<T> a) {
  wait_before();
  const int per_row = static_cast<int>(a.sums_stride / 8);
  const int64_t total = (a.live != nullptr ? static_cast<int64_t>(*a.live) : a.rows) * per_row;
  const int splits = a.live_k != nullptr ? min(a.splits, (max(*a.live_k, 1) + kPairK - 1) / kPairK) : a.splits;
  const float alpha = a.meta[1];
  for (int64_t x = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; x < total; x += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t i = total >> 32 == 0 ? static_cast<uint32_t>(x) / static_cast<uint32_t>(per_row) : x / per_row;
    const int col = static_cast<int>(x - i * per_row) * 8;
    const int64_t to = a.live != nullptr ? a.place[i] : i;
    float f[8] = {};
#pragma unroll 8
    for (int s = 0; s < splits; ++s) {
      const float4* p = reinterpret_cast<const float4*>(a.sums + (s * a.rows + i) * a.sums_stride + col);
      const float4 u = p[0], v = p[1];
      f[0] += u.x, f[1] += u.y, f[2] += u.z, f[3] += u.w, f[4] += v.x, f[5] += v.y, f[6] += v.z, f[7] += v.w;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] *= a.down != nullptr ? alpha * a.down[i] : alpha;
    Pack<T, 8> p;
    p.set(f);
    T* dst = a.out + to * a.stride + col;
    if (a.vec && col + 8 <= a.cols) p.store(dst);
    else p.store_some(dst, a.cols - col);
  }
}

// ------------------------------------------------------------------------------------------
// Host
// ------------------------------------------------------------------------------------------
template <int AM, int CTAS, class P0, class P1>
tbe_status launch_pair(const typename P0::Args& p0, const typename P1::Args& p1, int64_t items, const LossArgs& a, const DeviceInfo& dev,
                       cudaStream_t s) {
  auto* kernel = pair_mma_kernel<AM, CTAS, P0, P1>;
  constexpr size_t smem = PairTile<AM, CTAS>::kSmem;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem(kernel, smem, allowed);
  if (e != cudaSuccess) return cuda_status(e);
  const int64_t pairs = items < dev.sms / CTAS ? items : dev.sms / CTAS;
  return cuda_status(launch_after(kernel, static_cast<unsigned>(CTAS * pairs), kPairThreads, smem, s, p0, p1, a.stats));
}

template <int AM, int CTAS, class P>
tbe_status launch_product(const typename P::Args& p, const LossArgs& a, const DeviceInfo& dev, cudaStream_t s) {
  return launch_pair<AM, CTAS, P, NoProduct>(p, NoProduct::Args{}, p.g.items(), a, dev, s);
}

tbe_status launch_copy(const CopyArgs& p, const DeviceInfo& dev, cudaStream_t s) {
  const int64_t rows = p.tokens + (p.weight_copy != nullptr ? p.rows : 0);
  int64_t blocks = ceil_div(rows * (p.dim_pad / 8), 2 * kCopyThreads);
  if (p.hidden_low != nullptr && blocks < ceil_div(p.tokens, kCopyThreads / kWarp)) blocks = ceil_div(p.tokens, kCopyThreads / kWarp);
  if (blocks > dev.sms * 8) blocks = dev.sms * 8;
  return cuda_status(launch_after(loss_copy_kernel, static_cast<unsigned>(blocks), kCopyThreads, 0, s, p));
}

// Elements of hidden up to which the CTA that selects gathers them as well: 16 to a thread (and 4 rows to a warp where rows have a factor
// of their own), which takes less than a launch.  (us a gradient of 1000 rows x 64, so and by a launch: 64 tokens 24.9 and 26.6, 256
// tokens 25.3 and 26.8, 512 tokens 28.6 and 27.6, 1024 tokens 34.6 and 29.8.)
constexpr int64_t kAtOnce = 16 * kSelectThreads;

// Selects the tokens and gathers their rows.  The table's copy, where c has one, is made beside the selection.
template <bool BACKWARD>
tbe_status launch_select(const SelectArgs& p, CopyArgs& c, const DeviceInfo& dev, cudaStream_t s) {
  c.live = p.live, c.place = p.place, c.row = p.row;
  c.at_once = c.tokens * c.dim_pad <= kAtOnce && (c.hidden_low == nullptr || c.tokens <= 4 * (kSelectThreads / kWarp));
  int64_t blocks = c.weight_copy == nullptr ? 0 : ceil_div(c.rows * (c.dim_pad / 8), 2 * kSelectThreads);
  if (blocks > dev.sms * 2 - 1) blocks = dev.sms * 2 - 1;
  loss_select_kernel<BACKWARD><<<static_cast<unsigned>(1 + blocks), kSelectThreads, 0, s>>>(p, c);
  note_launch();
  const tbe_status st = cuda_status(cudaGetLastError());
  c.weight_copy = nullptr;
  return st != TBE_OK || c.at_once ? st : launch_copy(c, dev, s);
}

size_t place(size_t* at, int64_t bytes) {
  const size_t here = *at;
  *at += static_cast<size_t>(round_up(bytes, 256));
  return here;
}

// Rows that allow 16-byte stores.
int whole_stores(const void* p, int64_t stride) { return stride % 8 == 0 && is_aligned(p, 16); }

// Bytes of the softmax's parts that a piece of the table may take in the forward, 8 for each token and 128 rows: up to 2^32 logits are
// one piece.  (131072 x 131072 would take 1 GB in one, where the logits are not to be kept.)
constexpr int64_t kPartBytes = int64_t(256) << 20;

// Bytes of dz that a piece of the table may take.
constexpr int64_t kPieceBytes = int64_t(512) << 20;

// The forward selects the tokens that count from here on, which takes two launches, 7 to 10 us, and saves their share of the products;
// fewer are one to four tiles of rows.  (us a call, 1024 tokens, all rows and the selected ones: 131072 x 1024 186 and 151 with a third
// of padding, 175 and 185 with 2%; 50000 x 256 36.3 and 37.4, 36.2 and 43.6; 600 tokens with a third 29.9 and 33.1.)
constexpr int64_t kSelectTokens = 1024;

// Rows of A that a CTA copies in the forward's product of at most as many tokens.  (16 x 131072 x 1024: 56 us by 128, 47 by 32; beyond
// that single CTAs copy 128 up to 128 tokens, against pairs: 128 x 131072 x 1024 50.8 us and 55.4.)
constexpr int kFewTokens = 32;

// Blocks of k up to which one pair makes a whole tile of dhidden, with no sums to join after it.  (us a gradient, so and by sums: 4096 x
// 1536 x 1024 72 and 81, 300 x 1536 x 128 31.1 and 30.8, 300 x 2000 x 128 33.3 and 31.0, 300 x 3000 x 128 38.8 and 32.)
constexpr int kDirectBlocks = 24;

// Columns of a tile of few tokens' logits, which take as long as their rows of the table take through memory: the width with which
// the CTA with the most tiles has the fewest rows (131072 rows to 152 CTAs: 4 tiles of 224 each and not 4 of 256).
int even_width(int64_t rows, int workers) {
  int best = 256;
  int64_t least = INT64_MAX;
  for (int width = 256; width >= 128; width -= 32) {
    const int64_t most = ceil_div(ceil_div(rows, width), workers) * width;
    if (most < least) least = most, best = width;
  }
  return best;
}

// Columns of a tile of the gradients' products: as many tiles as 256 columns each would be, no wider than the rows need.
int gradient_width(int dim) { return static_cast<int>(round_up(ceil_div(dim, ceil_div(dim, 256)), 32)); }

template <typename T>
tbe_status loss_backward(const LossArgs& a, const LossBackwardLayout& l, const CUtensorMap* maps, const float* down, void* dhidden,
                         void* dweight, char* ws, const DeviceInfo& dev, cudaStream_t s) {
  const bool bf16 = a.dtype == TBE_BF16;
  const int N = static_cast<int>(a.tokens), m_tiles = static_cast<int>(ceil_div(N, kPairM));
  const int width = gradient_width(a.dim);
  const int d_tiles = static_cast<int>(ceil_div(a.dim, width)), d_blocks = static_cast<int>(ceil_div(a.dim, kPairK));
  float* meta = reinterpret_cast<float*>(ws + l.meta);
  const int* live = reinterpret_cast<const int*>(ws + l.live);
  const int* placed = reinterpret_cast<const int*>(ws + l.place);
  T* dz = reinterpret_cast<T*>(ws + l.dz);
  float* sums = reinterpret_cast<float*>(ws + l.sums);
  using Grad = Product<false, false, GradJob<T>>;
  using Sum = Product<false, true, SumJob>;
  using Direct = Product<false, true, OutJob<T>>;
  using Out = Product<true, true, OutJob<T>>;
  using SumOut = Product<true, true, SumJob>;
  tbe_status st;
  for (int64_t first = 0; first < a.rows; first += l.piece) {
    const int here = static_cast<int>(a.rows - first < l.piece ? a.rows - first : l.piece);
    const int v_tiles = static_cast<int>(ceil_div(here, 256)), f = static_cast<int>(first);
    typename Grad::Args ga{maps[0], maps[1],
                           PairShape{m_tiles, v_tiles, 1, d_blocks, 0, 0, f, 0, 256, 0, pair_idesc(bf16, 256, false, false), live, nullptr, 0},
                           {meta, live, reinterpret_cast<const float*>(ws + l.coef), reinterpret_cast<const float*>(ws + l.lse2),
                            reinterpret_cast<const int*>(ws + l.target), dz, l.dz_rows, f, here, a.scale * kLog2e}};
    if ((st = launch_product<128, 2, Grad>(ga, a, dev, s)) != TBE_OK) return st;
    // dhidden += dz [tokens, piece] by weight [piece, dim];  dweight = dz^T [piece, tokens] by hidden [tokens, dim]
    const PairShape sum{m_tiles, d_tiles, l.splits, static_cast<int>(ceil_div(here, kPairK)), 0, 0, 0, f, width, 0, pair_idesc(bf16, width, false, true),
                        live, nullptr, static_cast<int>(l.dz_rows)};
    typename Out::Args oa{maps[4], maps[5],
                          PairShape{v_tiles, d_tiles, 1, static_cast<int>(ceil_div(N, kPairK)), 0, 0, 0, 0, width, 1, pair_idesc(bf16, width, true, true),
                                    nullptr, live, static_cast<int>(l.dz_rows)},
                          {meta, static_cast<T*>(dweight), a.dweight_stride, first, a.rows, nullptr, nullptr, nullptr, a.dim, width,
                           whole_stores(dweight, a.dweight_stride)}};
    const int64_t items = static_cast<int64_t>(sum.items()) + oa.g.items();
    if (l.direct) {
      typename Direct::Args da{maps[2], maps[3], sum,
                               {meta, static_cast<T*>(dhidden), a.dhidden_stride, 0, a.tokens, placed, live, down, a.dim, width,
                                whole_stores(dhidden, a.dhidden_stride)}};
      if ((st = launch_pair<128, 2, Direct, Out>(da, oa, items, a, dev, s)) != TBE_OK) return st;
      continue;
    }
    Sum::Args sa{maps[2], maps[3], sum, {sums, l.dim_pad, N, first > 0, width}};
    if (l.out_splits > 1) {
      SumOut::Args wa{maps[4], maps[5], oa.g, {reinterpret_cast<float*>(ws + l.out_sums), l.dim_pad, here, 0, width}};
      wa.g.splits = l.out_splits;
      st = launch_pair<128, 2, Sum, SumOut>(sa, wa, static_cast<int64_t>(sum.items()) + wa.g.items(), a, dev, s);
    } else {
      st = launch_pair<128, 2, Sum, Out>(sa, oa, items, a, dev, s);
    }
    if (st != TBE_OK) return st;
  }
  if (l.direct) return TBE_OK;
  auto finish = [&](const float* from, const int* selected, void* out, int64_t rows, int64_t stride, int splits) {
    const bool by_token = selected != nullptr;
    const FinishArgs<T> fa{from, meta, selected, by_token ? nullptr : live, placed, by_token ? down : nullptr, static_cast<T*>(out), rows,
                           l.dim_pad, stride, splits, a.dim, whole_stores(out, stride)};
    int64_t blocks = ceil_div(rows * (l.dim_pad / 8), 256);
    if (blocks > dev.sms * 8) blocks = dev.sms * 8;
    return cuda_status(launch_after(loss_finish_kernel<T>, static_cast<unsigned>(blocks), 256, 0, s, fa));
  };
  st = finish(sums, live, dhidden, a.tokens, a.dhidden_stride, l.splits);
  if (st != TBE_OK || l.out_splits <= 1) return st;
  return finish(reinterpret_cast<float*>(ws + l.out_sums), nullptr, dweight, a.rows, a.dweight_stride, l.out_splits);
}

}  // namespace

bool encode_operand(CUtensorMap* map, const void* p, bool bf16, int64_t inner, int64_t outer, int64_t stride, int box_outer) {
  const auto encode = tensor_map_encoder();
  if (encode == nullptr) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[2] = {kPairK, static_cast<cuuint32_t>(box_outer)};
  const cuuint32_t estr[2] = {1, 1};
  return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(p), dims, strides,
                box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

LossForwardLayout loss_forward_layout(const LossArgs& a) {
  LossForwardLayout l{};
  size_t at = 0;
  const int64_t dim_pad = round_up(a.dim, 8);
  l.parts_rows = round_up(a.tokens > 0 ? a.tokens : 1, 32);
  int64_t most = kPartBytes / 16 / l.parts_rows;   // tiles of 256 rows, two parts to each; fewer are used where the pairs join theirs
  if (most < 1) most = 1;
  const int64_t tiles = ceil_div(a.rows, 256);
  l.piece = ceil_div(tiles, ceil_div(tiles, most)) * 256;
  l.parts = static_cast<int>(l.piece / 128);
  // As much as any smaller number of tokens may need.
  const int64_t whole = tiles * 16 * l.parts_rows, least = 16 * l.parts_rows, capped = least > kPartBytes ? least : kPartBytes;
  l.part = place(&at, (whole < capped ? whole : capped) + 8 * l.parts_rows);
  l.logit = place(&at, a.tokens * 4);
  l.ticket = place(&at, 256 + ceil_div(a.tokens, kWarp) * static_cast<int64_t>(sizeof(BlockSum)));  // and the blocks' sums
  l.live = place(&at, 4);
  l.place = place(&at, a.tokens * 4);
  l.target = place(&at, round_up(a.tokens, kPairM) * 4);
  l.row = place(&at, a.tokens * 4);
  l.hidden = place(&at, round_up(a.tokens, kPairM) * dim_pad * 2);
  l.weight = place(&at, a.copy_weight ? a.rows * dim_pad * 2 : 0);
  l.total = at;
  return l;
}

LossBackwardLayout loss_backward_layout(const LossArgs& a, const DeviceInfo& dev) {
  LossBackwardLayout l{};
  size_t at = 0;
  l.dim_pad = round_up(a.dim, 8);
  int64_t most = kPieceBytes / 2 / round_up(a.tokens > 0 ? a.tokens : 1, kPairM) / 256 * 256;
  if (most < 256) most = 256;
  if (most > (1 << 30)) most = 1 << 30;
  const int64_t pieces = ceil_div(a.rows, most);
  l.piece = round_up(ceil_div(a.rows, pieces), 256);
  const int64_t d_tiles = ceil_div(a.dim, gradient_width(a.dim)), blocks = ceil_div(l.piece, kPairK);
  const int64_t tiles = ceil_div(a.tokens, kPairM) * d_tiles, pairs = dev.sms / 2;
  // Where the table has few tiles, the sums over the tokens of dweight are split as well: no tile shall take more than twice a pair's
  // share (14732 x 17 x 48 bf16: 116 us by one pair's sum, 60 split).
  const int64_t out_tiles = ceil_div(l.piece, 256) * d_tiles, out_blocks = ceil_div(a.tokens, kPairK);
  const int64_t share = ceil_div(tiles * blocks + out_tiles * out_blocks, pairs);
  l.out_splits = 1;
  if (a.rows <= l.piece && out_blocks > 16 && out_blocks > 2 * share) {
    const int64_t n = ceil_div(out_blocks, share < 4 ? 4 : share), most = ceil_div(2 * pairs, out_tiles);
    l.out_splits = static_cast<int>(n < most ? n : most);
  }
  l.direct = a.rows <= l.piece && ceil_div(a.rows, kPairK) <= kDirectBlocks && l.out_splits == 1;
  l.splits = 1;
  if (!l.direct) {  // none of the tiles of dhidden's long sums shall take more than half of a pair's share of a piece's blocks
    const int64_t all = tiles * blocks + ceil_div(l.piece, 256) * d_tiles * ceil_div(a.tokens, kPairK);
    int64_t splits = all > 0 ? ceil_div(2 * pairs * blocks, all) : 1;
    if (splits > blocks / 2) splits = blocks / 2;
    // the last piece may be shorter: every split has to have a part of it
    const int64_t last = ceil_div(a.rows - (ceil_div(a.rows, l.piece) - 1) * l.piece, kPairK);
    if (splits > last) splits = last;
    if (splits > 1) l.splits = static_cast<int>(splits);
  }
  l.meta = place(&at, 16);
  l.live = place(&at, 4);
  l.place = place(&at, a.tokens * 4);
  l.dz_rows = round_up(a.tokens, kPairM);
  l.target = place(&at, l.dz_rows * 4);
  l.row = place(&at, a.tokens * 4);
  l.coef = place(&at, l.dz_rows * 4);
  l.down = place(&at, l.dz_rows * 4);
  l.lse2 = place(&at, l.dz_rows * 4);
  l.hidden = place(&at, l.dz_rows * l.dim_pad * 2);
  l.hidden_low = place(&at, a.dtype == TBE_F16 ? l.dz_rows * l.dim_pad * 2 : 0);
  l.weight = place(&at, a.copy_weight ? a.rows * l.dim_pad * 2 : 0);
  // What these two take varies with the number of tokens both ways: as much as any smaller number may need, so that a
  // workspace for the largest call serves every call.
  const int64_t whole = l.dz_rows * round_up(a.rows, 256) * 2, least = l.dz_rows * 512;
  const int64_t capped = least > kPieceBytes ? least : kPieceBytes;
  l.dz = place(&at, whole < capped ? whole : capped);
  // splits * tiles < 2 pairs + tiles; out_splits * out_tiles < 2 pairs + out_tiles, and those are at most pairs / 2 tiles, as
  // twice their blocks are more than a share
  const int64_t tile = int64_t(kPairM) * 256, row = (2 * pairs + 1) * l.dim_pad;
  const int64_t split = 2 * pairs * tile + a.tokens * l.dim_pad, out_split = 3 * pairs * tile;
  l.sums = place(&at, (split < a.tokens * row ? split : a.tokens * row) * 4);
  l.out_sums = place(&at, (out_split < a.rows * row ? out_split : a.rows * row) * 4);
  l.total = at;
  return l;
}

tbe_status launch_loss_forward(const LossArgs& a, const LossForwardLayout& l, const void* hidden, const void* weight,
                               const void* targets, float* loss, float* lse, float* mean, char* ws, const DeviceInfo& dev,
                               cudaStream_t s) {
  if (a.tokens == 0) return cuda_status(cudaMemsetAsync(mean, 0, 8, s));
  const bool bf16 = a.dtype == TBE_BF16, select = a.tokens >= kSelectTokens;
  const int dim_pad = static_cast<int>(round_up(a.dim, 8));
  int* live = reinterpret_cast<int*>(ws + l.live);
  int* selected = reinterpret_cast<int*>(ws + l.target);
  int* row = reinterpret_cast<int*>(ws + l.row);
  tbe_status st;
  int64_t hs = a.hidden_stride, wst = a.weight_stride;
  if (select || a.copy_hidden || a.copy_weight) {
    CopyArgs c{};
    c.hidden = static_cast<const uint16_t*>(hidden), c.weight = static_cast<const uint16_t*>(weight);
    c.hidden_copy = reinterpret_cast<uint16_t*>(ws + l.hidden);
    if (a.copy_weight) c.weight_copy = reinterpret_cast<uint16_t*>(ws + l.weight);
    c.tokens = a.tokens, c.rows = a.rows, c.hidden_stride = a.hidden_stride, c.weight_stride = a.weight_stride;
    c.dim = a.dim, c.dim_pad = dim_pad;
    if (select) {
      SelectArgs p{};
      p.targets = targets, p.tokens = a.tokens, p.rows = a.rows, p.itype = a.itype;
      p.live = live, p.place = reinterpret_cast<int*>(ws + l.place), p.target = selected, p.row = row;
      st = launch_select<false>(p, c, dev, s);
    } else {
      st = launch_copy(c, dev, s);
    }
    if (st != TBE_OK) return st;
    hidden = ws + l.hidden, hs = dim_pad;
    if (a.copy_weight) weight = ws + l.weight, wst = dim_pad;
  }
  const bool few = a.tokens <= kFewTokens, solo = a.tokens <= 128;
  const int m_tiles = static_cast<int>(ceil_div(a.tokens, kPairM)), workers = solo ? dev.sms : dev.sms / 2;
  uint32_t* ticket = reinterpret_cast<uint32_t*>(ws + l.ticket);
  float2* part = reinterpret_cast<float2*>(ws + l.part);
  float* target_logit = reinterpret_cast<float*>(ws + l.logit);
  CUtensorMap ma, mb;
  if (!encode_operand(&ma, hidden, bf16, a.dim, a.tokens, hs, few ? kFewTokens : 128)) return cuda_status(cudaErrorInvalidValue);
  using Stats = Product<false, false, StatsJob>;
  const unsigned blocks = static_cast<unsigned>(ceil_div(a.tokens, kWarp));
  for (int64_t first = 0; first < a.rows; first += l.piece) {
    const int64_t here = a.rows - first < l.piece ? a.rows - first : l.piece, tiles = ceil_div(here, 256);
    const bool carry = m_tiles == 1 && tiles > workers, last = first + here == a.rows;
    const int width = carry && solo ? even_width(here, workers) : 256, v_tiles = static_cast<int>(ceil_div(here, width));
    if (!encode_operand(&mb, weight, bf16, a.dim, a.rows, wst, solo ? width : 128)) return cuda_status(cudaErrorInvalidValue);
    const Stats::Args sa{ma, mb,
                         PairShape{m_tiles, v_tiles, 1, static_cast<int>(ceil_div(a.dim, kPairK)), 0, 0, static_cast<int>(first), 0, width, 0,
                                   pair_idesc(bf16, width, false, false, solo ? 1 : 2), select ? live : nullptr, nullptr, 0},
                         {targets, select ? selected : nullptr, live, part, target_logit, ticket, l.parts_rows, a.rows, first, first + here,
                          static_cast<int>(a.tokens), a.itype, carry, width, a.scale, a.scale * kLog2e}};
    st = few    ? launch_product<kFewTokens, 1, Stats>(sa, a, dev, s)
         : solo ? launch_product<128, 1, Stats>(sa, a, dev, s)
                : launch_product<128, 2, Stats>(sa, a, dev, s);
    if (st != TBE_OK) return st;
    const PartArgs parts{part, l.parts_rows, carry ? 2 * workers : static_cast<int>(2 * tiles), first > 0 ? l.parts : -1};
    if (!last) {
      const int* counting = select ? live : nullptr;
      st = cuda_status(launch_after(loss_fold_kernel, blocks, kJoinThreads, 0, s, parts, counting, a.tokens, l.parts));
      if (st != TBE_OK) return st;
      continue;
    }
    const JoinArgs ja{parts, target_logit, targets, select ? row : nullptr, loss, lse, mean, reinterpret_cast<BlockSum*>(ws + l.ticket + 256), ticket,
                      a.tokens, a.rows, a.itype, a.stats};
    st = cuda_status(launch_after(loss_join_kernel, blocks, kJoinThreads, 0, s, ja));
  }
  return st;
}

tbe_status launch_loss_backward(const LossArgs& a, const LossBackwardLayout& l, const void* hidden, const void* weight,
                                const void* targets, const float* lse, const float* dloss, const float* mean, void* dhidden,
                                void* dweight, char* ws, const DeviceInfo& dev, cudaStream_t s) {
  if (a.tokens == 0)  // a sum over no tokens
    return cuda_status(cudaMemset2DAsync(dweight, a.dweight_stride * 2, 0, static_cast<size_t>(a.dim) * 2, a.rows, s));
  const bool bf16 = a.dtype == TBE_BF16;
  SelectArgs p{};
  p.targets = targets, p.tokens = a.tokens, p.rows = a.rows, p.itype = a.itype;
  p.live = reinterpret_cast<int*>(ws + l.live), p.place = reinterpret_cast<int*>(ws + l.place);
  p.target = reinterpret_cast<int*>(ws + l.target), p.row = reinterpret_cast<int*>(ws + l.row);
  p.lse = lse, p.dloss = dloss, p.mean = mean, p.scale = a.scale;
  p.meta = reinterpret_cast<float*>(ws + l.meta), p.coef = reinterpret_cast<float*>(ws + l.coef);
  p.lse2 = reinterpret_cast<float*>(ws + l.lse2);
  CopyArgs c{};
  c.hidden = static_cast<const uint16_t*>(hidden), c.weight = static_cast<const uint16_t*>(weight);
  c.hidden_copy = reinterpret_cast<uint16_t*>(ws + l.hidden);
  if (a.copy_weight) c.weight_copy = reinterpret_cast<uint16_t*>(ws + l.weight);
  c.dhidden = static_cast<uint16_t*>(dhidden);
  c.tokens = a.tokens, c.rows = a.rows, c.hidden_stride = a.hidden_stride, c.weight_stride = a.weight_stride;
  c.dhidden_stride = a.dhidden_stride, c.dim = a.dim, c.dim_pad = static_cast<int>(l.dim_pad);
  const bool scaled = !bf16 && dloss != nullptr;
  if (scaled) {
    c.meta = p.meta, c.coef = p.coef, c.down = reinterpret_cast<float*>(ws + l.down);
    c.hidden_low = reinterpret_cast<uint16_t*>(ws + l.hidden_low);
    while (int64_t(1) << c.rows_log < a.rows) ++c.rows_log;
  }
  const tbe_status st = launch_select<true>(p, c, dev, s);
  if (st != TBE_OK) return st;
  const void* h = ws + l.hidden;
  const void* low = scaled ? ws + l.hidden_low : h;
  const int64_t wst = a.copy_weight ? l.dim_pad : a.weight_stride;
  if (a.copy_weight) weight = ws + l.weight;
  const void* dz = ws + l.dz;
  CUtensorMap maps[6];
  if (!encode_operand(&maps[0], h, bf16, a.dim, a.tokens, l.dim_pad, 128) || !encode_operand(&maps[1], weight, bf16, a.dim, a.rows, wst, 128) ||
      !encode_operand(&maps[2], dz, bf16, 64, l.piece / 64 * l.dz_rows, 64, 128) || !encode_operand(&maps[3], weight, bf16, a.dim, a.rows, wst, 64) ||
      !encode_operand(&maps[4], dz, bf16, 64, l.piece / 64 * l.dz_rows, 64, 64) || !encode_operand(&maps[5], low, bf16, a.dim, a.tokens, l.dim_pad, 64))
    return cuda_status(cudaErrorInvalidValue);
  if (bf16) return loss_backward<__nv_bfloat16>(a, l, maps, nullptr, dhidden, dweight, ws, dev, s);
  return loss_backward<__half>(a, l, maps, c.down, dhidden, dweight, ws, dev, s);
}

}  // namespace tbe
