// pair_mma.cuh -- matrix products on the fifth-generation tensor cores by pairs of CTAs: C tile of 256 x 256 =
// sum over k of A[256][k] B[256][k], 16-bit operands, fp32 accumulators, with an epilogue of the caller's.
//
// The two CTAs of a cluster sit on neighbouring SMs and work on one tile (tcgen05.mma.cta_group::2): each brings its
// 128 rows of A and its half of B's rows into its shared memory, so a CTA copies 128 rows of B where it would copy
// 256 alone: 64 bytes a clock at the full rate of a 256 x 256 tile, about what an SM can draw from L2.  Eleven
// warps: eight for the epilogue (warp w reads TMEM lanes 32 (w % 4) .. + 31 and half w / 4 of the columns), two threads that
// issue the TMA copies of a ring of stages of 64 k's, A's and B's, one (in the even CTA) that issues the products.  The
// accumulator takes all 512 columns of TMEM as two buffers, so that the products of the next tile run while the epilogue
// reads the last one.  The grid is persistent: pair p takes tiles p, p + pairs, ...  (4864 x 16384 x 4096 bf16 without an epilogue: 349 us,
// 1870 TFLOP/s, 97% of a library product of 8192^3; with no copies at all 330 us; with k = 1024 1790 TFLOP/s.)
//
// Every wait is bounded.  A role whose wait gives up leaves its loop, the others follow by their own limits, the copies
// in flight are given time to land, and TBE_STAT_WAIT_TIMEOUT is counted.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "cluster.cuh"

namespace tbe {

constexpr int kPairM = 256;            // rows of a tile; 128 to each CTA
constexpr int kPairK = 64;             // k's of a stage: 128 bytes, one row of the swizzle
constexpr int kEpiWarps = 8;
constexpr int kPairThreads = 32 * (kEpiWarps + 3);
constexpr uint32_t kPairWaitLimit = 1u << 22;

constexpr int kStagingBytes = 4096;    // of a warp of the epilogue: 32 rows of 64 16-bit elements

// AM: rows of A that a CTA copies.  With fewer than 128 (products of few rows, bound by B's way through memory) the products
// read what lies behind them as the others, whose results nobody looks at, and the ring has more stages.
// CTAS: 2, or 1 for products of up to 128 rows by single CTAs, each with all of a tile's B: a pair's product of 256 rows takes
// both SMs as long as one with 128 takes one SM (16 x 131072 x 2048: 99 us by pairs,
// 86 by single CTAs, 92% of the copy rate).
template <int AM = 128, int CTAS = 2>
struct PairTile {
  static constexpr int kA = AM * kPairK * 2;             // bytes of a CTA's part of a stage
  static constexpr int kB = 256 / CTAS * kPairK * 2;
  static constexpr int kStage = kA + kB;
  static constexpr int kStages = 196608 / kStage;        // 6 of 32 KB; single CTAs: 5 of 36 KB, 4 of 48 KB
  static_assert(kStage >= 128 * kPairK * 2, "the products read 128 rows of A from a stage's start");
  static constexpr int kSmem = kStages * kStage + kEpiWarps * kStagingBytes + 1024;  // and room to align to the swizzle's 1024 bytes
};

// A product: its tiles, and where it starts in A's and B's coordinates.  With `live`, the number of rows (m) or the length of
// the sums (k) is known on the device only: *live, taken as 1 at least; m_tiles and k_blocks are then the most they can be.
struct PairShape {
  int m_tiles, n_tiles, splits, k_blocks;   // k_blocks: of all splits together; splits <= k_blocks
  int a_m0, a_k0, b_n0, b_k0;
  int width;        // columns of a tile: a multiple of 32 up to 256
  int n_first;      // tiles go along n first, else along m; splits come last
  uint32_t idesc;
  const int* live_m;
  const int* live_k;
  int a_rows;       // 0, or A lies in blocks of 64 columns, each a_rows rows of 128 bytes: what a copy takes is contiguous then

  __device__ __forceinline__ void settle() {
    if (live_m != nullptr) m_tiles = (max(*live_m, 1) + kPairM - 1) / kPairM;
    if (live_k != nullptr) {
      k_blocks = (max(*live_k, 1) + kPairK - 1) / kPairK;
      splits = min(splits, k_blocks);
    }
  }
  __host__ __device__ __forceinline__ int items() const { return m_tiles * n_tiles * splits; }
};

// One or two products in a launch.  The pairs deal out the first one's tiles in turn; those that got one fewer (the lazy ones)
// take `extra` tiles of the second before the rest is dealt out, to the lazy ones first if lazy_first.
struct PairPlan {
  int pairs, extra, lazy_first;

  // The choice with which the last pair ends soonest, counting blocks of k and three more for a tile's other costs.
  __host__ __device__ static PairPlan two(const PairShape& g0, const PairShape& g1, int pairs) {
    const int n0 = g0.items(), n1 = g1.items(), c0 = g0.k_blocks / g0.splits + 3, c1 = g1.k_blocks / g1.splits + 3;
    const int each = n0 / pairs, busy = n0 - each * pairs, lazy = pairs - busy;
    PairPlan best{pairs, 0, 0};
    int64_t least = INT64_MAX;
    const int most = busy == 0 ? 0 : n1 / lazy, even = c0 / c1;
    for (int k = 0; k < 3; ++k) {
      int extra = k == 0 ? 0 : even + k - 1;
      extra = extra < most ? extra : most;
      const int rest = n1 - lazy * extra, round = rest / pairs, left = rest - round * pairs;
      for (int first = 0; first < 2; ++first) {
        const int64_t l = static_cast<int64_t>(each) * c0 + static_cast<int64_t>(extra + round + (first ? left > 0 : left > busy)) * c1;
        const int64_t b = busy == 0 ? 0 : static_cast<int64_t>(each + 1) * c0 + static_cast<int64_t>(round + (first ? left > lazy : left > 0)) * c1;
        const int64_t end = l > b ? l : b;
        if (end < least) least = end, best = PairPlan{pairs, extra, first};
      }
    }
    return best;
  }
};

// kind::f16 instruction descriptor: fp32 accumulator, 16-bit operands, M = 128 to a CTA.
inline uint32_t pair_idesc(bool bf16, int width, bool a_mn, bool b_mn, int ctas = 2) {
  const uint32_t t = bf16 ? 1 : 0;
  return (1u << 4) | (t << 7) | (t << 10) | (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
         (static_cast<uint32_t>(width >> 3) << 17) | (static_cast<uint32_t>(128 * ctas >> 4) << 24);
}

namespace pair {

// The same place in the even CTA's shared memory.
__device__ __forceinline__ uint32_t in_leader(uint32_t addr) { return cluster_address(addr, 0); }
// Orders this thread's shared memory accesses of its own CTA at most: what it has read of TMEM is ordered by fence_before, and a
// release to the cluster would wait for the epilogue's global stores (a quarter of a small product's time).
__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
template <int CTAS>
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if constexpr (CTAS == 1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
    return;
  }
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// Shared-memory descriptor of a 128-byte-swizzled operand tile.  K-major: rows of 64 k's, 8 of them (1024 bytes) to a
// swizzle atom.  MN-major: blocks of 64 (m or n) x 64 k's, a k to a row of 128 bytes, the blocks 8192 bytes apart.
template <bool MN>
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
  const uint64_t lbo = MN ? 8192 >> 4 : 1;
  return static_cast<uint64_t>((addr >> 4) & 0x3FFF) | (lbo << 16) | (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) |
         (uint64_t(2) << 61);
}
template <int CTAS>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  if constexpr (CTAS == 1) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
    return;
  }
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}
// Arrives on the barrier at this place in each CTA when the products issued so far are done.
template <int CTAS>
__device__ __forceinline__ void commit_all(uint64_t* bar) {
  if constexpr (CTAS == 1) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
    return;
  }
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 accumulator columns of this thread's TMEM lane: requested, and there after landed().
struct Columns {
  uint32_t r[32];
  __device__ __forceinline__ void request(uint32_t addr) {
    __syncwarp();
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
  }
  // The registers are operands, so that no use of them moves above the wait.
  __device__ __forceinline__ void landed() {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
  }
  __device__ __forceinline__ float get(int i) const { return __uint_as_float(r[i]); }
};

}  // namespace pair

// A tile, or a split's part of one: k blocks first .. last - 1.
struct PairItem {
  int m, n, split;
  __device__ __forceinline__ int first(const PairShape& g) const { return static_cast<int>(static_cast<int64_t>(g.k_blocks) * split / g.splits); }
  __device__ __forceinline__ int last(const PairShape& g) const { return static_cast<int>(static_cast<int64_t>(g.k_blocks) * (split + 1) / g.splits); }
};

// The tiles of a pair, in its order; every role of both CTAs walks them alike.
struct PairWalk {
  int item, end, stride;           // of the part being walked
  int item2, end2, stride2;        // the other part, taken before
  __device__ __forceinline__ static PairWalk first(int pair, const PairPlan& p, int items) {
    return PairWalk{pair, items, p.pairs, 0, 0, 1};
  }
  __device__ __forceinline__ static PairWalk second(int pair, const PairPlan& p, int items0, int items1) {
    const int busy = items0 % p.pairs, lazy = p.pairs - busy, taken = lazy * p.extra;
    const int turn = p.lazy_first ? (pair + lazy) % p.pairs : pair;   // the lazy ones are busy .. pairs - 1
    return PairWalk{taken + turn, items1, p.pairs, pair >= busy ? pair - busy : taken, taken, lazy};
  }
  __device__ __forceinline__ bool next(const PairShape& g, PairItem& i) {
    int t;
    if (item2 < end2) t = item2, item2 += stride2;
    else if (item < end) t = item, item += stride;
    else return false;
    const int tiles = g.m_tiles * g.n_tiles;
    i.split = g.splits > 1 ? t / tiles : 0;
    t -= i.split * tiles;
    if (g.n_first) i.m = t / g.n_tiles, i.n = t - i.m * g.n_tiles;
    else i.n = t / g.m_tiles, i.m = t - i.n * g.m_tiles;
    return true;
  }
};

// A product with its epilogue.  Job:
//   struct Args;  struct Row: what a thread needs of its row of a tile, Row::load(args, item, row) fetches it ahead;
//   struct State: what a thread carries from tile to tile;
//   tile(args, row_data, state, item, row, half, tmem, staging, release): row = this thread's row of the tile (0 .. 255), half =
//     which 128 of the columns, tmem = the address of its first column; release() once the columns are in registers;
//   finish(args, state, pair, row, half) after the last tile.  All 32 lanes of a warp call these together.
template <bool A_MN, bool B_MN, class J>
struct Product {
  static constexpr bool kAMN = A_MN, kBMN = B_MN, kNone = false;
  using Job = J;
  struct Args {
    CUtensorMap a, b;
    PairShape g;          // read by one thread of a CTA, which settles it
    typename J::Args job;
  };
};
struct NoProduct {
  static constexpr bool kNone = true;
  struct Args {
    int none;
  };
};

struct PairRole {
  uint64_t *full, *empty, *acc_full, *acc_empty;
  uint32_t ring, tmem, rank;
  uint32_t it, tile;   // stages and tiles so far
  bool failed;
};

// One of the two threads that issue copies: A's or B's.  A's also tells the barrier how many bytes a stage has.
template <int AM, int CTAS, class P, bool A>
__device__ __forceinline__ void pair_copy(const typename P::Args& p, const PairShape& g, PairWalk walk, PairRole& r) {
  using T = PairTile<AM, CTAS>;
  const uint32_t leader = pair::in_leader(smem_u32(r.full));
  // B with k across the rows comes in blocks of 64 columns, of which a narrow tile needs one
  const int blocks = A ? 2 : P::kBMN && g.width <= 128 ? 1 : 2;
  const uint32_t bytes = CTAS * (T::kA + (P::kBMN ? (g.width <= 128 ? T::kB / 2 : T::kB) : g.width / CTAS * kPairK * 2));
  PairItem i;
  while (!r.failed && walk.next(g, i)) {
    const int x = A ? g.a_m0 + i.m * kPairM + static_cast<int>(r.rank) * 128 : g.b_n0 + i.n * g.width + static_cast<int>(r.rank) * (g.width / CTAS);
    const int last = i.last(g);
    for (int kb = i.first(g); kb < last; ++kb, ++r.it) {
      const uint32_t st = r.it % T::kStages;
      if (!mbar_wait_bounded(&r.empty[st], ((r.it / T::kStages) & 1) ^ 1, kPairWaitLimit)) {
        r.failed = true;
        return;
      }
      if (A && r.rank == 0) mbar_arrive_expect_tx(&r.full[st], bytes);
      const uint32_t bar = leader + st * 8, to = r.ring + st * T::kStage + (A ? 0 : T::kA);
      const int k = (A ? g.a_k0 : g.b_k0) + kb * kPairK;
      const CUtensorMap* map = A ? &p.a : &p.b;
      if constexpr (A ? P::kAMN : P::kBMN) {
        for (int c = 0; c < blocks; ++c) {
          if (A && g.a_rows > 0) pair::tma_2d<CTAS>(to + c * 8192, map, 0, (x / 64 + c) * g.a_rows + k, bar);
          else pair::tma_2d<CTAS>(to + c * 8192, map, x + c * 64, k, bar);
        }
      } else {
        if (A && g.a_rows > 0) pair::tma_2d<CTAS>(to, map, 0, k / 64 * g.a_rows + x, bar);
        else pair::tma_2d<CTAS>(to, map, k, x, bar);
      }
    }
  }
}

// What is under way to this CTA's shared memory when its copies are all issued: the copies themselves, and the arrivals on `empty`,
// which the even CTA's products send to both CTAs.  Neither may find that the CTA has ended, and nothing orders those arrivals
// before the one on acc_full that the epilogue sees last.  A stage's arrival comes after both CTAs' copies of it have landed and
// been used, so the last round of arrivals is all there is to wait for.  Where a wait gave up it may never come; the
// copies that were issued land within microseconds all the same, and get a millisecond.
template <int ST>
__device__ __forceinline__ void pair_drain(PairRole& r) {
  for (uint32_t k = r.it < ST ? 0 : r.it - ST; k < r.it && !r.failed; ++k)
    r.failed = !mbar_wait_bounded(&r.empty[k % ST], (k / ST) & 1, kPairWaitLimit);
  if (r.failed)
    for (int i = 0; i < 1000; ++i) __nanosleep(1000);
}

template <int AM, int CTAS, class P>
__device__ __forceinline__ void pair_multiply(const PairShape& g, PairWalk walk, PairRole& r) {
  using T = PairTile<AM, CTAS>;
  PairItem i;
  for (; !r.failed && walk.next(g, i); ++r.tile) {
    const uint32_t buf = r.tile & 1, d = r.tmem + buf * 256;
    if (!mbar_wait_bounded(&r.acc_empty[buf], ((r.tile >> 1) & 1) ^ 1, kPairWaitLimit)) {
      r.failed = true;
      return;
    }
    pair::fence_after();
    const int first = i.first(g), last = i.last(g);
    for (int kb = first; kb < last; ++kb, ++r.it) {
      const uint32_t st = r.it % T::kStages;
      if (!mbar_wait_bounded(&r.full[st], (r.it / T::kStages) & 1, kPairWaitLimit)) {
        r.failed = true;
        return;
      }
      pair::fence_after();
      const uint64_t a = pair::operand_desc<P::kAMN>(r.ring + st * T::kStage), b = pair::operand_desc<P::kBMN>(r.ring + st * T::kStage + T::kA);
#pragma unroll
      for (int k = 0; k < kPairK / 16; ++k)  // 16 k's: 32 bytes along a row, or two groups of 8 rows
        pair::mma<CTAS>(d, a + k * ((P::kAMN ? 2048 : 32) >> 4), b + k * ((P::kBMN ? 2048 : 32) >> 4), g.idesc, kb > first || k > 0);
      pair::commit_all<CTAS>(&r.empty[st]);
    }
    pair::commit_all<CTAS>(&r.acc_full[buf]);
  }
}

template <int CTAS, class P>
__device__ __forceinline__ void pair_epilogue(const typename P::Args& p, const PairShape& g, PairWalk walk, PairRole& r, int pair, int w,
                                              int lane, uint32_t staging) {
  using Job = typename P::Job;
  const int row = static_cast<int>(r.rank) * 128 + (w % 4) * 32 + lane, half = w / 4;
  typename Job::State state{};
  PairItem i{}, next{};
  bool more = walk.next(g, i);
  typename Job::Row now{}, then{};
  if (more) now.load(p.job, i, row);
  while (more) {
    more = walk.next(g, next);
    if (more) then.load(p.job, next, row);   // the next tile's, while this one is waited for and worked on
    const uint32_t buf = r.tile & 1;
    r.failed = !mbar_wait_bounded(&r.acc_full[buf], (r.tile >> 1) & 1, kPairWaitLimit);
    r.failed = __any_sync(0xffffffffu, r.failed);
    if (r.failed) return;
    pair::fence_after();
    const uint32_t empty = pair::in_leader(smem_u32(&r.acc_empty[buf]));
    Job::tile(p.job, now, state, i, row, half, r.tmem + buf * 256 + half * 128 + (static_cast<uint32_t>((w % 4) * 32) << 16), staging,
              [&] {
                pair::fence_before();
                __syncwarp();
                if (lane == 0) pair::arrive_at(empty);
              });
    now = then, i = next, ++r.tile;
  }
  Job::finish(p.job, state, pair, row, half);
}

template <int AM, int CTAS, class P0, class P1>
__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(kPairThreads, 1)
    pair_mma_kernel(const __grid_constant__ typename P0::Args p0, const __grid_constant__ typename P1::Args p1,
                    unsigned long long* stats) {
  using T = PairTile<AM, CTAS>;
  static_assert((AM == 128 && CTAS == 2) || (!P0::kAMN && !P0::kBMN), "fewer rows of A, or single CTAs, with K-major operands only");
  constexpr int ST = T::kStages;
  extern __shared__ uint8_t s_raw[];
  __shared__ __align__(8) uint64_t full[ST], empty[ST], acc_full[2], acc_empty[2];
  __shared__ PairShape s_shape[2];
  __shared__ PairPlan s_plan;
  __shared__ uint32_t s_tmem;
  const uint32_t ring = (smem_u32(s_raw) + 1023u) & ~1023u;
  const int w = threadIdx.x / kWarp, lane = lane_id(), pair_id = blockIdx.x / CTAS, pairs = gridDim.x / CTAS;
  may_follow();

  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) mbar_init(&full[s], 1), mbar_init(&empty[s], 1);
    for (int s = 0; s < 2; ++s) mbar_init(&acc_full[s], 1), mbar_init(&acc_empty[s], CTAS * kEpiWarps);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    pair::prefetch_map(&p0.a), pair::prefetch_map(&p0.b);
    if constexpr (!P1::kNone) pair::prefetch_map(&p1.a), pair::prefetch_map(&p1.b);
  }
  if (w == 0) {
    if constexpr (CTAS == 1) {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem)) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem)) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
  }
  pair::fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist
  pair::fence_after();
  wait_before();   // what this kernel reads is complete from here on
  if (threadIdx.x == 32) {
    s_shape[0] = p0.g;
    s_shape[0].settle();
    s_plan = PairPlan{pairs, 0, 0};
    if constexpr (!P1::kNone) {
      s_shape[1] = p1.g;
      s_shape[1].settle();
      s_plan = PairPlan::two(s_shape[0], s_shape[1], pairs);
    }
  }
  __syncthreads();
  PairRole r{full, empty, acc_full, acc_empty, ring, s_tmem, cluster_rank(), 0, 0, false};
  const PairShape g0 = s_shape[0], g1 = s_shape[P1::kNone ? 0 : 1];
  const PairPlan plan = s_plan;
  const PairWalk walk0 = PairWalk::first(pair_id, plan, g0.items());
  PairWalk walk1 = walk0;
  if constexpr (!P1::kNone) walk1 = PairWalk::second(pair_id, plan, g0.items(), g1.items());

  if (w == kEpiWarps) {
    if (lane == 0) {
      pair_copy<AM, CTAS, P0, false>(p0, g0, walk0, r);
      if constexpr (!P1::kNone) pair_copy<AM, CTAS, P1, false>(p1, g1, walk1, r);
      pair_drain<ST>(r);
    }
    __syncwarp();
  } else if (w == kEpiWarps + 2) {
    if (lane == 0) {
      pair_copy<AM, CTAS, P0, true>(p0, g0, walk0, r);
      if constexpr (!P1::kNone) pair_copy<AM, CTAS, P1, true>(p1, g1, walk1, r);
      pair_drain<ST>(r);
    }
    __syncwarp();
  } else if (w == kEpiWarps + 1) {
    if (r.rank == 0 && lane == 0) {
      pair_multiply<AM, CTAS, P0>(g0, walk0, r);
      if constexpr (!P1::kNone) pair_multiply<AM, CTAS, P1>(g1, walk1, r);
    }
    __syncwarp();
  } else {
    const uint32_t staging = ring + ST * T::kStage + w * kStagingBytes;
    pair_epilogue<CTAS, P0>(p0, g0, walk0, r, pair_id, w, lane, staging);
    if constexpr (!P1::kNone)
      if (!r.failed) pair_epilogue<CTAS, P1>(p1, g1, walk1, r, pair_id, w, lane, staging);
  }
  if (r.failed && lane == 0) stat_add(stats, TBE_STAT_WAIT_TIMEOUT, 1);
  __syncwarp();
  pair::fence_before();
  cluster_sync();  // neither CTA ends, or frees its TMEM, while the other may still reach it
  pair::fence_after();
  if (w == 0) {
    if constexpr (CTAS == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(r.tmem) : "memory");
    else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(r.tmem) : "memory");
  }
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();  // NULL where the driver has none

// A [outer, inner] matrix of 16-bit elements, `stride` elements
// between rows, copied as boxes of 64 x box_outer with the 128-byte swizzle.  Elements outside the matrix read as 0.
bool encode_operand(CUtensorMap* map, const void* p, bool bf16, int64_t inner, int64_t outer, int64_t stride, int box_outer);

}  // namespace tbe
