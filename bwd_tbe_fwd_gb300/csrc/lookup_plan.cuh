// lookup_plan.cuh -- the cluster that sorts the tokens of a lookup's gradient: how many CTAs, and how many tokens to a thread.
#pragma once

#include <cstdint>
#include <initializer_list>

namespace tbe {

constexpr int kClusterThreads = 1024;
constexpr int kMaxCluster = 16;
constexpr int kMaxPerThread = 8;
constexpr int64_t kCtaTokens = int64_t(kClusterThreads) * kMaxPerThread;

struct SortPlan {
  int ctas;         // 0: no cluster, the tokens are sorted through memory
  int per_thread;   // 1, 2, 4 or 8
  int clusters;     // how many of them run at once
};

// As many CTAs as have tokens, up to 16, or up to 8 where there is much to set to zero, which takes longer than the sort and has more
// SMs beside smaller clusters (12345 tokens, 30 MB: 24.6 us a call with 8, 23.2 with 16; 65536 tokens, 268 MB: 86 and 90).
// Others, down to a single CTA, where at_once(ctas, per_thread) says that no such cluster can run (one of 16 needs that many
// SMs in one of the GPU's processing clusters), and none where the tokens do not fit what can.
template <typename F>
SortPlan plan_sort(int64_t tokens, bool long_zeros, F&& at_once) {
  for (int most : {long_zeros ? kMaxCluster / 2 : kMaxCluster, kMaxCluster, 8, 4, 2, 1}) {
    if (tokens > most * kCtaTokens) continue;
    SortPlan p{1, 1, 0};
    while (p.ctas < most && p.ctas * kClusterThreads < tokens) p.ctas *= 2;
    while (static_cast<int64_t>(p.ctas) * p.per_thread * kClusterThreads < tokens) p.per_thread *= 2;
    p.clusters = at_once(p.ctas, p.per_thread);
    if (p.clusters > 0) return p;
  }
  return SortPlan{0, 0, 0};
}

}  // namespace tbe
