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

// Whether the zeros of a gradient of so many bytes take longer than the sort, so that they want more SMs beside a smaller cluster: past
// 32768 tokens, eight of which a thread of 8 CTAs has to sort, that is much later.  (us a call with 8 and with 16 CTAs, by
// gradient: 12345 tokens 40 MB 24.8 and 24.0, 64 MB 26.9 and 27.4, 128 MB 39.2 and 41.1; 32000 tokens 64 MB 33.0 and 30.0, 96 MB
// 35.7 and 36.9; 45000 tokens 128 MB 51.5 and 44.9, 192 MB 58.0 and 55.7; 65536 tokens 128 MB 55.2 and 51.6, 192 MB 61.7 and 64.0.)
constexpr bool zeros_are_long(int64_t tokens, int64_t bytes) { return bytes > (int64_t(tokens > 4 * kCtaTokens ? 160 : 64) << 20); }

// As many CTAs as have tokens, up to 16, or up to 8 where there is much to set to zero.
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
