// The clusters that sort the tokens of a lookup's gradient, for GPUs on which clusters of any size up to a limit can run, or none:
// what is planned can run and holds the tokens, and nothing is planned only where nothing that can run does.  Prints "plans
// ok", or the first plan that is wrong.
#include <cstdio>
#include <initializer_list>

#include "lookup_plan.cuh"

using tbe::kClusterThreads;
using tbe::kCtaTokens;

namespace {

bool check(int64_t tokens, bool long_zeros, int largest, int most_per_thread) {
  auto at_once = [&](int ctas, int per_thread) { return ctas <= largest && per_thread <= most_per_thread ? 17 - ctas : 0; };
  const tbe::SortPlan p = tbe::plan_sort(tokens, long_zeros, at_once);
  const bool power = p.per_thread == 1 || p.per_thread == 2 || p.per_thread == 4 || p.per_thread == 8;
  bool ok;
  if (p.ctas > 0) {
    const int64_t room = int64_t(p.ctas) * p.per_thread * kClusterThreads;
    ok = p.ctas <= 16 && (p.ctas & (p.ctas - 1)) == 0 && power && at_once(p.ctas, p.per_thread) == p.clusters && p.clusters > 0 && tokens <= room;
  } else {
    ok = largest == 0 || tokens > int64_t(largest) * most_per_thread * kClusterThreads;
  }
  // where every cluster can run: the smallest of enough CTAs for a token to a thread, up to 16, or 8 beside long zeros
  if (ok && largest == 16 && most_per_thread == 8) {
    const int most = long_zeros && tokens <= 8 * kCtaTokens ? 8 : 16;
    ok = (p.ctas > 0) == (tokens <= 16 * kCtaTokens);
    if (p.ctas > 0) ok = ok && p.ctas <= most && (p.ctas == most || p.ctas * kClusterThreads >= tokens) && (p.ctas == 1 || p.ctas / 2 * kClusterThreads < tokens);
  }
  if (!ok) std::printf("%lld tokens, zeros %d, clusters up to %d of %d tokens a thread: %d CTAs, %d a thread, %d at once\n", (long long)tokens,
                       long_zeros, largest, most_per_thread, p.ctas, p.per_thread, p.clusters);
  return ok;
}

}  // namespace

int main() {
  for (int largest : {0, 1, 2, 4, 8, 16})
    for (int per_thread : {1, 2, 4, 8})
      for (bool zeros : {false, true})
        for (int64_t base = 1; base <= 1 << 20; base *= 2)
          for (int64_t tokens : {base - 1, base, base + 1, base + base / 2})
            if (tokens > 0 && !check(tokens, zeros, largest, per_thread)) return 1;
  static_assert(!tbe::zeros_are_long(1, 64 << 20) && tbe::zeros_are_long(32768, (64 << 20) + 1), "");
  static_assert(!tbe::zeros_are_long(32769, 160 << 20) && tbe::zeros_are_long(65536, (160 << 20) + 1), "");
  std::puts("plans ok");
  return 0;
}
