// Host-side check of the 4-bit linears' cluster choice (clusters.h) with a
// stand-in for the runtime's answer: the choice is the cheapest by a plain count, a
// failed question is that call's error and leaves nothing behind, an answer is
// asked for once, and a size of which none fits is passed over.  Built and run on the
// CPU by tests/test_cluster_choice.py; prints "ok ..." or the first failure.
#include <cstdio>

#include "clusters.h"

using namespace fp8bs;

static int g_asked = 0;
static int answer(int s) { return s == 1 ? 148 : 148 / s - (s & 1); }

#define REQUIRE(cond)                                        \
  do {                                                       \
    if (!(cond)) {                                           \
      std::printf("line %d: %s\n", __LINE__, #cond);         \
      return 1;                                              \
    }                                                        \
  } while (0)

int main() {
  auto good = [](int s, int* n) {
    ++g_asked;
    *n = answer(s);
    return cudaSuccess;
  };
  static ClusterSlots<4> slots;
  ClusterChoice c, again;

  // A question that fails, at the first size and at a later one.
  for (int failing : {1, 4}) {
    static ClusterSlots<1> fresh;
    auto bad = [&](int s, int* n) {
      *n = answer(s);
      return s == failing ? cudaErrorMemoryAllocation : cudaSuccess;
    };
    REQUIRE(choose_cluster(56, 144, 1, 12, 6, fresh.of(0), bad, &c) == cudaErrorMemoryAllocation);
    REQUIRE(fresh.of(0)[failing].load() == 0);
    REQUIRE(choose_cluster(56, 144, 1, 12, 6, fresh.of(0), good, &c) == cudaSuccess);
    for (int s = 1; s <= 8; ++s) {
      REQUIRE(fresh.of(0)[s].load() == answer(s));
      fresh.of(0)[s] = 0;
    }
  }

  long cases = 0;
  for (int64_t units : {1, 7, 56, 144, 576, 5000})
    for (int kblocks : {1, 2, 16, 56, 144})
      for (int warps : {1, 2, 8}) {
        REQUIRE(choose_cluster(units, kblocks, warps, 3, 6, slots.of(1), good, &c) == cudaSuccess);
        const int before = g_asked;
        REQUIRE(choose_cluster(units, kblocks, warps, 3, 6, slots.of(1), good, &again) == cudaSuccess);
        REQUIRE(g_asked == before && again.size == c.size && again.at_once == c.at_once);
        REQUIRE(c.size >= 1 && c.size <= 8 && c.at_once == answer(c.size));
        REQUIRE(c.size == 1 || c.size * warps <= kblocks);
        auto cost = [&](int s) {
          const int64_t rounds = (units + answer(s) - 1) / answer(s);
          return rounds * ((kblocks + s * warps - 1) / (s * warps) + 3 + (s > 1 ? 6 : 0));
        };
        for (int s = 1; s <= 8; ++s)
          if (s == 1 || s * warps <= kblocks) REQUIRE(cost(c.size) <= cost(s));
        ++cases;
      }

  // No room for some sizes, then for none.
  auto some = [](int s, int* n) { *n = s == 2 ? 10 : 0; return cudaSuccess; };
  REQUIRE(choose_cluster(10, 100, 1, 3, 0, slots.of(2), some, &c) == cudaSuccess && c.size == 2 && c.at_once == 10);
  auto none = [](int, int* n) { *n = 0; return cudaSuccess; };
  REQUIRE(choose_cluster(10, 100, 1, 3, 0, slots.of(3), none, &c) != cudaSuccess);
  std::printf("ok %ld choices\n", cases);
  return 0;
}
