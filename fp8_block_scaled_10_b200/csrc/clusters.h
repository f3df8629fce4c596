// How many CTAs of the 4-bit linears share the channels of a row block (a
// cluster), by what the GPU holds at once.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

namespace fp8bs {

constexpr int kMaxCluster = 8;

// Clusters of each size that the GPU holds at once for one kernel, as the runtime
// said: fewer than SMs / size where a size does not divide the SMs of a GPC.  Asked
// once per device and kernel; 0: not known yet, or none.
template <int kDevices>
struct ClusterSlots {
  std::atomic<int> n[kDevices][kMaxCluster + 1] = {};
  std::atomic<int>* of(int dev) { return n[dev]; }
};

struct ClusterChoice {
  int size;      // CTAs of a cluster
  int at_once;   // clusters of that size that fit at once
};

// The size that gives the least time, counted in 128-channel blocks of a warp (or
// CTA): rounds of the GPU's clusters times a share of the blocks, a fixed cost per
// round and, from two CTAs on, one for the join.  `query(size, &clusters)` asks the
// runtime.  A failed query is the call's error and is not remembered: a guess that
// stayed would slow every later call.
template <typename Query>
cudaError_t choose_cluster(int64_t units, int kblocks, int warps_k, int fixed, int join,
                           std::atomic<int>* known, Query query, ClusterChoice* choice) {
  int64_t best_cost = -1;
  *choice = ClusterChoice{0, 0};
  for (int s = 1; s <= kMaxCluster && (s == 1 || s * warps_k <= kblocks); ++s) {
    int at_once = known[s].load(std::memory_order_relaxed);
    if (at_once == 0) {
      const cudaError_t e = query(s, &at_once);
      if (e != cudaSuccess) {
        (void)cudaGetLastError();   // reported by this call, not by the next one
        return e;
      }
      known[s].store(at_once, std::memory_order_relaxed);
    }
    if (at_once < 1) continue;   // the GPU holds no cluster of this size
    const int64_t rounds = (units + at_once - 1) / at_once;
    const int64_t cost =
        rounds * ((kblocks + s * warps_k - 1) / (s * warps_k) + fixed + (s > 1 ? join : 0));
    if (best_cost < 0 || cost < best_cost) {
      *choice = ClusterChoice{s, at_once};
      best_cost = cost;
    }
  }
  return best_cost < 0 ? cudaErrorLaunchOutOfResources : cudaSuccess;
}

}  // namespace fp8bs
