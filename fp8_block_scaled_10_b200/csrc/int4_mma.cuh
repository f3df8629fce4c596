// Linear layers on 4-bit weights for more than 16 tokens (int4.cuh has the
// formula, the packed layout and the kernel for fewer): the same sums on the
// 5th-generation tensor core, with the weight rows as the 128-row operand and
// the tokens as columns.
//
// A weight tile of 128 rows x 128 channels arrives as 8 KB of codes (TMA), is
// expanded to bf16 integers in shared memory (32 KB, 128-byte swizzle) by four
// warps, and is multiplied by the tokens' tile (TMA): D[128 rows, 32 tokens] in
// TMEM.  Each group of G channels is a product of its own, which four other
// warps fold into fp32 registers by an FMA with the row's group scale.
//
// What binds it is the chain of hand-overs (codes, expanded tile, product, fold),
// not one stage: 18432 -> 18432 at 32 tokens takes 72 us; without the expansion's,
// the products' or the folding's work it took 58-64, without all three 51.  So
// two blocks make a step, with two waits (the expanded tiles with the tokens on
// one barrier, and free TMEM columns) and one commit for 16 MMAs; the commit's
// barrier tells the expanding warps, the token loads and the folding warps alike.
// (A step per block: 920 cycles each, against 1700 for two, 81 us.  Twice as many
// expanding warps, taking turns over two steps, gained 5 % more there and lost as
// much on small layers.  The expanded tiles in TMEM instead of shared memory gained
// 2-4 % with groups of 64 and 128 and lost 18 % with groups of 32, whose products
// then have room for one step only; a third step in flight gained nothing.)
// 18432 -> 7168 at 32 tokens (70 MB): 40.2 us, 1.7 TB/s.
#pragma once

#include <cooperative_groups.h>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "int4.cuh"
#include "sm100.cuh"

namespace fp8bs {
namespace w4 {

constexpr int kTileThreads = 512;
constexpr int kTok = 32;             // tokens per pass
constexpr int kRawStages = 6;        // code tiles in flight: 48 KB per SM
constexpr int kRawBytes = 128 * 64;
constexpr int kABytes = 128 * 256;   // an expanded tile; two per step, two steps
constexpr int kXBytes = kTok * 256;  // tokens x 128 channels; likewise
constexpr int kXOffset = 4 * kABytes;
constexpr int kRawOffset = kXOffset + 4 * kXBytes;
constexpr int kTileCtrl = kRawOffset + kRawStages * kRawBytes;
constexpr int kTileSmem = kTileCtrl + 256 + 1024;   // + alignment
static_assert(kTileSmem <= 227 * 1024, "shared memory");
static_assert(kTok * 128 * 4 <= kRawStages * kRawBytes, "the sums fit the code ring");

struct TileCtrl {
  uint64_t raw_full[kRawStages], raw_empty[kRawStages];
  uint64_t full[2];    // a step's tiles expanded and its tokens loaded
  uint64_t done[2];    // its MMAs complete: products there, tiles and tokens read
  uint64_t folded[2];  // its products read
  uint64_t flush;
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(TileCtrl) <= 256, "control block");

// D[tmem] (+)= A[smem] * B[smem]^T, both K-major bf16, fp32 accumulator.
__device__ __forceinline__ void mma_bf16_warp(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of kind::f16: D fp32, A and B bf16, both K-major.
__host__ __device__ constexpr uint32_t idesc_bf16_f32(int M, int N) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// One CTA: 128 weight rows (GATED: 64 of gate, then the same 64 of up) against
// 32 tokens, over its share of the channels; the CTAs of a cluster share a row
// tile's channels and join their sums as int4_linear_kernel does.  Step s has
// blocks 2 s and 2 s + 1 (the last may have one) and uses slot s % 2.  Waits are
// bounded: one that gives up reports FP8BS_ERR_TIMEOUT and makes every role leave
// its loop, and the CTA still takes part in its cluster's barriers.
template <int G, bool GATED>
__global__ void __launch_bounds__(kTileThreads, 1)
    int4_tile_kernel(const __grid_constant__ CUtensorMap tmap_q0,
                     const __grid_constant__ CUtensorMap tmap_q1,
                     const __grid_constant__ CUtensorMap tmap_x, const Params p) {
  namespace cg = cooperative_groups;
  constexpr int kGroups = 128 / G;
  constexpr int kMmas = 8 / kGroups;             // of a group, 16 channels each
  constexpr int kRows = GATED ? 64 : 128;        // rows of y per CTA
  constexpr int kStepCols = 2 * kGroups * kTok;  // TMEM columns of a step's products
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* x_tiles = smem + kXOffset;
  uint8_t* raw_tiles = smem + kRawOffset;
  TileCtrl* ctrl = reinterpret_cast<TileCtrl*>(smem + kTileCtrl);
  volatile int* abort_flag = &ctrl->abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  cg::cluster_group cluster = cg::this_cluster();
  const int splits = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const int n0 = static_cast<int>(blockIdx.x) / splits * kRows;
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * kTok;
  const int kblocks = p.K / 128;
  const int kb0 = static_cast<int>(static_cast<int64_t>(kblocks) * rank / splits);
  const int blocks = static_cast<int>(static_cast<int64_t>(kblocks) * (rank + 1) / splits) - kb0;
  const int steps = (blocks + 1) / 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kRawStages; ++s) {
      mbar_init(&ctrl->raw_full[s], 1);
      mbar_init(&ctrl->raw_empty[s], 4);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctrl->full[s], 9);     // eight expanding warps and the token loads
      mbar_init(&ctrl->done[s], 1);
      mbar_init(&ctrl->folded[s], 4);
    }
    mbar_init(&ctrl->flush, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_descriptor(&tmap_q0);
    if (GATED) tma_prefetch_descriptor(&tmap_q1);
    tma_prefetch_descriptor(&tmap_x);
  }
  if (warp == 1) {
    tmem_alloc(&ctrl->tmem_base, 2 * kStepCols);
    tmem_relinquish();
  }
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = ctrl->tmem_base;
  // Parity of the phase that step s completes in its slot; the wait for the
  // step before it in the slot passes at once in the first round.
  auto parity = [](int s) { return static_cast<uint32_t>((s >> 1) & 1); };

  float acc[kTok];   // folding warps: the sums of one row
#pragma unroll
  for (int c = 0; c < kTok; ++c) acc[c] = 0.0f;

  if (warp == 0) {
    // ------------------------------------------------------------ codes
    int i = 0;
    for (; i < blocks; ++i) {
      const int s = i % kRawStages;
      if (!mbar_wait_warp(&ctrl->raw_empty[s], ((i / kRawStages) & 1u) ^ 1u, abort_flag)) break;
      mbar_arrive_expect_tx_warp(&ctrl->raw_full[s], kRawBytes);
      const int32_t x = (kb0 + i) * 64;
      tma_load_2d_warp(raw_tiles + s * kRawBytes, &tmap_q0, &ctrl->raw_full[s], x, n0);
      if (GATED)
        tma_load_2d_warp(raw_tiles + s * kRawBytes + kRawBytes / 2, &tmap_q1, &ctrl->raw_full[s], x, n0);
    }
    if (*abort_flag)   // let the loads in flight land
      for (int j = max(0, i - kRawStages); j < i; ++j)
        mbar_wait(&ctrl->raw_full[j % kRawStages], (j / kRawStages) & 1u, nullptr);
  } else if (warp == 2) {
    // ------------------------------------------------------------ tokens
    int s = 0;
    for (; s < steps; ++s) {
      if (!mbar_wait_warp(&ctrl->done[s & 1], parity(s) ^ 1u, abort_flag)) break;
      const int nb = min(2, blocks - 2 * s);
      mbar_arrive_expect_tx_warp(&ctrl->full[s & 1], nb * kXBytes);
      for (int h = 0; h < 2 * nb; ++h)
        tma_load_2d_warp(x_tiles + (s & 1) * 2 * kXBytes + h * (kXBytes / 2), &tmap_x,
                         &ctrl->full[s & 1], (kb0 + 2 * s) * 128 + 64 * h, static_cast<int32_t>(m0));
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA
    constexpr uint32_t idesc = idesc_bf16_f32(128, kTok);
    for (int s = 0; s < steps; ++s) {
      const int slot = s & 1;
      if (!mbar_wait_warp(&ctrl->folded[slot], parity(s) ^ 1u, abort_flag)) break;
      if (!mbar_wait_warp(&ctrl->full[slot], parity(s), abort_flag)) break;
      tc_fence_after();
      const uint32_t a0 = smem_addr(smem + slot * 2 * kABytes);
      const uint32_t x0 = smem_addr(x_tiles + slot * 2 * kXBytes);
      const uint32_t d0 = tmem_base + slot * kStepCols;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        if (2 * s + b >= blocks) break;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_bf16_warp(d0 + (b * kGroups + k / kMmas) * kTok,
                        smem_desc_k_sw128(a0 + b * kABytes + (k / 4) * (kABytes / 2) + 32 * (k % 4)),
                        smem_desc_k_sw128(x0 + b * kXBytes + (k / 4) * (kXBytes / 2) + 32 * (k % 4)),
                        idesc, k % kMmas > 0 ? 1u : 0u);
      }
      mma_commit_warp(&ctrl->done[slot]);
    }
    // Every MMA must have finished before the TMEM columns are released.
    mma_commit_warp(&ctrl->flush);
    mbar_wait(&ctrl->flush, 0, nullptr);
    __syncwarp();
  } else if (warp >= 8) {
    // ------------------------------------------------------------ expansion
    // Thread = weight row: piece t, word j of its 64 bytes are channels 32 j + 8 t +
    // 0..7, 16 bytes of bf16, chunk 4 j + t of the row's 256.
    const int row = (warp & 3) * 32 + lane;
    const int b = (warp - 8) >> 2;   // block of the step
    uint32_t mask = 0x000F000Fu, exponent = 0x43004300u;
    asm volatile("" : "+r"(mask), "+r"(exponent));   // kept in registers
    for (int s = 0; s < steps; ++s) {
      const int i = 2 * s + b, sr = i % kRawStages;
      uint4 w[4];
      if (i < blocks) {
        if (!mbar_wait_warp(&ctrl->raw_full[sr], (i / kRawStages) & 1u, abort_flag)) break;
        const uint8_t* raw = raw_tiles + sr * kRawBytes + row * 64;
#pragma unroll
        for (int t = 0; t < 4; ++t)   // 64-byte swizzle
          w[t] = *reinterpret_cast<const uint4*>(raw + 16 * (t ^ ((row >> 1) & 3)));
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctrl->raw_empty[sr]);
      }
      if (!mbar_wait_warp(&ctrl->done[s & 1], parity(s) ^ 1u, abort_flag)) break;
      if (i < blocks) {
        uint8_t* dst = smem + ((s & 1) * 2 + b) * kABytes + row * 128;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const uint32_t v = j == 0 ? w[t].x : j == 1 ? w[t].y : j == 2 ? w[t].z : w[t].w;
            uint32_t c[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) c[e] = codes_bf16x2(v >> (4 * e), mask, exponent);
            const int chunk = 4 * j + t;   // 128-byte swizzle inside each half of the channels
            *reinterpret_cast<uint4*>(dst + (chunk >> 3) * (kABytes / 2) +
                                      16 * ((chunk & 7) ^ (row & 7))) = make_uint4(c[0], c[1], c[2], c[3]);
          }
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctrl->full[s & 1]);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ folding
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const int n = min(n0 + (GATED ? row & 63 : row), p.N - 1);
    const float* sp = (GATED && row >= 64 ? p.s[1] : p.s[0]) +
                      static_cast<int64_t>(n) * (p.K / G) + kb0 * kGroups;
    const int groups = blocks * kGroups;
    float next[2 * kGroups];   // the next step's scales
    auto load_scales = [&](int s) {
#pragma unroll
      for (int q = 0; q < 2 * kGroups; ++q)
        next[q] = 2 * kGroups * s + q < groups ? __ldca(sp + 2 * kGroups * s + q) : 0.0f;
    };
    load_scales(0);
    for (int s = 0; s < steps; ++s) {
      float sc[2 * kGroups];
#pragma unroll
      for (int q = 0; q < 2 * kGroups; ++q) sc[q] = next[q];
      load_scales(s + 1);
      if (!mbar_wait_warp(&ctrl->done[s & 1], parity(s), abort_flag)) break;
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < 2 * kGroups; ++q) {
        if (2 * kGroups * s + q < groups) {   // the same for the whole CTA
          uint32_t v[32];
          tmem_ld_32x32b_x32(lane_addr + (s & 1) * kStepCols + q * kTok, v);
          tmem_ld_wait(v);
#pragma unroll
          for (int c = 0; c < kTok; ++c) acc[c] = fmaf(sc[q], __uint_as_float(v[c]), acc[c]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctrl->folded[s & 1]);
    }
  }

  // After a wait that gave up, the tokens in flight still have to land.
  if (warp == 2 && *abort_flag)
    for (int s = max(0, steps - 2); s < steps; ++s) mbar_wait(&ctrl->full[s & 1], parity(s), nullptr);
  // The sums take the place of the codes, which have all been read: the last
  // group's product needed them.
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 2 * kStepCols);
  }
  float* sums = reinterpret_cast<float*>(raw_tiles);   // [token][128 rows]
  if (warp >= 4 && warp < 8) {
#pragma unroll
    for (int c = 0; c < kTok; ++c) sums[c * 128 + (warp & 3) * 32 + lane] = acc[c];
  }
  if (splits > 1) cluster.sync();
  else __syncthreads();
  // Four rows of one token per thread, shared out over the cluster's CTAs.
  for (int o = rank * kTileThreads + threadIdx.x; o < kRows / 4 * kTok; o += splits * kTileThreads) {
    const int token = o / (kRows / 4), r = 4 * (o % (kRows / 4));
    const int64_t m = m0 + token;
    const int n = n0 + r;
    if (m >= p.M || n >= p.N) continue;
    float v[4];
    const int at = token * 128 + r;
    if (splits == 1)
      join4<GATED, 64, 1>(v, [&](int) { return sums + at; }, 1);
    else
      join4<GATED, 64, 8>(
          v, [&](int k) { return cluster.map_shared_rank(sums, k < splits ? k : 0) + at; }, splits);
    store4(p, m, n, v);
  }
  if (splits > 1) cluster.sync();   // a CTA's sums stay until every CTA has read them
}

}  // namespace w4
}  // namespace fp8bs
