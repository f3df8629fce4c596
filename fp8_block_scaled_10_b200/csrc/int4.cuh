// Linear layers on 4-bit weights with group scales, up to 16 tokens (more:
// int4_mma.cuh): y[m, n] = sum_k x[m, k] s[n, k / G] (c[n, k] - 8), codes c in 0..15,
// fp32 scales per group of G = 32, 64 or 128 input channels.  Also the
// quantizer and its inverse.
//
// Packed layout of a row of K codes (K % 128 == 0, K/2 bytes): each 128
// channels are 64 bytes, word j (0..3) of 16-byte piece t (0..3) holds
// channels 32 j + 8 t + 0..7 of the block, nibble p of the word (low first)
// channel 2 p for p < 4 and 2 p - 7 above: the even channels in the low half
// word, the odd ones in the high half.  Lane t of a quad then reads its 16
// bytes of a row in one load; the words of one j over the quad are 32
// consecutive channels, so that a group of 32 is a whole number of matrix
// instructions; and (w >> 4 i) & 0x000F000F is a pair of adjacent channels.
#pragma once

#include <cooperative_groups.h>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gemm.cuh"
#include "quant.cuh"
#include "sm100.cuh"

namespace fp8bs {
namespace w4 {

// Two codes (bits 0-3 and 16-19) as the bf16 pair c - 8: 0x4300 | c is 128 + c,
// and the difference to 136 is exact.  Mask and exponent go in by one
// three-input operation (both constants in registers; written as C it becomes
// two): the integer pipe, 16 lanes per clock and scheduler, is the busiest.
__device__ __forceinline__ uint32_t codes_bf16x2(uint32_t w, uint32_t mask, uint32_t exponent) {
  uint32_t v;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(v) : "r"(w), "r"(mask), "r"(exponent));   // (w & mask) | exponent
  const __nv_bfloat162 d =
      __hsub2(*reinterpret_cast<__nv_bfloat162*>(&v), __float2bfloat162_rn(136.0f));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// d = A B + d, or A B where FIRST.
template <bool FIRST>
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (FIRST)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct Params {
  const __nv_bfloat16* x;   // [M, K]
  const uint8_t* q[2];      // packed [N, K/2]; GATED: gate, up
  const float* s[2];        // [N, K/G]
  void* y;                  // [M, N], bf16 or (y_f32) fp32
  int y_f32;
  int64_t M;
  int N;
  int K;
};

constexpr int kThreads = 256;
constexpr int kWarps = 8;

// NT: tiles of 8 tokens.  One token tile is bound by the weight stream alone: the
// eight warps of a CTA share the channels of its rows, which gives the most
// CTAs, and x stays in L1.  More tokens would make the CTAs' reads of x from L2
// (2 M K bytes each) pass the weight stream: there four warps lie along the rows
// and share the blocks of x, which are copied to shared memory with the weights.
template <int NT, int G, bool GATED>
struct Cfg {
  static constexpr bool kShareX = NT > 1;
  static constexpr int kTiles = 2;                         // 16-row weight tiles per warp
  static constexpr int WR = kShareX ? 4 : 1;               // warps along the rows
  static constexpr int WK = kWarps / WR;                   // warps along the channels
  static constexpr int kGroups = 128 / G;                  // scales per row and block
  static constexpr int kWarpRows = GATED ? 16 : 16 * kTiles;   // rows of y per warp
  static constexpr int kRows = kWarpRows * WR;             // rows of y per CTA
  static constexpr int kWarpSums = kTiles * NT * 128;
  static constexpr int kSums = WR * kWarpSums;
  static constexpr int kUp = 8 * NT * 16;                  // GATED: from a gate sum to its up sum
  static constexpr int kStageBytes = kTiles * 2 * 512 + kTiles * 2 * 8 * kGroups * 4;   // of a warp
  static constexpr int kScales = kTiles * 2 * 512;         // where a stage's scales start
  static constexpr int kXBytes = kShareX ? NT * 2048 : 0;  // of WR warps: [8 NT tokens][128] bf16
  static constexpr int kSumBuffers = kShareX ? 1 : 2;
  static constexpr int kSumBytes = 4 * WK * kSums * kSumBuffers;
  // Stages that let two CTAs share an SM's 227 KB, four at most.
  static constexpr int kFit = (227 * 1024 / 2 - 1024 - kSumBytes) / (kWarps * kStageBytes + WK * kXBytes);
  static constexpr int kStages = kFit > 4 ? 4 : kFit;
  static constexpr int kRingBytes = kStages * (kWarps * kStageBytes + WK * kXBytes);
  static constexpr int kSmem = kRingBytes + kSumBytes;
  static_assert(WK > 1 && kStages >= 2 && 2 * (kSmem + 1024) <= 227 * 1024, "two CTAs per SM");
};

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// silu(g) u = g e / (1 + e) u with e = exp(g) for g < 0, and g / (1 + e) u with e = exp(-g)
// above, within 2^-20 relative: fp32 outputs are stored as they are, so the
// gate of the bf16 epilogues (gemm.cuh, 2^-17 and nothing below -87) will not do.
// In units of 2^-24: expf 4 at most, the reciprocal 2 (1 + e is in [1, 2]), the sum and
// the products 1 each.  Far out exp(g) would be subnormal: there its square root is
// multiplied in twice, 15 in all (1 + e is 1).  Once per output: 4 tokens, 7168 ->
// 2048 in groups of 32, weights from memory, 9.0 us as with the fast gate (9.2 with
// an IEEE division).
__device__ __forceinline__ float gated_wide(float g, float u) {
  const bool far = g < -80.0f;
  const float e = expf(far ? 0.5f * g : -fabsf(g));
  const float h = (g < 0.0f ? g * e : g) * gemm::rcp_ftz(1.0f + e) * u;
  return far ? h * e : h;
}

// Four outputs: the sums at from(0), from(1), .. from(n - 1) added in this order
// (n <= MOST; GATED: the up sums lie UP floats behind, and the gate is applied).
template <bool GATED, int UP, int MOST, typename From>
__device__ __forceinline__ void join4(float (&v)[4], From from, int n) {
  float4 total[GATED ? 2 : 1];
#pragma unroll
  for (int i = 0; i < (GATED ? 2 : 1); ++i) {
    float4 a[MOST];
#pragma unroll
    for (int k = 0; k < MOST; ++k) a[k] = *reinterpret_cast<const float4*>(from(k) + i * UP);
    total[i] = a[0];
#pragma unroll
    for (int k = 1; k < MOST; ++k)
      if (k < n) {
        total[i].x += a[k].x;
        total[i].y += a[k].y;
        total[i].z += a[k].z;
        total[i].w += a[k].w;
      }
  }
  v[0] = total[0].x; v[1] = total[0].y; v[2] = total[0].z; v[3] = total[0].w;
  if constexpr (GATED) {
    v[0] = gated_wide(v[0], total[1].x);
    v[1] = gated_wide(v[1], total[1].y);
    v[2] = gated_wide(v[2], total[1].z);
    v[3] = gated_wide(v[3], total[1].w);
  }
}

// Stores four outputs of token m, rows n..n+3.
__device__ __forceinline__ void store4(const Params& p, int64_t m, int n, const float (&v)[4]) {
  if (p.y_f32) {
    float* y = static_cast<float*>(p.y) + m * p.N + n;
    if (p.N % 4 == 0) {
      *reinterpret_cast<float4*>(y) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < p.N) y[e] = v[e];
    }
  } else {
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) + m * p.N + n;
    if (p.N % 4 == 0) {
      *reinterpret_cast<uint2*>(y) =
          make_uint2(gemm::pack_bf16x2(v[0], v[1]), gemm::pack_bf16x2(v[2], v[3]));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < p.N) y[e] = __float2bfloat16_rn(v[e]);
    }
  }
}

// Barrier of THREADS threads (whole warps).
template <int THREADS>
__device__ __forceinline__ void group_sync(int id) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(THREADS) : "memory");
}

// The bound is the weight stream.  A CTA walks blocks of kRows rows against one
// tile of 8 NT tokens; the warps along K, and the CTAs of a cluster when the
// rows alone do not fill the GPU, take 128-channel blocks in turn and join
// their sums in a fixed order: in shared memory, then over the cluster's
// distributed shared memory, so there is no workspace and no second launch.
// Blocks are copied (cp.async) into a ring, kStages - 1 ahead and on into the
// next row block, so the stream does not stop for the joins; a lane copies the
// weight bytes that it will use itself.
// A warp multiplies 16-row tiles by mma.sync m16n8k16, whose operands are
// expanded in registers: codes become exact bf16 integers in three instructions
// per pair, sums of one group are kept in fp32 and enter the row's sum by an fp32
// FMA with the group's scale.  (Through tcgen05 the expanded weights pass shared
// memory and a product costs the same for 1 token as for 32; measured at 16
// tokens, this kernel against that: 7168 -> 18432 24.4 / 30.6 us, 18432 -> 7168
// 26.1 / 38.7, gated 7168 -> 2048 10.4 / 11.7; at 32, in two passes' worth of
// tiles, 41.4 / 40.2 and 17.3 / 12.2.)
// One token, 7168 -> 18432 (70 MB): 17.8 us, 3.9 TB/s; 55 % of the
// issue slots are taken, and 43 % of the instructions are the integer pipe's, which
// expands the codes at half rate; the rest is the start and the join of a kernel
// this short.
template <int NT, int G, bool GATED>
__global__ void __launch_bounds__(kThreads, 2)
    int4_linear_kernel(const Params p) {
  namespace cg = cooperative_groups;
  using C = Cfg<NT, G, GATED>;
  constexpr int kGroups = C::kGroups;
  constexpr int kTiles = C::kTiles;
  extern __shared__ __align__(128) uint8_t smem[];
  float* red = reinterpret_cast<float*>(smem + C::kRingBytes);   // [kSumBuffers][WK][kSums]
  pdl_trigger();
  pdl_wait();
  cg::cluster_group cluster = cg::this_cluster();
  const int splits = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wr = warp % C::WR, wk = warp / C::WR;
  const int g = lane >> 2, t = lane & 3;
  const int kblocks = p.K / 128;
  const int64_t row_bytes = p.K / 2;
  const int groups_k = p.K / G;
  const int row_blocks = (p.N + C::kRows - 1) / C::kRows;
  const int rb0 = static_cast<int>(blockIdx.x) / splits;
  const int rb_step = static_cast<int>(gridDim.x) / splits;
  const int kb0 = rank * C::WK + wk, kb_step = splits * C::WK;

  const uint32_t ring = smem_addr(smem) + warp * (C::kStages * C::kStageBytes);
  const uint8_t* ring_p = smem + warp * (C::kStages * C::kStageBytes);

  // x ring of the WR warps that share a channel block; piece c (16 bytes) of token
  // m lies at c ^ 4 (m % 2), so that the fragments' reads (four pieces of eight
  // tokens) touch each bank once.
  const int xring = kWarps * C::kStages * C::kStageBytes + wk * (C::kStages * C::kXBytes);
  constexpr int kGroupThreads = 32 * C::WR;
  const int tid = threadIdx.x % kGroupThreads;
  const uint32_t xdst = smem_addr(smem) + xring + (tid >> 4) * 256 + 16 * ((tid & 15) ^ (4 * ((tid >> 4) & 1)));
  const __nv_bfloat16* xq[NT];   // copy sources: token 8 c + tid / 16, piece tid % 16
  auto token = [&](int c, int m) -> int64_t { return 8 * c + m < p.M ? 8 * c + m : 0; };

  // Copy cursor: row block, channel block, and pointers to this lane's weight rows
  // and its share of the scales (tile t / 2, half t % 2, row g) at that block.
  // Rows past N read row N - 1; their sums are not stored.  (Pointers are kept
  // and stepped: made anew from indices they took as many operations as the codes.)
  int prb = rb0, pkb = kb0;
  const uint8_t* wp[kTiles][2];
  const float* sp = nullptr;
  auto row_of = [&](int i, int h) -> int64_t {
    return min(prb * C::kRows + wr * C::kWarpRows + (GATED ? 0 : 16 * i) + 8 * h + g, p.N - 1);
  };
  auto point = [&]() {
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        wp[i][h] = p.q[GATED ? i : 0] + row_of(i, h) * row_bytes + 16 * t + kb0 * 64;
    sp = (GATED && t >= 2 ? p.s[1] : p.s[0]) + row_of((t >> 1) % kTiles, t & 1) * groups_k + kb0 * kGroups;
    if constexpr (C::kShareX) {
#pragma unroll
      for (int c = 0; c < NT; ++c)
        xq[c] = p.x + token(c, tid >> 4) * p.K + 8 * (tid & 15) + kb0 * 128;
    }
  };
  int pstage = 0;
  auto issue = [&]() {
    const uint32_t pat = ring + pstage * C::kStageBytes;
    if (prb < row_blocks) {
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          copy_async<16>(pat + (2 * i + h) * 512 + 16 * lane, wp[i][h]);
          wp[i][h] += kb_step * 64;
        }
      if (t < 2 * kTiles) copy_async<4 * kGroups>(pat + C::kScales + (t * 8 + g) * (4 * kGroups), sp);
      sp += kb_step * kGroups;
      if constexpr (C::kShareX) {
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          copy_async<16>(xdst + pstage * C::kXBytes + c * 2048, xq[c]);
          xq[c] += kb_step * 128;
        }
      }
      pkb += kb_step;
      if (pkb >= kblocks) {
        prb += rb_step;
        pkb = kb0;
        if (prb < row_blocks) point();
      }
    }
    copy_commit();
    if (++pstage == C::kStages) pstage = 0;
  };
  // A warp past the last channel block copies and multiplies nothing.
  if (kb0 >= kblocks) prb = row_blocks;
  if (prb < row_blocks) point();
#pragma unroll
  for (int d = 0; d < C::kStages - 1; ++d) issue();

  // x of one token tile, a block ahead: lane (g, t) holds channels 32 j + 8 t +
  // 0..7 of a block of token g.  Lanes past the last token read token 0 (so do
  // the copies above): a token's sums depend on its own x alone, and theirs are
  // not stored.
  const __nv_bfloat16* xp = p.x + token(0, g) * p.K + 8 * t + min(kb0, kblocks - 1) * 128;
  uint4 xn[4];
  auto load_x = [&]() {
#pragma unroll
    for (int j = 0; j < 4; ++j) xn[j] = __ldca(reinterpret_cast<const uint4*>(xp + 32 * j));
  };
  if (!C::kShareX) load_x();
  uint32_t mask = 0x000F000Fu, exponent = 0x43004300u;
  asm volatile("" : "+r"(mask), "+r"(exponent));   // kept in registers

  // Output o of a row block: token, row of y (the first of four) and the place of
  // its sums; false past the last token or row.
  auto place = [&](int o, int rb, int& at, int64_t& m, int& n) {
    const int tok = o / (C::kRows / 4), r = 4 * (o % (C::kRows / 4));
    m = tok;
    n = rb * C::kRows + r;
    const int wrow = r % C::kWarpRows;
    at = (r / C::kWarpRows) * C::kWarpSums + ((GATED ? 0 : wrow / 16) * 8 * NT + tok) * 16 + wrow % 16;
    return m < p.M && n < p.N;
  };
  int stage = 0, buffer = 0;
  for (int rb = rb0; rb < row_blocks; rb += rb_step) {
    float acc[kTiles][NT][4];
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][c][e] = 0.0f;
#pragma unroll 1
    for (int kb = kb0; kb < kblocks; kb += kb_step) {
      copy_wait<C::kStages - 2>();
      // What the other lanes (warps) copied has arrived, and all have read the
      // stage that is copied into next.
      if (C::kShareX) group_sync<kGroupThreads>(1 + wk);
      else __syncwarp();
      issue();
      const uint8_t* at = ring_p + stage * C::kStageBytes;
      const uint8_t* xs = smem + xring + stage * C::kXBytes + g * 256;
      if (++stage == C::kStages) stage = 0;
      uint4 w[kTiles][2];
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[i][h] = *reinterpret_cast<const uint4*>(at + (2 * i + h) * 512 + 16 * lane);
      // channels to the next block of x: on, or back to the first (the next row block)
      const int xstep = kb + kb_step < kblocks ? kb_step * 128 : (kb0 - kb) * 128;
      uint4 x1[4];
      if constexpr (!C::kShareX) {
#pragma unroll
        for (int j = 0; j < 4; ++j) x1[j] = xn[j];
        xp += xstep;
        load_x();
      }
      float part[kTiles][NT][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        constexpr int kPerGroup = 4 / kGroups;   // j's of a group
        uint4 xb[NT];
        if constexpr (C::kShareX) {
#pragma unroll
          for (int c = 0; c < NT; ++c)
            xb[c] = *reinterpret_cast<const uint4*>(xs + c * 2048 + 16 * ((4 * j + t) ^ (4 * (g & 1))));
        } else {
          xb[0] = x1[j];
        }
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          const uint32_t lo = j == 0 ? w[i][0].x : j == 1 ? w[i][0].y : j == 2 ? w[i][0].z : w[i][0].w;
          const uint32_t hi = j == 0 ? w[i][1].x : j == 1 ? w[i][1].y : j == 2 ? w[i][1].z : w[i][1].w;
          uint32_t al[4], ah[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            al[e] = codes_bf16x2(lo >> (4 * e), mask, exponent);
            ah[e] = codes_bf16x2(hi >> (4 * e), mask, exponent);
          }
#pragma unroll
          for (int c = 0; c < NT; ++c) {
            if (j % kPerGroup == 0) mma_bf16<true>(part[i][c], al[0], ah[0], al[1], ah[1], xb[c].x, xb[c].y);
            else mma_bf16<false>(part[i][c], al[0], ah[0], al[1], ah[1], xb[c].x, xb[c].y);
            mma_bf16<false>(part[i][c], al[2], ah[2], al[3], ah[3], xb[c].z, xb[c].w);
          }
        }
        if (j % kPerGroup == kPerGroup - 1) {
          const int gi = j / kPerGroup;
#pragma unroll
          for (int i = 0; i < kTiles; ++i) {
            float sc[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
              sc[h] = *reinterpret_cast<const float*>(at + C::kScales + (((2 * i + h) * 8 + g) * kGroups + gi) * 4);
#pragma unroll
            for (int c = 0; c < NT; ++c)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[i][c][e] = fmaf(sc[e >> 1], part[i][c][e], acc[i][c][e]);
          }
        }
      }
    }

    // Sum e of (tile i, token tile c) of a lane: row 8 (e / 2) + g of the tile,
    // token 8 c + 2 t + e % 2.  Stored as [warp along rows][tile][token][row].
    float* sums = red + buffer * (C::WK * C::kSums);
    if (C::kSumBuffers == 2) buffer ^= 1;
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sums[wk * C::kSums + wr * C::kWarpSums + (i * 8 * NT + 8 * c + 2 * t + (e & 1)) * 16 +
               8 * (e >> 1) + g] = acc[i][c][e];
    __syncthreads();
    // Four rows of one token per thread.  With two buffers a warp goes on to the
    // next row block at once: the buffer is written again only after the next
    // barrier, which every warp reaches when it has read this one.
    if (splits == 1) {
      for (int o = threadIdx.x; o < C::kRows * 2 * NT; o += kThreads) {
        int at;
        int64_t m;
        int n;
        if (!place(o, rb, at, m, n)) continue;
        float v[4];
        join4<GATED, C::kUp, C::WK>(v, [&](int k) { return sums + k * C::kSums + at; }, C::WK);
        store4(p, m, n, v);
      }
      if (C::kSumBuffers == 1) __syncthreads();
    } else {
      // The CTA's own sum first, over the first warp's; then the cluster's, shared
      // out over its CTAs, with the loads of all CTAs' sums in flight together.
      for (int v = threadIdx.x; v < C::kSums; v += kThreads) {
        float sum = sums[v];
#pragma unroll
        for (int k = 1; k < C::WK; ++k) sum += sums[k * C::kSums + v];
        sums[v] = sum;
      }
      cluster.sync();
      for (int o = rank * kThreads + threadIdx.x; o < C::kRows * 2 * NT; o += splits * kThreads) {
        int at;
        int64_t m;
        int n;
        if (!place(o, rb, at, m, n)) continue;
        float v[4];
        join4<GATED, C::kUp, 8>(
            v, [&](int k) { return cluster.map_shared_rank(sums, k < splits ? k : 0) + at; }, splits);
        store4(p, m, n, v);
      }
      if (C::kSumBuffers == 1) cluster.sync();
    }
  }
  copy_wait<0>();
  if (splits > 1) cluster.sync();   // a CTA's sums stay until every CTA has read them
}

// ---------------------------------------------------------------------------
// Quantizer and its inverse
// ---------------------------------------------------------------------------
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
  const float4 b = __ldcs(reinterpret_cast<const float4*>(p + 4));
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}

// A word of codes 8 + clamp(rne(v / s), -8, 7), by the IEEE quotients: with r the
// correctly rounded 1 / s, one step t + r (v - s t) from t = v r (off by 1.5
// units in the last place at most) gives a neighbour of v / s, and a second one
// the correctly rounded quotient (Markstein, "Computation of elementary functions
// on the IBM RISC System/6000 processor", 1990; the remainders are exact where
// the rounding to an integer depends on them: |v| > s / 4 >= 3e-6).  Added to
// 1.5 2^23 it is rounded to an integer, which stands in the low bits; |v / s| is
// 7 at most.  Infinite scales and NaN take the division.
__device__ __forceinline__ uint32_t code_word(const float (&v)[8], float s, float r) {
  uint32_t word = 0;
  bool special = false;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float t = v[e] * r;
    t = fmaf(fmaf(-t, s, v[e]), r, t);
    t = fmaf(fmaf(-t, s, v[e]), r, t);
    special |= !(fabsf(t) < 8.0f);
    word |= ((__float_as_uint(t + 12582912.0f) + 8u) & 15u) << (4 * (e / 2 + 4 * (e & 1)));
  }
  if (special) {
    word = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = 8 + static_cast<int>(fminf(fmaxf(rintf(__fdiv_rn(v[e], s)), -8.0f), 7.0f));
      word |= static_cast<uint32_t>(c) << (4 * (e / 2 + 4 * (e & 1)));
    }
  }
  return word;
}

// Word i of the codes, counted along the channels (8 each): block i / 16,
// j = i / 4 % 4, t = i % 4; its place in memory.
__device__ __forceinline__ int64_t word_place(int64_t i) {
  return (i & ~int64_t(15)) + 4 * (i & 3) + ((i >> 2) & 3);
}

// s = max(amax of the group, 1e-4) / 7, c = 8 + clamp(rne(w / s), -8, 7) (IEEE
// fp32 divisions).  A thread makes kQuantWords words of 8 channels, 256 words
// apart, with all loads before the first use; G / 8 neighbouring lanes make a
// group.  Memory bound on fp32 weights ([18432, 7168] in groups of 128: 97 us, 6.2
// TB/s), near the issue rate on bf16 ones (92 us, 3.6 TB/s).  (One load in flight
// per warp and a division per element: 183 and 187 us.)
constexpr int kQuantWords = 4;
template <typename T, int G>
__global__ void __launch_bounds__(256)
    quant_int4_kernel(const T* __restrict__ w, uint32_t* __restrict__ q, float* __restrict__ s,
                      int64_t nwords) {
  pdl_trigger();
  pdl_wait();
  constexpr int kCta = 256 * kQuantWords;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * kCta; base < nwords;
       base += static_cast<int64_t>(gridDim.x) * kCta) {
    float v[kQuantWords][8];
#pragma unroll
    for (int u = 0; u < kQuantWords; ++u) {
      const int64_t i = base + u * 256 + threadIdx.x;
      if (i < nwords) {
        load8(w + 8 * i, v[u]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[u][e] = 0.0f;
      }
    }
#pragma unroll
    for (int u = 0; u < kQuantWords; ++u) {
      const int64_t i = base + u * 256 + threadIdx.x;
      float amax = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[u][e]));
#pragma unroll
      for (int off = G / 16; off >= 1; off >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, off));
      const float sc = __fdiv_rn(fmaxf(amax, 1e-4f), 7.0f);
      const uint32_t word = code_word(v[u], sc, __frcp_rn(sc));
      if (i < nwords) {
        q[word_place(i)] = word;
        if (i % (G / 8) == 0) s[i / (G / 8)] = sc;
      }
    }
  }
}

// y = (c - 8) s: the fp32 product, rounded to bf16 or stored.  A thread stores
// 16 bytes: a word's 8 channels in bf16, half of them in fp32.  Bound by the
// stores ([18432, 7168]: bf16 60 us, 5.6 TB/s; fp32 111 us, 5.5 TB/s, 150 us with
// 32 bytes per thread).  In bf16 the loads of two words are in flight before the
// first store, which no later load passes (one word: 65 us); in fp32, with half the
// loads per byte stored, two took 112.
template <typename T>
__global__ void __launch_bounds__(256)
    dequant_int4_kernel(const uint8_t* __restrict__ q, const float* __restrict__ s,
                        T* __restrict__ y, int64_t nwords, int lg) {
  pdl_trigger();
  pdl_wait();
  constexpr int kHalves = static_cast<int>(sizeof(T)) / 2, kV = 8 / kHalves;
  constexpr int kDequantWords = 2 / kHalves;
  const int64_t items = kHalves * nwords, step = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; first < items;
       first += kDequantWords * step) {
    uint32_t w[kDequantWords];
    float sc[kDequantWords];
#pragma unroll
    for (int u = 0; u < kDequantWords; ++u) {
      const int64_t o = first + u * step, i = o / kHalves;
      w[u] = 0;
      sc[u] = 0.0f;
      if (o < items) {
        // the upper four channels are nibbles 2, 3 and 6, 7
        w[u] = __ldca(reinterpret_cast<const uint32_t*>(q) + word_place(i)) >>
               (8 * static_cast<int>(o % kHalves));
        sc[u] = __ldca(s + ((8 * i) >> lg));
      }
    }
#pragma unroll
    for (int u = 0; u < kDequantWords; ++u) {
      const int64_t o = first + u * step;
      if (o >= items) break;
      float v[kV];
#pragma unroll
      for (int e = 0; e < kV; ++e)
        v[e] = static_cast<float>(static_cast<int>((w[u] >> (4 * (e / 2 + 4 * (e & 1)))) & 15u) - 8) * sc[u];
      if constexpr (sizeof(T) == 2) {
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = gemm::pack_bf16x2(v[2 * e], v[2 * e + 1]);
        __stcs(reinterpret_cast<uint4*>(y + 8 * o), make_uint4(h[0], h[1], h[2], h[3]));
      } else {
        __stcs(reinterpret_cast<float4*>(y + 4 * o), make_float4(v[0], v[1], v[2], v[3]));
      }
    }
  }
}

}  // namespace w4
}  // namespace fp8bs
