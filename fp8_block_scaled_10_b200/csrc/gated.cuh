// Kernels around the gate of a feed-forward block, h = silu(g) u with
// g = A Wg^T and u = A Wu^T (the products themselves are gemm.cuh's GATED
// instantiations):
//   gated_reduce_kernel     sums a K split's or split tail's FP32 partials of
//                           g and u and applies the gate;
//   gated_backward_kernel   the gate's backward pass in bf16;
//   gated_backward_quant_kernel  the same with the gradients quantized for
//                           the activation- and weight-gradient GEMMs.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gemm.cuh"
#include "quant.cuh"
#include "sm100.cuh"

namespace fp8bs {
namespace gated {

using gemm::gated_f32;
using gemm::pack_bf16x2;
using gemm::sigmoid_f32;

// ---------------------------------------------------------------------------
// Reduction of the FP32 partials of gated launches
// ---------------------------------------------------------------------------
// K split: partials [splits][M][2 Np], Np = N rounded up to 128.  Split tail
// (tail_tiles > 0): partials [tail_tiles][splits][128][256], the whole tile,
// gate columns first.  Outputs as the GEMM's own epilogue writes them: h bf16
// (y), the bf16 pre-activations (gu, nullable), or act_quant'ed codes of the
// bf16 h (q, s; y nullable).
struct ReduceParams {
  const float* ws;
  __nv_bfloat16* y;
  __nv_bfloat16* gu;
  uint8_t* q;
  float* s;
  int q_ue8m0;
  int64_t M;
  int N;
  int splits;
  int m_tiles, n_tiles, n_group, full_units, tail_tiles;
};

// One warp per row and 128-column block, four columns per lane: a block's
// maximum is then a warp reduction.  Memory bound,
// and a latency at decode sizes, where the partials come from L2.
__global__ void __launch_bounds__(256) gated_reduce_kernel(const ReduceParams p) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * 8;
  const int nblk = (p.N + 127) / 128;
  const int64_t items = p.tail_tiles > 0 ? static_cast<int64_t>(p.tail_tiles) * 128 : p.M * nblk;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); i < items;
       i += nwarps) {
    int64_t row;
    int blk;
    const float* base;
    int64_t up, step;   // offset of up from gate, and from one split to the next
    const int c = 4 * lane;
    if (p.tail_tiles > 0) {
      const int tt = static_cast<int>(i >> 7), r = static_cast<int>(i & 127);
      int m_tile;
      gemm::tile_mn(p.full_units + tt, p.m_tiles, p.n_tiles, p.n_group, m_tile, blk);
      row = static_cast<int64_t>(m_tile) * 128 + r;
      if (row >= p.M) continue;   // the same for the whole warp
      base = p.ws + (static_cast<int64_t>(tt) * p.splits * 128 + r) * 256 + c;
      up = 128;
      step = 128 * 256;
    } else {
      row = i / nblk;
      blk = static_cast<int>(i - row * nblk);
      up = static_cast<int64_t>(nblk) * 128;
      base = p.ws + row * 2 * up + static_cast<int64_t>(blk) * 128 + c;
      step = p.M * 2 * up;
    }
    const int64_t col = static_cast<int64_t>(blk) * 128 + c;
    float g[4] = {0.f, 0.f, 0.f, 0.f}, u[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int sp = 0; sp < p.splits; ++sp) {
      const float4 a = __ldcg(reinterpret_cast<const float4*>(base + sp * step));
      const float4 b = __ldcg(reinterpret_cast<const float4*>(base + sp * step + up));
      g[0] += a.x; g[1] += a.y; g[2] += a.z; g[3] += a.w;
      u[0] += b.x; u[1] += b.y; u[2] += b.z; u[3] += b.w;
    }
    const uint32_t h0 = pack_bf16x2(gated_f32(g[0], u[0]), gated_f32(g[1], u[1]));
    const uint32_t h1 = pack_bf16x2(gated_f32(g[2], u[2]), gated_f32(g[3], u[3]));
    const bool vec = (p.N % 4) == 0 && col + 4 <= p.N;
    auto store4 = [&](__nv_bfloat16* dst, uint32_t a, uint32_t b) {
      if (vec) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(a, b);
      } else {
        uint16_t* d = reinterpret_cast<uint16_t*>(dst);
        const uint32_t w[2] = {a, b};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (col + j < p.N) d[j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
      }
    };
    if (p.gu != nullptr) {
      store4(p.gu + row * 2 * p.N + col, pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3]));
      store4(p.gu + row * 2 * p.N + p.N + col, pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3]));
    }
    if (p.q != nullptr) {   // N % 128 == 0
      float v[8] = {__uint_as_float(h0 << 16), __uint_as_float(h0 & 0xFFFF0000u),
                    __uint_as_float(h1 << 16), __uint_as_float(h1 & 0xFFFF0000u),
                    0.f, 0.f, 0.f, 0.f};
      float amax = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, off));
      const float sc = block_scale(amax, p.q_ue8m0 != 0);
      const float r = __frcp_rn(sc);
      const uint2 cd = p.q_ue8m0 ? quantize8<true>(v, sc, r) : quantize8<false>(v, sc, r);
      *reinterpret_cast<uint32_t*>(p.q + row * p.N + col) = cd.x;
      if (lane == 0) p.s[row * nblk + blk] = sc;
    }
    if (p.y != nullptr) store4(p.y + row * p.N + col, h0, h1);
  }
}

// ---------------------------------------------------------------------------
// Backward pass of the gate
// ---------------------------------------------------------------------------
// With p = sigmoid(g):  dg = dh u p (1 + g (1 - p)),  du = dh g p,  h = g p u.
struct GateGrad {
  float dg, du, h;
};
__device__ __forceinline__ GateGrad gate_grad(float g, float u, float dh) {
  const float p = sigmoid_f32(g);
  const float gp = g * p;
  GateGrad o;
  o.du = dh * gp;
  o.dg = dh * u * fmaf(gp, 1.0f - p, p);
  o.h = gp * u;
  return o;
}

// The same for two elements in packed fp32 arithmetic, all three negated (which
// costs nothing: the negation goes into the reciprocal's argument), as
// neg_quotient2 takes them.
struct NegGateGrad2 {
  float2 dg, du, h;
};
__device__ __forceinline__ NegGateGrad2 neg_gate_grad2(float2 g, float2 u, float2 dh) {
  const float2 one = make_float2(1.0f, 1.0f), minus = make_float2(-1.0f, -1.0f);
  const float2 y = __fmul2_rn(g, make_float2(-gemm::kLog2e, -gemm::kLog2e));
  const float2 d = __ffma2_rn(make_float2(gemm::exp2_ftz(y.x), gemm::exp2_ftz(y.y)), minus, minus);
  const float2 p = make_float2(gemm::rcp_ftz(d.x), gemm::rcp_ftz(d.y));   // -sigmoid(g)
  const float2 gp = __fmul2_rn(g, p);
  NegGateGrad2 o;
  o.du = __fmul2_rn(dh, gp);
  o.h = __fmul2_rn(gp, u);
  o.dg = __fmul2_rn(__fmul2_rn(dh, u), __ffma2_rn(gp, __fadd2_rn(one, p), p));
  return o;
}

// Quotients x / s of two values from their negations y = -x and nr = -RN(1 / s):
// one of quotient2's two correction steps (quant.cuh), with the residual q s - x
// in the place of x - q s.  The estimate is off by two ulps at most, so the step
// leaves an error of 2^-22 ulp before its rounding: the result is the correctly
// rounded quotient unless x / s lies that near to the middle of two fp32 numbers,
// and then one of the two.  (The values come from an approximate sigmoid, 2^-21
// off themselves or more; the second step would change nothing but the time, 233 us
// instead of 204 at [4096, 18432], where fp32 operations are what binds.)
// With these signs a zero keeps its sign (-0: 0 * nr = -0, the residual -0 + 0 = 0,
// and 0 nr + -0 = -0), so there is none to put back.  s is 0 where the scale is
// infinite (the estimate then stands, as in quantize8).
__device__ __forceinline__ float2 neg_quotient2(float2 y, float2 nr, float2 s) {
  const float2 q = __fmul2_rn(y, nr);
  return __ffma2_rn(__ffma2_rn(q, s, y), nr, q);
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// bf16 gu [M, 2N] (gate columns first), dh [M, N] -> dgu [M, 2N] and, unless
// h is null, h [M, N].  A stream of 6 bytes in and 4 or 6 out per element: eight
// columns per thread where N % 8 == 0 and all tensors are 16-byte aligned.  [4096,
// 18432]: 116 us without h, 148 with it, 6.5 and 6.1 TB/s.
__global__ void __launch_bounds__(256)
    gated_backward_kernel(const __nv_bfloat16* __restrict__ gu, const __nv_bfloat16* __restrict__ dh,
                          __nv_bfloat16* __restrict__ dgu, __nv_bfloat16* __restrict__ h, int64_t M,
                          int64_t N) {
  pdl_trigger();
  pdl_wait();
  const int64_t per_row = N / 8;
  const int64_t items = M * per_row;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < items;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t row = i / per_row;
    const int64_t col = (i - row * per_row) * 8;
    const __nv_bfloat16* gp = gu + row * 2 * N + col;
    __nv_bfloat16* dp = dgu + row * 2 * N + col;
    const uint4 g4 = __ldcs(reinterpret_cast<const uint4*>(gp));
    const uint4 u4 = __ldcs(reinterpret_cast<const uint4*>(gp + N));
    const uint4 d4 = __ldcs(reinterpret_cast<const uint4*>(dh + row * N + col));
    const uint32_t gw[4] = {g4.x, g4.y, g4.z, g4.w}, uw[4] = {u4.x, u4.y, u4.z, u4.w};
    const uint32_t dw[4] = {d4.x, d4.y, d4.z, d4.w};
    uint32_t a[4], b[4], c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const GateGrad lo = gate_grad(bf_lo(gw[j]), bf_lo(uw[j]), bf_lo(dw[j]));
      const GateGrad hi = gate_grad(bf_hi(gw[j]), bf_hi(uw[j]), bf_hi(dw[j]));
      a[j] = pack_bf16x2(lo.dg, hi.dg);
      b[j] = pack_bf16x2(lo.du, hi.du);
      c[j] = pack_bf16x2(lo.h, hi.h);
    }
    __stcs(reinterpret_cast<uint4*>(dp), make_uint4(a[0], a[1], a[2], a[3]));
    __stcs(reinterpret_cast<uint4*>(dp + N), make_uint4(b[0], b[1], b[2], b[3]));
    if (h != nullptr)
      __stcs(reinterpret_cast<uint4*>(h + row * N + col), make_uint4(c[0], c[1], c[2], c[3]));
  }
}

// The same for any N and alignment: a CTA takes 2048 columns of a row, eight per
// thread, 256 columns apart (2-byte accesses along the row, all loads before the
// first use; the row and column are the CTA's, so there is no division per element).
// The loads stay in L1: neighbouring warps share the sectors at their ends (streaming
// loads: 209 and 274 us).
// [4096, 18431]: 163 us without h, 207 with it; bound by the accesses, four times as
// many as the wide kernel's per byte.
constexpr int kAnyCols = 8 * 256;
__global__ void __launch_bounds__(256)
    gated_backward_any_kernel(const __nv_bfloat16* __restrict__ gu,
                              const __nv_bfloat16* __restrict__ dh, __nv_bfloat16* __restrict__ dgu,
                              __nv_bfloat16* __restrict__ h, int64_t M, int64_t N) {
  pdl_trigger();
  pdl_wait();
  const int64_t per_row = (N + kAnyCols - 1) / kAnyCols;
  for (int64_t i = blockIdx.x; i < M * per_row; i += gridDim.x) {
    const int64_t row = i / per_row;
    const int64_t col = (i - row * per_row) * kAnyCols + threadIdx.x;
    const __nv_bfloat16* gp = gu + row * 2 * N + col;
    const __nv_bfloat16* dhp = dh + row * N + col;
    __nv_bfloat16 g[8], u[8], d[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      g[j] = u[j] = d[j] = __nv_bfloat16(0.0f);
      if (col + 256 * j < N) {
        g[j] = __ldca(gp + 256 * j);
        u[j] = __ldca(gp + N + 256 * j);
        d[j] = __ldca(dhp + 256 * j);
      }
    }
    __nv_bfloat16* dp = dgu + row * 2 * N + col;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (col + 256 * j >= N) break;
      const GateGrad o = gate_grad(__bfloat162float(g[j]), __bfloat162float(u[j]), __bfloat162float(d[j]));
      dp[256 * j] = __float2bfloat16_rn(o.dg);
      dp[N + 256 * j] = __float2bfloat16_rn(o.du);
      if (h != nullptr) h[row * N + col + 256 * j] = __float2bfloat16_rn(o.h);
    }
  }
}

// The gradients quantized for the two gradient GEMMs, straight from fp32 (no
// rounding to bf16 before the codes: one rounding less than quantizing a bf16
// gradient, and no bf16 gradient in memory):
//   q  [M, 2N],  s  [M, 2N/128]     dgu by 1 x 128 blocks   (activation gradient)
//   qt [2N, Mp], st [2N, Mp/128]    dgu^T by 128 x 1 blocks (weight gradient of gate and up)
//   ht [N, Mp],  hts [N, Mp/128]    h^T by 128 x 1 blocks   (weight gradient of down)
// Mp = M rounded up to 128; the codes of rows past M are zero, so the weight
// gradient GEMM's sum over Mp tokens is the sum over M.
//
// A CTA walks 128 x 128 tiles.  Warp w holds rows 8w..8w+7 and lane l columns
// 4l..4l+3 with all three results in fp32 registers (8 x 4 x 3), so each
// input is read once and exp is computed once.  A row block's maximum is a
// warp reduction; a column block's is the thread's maximum over its rows,
// joined over the 16 warps through shared memory.  Codes of the transposed
// outputs are turned 4 x 4 in registers, then in shared memory (8-byte pieces
// of 8 rows, exclusive-or'ed with the column group, so neither side has bank
// conflicts), and stored 128 bytes per column.  16 warps of 96 results each
// fill the register file, so one CTA runs per SM, and the next tile's inputs
// are copied to shared memory by TMA while this tile is quantized.  [4096,
// 18432]: 204 us, 4.1 TB/s; bound by instructions, not bytes (three results, each
// scaled and rounded along rows or columns or both: half of the issue slots are
// taken, at 4 warps per scheduler; 38 % of the instructions are the ALU pipe's, 39 %
// the FMA pipe's).  (A bulk copy per row measured 658 us: 384 of them per tile.)
constexpr int kBqThreads = 512;
constexpr int kBqInBytes = 3 * 128 * 256;      // g, u, dh: [128 rows][128] bf16
constexpr int kBqTurned = 3 * 128 * 128;       // codes of dg, du, h: [128 columns][128 rows]
constexpr int kBqPart = 3 * 16 * 128 * 4;      // column maxima per warp
constexpr int kBqScale = 2 * 3 * 128 * 4;      // column scales and their negated reciprocals
constexpr int kBqSmem = kBqInBytes + kBqTurned + kBqPart + kBqScale + 16;

// max |v| over the warp (NaN dropped, as fmaxf does).
__device__ __forceinline__ float warp_max_abs(float v) {
  float m;
  asm volatile("redux.sync.max.abs.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}

// max(|a|, |b|, |c|), NaN dropped.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float m;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
  return m;
}

// Codes of two pairs given negated, each value with its own scale.
template <bool UE>
__device__ __forceinline__ uint32_t neg_codes4(const float (&y)[4], const float2 (&nr)[2],
                                               const float2 (&s)[2]) {
  float2 t[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float2 v = make_float2(y[2 * j], y[2 * j + 1]);
    t[j] = UE ? __fmul2_rn(v, nr[j]) : neg_quotient2(v, nr[j], s[j]);
  }
  return e4m3x2(t[0].x, t[0].y) | (e4m3x2(t[1].x, t[1].y) << 16);
}

__device__ __forceinline__ float finite_scale(float s) { return isinf(s) ? 0.0f : s; }

template <bool UE>
__global__ void __launch_bounds__(kBqThreads, 1)
    gated_backward_quant_kernel(const __grid_constant__ CUtensorMap tmap_gu,
                                const __grid_constant__ CUtensorMap tmap_dh,
                                uint8_t* __restrict__ q, float* __restrict__ s,
                                uint8_t* __restrict__ qt, float* __restrict__ st,
                                uint8_t* __restrict__ ht, float* __restrict__ hts, int64_t M,
                                int64_t N) {
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* in = smem;
  uint8_t* turned = smem + kBqInBytes;
  float* part = reinterpret_cast<float*>(smem + kBqInBytes + kBqTurned);
  float* csc = part + 3 * 16 * 128;   // per column: scale (0 for an infinite one), -1 / scale
  float* cnr = csc + 3 * 128;
  uint64_t* bar = reinterpret_cast<uint64_t*>(cnr + 3 * 128);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(bar, 1);
    fence_barrier_init();
  }
  pdl_trigger();
  pdl_wait();
  __syncthreads();
  const int64_t mt = (M + 127) / 128, nt = N / 128;
  const int64_t Mp = mt * 128;
  const int64_t tiles = mt * nt;

  // Thread 0 starts a tile's copies (rows past M arrive as zeros).
  auto start = [&](int64_t tile) {
    const int64_t m_tile = tile / nt, n_tile = tile - m_tile * nt;
    const int32_t x = static_cast<int32_t>(n_tile * 128), y = static_cast<int32_t>(m_tile * 128);
    mbar_arrive_expect_tx(bar, kBqInBytes);
    tma_load_2d(in, &tmap_gu, bar, x, y);
    tma_load_2d(in + 32768, &tmap_gu, bar, static_cast<int32_t>(N) + x, y);
    tma_load_2d(in + 65536, &tmap_dh, bar, x, y);
  };
  if (threadIdx.x == 0 && blockIdx.x < tiles) start(blockIdx.x);
  uint32_t phase = 0;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t m_tile = tile / nt, n_tile = tile - m_tile * nt;
    const int64_t row0 = m_tile * 128 + warp * 8;
    const int64_t col = n_tile * 128 + 4 * lane;
    // No barrier here: a warp starts on its rows as soon as they are there, while
    // others still store the previous tile (what they read is written again only
    // behind the next two barriers).
    const bool ok = mbar_wait(bar, phase, nullptr);
    phase ^= 1u;
    float v[3][8][4];   // -dg, -du, -h
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint8_t* at = in + (warp * 8 + i) * 256 + 8 * lane;
      const uint2 gr = *reinterpret_cast<const uint2*>(at);
      const uint2 ur = *reinterpret_cast<const uint2*>(at + 32768);
      const uint2 dr = *reinterpret_cast<const uint2*>(at + 65536);
      const uint32_t gw[2] = {gr.x, gr.y}, uw[2] = {ur.x, ur.y}, dw[2] = {dr.x, dr.y};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const NegGateGrad2 o = neg_gate_grad2(make_float2(bf_lo(gw[j]), bf_hi(gw[j])),
                                       make_float2(bf_lo(uw[j]), bf_hi(uw[j])),
                                       make_float2(bf_lo(dw[j]), bf_hi(dw[j])));
        v[0][i][2 * j] = o.dg.x;
        v[0][i][2 * j + 1] = o.dg.y;
        v[1][i][2 * j] = o.du.x;
        v[1][i][2 * j + 1] = o.du.y;
        v[2][i][2 * j] = o.h.x;
        v[2][i][2 * j + 1] = o.h.y;
      }
    }
    // 128 x 1 blocks: this thread's share of the maxima.
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      float cm[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        cm[j] = max3_abs(v[k][0][j], v[k][1][j], v[k][2][j]);
        cm[j] = max3_abs(cm[j], v[k][3][j], v[k][4][j]);
        cm[j] = max3_abs(cm[j], v[k][5][j], v[k][6][j]);
        cm[j] = fmaxf(cm[j], fabsf(v[k][7][j]));
      }
      *reinterpret_cast<float4*>(part + (k * 16 + warp) * 128 + 4 * lane) =
          make_float4(cm[0], cm[1], cm[2], cm[3]);
    }
    // The inputs and the previous tile's codes have been read.  (A wait that gave
    // up has reported FP8BS_ERR_TIMEOUT; the copies in flight still have to land
    // before the CTA may leave.)
    if (!__syncthreads_and(ok)) {
      mbar_wait(bar, phase ^ 1u, nullptr);
      return;
    }
    if (threadIdx.x == 0 && tile + gridDim.x < tiles) start(tile + gridDim.x);
    if (threadIdx.x < 384) {
      const int k = threadIdx.x >> 7, c = threadIdx.x & 127;
      float m = 0.0f;
#pragma unroll
      for (int w = 0; w < 16; ++w) m = fmaxf(m, part[(k * 16 + w) * 128 + c]);
      const float sc = block_scale(m, UE);
      csc[threadIdx.x] = finite_scale(sc);
      cnr[threadIdx.x] = -__frcp_rn(sc);
      float* dst = k < 2 ? st + (k * N + n_tile * 128) * mt : hts + n_tile * 128 * mt;
      dst[c * mt + m_tile] = sc;
    }
    // 1 x 128 blocks: the warp's rows, 16 blocks.  Lane 8 k + i makes the scale of
    // row i of output k, once for the warp.
    float amax = 0.0f;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float m = warp_max_abs(
            fmaxf(max3_abs(v[k][i][0], v[k][i][1], v[k][i][2]), fabsf(v[k][i][3])));
        if (lane == 8 * k + i) amax = m;
      }
    const float sc = block_scale(amax, UE);
    const float fin = finite_scale(sc), rcp = -__frcp_rn(sc);
    if (lane < 16 && row0 + (lane & 7) < M)
      s[(row0 + (lane & 7)) * (2 * nt) + (lane >> 3) * nt + n_tile] = sc;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float sk = __shfl_sync(0xFFFFFFFFu, fin, 8 * k + i);
        const float r = __shfl_sync(0xFFFFFFFFu, rcp, 8 * k + i);
        const int64_t row = row0 + i;
        if (row < M) {
          const float2 r2[2] = {make_float2(r, r), make_float2(r, r)};
          const float2 n2[2] = {make_float2(sk, sk), make_float2(sk, sk)};
          __stcs(reinterpret_cast<uint32_t*>(q + row * 2 * N + k * N + col),
                 neg_codes4<UE>(v[k][i], r2, n2));
        }
      }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const float4 nc = *reinterpret_cast<const float4*>(csc + k * 128 + 4 * lane);
      const float4 rc = *reinterpret_cast<const float4*>(cnr + k * 128 + 4 * lane);
      const float2 r2[2] = {make_float2(rc.x, rc.y), make_float2(rc.z, rc.w)};
      const float2 n2[2] = {make_float2(nc.x, nc.y), make_float2(nc.z, nc.w)};
      uint32_t w[2][4];   // [rows 0-3, 4-7][column]
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        uint32_t c[4];    // [row]: four columns' codes
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = neg_codes4<UE>(v[k][4 * b + i], r2, n2);
        const uint32_t x0 = __byte_perm(c[0], c[1], 0x5140), x1 = __byte_perm(c[0], c[1], 0x7362);
        const uint32_t y0 = __byte_perm(c[2], c[3], 0x5140), y1 = __byte_perm(c[2], c[3], 0x7362);
        w[b][0] = __byte_perm(x0, y0, 0x5410);
        w[b][1] = __byte_perm(x0, y0, 0x7632);
        w[b][2] = __byte_perm(x1, y1, 0x5410);
        w[b][3] = __byte_perm(x1, y1, 0x7632);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint2*>(turned + k * 16384 + (4 * lane + j) * 128 +
                                  8 * (warp ^ (lane & 15))) = make_uint2(w[0][j], w[1][j]);
    }
    __syncthreads();
    // A warp stores 24 columns (8 of each output), four at a time: lane / 8 is
    // the column, lane % 8 its 16-byte piece (two 8-byte ones of 8 rows).
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      uint8_t* dst = k < 2 ? qt + (k * N + n_tile * 128) * Mp : ht + n_tile * 128 * Mp;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int c = warp * 8 + 4 * b + (lane >> 3), piece = lane & 7;
        const int key = (c >> 2) & 15;
        const uint8_t* from = turned + k * 16384 + c * 128;
        const uint2 lo = *reinterpret_cast<const uint2*>(from + 8 * ((2 * piece) ^ key));
        const uint2 hi = *reinterpret_cast<const uint2*>(from + 8 * ((2 * piece + 1) ^ key));
        __stcs(reinterpret_cast<uint4*>(dst + c * Mp + m_tile * 128 + 16 * piece),
               make_uint4(lo.x, lo.y, hi.x, hi.y));
      }
    }
  }
}

}  // namespace gated
}  // namespace fp8bs
