// The global norm of a set of gradient tensors and their clipping:
//   norm = sqrt(sum of squares over all elements of all tensors),
//   out  = grad * min(1, max_norm / (norm + 1e-6)).
// Two launches: partial sums per CTA, then a pass that joins the partials (in
// one order, so the norm has the same bits every time) and scales.  Both are
// streams over the tensors cut into chunks; the second pass walks the chunks
// from the last one back, so that what the first pass left in the L2 is read
// there.  The norm alone: 64 x [7168, 2048] fp32 (3.8 GB) in 624 us, 6.0 TB/s.
// Clipping 396 M fp32 gradients (1.59 GB read twice and written once): 751 us, 6.3
// TB/s.  40 tensors, 600 thousand elements: 10 us, two launches' latency.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gemm.cuh"
#include "sm100.cuh"

namespace fp8bs {
namespace clip {

constexpr int kThreads = 512;
constexpr int kChunk = 16384;        // elements of a chunk
constexpr int kMaxTensors = 128;     // of one launch: the table fits 4 KB of kernel arguments

// CTAs of a launch over `chunks` chunks: two per SM.  CTA b of every launch of a call
// sums into slot b, so a call of any number of tensors has 2 sms partials: the
// launches follow one another on the stream, which fixes the order of the sum.
// (Slots of their own for every launch would have to be few per launch to stay
// few: with 2368 in all, 1.6 GB in 2000 tensors took 557 us, now 367, and 8.2 GB in
// 5120 tensors 5.6 ms, now 1.6.)
__host__ __device__ constexpr int max_ctas(int sms) { return 2 * sms; }
__host__ __device__ constexpr int launch_ctas(int chunks, int sms) {
  return chunks < max_ctas(sms) ? chunks : max_ctas(sms);
}

// Tensors of one launch.  Chunk c belongs to the tensor i with
// first[i] <= c < first[i + 1].
struct Table {
  const void* in[kMaxTensors];
  void* out[kMaxTensors];
  int64_t n[kMaxTensors];
  int first[kMaxTensors + 1];
  uint32_t in_bf16[kMaxTensors / 32];
  uint32_t out_bf16[kMaxTensors / 32];
  int count;
};

__device__ __forceinline__ int tensor_of(const Table& t, int chunk) {
  int a = 0, b = t.count;
  while (b - a > 1) {
    const int mid = (a + b) >> 1;
    if (t.first[mid] <= chunk) a = mid; else b = mid;
  }
  return a;
}

__device__ __forceinline__ bool bit(const uint32_t* w, int i) { return (w[i >> 5] >> (i & 31)) & 1u; }

__device__ __forceinline__ void load_vec(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load_vec(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void store_vec(float* p, const float (&v)[8]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
  __stcs(reinterpret_cast<float4*>(p + 4), make_float4(v[4], v[5], v[6], v[7]));
}
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&v)[8]) {
  __stcs(reinterpret_cast<uint4*>(p),
         make_uint4(gemm::pack_bf16x2(v[0], v[1]), gemm::pack_bf16x2(v[2], v[3]),
                    gemm::pack_bf16x2(v[4], v[5]), gemm::pack_bf16x2(v[6], v[7])));
}
__device__ __forceinline__ float load_one(const float* p) { return *p; }
__device__ __forceinline__ float load_one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_one(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_one(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ bool aligned(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

// Squares in 64 bits: neither a large gradient's square overflows nor a small
// one's vanishes, and the sum of 10^9 of them keeps more bits than the
// result.  (64-bit FMAs keep up with the stream: 6 elements per clock and SM
// arrive, 64 can be added.)
template <typename T>
__device__ __forceinline__ double chunk_squares(const T* p, int64_t n) {
  double acc[4] = {0.0, 0.0, 0.0, 0.0};
  if (aligned(p)) {
    const int64_t nv = n / 8;
#pragma unroll 2
    for (int64_t i = threadIdx.x; i < nv; i += kThreads) {
      float v[8];
      load_vec(p + 8 * i, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j & 3] = fma(static_cast<double>(v[j]), static_cast<double>(v[j]), acc[j & 3]);
    }
    for (int64_t i = 8 * nv + threadIdx.x; i < n; i += kThreads) {
      const double v = load_one(p + i);
      acc[0] = fma(v, v, acc[0]);
    }
  } else {
    for (int64_t i = threadIdx.x; i < n; i += kThreads) {
      const double v = load_one(p + i);
      acc[0] = fma(v, v, acc[0]);
    }
  }
  return (acc[0] + acc[1]) + (acc[2] + acc[3]);
}

// Sum over the CTA's threads, in a fixed order; in every thread.
__device__ __forceinline__ double cta_sum(double v, double* smem) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
  if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = v;
  __syncthreads();
  double sum = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) sum += smem[w];
  __syncthreads();
  return sum;
}

// `used`: the slots that earlier launches of the call have written.
__global__ void __launch_bounds__(kThreads)
    norm_partial_kernel(const __grid_constant__ Table t, double* partials, int used) {
  __shared__ double smem[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  double sum = 0.0;
  const int chunks = t.first[t.count];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int i = tensor_of(t, c);
    const int64_t at = static_cast<int64_t>(c - t.first[i]) * kChunk;
    const int64_t n = min(static_cast<int64_t>(kChunk), t.n[i] - at);
    sum += bit(t.in_bf16, i) ? chunk_squares(static_cast<const __nv_bfloat16*>(t.in[i]) + at, n)
                             : chunk_squares(static_cast<const float*>(t.in[i]) + at, n);
  }
  sum = cta_sum(sum, smem);
  if (threadIdx.x == 0) {
    if (static_cast<int>(blockIdx.x) < used) sum += __ldcg(partials + blockIdx.x);
    partials[blockIdx.x] = sum;
  }
}

__device__ __forceinline__ double norm_of(const double* partials, int n, double* smem) {
  double v = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) v += __ldcg(partials + i);
  return sqrt(cta_sum(v, smem));
}

__global__ void __launch_bounds__(kThreads)
    norm_final_kernel(const double* __restrict__ partials, int n, float* __restrict__ norm) {
  __shared__ double smem[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  const double v = norm_of(partials, n, smem);
  if (threadIdx.x == 0) *norm = static_cast<float>(v);
}

template <typename TI, typename TO>
__device__ __forceinline__ void scale_chunk(const TI* p, TO* o, int64_t n, float scale) {
  int64_t done = 0;
  if (aligned(p) && aligned(o)) {
    const int64_t nv = n / 8;
#pragma unroll 2
    for (int64_t i = threadIdx.x; i < nv; i += kThreads) {
      float v[8];
      load_vec(p + 8 * i, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= scale;
      store_vec(o + 8 * i, v);
    }
    done = 8 * nv;
  }
  for (int64_t i = done + threadIdx.x; i < n; i += kThreads) store_one(o + i, load_one(p + i) * scale);
}

// A norm that is NaN scales by NaN, an infinite one by 0 whatever the bound (an
// infinite gradient then becomes NaN): nothing that went wrong is passed on as a
// plausible step.  In place and with nothing to clip, nothing is written:
// times 1 is the value that stands there.
__global__ void __launch_bounds__(kThreads)
    clip_scale_kernel(const __grid_constant__ Table t, const double* __restrict__ partials, int n,
                      double max_norm, float* __restrict__ norm) {
  __shared__ double smem[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  const double v = norm_of(partials, n, smem);
  if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(v);
  const double r = isinf(v) ? 0.0 : max_norm / (v + 1e-6);
  const float scale = r >= 1.0 ? 1.0f : static_cast<float>(r);
  const int chunks = t.first[t.count];
  for (int c = chunks - 1 - static_cast<int>(blockIdx.x); c >= 0; c -= gridDim.x) {
    const int i = tensor_of(t, c);
    const int64_t at = static_cast<int64_t>(c - t.first[i]) * kChunk;
    const int64_t m = min(static_cast<int64_t>(kChunk), t.n[i] - at);
    if (scale == 1.0f && t.in[i] == t.out[i]) continue;
    const bool ib = bit(t.in_bf16, i), ob = bit(t.out_bf16, i);
    using B = __nv_bfloat16;
    if (ib && ob) scale_chunk(static_cast<const B*>(t.in[i]) + at, static_cast<B*>(t.out[i]) + at, m, scale);
    else if (ib) scale_chunk(static_cast<const B*>(t.in[i]) + at, static_cast<float*>(t.out[i]) + at, m, scale);
    else if (ob) scale_chunk(static_cast<const float*>(t.in[i]) + at, static_cast<B*>(t.out[i]) + at, m, scale);
    else scale_chunk(static_cast<const float*>(t.in[i]) + at, static_cast<float*>(t.out[i]) + at, m, scale);
  }
}

}  // namespace clip
}  // namespace fp8bs
