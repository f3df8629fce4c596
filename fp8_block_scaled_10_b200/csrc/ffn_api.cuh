// Entry points of the feed-forward operators (declared in include/fp8bs.h):
// the gated projections and the gate's backward pass, the linear layers on
// 4-bit weights, the gradient norm and clipping.  Part of fp8bs.cu's
// translation unit: it uses that file's checks, launches and tensor maps.
#pragma once

namespace fp8bs {
namespace {

// ---------------------------------------------------------------------------
// Gated projections
// ---------------------------------------------------------------------------
struct GatedOperands {
  const uint8_t* a;
  const float* a_s;
  const uint8_t* gate;
  const float* gate_s;
  const uint8_t* up;
  const float* up_s;
};

struct GatedOutputs {
  uint16_t* h = nullptr;    // bf16 [M, N]
  uint16_t* gu = nullptr;   // bf16 [M, 2N]
  uint8_t* q = nullptr;     // FP8 output: codes [M, N] and scales [M, N / 128]
  float* s = nullptr;
  bool ue8m0 = false;
};

// An empty problem: well-formed sizes and no rows (empty tensors have no
// address, so the pointers are not looked at).
bool gated_empty(int64_t M, int64_t N, int64_t K) {
  return M == 0 && N > 0 && N <= (1 << 30) && K > 0 && K % 128 == 0;
}

fp8bs_status check_gated(const GatedOperands& o, const void* out, int64_t N, int64_t K) {
  fp8bs_status r = check_gemm_operands(o.a, o.a_s, o.gate, o.gate_s, out, N, K);
  if (r != FP8BS_OK) return r;
  return check_gemm_operands(o.a, o.a_s, o.up, o.up_s, out, N, K);
}

// The gu map: bf16 [M, 2N] in boxes of 32 rows x 32 columns, 64-byte swizzle.
// Boxes of gate columns must not reach into the up columns: N % 32 == 0, else
// the epilogue stores directly.
fp8bs_status make_tmap_gu(CUtensorMap* map, const uint16_t* gu, int64_t M, int64_t N, int* gu_tma) {
  memset(map, 0, sizeof(*map));
  *gu_tma = 0;
  if (gu == nullptr || N % 32 != 0) return FP8BS_OK;
  return make_tmap_out(map, gu, nullptr, M, 2 * N, 1, gu_tma);
}

// bf16 [rows, cols] read in boxes of 128 x 128, not swizzled; rows past the last
// read as zero.
fp8bs_status make_tmap_bf16(CUtensorMap* map, const uint16_t* base, int64_t rows, int64_t cols) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * 2u};
  const cuuint32_t box[2] = {128u, 128u};
  const cuuint32_t elem[2] = {1u, 1u};
  const CUresult cr = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(base),
                               dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                               CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (cr != CUDA_SUCCESS) return fail(FP8BS_ERR_CUDA, "cuTensorMapEncodeTiled (bf16) failed (%d)", (int)cr);
  return FP8BS_OK;
}

template <int AR, bool G>
cudaError_t launch_gated(const CUtensorMap& ta, const CUtensorMap& tg, const CUtensorMap& ty,
                         const CUtensorMap& tu, const CUtensorMap& tgu, const gemm::Params& p,
                         int grid, cudaStream_t st) {
  using C = gemm::Cfg<256, AR>;
  return launch(gemm::fp8_gemm_kernel<256, G, AR, false, false, false, true>, grid, C::kThreads,
                C::gated_smem_bytes(G), st, ta, tg, ty, tu, tgu, p);
}

// FP32 partials of a gated plan: 2 Np columns, Np = N rounded up to whole tiles.
int64_t gated_partial_cols(int64_t N) { return 2 * 128 * ((N + 127) / 128); }
size_t gated_workspace(const Plan& pl, int64_t M, int64_t N) {
  return plan_workspace(pl, M, gated_partial_cols(N));
}

fp8bs_status run_gated(const GatedOperands& o, int64_t M, int64_t N, int64_t K,
                       const GatedOutputs& out, void* ws, size_t ws_bytes, cudaStream_t st) {
  if (gated_empty(M, N, K)) return FP8BS_OK;
  fp8bs_status r = check_gated(o, out.q ? static_cast<const void*>(out.q) : out.h, N, K);
  if (r != FP8BS_OK) return r;
  if (!aligned16(out.h) || !aligned16(out.gu))
    return fail(FP8BS_ERR_INVALID_ARG, "h and gu must be 16-byte aligned");
  if (M < 0 || M >= (int64_t(1) << 31) - 128) return fail(FP8BS_ERR_INVALID_ARG, "M out of range");
  if (gemm_too_large(M, N)) return fail(FP8BS_ERR_INVALID_ARG, "M x N too large (tile count)");
  int dev;
  DeviceInfo* info;
  if ((r = device_setup(&dev, &info)) != FP8BS_OK) return r;
  const Plan pl = plan_gemm(M, N, K, info->sms, GemmKind::kGated);
  const size_t need = gated_workspace(pl, M, N);
  if (need > 0 && (ws == nullptr || ws_bytes < need || !aligned16(ws)))
    return fail(FP8BS_ERR_WORKSPACE, "workspace of %zu bytes (16-byte aligned) required", need);
  CUtensorMap ta, tg, tu, ty, tgu;
  gemm::Params p{};
  const int a_rows = a_rows_for(M);
  if ((r = make_tmap(&ta, o.a, M, K, a_rows)) != FP8BS_OK) return r;
  if ((r = make_tmap(&tg, o.gate, N, K, 128)) != FP8BS_OK) return r;
  if ((r = make_tmap(&tu, o.up, N, K, 128)) != FP8BS_OK) return r;
  if ((r = make_tmap_gu(&tgu, out.gu, M, N, &p.gu_tma)) != FP8BS_OK) return r;
  memset(&ty, 0, sizeof(ty));
  if (pl.splits > 1) {
    // FP32 partials; the reduction writes the outputs.
    if ((r = make_tmap_out(&ty, nullptr, ws, M, gated_partial_cols(N), pl.splits, &p.y_tma)) != FP8BS_OK)
      return r;
  } else if (out.q != nullptr) {
    if ((r = make_tmap_codes(&ty, out.q, M, N)) != FP8BS_OK) return r;
    p.y_tma = 3;
  } else if ((r = make_tmap_out(&ty, out.h, nullptr, M, N, 1, &p.y_tma)) != FP8BS_OK) {
    return r;
  }
  p.sa = o.a_s;
  p.sw = o.gate_s;
  p.sw_up = o.up_s;
  p.y = reinterpret_cast<__nv_bfloat16*>(out.h);
  p.gu = reinterpret_cast<__nv_bfloat16*>(out.gu);
  p.q_out = out.q;
  p.s_out = out.s;
  p.q_ue8m0 = out.ue8m0 ? 1 : 0;
  p.ws = static_cast<float*>(ws);
  set_schedule(p, pl, M, N, K);
  p.tail_ws = pl.tail_splits > 0 ? static_cast<float*>(ws) : nullptr;
  cudaError_t e = a_rows == 16   ? launch_gated<16, false>(ta, tg, ty, tu, tgu, p, pl.grid, st)
                  : a_rows == 64 ? launch_gated<64, false>(ta, tg, ty, tu, tgu, p, pl.grid, st)
                                 : launch_gated<128, false>(ta, tg, ty, tu, tgu, p, pl.grid, st);
  if (e != cudaSuccess) return cuda_fail(e, "fp8_gemm_gated launch");
  if (need > 0) {
    gated::ReduceParams rp{};
    rp.ws = static_cast<const float*>(ws);
    rp.y = p.y;
    rp.gu = p.gu;
    rp.q = out.q;
    rp.s = out.s;
    rp.q_ue8m0 = p.q_ue8m0;
    rp.M = M;
    rp.N = static_cast<int>(N);
    rp.splits = pl.tail_splits > 0 ? pl.tail_splits : pl.splits;
    rp.m_tiles = pl.m_tiles;
    rp.n_tiles = pl.n_tiles;
    rp.n_group = pl.n_group;
    rp.full_units = pl.full_units;
    rp.tail_tiles = pl.tail_tiles;
    const int64_t warps = pl.tail_tiles > 0 ? int64_t(pl.tail_tiles) * 128 : M * ((N + 127) / 128);
    e = launch(gated::gated_reduce_kernel, grid_for(warps, 8, info->sms * 8), 256, 0, st, rp);
    if (e != cudaSuccess) return cuda_fail(e, "gated reduce launch");
  }
  return FP8BS_OK;
}

// Workspace of the whole block: codes and scales of x and of h, and the split
// scratch that its two GEMMs use in turn (the stream orders them).
struct FfnScratch {
  size_t xq, xs, hq, hs, ws, ws_bytes, bytes;
};

FfnScratch ffn_scratch(int64_t M, int64_t N, int64_t K, int64_t K_out, int sms) {
  FfnScratch f{};
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t p = at;
    at = (at + n + 255) & ~static_cast<size_t>(255);
    return p;
  };
  f.xq = take(static_cast<size_t>(M) * K);
  f.xs = take(static_cast<size_t>(M) * (K / 128) * 4);
  f.hq = take(static_cast<size_t>(M) * N);
  f.hs = take(static_cast<size_t>(M) * (N / 128) * 4);
  f.ws_bytes = std::max(gated_workspace(plan_gemm(M, N, K, sms, GemmKind::kGated), M, N),
                        plan_workspace(plan_gemm(M, K_out, N, sms), M, K_out));
  f.ws = take(f.ws_bytes);
  f.bytes = at;
  return f;
}

// ---------------------------------------------------------------------------
// 4-bit linears
// ---------------------------------------------------------------------------
int int4_group_log2(int64_t group) { return group == 32 ? 5 : group == 64 ? 6 : group == 128 ? 7 : -1; }

fp8bs_status check_int4(int64_t N, int64_t K, int64_t group) {
  if (int4_group_log2(group) < 0)
    return fail(FP8BS_ERR_UNSUPPORTED, "group=%lld (32, 64 and 128 are implemented)", (long long)group);
  if (K <= 0 || K % 128 != 0 || K > (1 << 24))
    return fail(FP8BS_ERR_INVALID_ARG, "K=%lld must be a positive multiple of 128, 2^24 at most", (long long)K);
  if (N < 0 || N > (1 << 30)) return fail(FP8BS_ERR_INVALID_ARG, "N=%lld out of range", (long long)N);
  return FP8BS_OK;
}

// Launch of a 4-bit linear kernel in clusters of `splits` CTAs along x.
struct Int4Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  Int4Launch(int threads, int smem, cudaStream_t st) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
  }
  void grid(int64_t clusters, int splits, int64_t passes) {
    attr[1].val.clusterDim.x = static_cast<unsigned>(splits);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * splits), static_cast<unsigned>(passes));
  }
};

// The runtime's answer for one kernel: clusters of `size` CTAs that the GPU holds at once.
template <typename Kernel>
auto cluster_query(Kernel* kernel, const Int4Launch& like) {
  return [kernel, &like](int size, int* clusters) {
    Int4Launch l = like;
    l.cfg.attrs = l.attr;
    l.grid(1, size, 1);
    return cudaOccupancyMaxActiveClusters(clusters, kernel, &l.cfg);
  };
}

template <int NT, int G, bool GATED>
cudaError_t launch_int4(const w4::Params& p, int dev, cudaStream_t st) {
  using C = w4::Cfg<NT, G, GATED>;
  static ClusterSlots<kMaxDevices> slots;
  auto kernel = w4::int4_linear_kernel<NT, G, GATED>;
  Int4Launch l(w4::kThreads, C::kSmem, st);
  const int64_t blocks = (p.N + C::kRows - 1) / C::kRows;
  // Measured: a join costs about 3 blocks of a warp, with or without a cluster.
  ClusterChoice c;
  const cudaError_t e =
      choose_cluster(blocks, p.K / 128, C::WK, 3, 0, slots.of(dev), cluster_query(kernel, l), &c);
  if (e != cudaSuccess) return e;
  // A cluster walks several row blocks where there are more than fit.
  l.grid(std::min<int64_t>(blocks, c.at_once), c.size, 1);
  return cudaLaunchKernelEx(&l.cfg, kernel, p);
}

// The tensor-core form: 128 weight rows per CTA, one CTA per SM.
template <int G, bool GATED>
cudaError_t launch_int4_tile(const CUtensorMap& q0, const CUtensorMap& q1, const CUtensorMap& x,
                             const w4::Params& p, int dev, cudaStream_t st) {
  static ClusterSlots<kMaxDevices> slots;
  auto kernel = w4::int4_tile_kernel<G, GATED>;
  Int4Launch l(w4::kTileThreads, w4::kTileSmem, st);
  const int rows = GATED ? 64 : 128;
  const int64_t tiles = (p.N + rows - 1) / rows;
  const int64_t passes = (p.M + w4::kTok - 1) / w4::kTok;
  // Measured: a CTA's start and end cost 12 of its blocks (0.45 us each), a
  // cluster's join 6 more.
  ClusterChoice c;
  const cudaError_t e =
      choose_cluster(tiles * passes, p.K / 128, 1, 12, 6, slots.of(dev), cluster_query(kernel, l), &c);
  if (e != cudaSuccess) return e;
  l.grid(tiles, c.size, passes);
  return cudaLaunchKernelEx(&l.cfg, kernel, q0, q1, x, p);
}

// Codes [N, K/2] in boxes of `rows` x 64 bytes, 64-byte swizzle.
fp8bs_status make_tmap_int4(CUtensorMap* map, const uint8_t* q, int64_t N, int64_t K, int rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K / 2), static_cast<cuuint64_t>(N)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K / 2)};
  const cuuint32_t box[2] = {64u, static_cast<cuuint32_t>(rows)};
  const cuuint32_t elem[2] = {1u, 1u};
  const CUresult cr = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(q), dims,
                               strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                               CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (cr != CUDA_SUCCESS) return fail(FP8BS_ERR_CUDA, "cuTensorMapEncodeTiled (int4) failed (%d)", (int)cr);
  return FP8BS_OK;
}

// Tokens [M, K] bf16 in boxes of `tokens` x 64 channels, 128-byte swizzle;
// tokens past the last read as zero.
fp8bs_status make_tmap_tokens(CUtensorMap* map, const uint16_t* x, int64_t M, int64_t K, int tokens) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(M)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K) * 2u};
  const cuuint32_t box[2] = {64u, static_cast<cuuint32_t>(tokens)};
  const cuuint32_t elem[2] = {1u, 1u};
  const CUresult cr = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(x),
                               dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (cr != CUDA_SUCCESS) return fail(FP8BS_ERR_CUDA, "cuTensorMapEncodeTiled (tokens) failed (%d)", (int)cr);
  return FP8BS_OK;
}

// Up to 16 tokens: the weight stream through mma.sync's small tiles.  More: the
// tensor-core form, 32 tokens per pass.  (Both sides of the limit were measured:
// the kernel's comment has the figures.)
template <bool GATED, int G>
fp8bs_status launch_int4_group(const w4::Params& p, int dev, cudaStream_t st) {
  cudaError_t e;
  if (p.M <= 8) {
    e = launch_int4<1, G, GATED>(p, dev, st);
  } else if (p.M <= 16) {
    e = launch_int4<2, G, GATED>(p, dev, st);
  } else {
    CUtensorMap q0, q1, x;
    fp8bs_status r;
    const int rows = GATED ? 64 : 128;
    if ((r = make_tmap_int4(&q0, p.q[0], p.N, p.K, rows)) != FP8BS_OK) return r;
    if ((r = make_tmap_int4(&q1, GATED ? p.q[1] : p.q[0], p.N, p.K, rows)) != FP8BS_OK) return r;
    if ((r = make_tmap_tokens(&x, reinterpret_cast<const uint16_t*>(p.x), p.M, p.K, w4::kTok)) != FP8BS_OK)
      return r;
    e = launch_int4_tile<G, GATED>(q0, q1, x, p, dev, st);
  }
  if (e != cudaSuccess) return cuda_fail(e, "int4_linear launch");
  return FP8BS_OK;
}

template <bool GATED>
fp8bs_status launch_int4_any(const w4::Params& p, int64_t group, int dev, cudaStream_t st) {
  return group == 32   ? launch_int4_group<GATED, 32>(p, dev, st)
         : group == 64 ? launch_int4_group<GATED, 64>(p, dev, st)
                       : launch_int4_group<GATED, 128>(p, dev, st);
}

// Documented limit; the grid's y would hold 65535 passes.
constexpr int64_t kInt4MaxTokens = 524280;
static_assert(kInt4MaxTokens <= 65535ll * w4::kTok, "passes of one launch");

fp8bs_status run_int4(const uint16_t* x, int64_t M, const uint8_t* q0, const float* s0,
                      const uint8_t* q1, const float* s1, bool gated, int64_t N, int64_t K,
                      int64_t group, void* y, fp8bs_dtype y_dtype, cudaStream_t st) {
  fp8bs_status r = check_int4(N, K, group);
  if (r != FP8BS_OK) return r;
  if (M < 0 || M > kInt4MaxTokens) return fail(FP8BS_ERR_INVALID_ARG, "M=%lld out of range", (long long)M);
  if (y_dtype != FP8BS_DTYPE_BF16 && y_dtype != FP8BS_DTYPE_F32)
    return fail(FP8BS_ERR_INVALID_ARG, "y_dtype");
  if (M == 0 || N == 0) return FP8BS_OK;
  if (!x || !q0 || !s0 || !y || (gated && (!q1 || !s1)))
    return fail(FP8BS_ERR_INVALID_ARG, "null operand pointer");
  if (!aligned16(x) || !aligned16(q0) || !aligned16(q1) || !aligned16(s0) || !aligned16(s1) || !aligned16(y))
    return fail(FP8BS_ERR_INVALID_ARG, "operands must be 16-byte aligned");
  int dev;
  DeviceInfo* info;
  if ((r = device_setup(&dev, &info)) != FP8BS_OK) return r;
  w4::Params p{};
  p.x = reinterpret_cast<const __nv_bfloat16*>(x);
  p.q[0] = q0;
  p.q[1] = q1;
  p.s[0] = s0;
  p.s[1] = s1;
  p.y = y;
  p.M = M;
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.y_f32 = y_dtype == FP8BS_DTYPE_F32 ? 1 : 0;
  return gated ? launch_int4_any<true>(p, group, dev, st)
               : launch_int4_any<false>(p, group, dev, st);
}

template <typename T>
cudaError_t launch_quant_int4(const T* w, uint8_t* q, float* s, int64_t words, int64_t group,
                              int sms, cudaStream_t st) {
  const int grid = grid_for(words, 256 * w4::kQuantWords, sms * 8);
  uint32_t* q4 = reinterpret_cast<uint32_t*>(q);
  return group == 32   ? launch(w4::quant_int4_kernel<T, 32>, grid, 256, 0, st, w, q4, s, words)
         : group == 64 ? launch(w4::quant_int4_kernel<T, 64>, grid, 256, 0, st, w, q4, s, words)
                       : launch(w4::quant_int4_kernel<T, 128>, grid, 256, 0, st, w, q4, s, words);
}

// ---------------------------------------------------------------------------
// Gradient norm and clipping
// ---------------------------------------------------------------------------
struct Range {
  uintptr_t lo, hi;
  int64_t index;
  bool operator<(const Range& o) const { return lo < o.lo; }
};

fp8bs_status check_grads(const void* const* grads, const int64_t* numel, const fp8bs_dtype* dtypes,
                         int64_t n) {
  if (n < 0 || n > (1 << 20)) return fail(FP8BS_ERR_INVALID_ARG, "n=%lld tensors", (long long)n);
  if (n > 0 && (!grads || !numel || !dtypes)) return fail(FP8BS_ERR_INVALID_ARG, "null array");
  int64_t chunks = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (numel[i] < 0 || numel[i] > (int64_t(1) << 42))
      return fail(FP8BS_ERR_INVALID_ARG, "tensor %lld: %lld elements", (long long)i, (long long)numel[i]);
    if (dtypes[i] != FP8BS_DTYPE_BF16 && dtypes[i] != FP8BS_DTYPE_F32)
      return fail(FP8BS_ERR_INVALID_ARG, "tensor %lld: dtype", (long long)i);
    if (numel[i] > 0 && !grads[i]) return fail(FP8BS_ERR_INVALID_ARG, "tensor %lld: null pointer", (long long)i);
    const uintptr_t mask = dtypes[i] == FP8BS_DTYPE_BF16 ? 1u : 3u;
    if (reinterpret_cast<uintptr_t>(grads[i]) & mask)
      return fail(FP8BS_ERR_INVALID_ARG, "tensor %lld is not aligned to its type", (long long)i);
    chunks += (numel[i] + clip::kChunk - 1) / clip::kChunk;
    if (chunks >= (int64_t(1) << 31) - 1) return fail(FP8BS_ERR_INVALID_ARG, "too many elements");
  }
  return FP8BS_OK;
}

// No output may share memory with another output, nor with another tensor's
// gradient, nor with part of its own: two CTAs would then write, or write and
// read, the same element.  An output may be its own gradient.
fp8bs_status check_outputs(const void* const* grads, void* const* outs, const int64_t* numel,
                           const fp8bs_dtype* dtypes, const fp8bs_dtype* out_dtypes, int64_t n) {
  if (n == 0) return FP8BS_OK;
  // (No exception may leave the C entry that this is called from.)
  const std::unique_ptr<Range[]> ranges(new (std::nothrow) Range[static_cast<size_t>(n)]);
  if (!ranges) return fail(FP8BS_ERR_WORKSPACE, "no host memory for the ranges of %lld outputs", (long long)n);
  Range* const r = ranges.get();
  Range* end = r;
  auto bytes = [](fp8bs_dtype t) { return t == FP8BS_DTYPE_BF16 ? 2 : 4; };
  for (int64_t i = 0; i < n; ++i) {
    if (numel[i] == 0) continue;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(outs[i]);
    *end++ = {lo, lo + static_cast<uintptr_t>(numel[i]) * bytes(out_dtypes[i]), i};
  }
  std::sort(r, end);
  for (const Range* o = r + 1; o < end; ++o)
    if (o->lo < o[-1].hi)
      return fail(FP8BS_ERR_INVALID_ARG, "outputs %lld and %lld overlap", (long long)o[-1].index,
                  (long long)o->index);
  for (int64_t i = 0; i < n; ++i) {
    if (numel[i] == 0) continue;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(grads[i]);
    const uintptr_t hi = lo + static_cast<uintptr_t>(numel[i]) * bytes(dtypes[i]);
    const Range* it = std::upper_bound(r, end, Range{lo, 0, 0});
    if (it != r) --it;
    for (; it != end && it->lo < hi; ++it) {
      if (it->hi <= lo) continue;
      if (it->index == i && outs[i] == grads[i] && out_dtypes[i] == dtypes[i]) continue;
      return fail(FP8BS_ERR_INVALID_ARG, "output %lld overlaps gradient %lld", (long long)it->index,
                  (long long)i);
    }
  }
  return FP8BS_OK;
}

// The table of tensors [i0, i1), outputs optional.
void fill_table(clip::Table* t, const void* const* grads, void* const* outs, const int64_t* numel,
                const fp8bs_dtype* dtypes, const fp8bs_dtype* out_dtypes, int64_t i0, int64_t i1) {
  memset(t, 0, sizeof(*t));
  int chunks = 0;
  for (int64_t i = i0; i < i1; ++i) {
    if (numel[i] == 0) continue;
    const int k = t->count++;
    t->in[k] = grads[i];
    t->out[k] = outs ? outs[i] : nullptr;
    t->n[k] = numel[i];
    t->first[k] = chunks;
    if (dtypes[i] == FP8BS_DTYPE_BF16) t->in_bf16[k >> 5] |= 1u << (k & 31);
    if (outs && out_dtypes[i] == FP8BS_DTYPE_BF16) t->out_bf16[k >> 5] |= 1u << (k & 31);
    chunks += static_cast<int>((numel[i] + clip::kChunk - 1) / clip::kChunk);
  }
  t->first[t->count] = chunks;
}

// Launches the partial sums; *partials receives the number of their slots.
fp8bs_status run_norm_partials(const void* const* grads, const int64_t* numel,
                               const fp8bs_dtype* dtypes, int64_t n, double* ws, int sms,
                               cudaStream_t st, int* partials) {
  *partials = 0;
  for (int64_t i = 0; i < n; i += clip::kMaxTensors) {
    clip::Table t;
    fill_table(&t, grads, nullptr, numel, dtypes, nullptr, i, std::min<int64_t>(n, i + clip::kMaxTensors));
    if (t.first[t.count] == 0) continue;
    const int grid = clip::launch_ctas(t.first[t.count], sms);
    const cudaError_t e = launch(clip::norm_partial_kernel, grid, clip::kThreads, 0, st, t, ws, *partials);
    if (e != cudaSuccess) return cuda_fail(e, "grad_norm launch");
    *partials = std::max(*partials, grid);
  }
  return FP8BS_OK;
}

size_t norm_workspace(int sms) { return sizeof(double) * static_cast<size_t>(clip::max_ctas(sms)); }

}  // namespace
}  // namespace fp8bs

extern "C" {

size_t fp8bs_gemm_gated_workspace_size(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0 || K % 128 != 0 || gemm_too_large(M, N)) return 0;
  int dev;
  DeviceInfo* info;
  if (device_setup(&dev, &info) != FP8BS_OK) return 0;
  return gated_workspace(plan_gemm(M, N, K, info->sms, GemmKind::kGated), M, N);
}

fp8bs_status fp8bs_fp8_gemm_gated(const uint8_t* a, const float* a_s, const uint8_t* w_gate,
                                  const float* w_gate_s, const uint8_t* w_up, const float* w_up_s,
                                  int64_t M, int64_t N, int64_t K, uint16_t* h, uint16_t* gu,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  GatedOutputs out;
  out.h = h;
  out.gu = gu;
  return run_gated({a, a_s, w_gate, w_gate_s, w_up, w_up_s}, M, N, K, out, workspace,
                   workspace_bytes, as_stream(stream));
}

fp8bs_status fp8bs_fp8_gemm_gated_quant(const uint8_t* a, const float* a_s, const uint8_t* w_gate,
                                        const float* w_gate_s, const uint8_t* w_up,
                                        const float* w_up_s, int64_t M, int64_t N, int64_t K,
                                        fp8bs_scale_fmt out_fmt, uint8_t* q_out, float* s_out,
                                        uint16_t* h, void* workspace, size_t workspace_bytes,
                                        void* stream) {
  if (N <= 0 || N % 128 != 0)
    return fail(FP8BS_ERR_INVALID_ARG, "N=%lld must be a multiple of 128 (1x128 output blocks)",
                (long long)N);
  if (out_fmt != FP8BS_SCALE_FMT_NONE && out_fmt != FP8BS_SCALE_FMT_UE8M0)
    return fail(FP8BS_ERR_INVALID_ARG, "out_fmt");
  if (gated_empty(M, N, K)) return FP8BS_OK;
  if (q_out == nullptr) return fail(FP8BS_ERR_INVALID_ARG, "null operand pointer");
  if (s_out == nullptr || (reinterpret_cast<uintptr_t>(s_out) & 3u))
    return fail(FP8BS_ERR_INVALID_ARG, "s_out must be a 4-byte aligned device pointer");
  GatedOutputs out;
  out.h = h;
  out.q = q_out;
  out.s = s_out;
  out.ue8m0 = out_fmt == FP8BS_SCALE_FMT_UE8M0;
  return run_gated({a, a_s, w_gate, w_gate_s, w_up, w_up_s}, M, N, K, out, workspace,
                   workspace_bytes, as_stream(stream));
}

size_t fp8bs_gated_ffn_workspace_size(int64_t M, int64_t N, int64_t K, int64_t K_out) {
  if (M <= 0 || N <= 0 || N % 128 != 0 || K <= 0 || K % 128 != 0 || K_out <= 0 ||
      gemm_too_large(M, N) || gemm_too_large(M, K_out))
    return 0;
  int dev;
  DeviceInfo* info;
  if (device_setup(&dev, &info) != FP8BS_OK) return 0;
  return ffn_scratch(M, N, K, K_out, info->sms).bytes;
}

fp8bs_status fp8bs_fp8_gated_ffn(const uint16_t* x, int64_t M, int64_t K, const float* x_scales,
                                 int64_t x_scales_row_stride, fp8bs_scale_fmt fmt,
                                 const uint8_t* w_gate, const float* w_gate_s, const uint8_t* w_up,
                                 const float* w_up_s, int64_t N, const uint8_t* w_down,
                                 const float* w_down_s, int64_t K_out, uint16_t* y, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  if (K <= 0 || K % 128 != 0 || N <= 0 || N % 128 != 0)
    return fail(FP8BS_ERR_INVALID_ARG, "K=%lld and N=%lld must be positive multiples of 128",
                (long long)K, (long long)N);
  if (K > (1 << 30) || N > (1 << 30) || K_out <= 0 || K_out > (1 << 30))
    return fail(FP8BS_ERR_INVALID_ARG, "size out of range");
  if (fmt != FP8BS_SCALE_FMT_NONE && fmt != FP8BS_SCALE_FMT_UE8M0)
    return fail(FP8BS_ERR_INVALID_ARG, "scale_fmt");
  if (M < 0 || M >= (int64_t(1) << 31) - 128 || gemm_too_large(M, N) || gemm_too_large(M, K_out))
    return fail(FP8BS_ERR_INVALID_ARG, "M=%lld out of range", (long long)M);
  if (M == 0) return FP8BS_OK;
  // Everything is checked before the first launch.
  fp8bs_status r = check_gemm_operands(w_gate, w_gate_s, w_up, w_up_s, y, N, K);
  if (r != FP8BS_OK) return r;
  if ((r = check_gemm_operands(w_down, w_down_s, w_down, w_down_s, y, K_out, N)) != FP8BS_OK) return r;
  if (!x || !aligned16(x)) return fail(FP8BS_ERR_INVALID_ARG, "x must be a 16-byte aligned device pointer");
  if (x_scales != nullptr && ((reinterpret_cast<uintptr_t>(x_scales) & 3u) ||
                              (x_scales_row_stride != 0 && x_scales_row_stride < K / 128)))
    return fail(FP8BS_ERR_INVALID_ARG, "x_scales: alignment or row stride");
  int dev;
  DeviceInfo* info;
  if ((r = device_setup(&dev, &info)) != FP8BS_OK) return r;
  const FfnScratch w = ffn_scratch(M, N, K, K_out, info->sms);
  if (!workspace || workspace_bytes < w.bytes || !aligned16(workspace))
    return fail(FP8BS_ERR_WORKSPACE, "workspace of %zu bytes (16-byte aligned) required", w.bytes);
  uint8_t* base = static_cast<uint8_t*>(workspace);
  uint8_t* xq = base + w.xq;
  float* xs = reinterpret_cast<float*>(base + w.xs);
  r = x_scales != nullptr
          ? fp8bs_act_quant_static(x, FP8BS_DTYPE_BF16, M, K, 128, x_scales, x_scales_row_stride, xq,
                                   xs, stream)
          : run_act_quant(x, FP8BS_DTYPE_BF16, M, K, 128, fmt, xq, xs, as_stream(stream));
  if (r != FP8BS_OK) return r;
  GatedOutputs out;
  out.q = base + w.hq;
  out.s = reinterpret_cast<float*>(base + w.hs);
  out.ue8m0 = fmt == FP8BS_SCALE_FMT_UE8M0;
  r = run_gated({xq, xs, w_gate, w_gate_s, w_up, w_up_s}, M, N, K, out, base + w.ws, w.ws_bytes,
                as_stream(stream));
  if (r != FP8BS_OK) return r;
  return run_gemm(out.q, out.s, w_down, w_down_s, M, K_out, N, y, base + w.ws, w.ws_bytes,
                  as_stream(stream));
}

fp8bs_status fp8bs_fp8_gemm_grouped_gated(int64_t G, const int64_t* m_offsets, int64_t M_total,
                                          const uint8_t* a, const float* a_s,
                                          const uint8_t* w_gate, const float* w_gate_s,
                                          const uint8_t* w_up, const float* w_up_s, int64_t N,
                                          int64_t K, uint16_t* h, void* stream) {
  if (G < 1 || G > gemm::kMaxGroups) return fail(FP8BS_ERR_INVALID_ARG, "G=%lld out of [1, %d]", (long long)G, gemm::kMaxGroups);
  if (!m_offsets || (reinterpret_cast<uintptr_t>(m_offsets) & 7u))
    return fail(FP8BS_ERR_INVALID_ARG, "m_offsets must be an 8-byte aligned device pointer");
  if (gated_empty(M_total, N, K)) return FP8BS_OK;
  fp8bs_status r = check_gated({a, a_s, w_gate, w_gate_s, w_up, w_up_s}, h, N, K);
  if (r != FP8BS_OK) return r;
  if (M_total < 0 || M_total >= (int64_t(1) << 31)) return fail(FP8BS_ERR_INVALID_ARG, "M_total out of range");
  if (G * N > (int64_t(1) << 31)) return fail(FP8BS_ERR_INVALID_ARG, "G*N too large");
  int dev;
  DeviceInfo* info;
  if ((r = device_setup(&dev, &info)) != FP8BS_OK) return r;
  CUtensorMap ta, tg, tu, ty;
  gemm::Params p{};
  if ((r = make_tmap(&ta, a, M_total, K, 128)) != FP8BS_OK) return r;
  if ((r = make_tmap(&tg, w_gate, G * N, K, 128)) != FP8BS_OK) return r;
  if ((r = make_tmap(&tu, w_up, G * N, K, 128)) != FP8BS_OK) return r;
  if ((r = make_tmap_out(&ty, h, nullptr, M_total, N, 1, &p.y_tma)) != FP8BS_OK) return r;
  p.sa = a_s;
  p.sw = w_gate_s;
  p.sw_up = w_up_s;
  p.y = reinterpret_cast<__nv_bfloat16*>(h);
  p.m_offsets = m_offsets;
  p.M = M_total;
  p.N = static_cast<int>(N);
  p.kbn = static_cast<int>(K / 128);
  p.nbn = static_cast<int>((N + 127) / 128);
  p.n_tiles = p.nbn;
  p.n_group = 1;
  p.splits = 1;
  p.kb_per_split = p.kbn;
  p.groups = static_cast<int>(G);
  // Units are only known on the device; an upper bound sizes the grid.
  const int64_t max_units = ((M_total + 127) / 128 + G) * p.n_tiles;
  if (max_units >= (int64_t(1) << 26))
    return fail(FP8BS_ERR_INVALID_ARG, "M_total x N too large (tile count)");
  const int grid = static_cast<int>(std::min<int64_t>(max_units, info->sms));
  const cudaError_t e = launch_gated<128, true>(ta, tg, ty, tu, kNoMap, p, grid, as_stream(stream));
  if (e != cudaSuccess) return cuda_fail(e, "fp8_gemm_grouped_gated launch");
  return FP8BS_OK;
}

fp8bs_status fp8bs_gated_backward(const uint16_t* gu, const uint16_t* dh, int64_t M, int64_t N,
                                  uint16_t* dgu, uint16_t* h, void* stream) {
  if (M < 0 || N < 0) return fail(FP8BS_ERR_INVALID_ARG, "negative size");
  if (M == 0 || N == 0) return FP8BS_OK;
  if (M > (int64_t(1) << 31) || N > (1 << 30)) return fail(FP8BS_ERR_INVALID_ARG, "size out of range");
  if (!gu || !dh || !dgu) return fail(FP8BS_ERR_INVALID_ARG, "null pointer");
  for (const void* v : {static_cast<const void*>(gu), static_cast<const void*>(dh),
                        static_cast<const void*>(dgu), static_cast<const void*>(h)})
    if (reinterpret_cast<uintptr_t>(v) & 1u)
      return fail(FP8BS_ERR_INVALID_ARG, "operands must be aligned to their 2-byte elements");
  // 16-byte accesses where every row starts on 16 bytes (N % 8 == 0: all rows do if
  // the tensors do), else 2-byte ones ([4096, 18432] with h: 148 and 184 us).
  const bool wide = N % 8 == 0 && aligned16(gu) && aligned16(dh) && aligned16(dgu) && aligned16(h);
  int dev;
  DeviceInfo* info;
  fp8bs_status r = device_setup(&dev, &info);
  if (r != FP8BS_OK) return r;
  using B = __nv_bfloat16;
  const B* g = reinterpret_cast<const B*>(gu);
  const B* d = reinterpret_cast<const B*>(dh);
  B* o = reinterpret_cast<B*>(dgu);
  B* hh = reinterpret_cast<B*>(h);
  const cudaError_t e =
      wide
          ? launch(gated::gated_backward_kernel, grid_for(M * (N / 8), 256, info->sms * 8), 256, 0,
                   as_stream(stream), g, d, o, hh, M, N)
          : launch(gated::gated_backward_any_kernel,
                   grid_for(M * ((N + gated::kAnyCols - 1) / gated::kAnyCols), 1, info->sms * 8), 256,
                   0, as_stream(stream), g, d, o, hh, M, N);
  if (e != cudaSuccess) return cuda_fail(e, "gated_backward launch");
  return FP8BS_OK;
}

fp8bs_status fp8bs_gated_backward_quant(const uint16_t* gu, const uint16_t* dh, int64_t M, int64_t N,
                                        fp8bs_scale_fmt fmt, uint8_t* q, float* s, uint8_t* qt,
                                        float* st, uint8_t* ht, float* hts, void* stream) {
  if (M < 0 || M > (int64_t(1) << 31)) return fail(FP8BS_ERR_INVALID_ARG, "M out of range");
  if (N <= 0 || N % 128 != 0 || N > (1 << 30))
    return fail(FP8BS_ERR_INVALID_ARG, "N=%lld must be a positive multiple of 128", (long long)N);
  if (fmt != FP8BS_SCALE_FMT_NONE && fmt != FP8BS_SCALE_FMT_UE8M0)
    return fail(FP8BS_ERR_INVALID_ARG, "scale_fmt");
  if (M == 0) return FP8BS_OK;
  if (!gu || !dh || !q || !s || !qt || !st || !ht || !hts)
    return fail(FP8BS_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(gu) || !aligned16(dh) || !aligned16(q) || !aligned16(qt) || !aligned16(ht))
    return fail(FP8BS_ERR_INVALID_ARG, "gu, dh, q, qt and ht must be 16-byte aligned");
  for (const float* f : {s, st, hts})
    if (reinterpret_cast<uintptr_t>(f) & 3u)
      return fail(FP8BS_ERR_INVALID_ARG, "scale pointers must be 4-byte aligned");
  int dev;
  DeviceInfo* info;
  fp8bs_status r = device_setup(&dev, &info);
  if (r != FP8BS_OK) return r;
  const int64_t tiles = ((M + 127) / 128) * (N / 128);
  const int grid = grid_for(tiles, 1, info->sms);
  CUtensorMap g, d;
  if ((r = make_tmap_bf16(&g, gu, M, 2 * N)) != FP8BS_OK) return r;
  if ((r = make_tmap_bf16(&d, dh, M, N)) != FP8BS_OK) return r;
  const cudaError_t e =
      fmt == FP8BS_SCALE_FMT_UE8M0
          ? launch(gated::gated_backward_quant_kernel<true>, grid, gated::kBqThreads, gated::kBqSmem,
                   as_stream(stream), g, d, q, s, qt, st, ht, hts, M, N)
          : launch(gated::gated_backward_quant_kernel<false>, grid, gated::kBqThreads, gated::kBqSmem,
                   as_stream(stream), g, d, q, s, qt, st, ht, hts, M, N);
  if (e != cudaSuccess) return cuda_fail(e, "gated_backward_quant launch");
  return FP8BS_OK;
}

fp8bs_status fp8bs_weight_quant_int4(const void* w, fp8bs_dtype w_dtype, int64_t N, int64_t K,
                                     int64_t group, uint8_t* q, float* s, void* stream) {
  fp8bs_status r = check_int4(N, K, group);
  if (r != FP8BS_OK) return r;
  if (w_dtype != FP8BS_DTYPE_BF16 && w_dtype != FP8BS_DTYPE_F32)
    return fail(FP8BS_ERR_INVALID_ARG, "w_dtype");
  if (N == 0) return FP8BS_OK;
  if (!w || !q || !s) return fail(FP8BS_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(w) || !aligned16(q) || (reinterpret_cast<uintptr_t>(s) & 3u))
    return fail(FP8BS_ERR_INVALID_ARG, "w and q must be 16-byte aligned, s 4-byte aligned");
  int dev;
  DeviceInfo* info;
  if ((r = device_setup(&dev, &info)) != FP8BS_OK) return r;
  const int64_t words = N * (K / 8);
  const cudaError_t e =
      w_dtype == FP8BS_DTYPE_BF16
          ? launch_quant_int4(static_cast<const __nv_bfloat16*>(w), q, s, words, group, info->sms, as_stream(stream))
          : launch_quant_int4(static_cast<const float*>(w), q, s, words, group, info->sms, as_stream(stream));
  if (e != cudaSuccess) return cuda_fail(e, "weight_quant_int4 launch");
  return FP8BS_OK;
}

fp8bs_status fp8bs_weight_dequant_int4(const uint8_t* q, const float* s, int64_t N, int64_t K,
                                       int64_t group, void* y, fp8bs_dtype y_dtype, void* stream) {
  fp8bs_status r = check_int4(N, K, group);
  if (r != FP8BS_OK) return r;
  if (y_dtype != FP8BS_DTYPE_BF16 && y_dtype != FP8BS_DTYPE_F32)
    return fail(FP8BS_ERR_INVALID_ARG, "y_dtype");
  if (N == 0) return FP8BS_OK;
  if (!q || !s || !y) return fail(FP8BS_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(q) || !aligned16(y) || (reinterpret_cast<uintptr_t>(s) & 3u))
    return fail(FP8BS_ERR_INVALID_ARG, "q and y must be 16-byte aligned, s 4-byte aligned");
  int dev;
  DeviceInfo* info;
  if ((r = device_setup(&dev, &info)) != FP8BS_OK) return r;
  const int64_t words = N * (K / 8);
  const int grid = grid_for(y_dtype == FP8BS_DTYPE_F32 ? 2 * words : words, 256, info->sms * 8);
  const int lg = int4_group_log2(group);
  const cudaError_t e =
      y_dtype == FP8BS_DTYPE_BF16
          ? launch(w4::dequant_int4_kernel<__nv_bfloat16>, grid, 256, 0, as_stream(stream), q, s,
                   static_cast<__nv_bfloat16*>(y), words, lg)
          : launch(w4::dequant_int4_kernel<float>, grid, 256, 0, as_stream(stream), q, s,
                   static_cast<float*>(y), words, lg);
  if (e != cudaSuccess) return cuda_fail(e, "weight_dequant_int4 launch");
  return FP8BS_OK;
}

fp8bs_status fp8bs_int4_linear(const uint16_t* x, int64_t M, const uint8_t* q, const float* s,
                               int64_t N, int64_t K, int64_t group, void* y, fp8bs_dtype y_dtype,
                               void* stream) {
  return run_int4(x, M, q, s, nullptr, nullptr, false, N, K, group, y, y_dtype, as_stream(stream));
}

fp8bs_status fp8bs_int4_linear_gated(const uint16_t* x, int64_t M, const uint8_t* q_gate,
                                     const float* s_gate, const uint8_t* q_up, const float* s_up,
                                     int64_t N, int64_t K, int64_t group, void* h,
                                     fp8bs_dtype h_dtype, void* stream) {
  return run_int4(x, M, q_gate, s_gate, q_up, s_up, true, N, K, group, h, h_dtype, as_stream(stream));
}

size_t fp8bs_grad_norm_workspace_size(int64_t n) {
  if (n <= 0) return 0;
  int dev;
  DeviceInfo* info;
  if (device_setup(&dev, &info) != FP8BS_OK) return 0;
  return norm_workspace(info->sms);
}

fp8bs_status fp8bs_grad_norm(const void *const *grads, const int64_t* numel,
                             const fp8bs_dtype* dtypes, int64_t n, float* norm, void* workspace,
                             size_t workspace_bytes, void* stream) {
  fp8bs_status r = check_grads(grads, numel, dtypes, n);
  if (r != FP8BS_OK) return r;
  if (!norm || (reinterpret_cast<uintptr_t>(norm) & 3u))
    return fail(FP8BS_ERR_INVALID_ARG, "norm must be a 4-byte aligned device pointer");
  int dev;
  DeviceInfo* info;
  if ((r = device_setup(&dev, &info)) != FP8BS_OK) return r;
  if (n > 0 && (!workspace || workspace_bytes < norm_workspace(info->sms) ||
                (reinterpret_cast<uintptr_t>(workspace) & 7u)))
    return fail(FP8BS_ERR_WORKSPACE, "workspace of %zu bytes (8-byte aligned) required",
                norm_workspace(info->sms));
  int partials = 0;
  double* ws = static_cast<double*>(workspace);
  if ((r = run_norm_partials(grads, numel, dtypes, n, ws, info->sms, as_stream(stream), &partials)) != FP8BS_OK)
    return r;
  const cudaError_t e = launch(clip::norm_final_kernel, 1, clip::kThreads, 0, as_stream(stream),
                               static_cast<const double*>(ws), partials, norm);
  if (e != cudaSuccess) return cuda_fail(e, "grad_norm final launch");
  return FP8BS_OK;
}

fp8bs_status fp8bs_clip_grads(const void *const *grads, void *const *outs, const int64_t* numel,
                              const fp8bs_dtype* dtypes, const fp8bs_dtype* out_dtypes, int64_t n,
                              const double* max_norm, float* norm, void* workspace,
                              size_t workspace_bytes, void* stream) {
  fp8bs_status r = check_grads(grads, numel, dtypes, n);
  if (r != FP8BS_OK) return r;
  if (n > 0 && !out_dtypes) return fail(FP8BS_ERR_INVALID_ARG, "null array");
  if ((r = check_grads(const_cast<const void* const*>(outs), numel, out_dtypes, n)) != FP8BS_OK) return r;
  if (!max_norm || !(*max_norm >= 0.0))
    return fail(FP8BS_ERR_INVALID_ARG, "max_norm must point to a number that is not negative");
  if (!norm || (reinterpret_cast<uintptr_t>(norm) & 3u))
    return fail(FP8BS_ERR_INVALID_ARG, "norm must be a 4-byte aligned device pointer");
  if ((r = check_outputs(grads, outs, numel, dtypes, out_dtypes, n)) != FP8BS_OK) return r;
  int dev;
  DeviceInfo* info;
  if ((r = device_setup(&dev, &info)) != FP8BS_OK) return r;
  if (n > 0 && (!workspace || workspace_bytes < norm_workspace(info->sms) ||
                (reinterpret_cast<uintptr_t>(workspace) & 7u)))
    return fail(FP8BS_ERR_WORKSPACE, "workspace of %zu bytes (8-byte aligned) required",
                norm_workspace(info->sms));
  cudaStream_t stm = as_stream(stream);
  int partials = 0;
  double* ws = static_cast<double*>(workspace);
  if ((r = run_norm_partials(grads, numel, dtypes, n, ws, info->sms, stm, &partials)) != FP8BS_OK) return r;
  cudaError_t e;
  if (partials == 0) {   // nothing to scale: the norm of no elements
    e = launch(clip::norm_final_kernel, 1, clip::kThreads, 0, stm, static_cast<const double*>(ws), 0, norm);
    if (e != cudaSuccess) return cuda_fail(e, "grad_norm final launch");
    return FP8BS_OK;
  }
  float* norm_out = norm;   // written by the first launch
  // Last tensors first: they were read last.
  const int64_t last = (n - 1) / clip::kMaxTensors * clip::kMaxTensors;
  for (int64_t i = last; i >= 0; i -= clip::kMaxTensors) {
    clip::Table t;
    fill_table(&t, grads, outs, numel, dtypes, out_dtypes, i, std::min<int64_t>(n, i + clip::kMaxTensors));
    if (t.first[t.count] == 0) continue;
    const int grid = clip::launch_ctas(t.first[t.count], info->sms);
    e = launch(clip::clip_scale_kernel, grid, clip::kThreads, 0, stm, t, static_cast<const double*>(ws),
               partials, *max_norm, norm_out);
    if (e != cudaSuccess) return cuda_fail(e, "clip_grads launch");
    norm_out = nullptr;
  }
  return FP8BS_OK;
}

}  // extern "C"
