// Host side of the 16-bit ragged products, the SwiGLU checkpoint and the
// 4-bit operators: argument checks, tensor maps, launches.  Included by
// mxmoe.cu after its shared helpers.
#pragma once

namespace {

int check_dtype(int dtype) {
  if (dtype != MXMOE_BF16 && dtype != MXMOE_FP16)
    return fail(MXMOE_ERR_ARG, "dtype=%d must be MXMOE_BF16 or MXMOE_FP16", dtype);
  return MXMOE_OK;
}

// Allow `bytes` of dynamic shared memory for a kernel, once per device.
template <typename K>
int ensure_smem(K kern, std::atomic<uint64_t>& done, int bytes) {
  int dev = 0;
  MX_CHECK_CUDA(cudaGetDevice(&dev), "cudaGetDevice");
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (!(done.load(std::memory_order_acquire) & bit)) {
    MX_CHECK_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes), "cudaFuncSetAttribute");
    done.fetch_or(bit, std::memory_order_release);
  }
  return MXMOE_OK;
}

// A launch that may start while the one before it in the stream drains
// (`after`: that one is this call's own and announced it).
template <typename K, typename... A>
cudaError_t launch_after(K kern, dim3 grid, int threads, int smem, cudaStream_t stream, bool after, A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = after ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// ---------------------------------------------------------------- ragged products
constexpr size_t kRaggedHeader = 256;   // of the workspace: join_kernel's flag

// Units that share a tile's contraction (1: no split): few tiles leave pairs of
// SMs without work.  As many units as there are pairs, each with eight K blocks
// or more, where the contraction has at least 48 blocks: the join's launch and
// workspace cost the caller 5 us, and a lone tile takes 4 us and 0.22 us a block.
// On the GPU, split against not: weight gradient 24 x 704 of 31134 rows (3 tiles
// of 487 blocks) 23 / 141 us, forward 128 rows x 2048 x 7168 (8 tiles of 112)
// 15.5 / 28.8, one row x 4096 x 4096 (16 of 64) 12.4 / 17.9; with 32 blocks the
// calls take 13.7 us split and 11.4 not.
int ragged_splits(int64_t tiles, int64_t blocks) {
  constexpr int64_t pairs = 74;          // of a B200: the size must not depend on the device that is current
  if (blocks < 48) return 1;
  return int(std::max<int64_t>(1, std::min<int64_t>(pairs / std::max<int64_t>(1, tiles), blocks / 8)));
}
int64_t ragged_tiles(int64_t M, int64_t N, int64_t K, int E, int which) {
  using C = ragged::Cfg;
  const int64_t rt = ((which == 1 ? K : N) + C::BM - 1) / C::BM;
  // every segment's last tile may be short
  return which == 2 ? int64_t(E) * rt * ((K + C::BN - 1) / C::BN) : (M / C::BN + std::min<int64_t>(E, M)) * rt;
}
int64_t ragged_blocks(int64_t M, int64_t N, int64_t K, int which) {
  return ((which == 0 ? K : which == 1 ? N : M) + ragged::kBK - 1) / ragged::kBK;
}
int64_t ragged_values(int64_t M, int64_t N, int64_t K, int E, int which) {
  return which == 2 ? int64_t(E) * N * K : M * (which == 1 ? K : N);
}

// A workspace (may be NULL) of the size for this call lets the product be
// split; without one it runs unsplit.
int ragged_workspace(ragged::Params* p, int64_t M, int64_t N, int64_t K, int E, int which, void* workspace,
                     size_t bytes) {
  p->splits = 1;
  const size_t need = mxmoe_ragged_workspace_size(M, N, K, E, which);
  if (!workspace || need == 0) return MXMOE_OK;
  if (bytes < need) return fail(MXMOE_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed", bytes, need);
  if (!aligned16(workspace)) return fail(MXMOE_ERR_ALIGN, "workspace is not 16-byte aligned");
  p->splits = ragged_splits(ragged_tiles(M, N, K, E, which), ragged_blocks(M, N, K, which));
  p->ok = static_cast<int*>(workspace);
  p->sums = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kRaggedHeader);
  return MXMOE_OK;
}

// 16-bit map of rank 2 or 3 ([z,] y, x), dense rows.
int make_map16(CUtensorMap* map, int dtype, const void* base, int rank, int64_t x, int64_t y, int64_t z, uint32_t bx,
               uint32_t by, CUtensorMapSwizzle swizzle, const char* what) {
  EncodeTiledFn enc;
  MX_TRY(get_encode(&enc));
  cuuint64_t dims[3] = {cuuint64_t(x), cuuint64_t(y), cuuint64_t(z)};
  cuuint64_t strides[2] = {cuuint64_t(x * 2), cuuint64_t(x * y * 2)};
  cuuint32_t box[3] = {bx, by, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(map, dtype == MXMOE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                   cuuint32_t(rank), const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(MXMOE_ERR_CUDA, "cuTensorMapEncodeTiled (%s) failed (%d)", what, int(r));
  return MXMOE_OK;
}

template <int kMode, int kDt, bool kPair>
int launch_ragged_dt(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mo, const ragged::Params& p,
                     int64_t max_tiles, const DevInfo* d, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  auto kern = ragged::ragged_gemm_kernel<kMode, kDt, kPair>;
  MX_TRY(ensure_smem(kern, done, ragged::Cfg::SMEM_BYTES));
  max_tiles *= p.splits;
  if (max_tiles > 0x7FFFFFFF) return fail(MXMOE_ERR_SHAPE, "%lld tiles: too large", (long long)max_tiles);
  // clusters of two CTAs, as many as can be resident
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(384, 1, 1);
  cfg.dynamicSmemBytes = ragged::Cfg::SMEM_BYTES;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(unsigned(2 * std::min<int64_t>(max_tiles, d->sms / 2)), 1, 1);
  MX_CHECK_CUDA(cudaLaunchKernelEx(&cfg, kern, ma, mb, mo, p), "ragged product launch");
  if (p.splits > 1) {
    constexpr bool kW = kMode == ragged::kWgrad;
    const int64_t values = int64_t(p.rows) * (kW ? int64_t(p.cols) * p.E : p.M);
    MX_CHECK_CUDA(launch_after(ragged::join_kernel<kW, kDt>, dim3(unsigned((values / 8 + 255) / 256)), 256, 0, stream, true, p),
                  "ragged join launch");
  }
  MX_CHECK_CUDA(cudaGetLastError(), "ragged product launch");
  return MXMOE_OK;
}

template <int kMode, bool kPair>
int launch_ragged(int dtype, const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mo,
                  const ragged::Params& p, int64_t max_tiles, const DevInfo* d, cudaStream_t stream) {
  return dtype == MXMOE_BF16 ? launch_ragged_dt<kMode, kBF16, kPair>(ma, mb, mo, p, max_tiles, d, stream)
                             : launch_ragged_dt<kMode, kFP16, kPair>(ma, mb, mo, p, max_tiles, d, stream);
}

int check_ragged(int64_t M, int64_t N, int64_t K, int E, const int32_t* offsets, int dtype) {
  MX_TRY(check_dtype(dtype));
  // (token numbers are 32-bit in the kernel, up to a tile past the last row)
  if (M < 0 || M > (int64_t(1) << 31) - 1024) return fail(MXMOE_ERR_SHAPE, "M=%lld must be in [0, 2^31 - 1024]", (long long)M);
  if (E <= 0 || E > ragged::kMaxE) return fail(MXMOE_ERR_SHAPE, "E=%d must be in [1, %d]", E, ragged::kMaxE);
  MX_TRY(check_mult("N", N, 8));
  MX_TRY(check_mult("K", K, 8));
  if (N >= (int64_t(1) << 30) || K >= (int64_t(1) << 30)) return fail(MXMOE_ERR_SHAPE, "N and K must be below 2^30");
  if (!offsets) return fail(MXMOE_ERR_NULL, "expert_offsets is NULL");
  return MXMOE_OK;
}

// ---------------------------------------------------------------- 4-bit matvec
// Slots that share one pass over an expert's weights: eight, or as many as
// shared memory holds next to the rings (0: not even one).
int mv_group(int64_t K, int E, int S, int pieces) {
  for (int g = 8; g >= 1; g >>= 1)
    if (mv_smem(K, g, E, S, pieces) <= 232448 - 1024) return g;
  return 0;
}

template <int kDt, bool kGated, int kOut>
int launch_mv(MvArgs a, const DevInfo* d, cudaStream_t stream, bool after = false) {
  static std::atomic<uint64_t> done{0};
  auto kern = fp4_matvec_kernel<kDt, kGated, kOut>;
  MX_TRY(ensure_smem(kern, done, 232448 - 1024));
  a.group = mv_group(a.K, a.E, a.S, a.pieces);
  if (a.group == 0) return fail(MXMOE_ERR_SHAPE, "K=%d with E=%d and %d slots does not fit shared memory", a.K, a.E, a.S);
  // As many warps share a tile as leave each four cells or more of it.  On the GPU,
  // one / two / four warps, one slot for each of 8 experts of 4096 rows: K = 256 6.0 /
  // 7.0 / 6.9 us, 512 7.0 / 7.5 / 8.3, 1024 8.9 / 9.1 / 9.2, 2048 12.8 / 12.5 / 12.3,
  // 7168 37 / 32 / 29; for 48 of 64 experts: 2048 rows, K = 1024 16.3 / 17.0 / 18.0,
  // 4096 rows, K = 7168 136 / 127 / 125.  Between 1024 and 2048 it hardly matters to few
  // tiles, and many would rather be one warp's (7168 rows, K = 2048 66 / 72 / 74).
  a.team_log2 = kMvWarps % 4 == 0 ? 2 : 0;
  while (a.team_log2 > 0 && (4 << a.team_log2) > a.K / 128) --a.team_log2;
  const int grid = int(std::min<int64_t>(int64_t(a.S) * a.tiles, d->sms));
  MX_CHECK_CUDA(launch_after(kern, dim3(grid), kMvThreads, mv_smem(a.K, a.group, a.E, a.S, a.pieces), stream, after, a), "4-bit matvec launch");
  return MXMOE_OK;
}

int check_mv(int64_t S, int E) {
  if (S < 0 || S > kMvMaxSlots)
    return fail(MXMOE_ERR_SHAPE, "%lld slots: at most %d (use the grouped GEMMs for more)", (long long)S, kMvMaxSlots);
  if (E <= 0 || E > kMvMaxE) return fail(MXMOE_ERR_SHAPE, "E=%d must be in [1, %d]", E, kMvMaxE);
  return MXMOE_OK;
}

int ckpt_args(CkptArgs* a, int64_t rows, int64_t F, const int32_t* rows_dev, int64_t* blocks) {
  if (rows < 0) return fail(MXMOE_ERR_SHAPE, "rows=%lld must not be negative", (long long)rows);
  MX_TRY(check_mult("F", F, 8));
  if (F >= (int64_t(1) << 28)) return fail(MXMOE_ERR_SHAPE, "F=%lld too large", (long long)F);
  a->rows = rows;
  a->rows_dev = rows_dev;
  a->F = uint32_t(F);
  a->units = uint32_t((F + 31) / 32 * 4);
  if (rows > (int64_t(1) << 62) / a->units) return fail(MXMOE_ERR_SHAPE, "rows=%lld too large", (long long)rows);
  *blocks = (rows * a->units + 256 * kCkptUnits - 1) / (256 * kCkptUnits);
  if (*blocks > 0x7FFFFFFF) return fail(MXMOE_ERR_SHAPE, "rows=%lld x F=%lld: too large", (long long)rows, (long long)F);
  return MXMOE_OK;
}

int check_fp4(int64_t batch, int64_t rows, int64_t cols, int layout) {
  if (layout < MXFP4_PLAIN || layout > MXFP4_TILE_GATED) return fail(MXMOE_ERR_ARG, "layout=%d invalid", layout);
  if (batch <= 0 || rows <= 0) return fail(MXMOE_ERR_SHAPE, "batch=%lld and rows=%lld must be positive", (long long)batch, (long long)rows);
  MX_TRY(check_mult("cols", cols, layout == MXFP4_PLAIN ? 32 : 128));
  if (layout != MXFP4_PLAIN) MX_TRY(check_mult("rows", rows, 16));
  if (cols >= (int64_t(1) << 30) || rows > (int64_t(1) << 60) / cols || batch > (int64_t(1) << 60) / cols / rows ||
      (batch * rows * cols / 8 + 255) / 256 > 0x7FFFFFFF)
    return fail(MXMOE_ERR_SHAPE, "tensor too large");
  return MXMOE_OK;
}

struct DecodeWs {
  float* h;   // [S, F]
  float* y;   // [S, D]
};
size_t carve_decode(uint8_t* base, int64_t S, int64_t D, int64_t F, DecodeWs* w) {
  Carver c{base};
  w->h = c.take<float>(size_t(S) * F * 4);
  w->y = c.take<float>(size_t(S) * D * 4);
  return c.off + 256;
}

}  // namespace

extern "C" {

size_t mxmoe_ragged_workspace_size(int64_t M, int64_t N, int64_t K, int E, int which) {
  if (M <= 0 || N <= 0 || K <= 0 || E <= 0 || E > ragged::kMaxE || which < 0 || which > 2 || N >= (int64_t(1) << 30) || K >= (int64_t(1) << 30) ||
      M > (int64_t(1) << 31))
    return 0;
  const int splits = ragged_splits(ragged_tiles(M, N, K, E, which), ragged_blocks(M, N, K, which));
  return splits > 1 ? kRaggedHeader + size_t(splits) * ragged_values(M, N, K, E, which) * 4 : 0;
}

int mxmoe_ragged_gemm(const void* a, int64_t M, const void* w, int E, int64_t N, int64_t K,
                      const int32_t* expert_offsets, int transpose_w, int dtype, void* out, void* workspace,
                      size_t workspace_bytes, cudaStream_t stream) {
  MX_TRY(check_ragged(M, N, K, E, expert_offsets, dtype));
  if (transpose_w != 0 && transpose_w != 1) return fail(MXMOE_ERR_ARG, "transpose_w=%d must be 0 or 1", transpose_w);
  if (M == 0) return MXMOE_OK;
  MX_TRY(check_ptrs({{"a", a}, {"w", w}, {"out", out}}));
  ragged::Params p{};
  p.E = E;
  p.M = M;
  p.offsets = expert_offsets;
  p.out = static_cast<uint16_t*>(out);
  p.rows = int(transpose_w ? K : N);
  p.kext = int(transpose_w ? N : K);
  MX_TRY(ragged_workspace(&p, M, N, K, E, transpose_w, workspace, workspace_bytes));
  DevInfo* d;
  MX_TRY(device_info(&d));
  CUtensorMap ma, mb, mo;
  MX_TRY(make_map16(&ma, dtype, w, 3, K, N, E, 64, transpose_w ? 64 : 128, CU_TENSOR_MAP_SWIZZLE_128B, "weights"));
  MX_TRY(make_map16(&mb, dtype, a, 2, p.kext, M, 1, 64, ragged::Cfg::kBox, CU_TENSOR_MAP_SWIZZLE_128B, "tokens"));
  mo = mb;   // (fewer than 32 tokens: no chunk of 32 to store)
  if (M >= 32) MX_TRY(make_map16(&mo, dtype, out, 2, p.rows, M, 1, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B, "output"));
  const int64_t tiles = ragged_tiles(M, N, K, E, transpose_w);
  return transpose_w ? launch_ragged<ragged::kDgrad, true>(dtype, ma, mb, mo, p, tiles, d, stream)
                     : launch_ragged<ragged::kFwd, true>(dtype, ma, mb, mo, p, tiles, d, stream);
}

int mxmoe_ragged_gemm_wgrad(const void* g, int64_t N, const void* a, int64_t K, int64_t M,
                            const int32_t* expert_offsets, int E, int dtype, void* dw, void* workspace,
                            size_t workspace_bytes, cudaStream_t stream) {
  MX_TRY(check_ragged(M, N, K, E, expert_offsets, dtype));
  MX_TRY(check_ptrs({{"dw", dw}}));
  DevInfo* d;
  if (M == 0) {
    MX_TRY(device_info(&d));
    MX_CHECK_CUDA(cudaMemsetAsync(dw, 0, size_t(E) * N * K * 2, stream), "cudaMemsetAsync");
    return MXMOE_OK;
  }
  MX_TRY(check_ptrs({{"g", g}, {"a", a}}));
  ragged::Params p{};
  p.E = E;
  p.M = M;
  p.offsets = expert_offsets;
  p.rows = int(N);
  p.cols = int(K);
  p.out = static_cast<uint16_t*>(dw);
  MX_TRY(ragged_workspace(&p, M, N, K, E, 2, workspace, workspace_bytes));
  MX_TRY(device_info(&d));
  CUtensorMap ma, mb, mo;
  MX_TRY(make_map16(&ma, dtype, g, 2, N, M, 1, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B, "gradients"));
  MX_TRY(make_map16(&mb, dtype, a, 2, K, M, 1, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B, "tokens"));
  // Boxes of 64 columns leave whole 128-byte lines, but tie two epilogue warps to
  // each other.  They gain where rows start off the 32-byte sectors (44 experts of 31
  // rows, 456 x 6776: 79 / 95 us) and where tiles have six K blocks or more on average
  // (64 x 1408 x 2048: 469 rows an expert 159 / 168, 768 rows x 2816 429 / 447);
  // shorter tiles wait for the epilogue (312 rows 127 / 125, 94 rows of 2048 x 2048
  // 127 / 121, one row of 4096 x 2048 209 / 178).
  const bool pair = K % 16 != 0 || M >= int64_t(400) * E;
  MX_TRY(make_map16(&mo, dtype, dw, 3, K, N, E, pair ? 64 : 32, 32,
                    pair ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, "weight gradients"));
  const int64_t tiles = ragged_tiles(M, N, K, E, 2);
  return pair ? launch_ragged<ragged::kWgrad, true>(dtype, ma, mb, mo, p, tiles, d, stream)
              : launch_ragged<ragged::kWgrad, false>(dtype, ma, mb, mo, p, tiles, d, stream);
}

int mxfp8_swiglu_ckpt(const void* h13, int64_t rows, int64_t F, const int32_t* rows_dev, int dtype, void* h,
                      uint8_t* codes, uint8_t* scales, cudaStream_t stream) {
  MX_TRY(check_dtype(dtype));
  CkptArgs a{};
  int64_t blocks;
  MX_TRY(ckpt_args(&a, rows, F, rows_dev, &blocks));
  if (rows == 0) return MXMOE_OK;
  MX_TRY(check_ptrs({{"h13", h13}, {"h", h}, {"codes", codes}}));
  if (!scales) return fail(MXMOE_ERR_NULL, "scales is NULL");
  DevInfo* d;
  MX_TRY(device_info(&d));
  a.in = static_cast<const uint16_t*>(h13);
  a.h = static_cast<uint16_t*>(h);
  a.codes = codes;
  a.scales = scales;
  if (dtype == MXMOE_BF16) swiglu_ckpt_kernel<kBF16><<<unsigned(blocks), 256, 0, stream>>>(a);
  else swiglu_ckpt_kernel<kFP16><<<unsigned(blocks), 256, 0, stream>>>(a);
  MX_CHECK_CUDA(cudaGetLastError(), "SwiGLU checkpoint launch");
  return MXMOE_OK;
}

int mxfp8_swiglu_ckpt_bwd(const void* dh, const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t F,
                          const int32_t* rows_dev, int dtype, void* dh13, void* h, cudaStream_t stream) {
  MX_TRY(check_dtype(dtype));
  CkptArgs a{};
  int64_t blocks;
  MX_TRY(ckpt_args(&a, rows, F, rows_dev, &blocks));
  if (rows == 0) return MXMOE_OK;
  MX_TRY(check_ptrs({{"dh", dh}, {"codes", codes}, {"dh13", dh13}}));
  if (!scales) return fail(MXMOE_ERR_NULL, "scales is NULL");
  if (h && !aligned16(h)) return fail(MXMOE_ERR_ALIGN, "h is not 16-byte aligned");
  DevInfo* d;
  MX_TRY(device_info(&d));
  a.in = static_cast<const uint16_t*>(dh);
  a.codes = const_cast<uint8_t*>(codes);
  a.scales = const_cast<uint8_t*>(scales);
  a.dh13 = static_cast<uint16_t*>(dh13);
  a.h = static_cast<uint16_t*>(h);
  if (dtype == MXMOE_BF16) swiglu_ckpt_bwd_kernel<kBF16><<<unsigned(blocks), 256, 0, stream>>>(a);
  else swiglu_ckpt_bwd_kernel<kFP16><<<unsigned(blocks), 256, 0, stream>>>(a);
  MX_CHECK_CUDA(cudaGetLastError(), "SwiGLU checkpoint backward launch");
  return MXMOE_OK;
}

int mxfp4_quantize(const void* x, int64_t batch, int64_t rows, int64_t cols, int dtype, int layout, uint8_t* codes,
                   uint8_t* scales, cudaStream_t stream) {
  MX_TRY(check_dtype(dtype));
  MX_TRY(check_fp4(batch, rows, cols, layout));
  MX_TRY(check_ptrs({{"x", x}, {"codes", codes}, {"scales", scales}}));
  DevInfo* d;
  MX_TRY(device_info(&d));
  const int64_t per = 256 * kFp4Units;
  const unsigned blocks = unsigned((batch * rows * (cols / 8) + per - 1) / per);
  const auto* in = static_cast<const uint16_t*>(x);
  if (dtype == MXMOE_BF16) fp4_quantize_kernel<kBF16><<<blocks, 256, 0, stream>>>(in, batch, rows, cols, layout, codes, scales);
  else fp4_quantize_kernel<kFP16><<<blocks, 256, 0, stream>>>(in, batch, rows, cols, layout, codes, scales);
  MX_CHECK_CUDA(cudaGetLastError(), "4-bit cast launch");
  return MXMOE_OK;
}

int mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, int dtype, void* out,
                     cudaStream_t stream) {
  MX_TRY(check_dtype(dtype));
  MX_TRY(check_fp4(1, rows, cols, MXFP4_PLAIN));
  MX_TRY(check_ptrs({{"codes", codes}, {"scales", scales}, {"out", out}}));
  DevInfo* d;
  MX_TRY(device_info(&d));
  const int64_t units = rows * (cols / 8);
  const int64_t per = 256 * kFp4Units;
  const unsigned blocks = unsigned((units + per - 1) / per);
  const auto* c = reinterpret_cast<const uint32_t*>(codes);
  auto* o = static_cast<uint4*>(out);
  if (dtype == MXMOE_BF16) fp4_dequantize_kernel<kBF16><<<blocks, 256, 0, stream>>>(c, scales, units, o);
  else fp4_dequantize_kernel<kFP16><<<blocks, 256, 0, stream>>>(c, scales, units, o);
  MX_CHECK_CUDA(cudaGetLastError(), "4-bit decode launch");
  return MXMOE_OK;
}

int mxfp4_expert_matvec(const void* x, int64_t S, int64_t K, const int32_t* expert_ids, const uint8_t* codes,
                        const uint8_t* scales, int E, int64_t N, int dtype, void* y, cudaStream_t stream) {
  MX_TRY(check_dtype(dtype));
  MX_TRY(check_mv(S, E));
  MX_TRY(check_mult("K", K, 128));
  MX_TRY(check_mult("N", N, 16));
  if (K >= (1 << 24) || N >= (1 << 28) || S * (N / 16) > 0x7FFFFFFF) return fail(MXMOE_ERR_SHAPE, "K=%lld N=%lld: too large", (long long)K, (long long)N);
  if (S > 0 && mv_group(K, E, int(S), 1) == 0) return fail(MXMOE_ERR_SHAPE, "K=%lld does not fit shared memory", (long long)K);
  if (S == 0) return MXMOE_OK;
  MX_TRY(check_ptrs({{"x", x}, {"codes", codes}, {"scales", scales}, {"y", y}}));
  if (!expert_ids) return fail(MXMOE_ERR_NULL, "expert_ids is NULL");
  DevInfo* d;
  MX_TRY(device_info(&d));
  MvArgs a{};
  a.x = x;
  a.ids = expert_ids;
  a.S = int(S);
  a.x_div = 1;
  a.pieces = 1;
  a.E = E;
  a.tiles = int(N / 16);
  a.K = int(K);
  a.codes = codes;
  a.scales = scales;
  a.out = y;
  return dtype == MXMOE_BF16 ? launch_mv<kBF16, false, kBF16>(a, d, stream) : launch_mv<kFP16, false, kFP16>(a, d, stream);
}

size_t mxfp4_decode_workspace_size(int64_t T, int top_k, int64_t D, int64_t F) {
  if (T <= 0 || top_k <= 0 || D <= 0 || F <= 0 || T > kMvMaxSlots || T * top_k > kMvMaxSlots || D >= (1 << 24) ||
      F >= (1 << 24))
    return 0;
  DecodeWs w;
  return carve_decode(nullptr, T * top_k, D, F, &w);
}

int moe_layer_decode_fp4(const void* x_tokens, int64_t T, int64_t D, const int32_t* topk_ids,
                         const float* topk_weights, int top_k, const mxmoe_q4weights* qw, int E, int64_t F, int dtype,
                         void* out_tokens, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  MX_TRY(check_dtype(dtype));
  if (T < 0 || top_k <= 0 || top_k > E || T > kMvMaxSlots)
    return fail(MXMOE_ERR_SHAPE, "T=%lld top_k=%d (1..E) E=%d", (long long)T, top_k, E);
  const int64_t S = T * top_k;
  MX_TRY(check_mv(S, E));
  MX_TRY(check_mult("D", D, 128));
  MX_TRY(check_mult("F", F, 128));
  if (D >= (1 << 24) || F >= (1 << 24) || S * (std::max(D, F) / 8) > 0x7FFFFFFF) return fail(MXMOE_ERR_SHAPE, "D=%lld F=%lld: too large", (long long)D, (long long)F);
  if (T == 0) return MXMOE_OK;
  // h goes in as two f16 pieces; for a bf16 result as one (11 bits, an eighth of that
  // result's rounding) where shared memory does not hold two of a row
  const int pieces = dtype == MXMOE_BF16 && mv_group(F, E, int(S), 2) == 0 ? 1 : 2;
  if (mv_group(D, E, int(S), 1) == 0 || mv_group(F, E, int(S), pieces) == 0)
    return fail(MXMOE_ERR_SHAPE, "D=%lld F=%lld with %lld slots does not fit shared memory", (long long)D, (long long)F, (long long)S);
  if (!qw) return fail(MXMOE_ERR_NULL, "qweights is NULL");
  MX_TRY(check_ptrs({{"x_tokens", x_tokens}, {"out_tokens", out_tokens}, {"qw.w13_codes", qw->w13_codes},
                     {"qw.w13_scales", qw->w13_scales}, {"qw.w2_codes", qw->w2_codes}, {"qw.w2_scales", qw->w2_scales}}));
  if (!topk_ids || !topk_weights) return fail(MXMOE_ERR_NULL, "topk_ids/topk_weights is NULL");
  DecodeWs ws;
  const size_t need = carve_decode(nullptr, S, D, F, &ws);
  if (!workspace || workspace_bytes < need)
    return fail(MXMOE_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed", workspace_bytes, need);
  carve_decode(align_ws(workspace), S, D, F, &ws);
  DevInfo* d;
  MX_TRY(device_info(&d));
  MvArgs a{};
  a.ids = topk_ids;
  a.S = int(S);
  a.E = E;
  // FC1 + SwiGLU: h [S, F] in fp32
  a.pieces = 1;
  a.x = x_tokens;
  a.x_div = top_k;
  a.tiles = int(F / 8);
  a.K = int(D);
  a.codes = qw->w13_codes;
  a.scales = qw->w13_scales;
  a.out = ws.h;
  MX_TRY((dtype == MXMOE_BF16 ? launch_mv<kBF16, true, kF32>(a, d, stream) : launch_mv<kFP16, true, kF32>(a, d, stream)));
  // FC2: y [S, D] in fp32
  a.pieces = pieces;
  a.x = ws.h;
  a.x_div = 1;
  a.tiles = int(D / 16);
  a.K = int(F);
  a.codes = qw->w2_codes;
  a.scales = qw->w2_scales;
  a.out = ws.y;
  MX_TRY((launch_mv<kF32, false, kF32>(a, d, stream, true)));
  const dim3 grid(unsigned((D / 4 + 127) / 128), unsigned(T));
  auto* o = static_cast<uint16_t*>(out_tokens);
  const auto combine = dtype == MXMOE_BF16 ? fp4_combine_kernel<kBF16> : fp4_combine_kernel<kFP16>;
  MX_CHECK_CUDA(launch_after(combine, grid, 128, 0, stream, true, static_cast<const float*>(ws.y), topk_ids, topk_weights,
                             top_k, E, int(D), o), "decode combine launch");
  return MXMOE_OK;
}

}  // extern "C"
