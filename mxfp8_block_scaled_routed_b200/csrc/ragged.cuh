// Grouped 16-bit products over ragged expert segments on the sm_100a tensor
// cores (tcgen05 kind::f16, fp32 accumulators in TMEM, TMA-fed tiles).
//
//   kFwd    out[m, n] = sum_k a[m, k] W[e, n, k]   for the rows m of expert e
//   kDgrad  out[m, k] = sum_n g[m, n] W[e, n, k]
//   kWgrad  dW[e, n, k] = sum_m g[m, n] a[m, k]    over the rows m of expert e
//
// Segments have any length (no padding) and start at any row.  TMA boxes may
// start at any row, so a tile simply reads from its first token on:
//  * kFwd / kDgrad put the weights on the MMA's M side (128 rows a CTA) and the
//    tokens on its N side, whose width is the instruction's and not the
//    kernel's: a segment's last tile runs an MMA of its own rows rounded up to
//    16, so a ragged tail costs its own columns only.  A tile's columns past
//    the segment hold the next expert's tokens; they are not stored.
//  * kWgrad contracts over the tokens.  A segment's last K block is cut at the
//    next multiple of 16 tokens, and the issuing warp clears the up to 15 rows
//    past the end in both operands first (they may hold NaN: a product with
//    zero would not do).
// Operands are read as they lie: W for kFwd and the token matrices are K-major
// (128-byte swizzled rows of 64 values); W for kDgrad and both operands of
// kWgrad are MN-major (boxes of 64 values of the M or N extent by 64 of K).
//
// CTA = 12 warps: warp 0 issues TMA, warp 1 issues MMAs, warp 2 owns TMEM,
// warps 4..11 are the epilogue (warp 4 + q and
// 8 + q read TMEM lanes 32 q.., alternating 32-column chunks).  Two
// accumulators of up to 256 columns: a tile's epilogue runs beside the next
// tile's MMAs.
#pragma once
#include <cuda.h>
#include "half16.cuh"
#include "sm100.cuh"

namespace mxmoe::ragged {

using namespace mxmoe::sm100;

enum Mode : int { kFwd = 0, kDgrad = 1, kWgrad = 2 };

constexpr int kErrOffsets = 4, kErrTimeout = 7;
constexpr int kMaxE = 1024;
constexpr int kBK = 64;                        // K values per stage (128 bytes of a K-major row)

struct Params {
  int E;
  int64_t M;                 // token rows of the buffers (bounds the offsets)
  int rows;                  // M-side extent of one expert's output (kFwd N, kDgrad K, kWgrad N)
  int cols;                  // kWgrad: N-side extent (K); else unused
  int kext;                  // contraction extent (kFwd K, kDgrad N; kWgrad: per segment)
  const int32_t* offsets;
  uint16_t* out;             // kFwd / kDgrad: [M, rows]
};

struct Cfg {
  static constexpr int BM = 128, BN = 256;
  static constexpr int A_BYTES = BM * kBK * 2, B_BYTES = BN * kBK * 2;
  static constexpr int kStages = 4;
  static constexpr int OFF_A = 0, OFF_B = kStages * A_BYTES;
  static constexpr int OFF_EPI = OFF_B + kStages * B_BYTES;
  static constexpr int EPI_WARP_BYTES = 2048;  // one 32 x 32 block of 16-bit outputs per warp
  static constexpr int OFF_BAR = OFF_EPI + 8 * EPI_WARP_BYTES;
  static constexpr int NUM_BARS = 2 * kStages + 4;
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int OFF_TAB = OFF_MISC + 16;   // offsets [E + 1], first token tile of each expert [E + 1]
  static constexpr int SMEM_BYTES = OFF_TAB + 2 * (kMaxE + 1) * 4 + 1024;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

// Instruction descriptor, kind::f16: fp32 accumulator (bit 4), A and B type at
// 7 and 10 (0 f16, 1 bf16), MN-major A / B at 15 / 16, N >> 3 at 17, M >> 4 at 24.
__device__ __forceinline__ uint32_t f16_idesc(int dt_bits, bool a_mn, bool b_mn, uint32_t M, uint32_t N) {
  return (1u << 4) | (uint32_t(dt_bits) << 7) | (uint32_t(dt_bits) << 10) | (uint32_t(a_mn) << 15) |
         (uint32_t(b_mn) << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tma_store_3d(const void* tmap, uint32_t src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(tmap), "r"(x),
               "r"(y), "r"(z), "r"(src)
               : "memory");
}

struct Tile {
  int e;
  int nk;       // K blocks
  int r0;       // first M-side row (of the expert's matrix)
  int n;        // N-side columns (tokens; kWgrad: columns of K)
  int64_t t0;   // first token (kFwd / kDgrad: of the tile; kWgrad: of the segment)
  int c0;       // kWgrad: first N-side column
  int len;      // kWgrad: tokens of the segment
};

// Tile t.  kFwd / kDgrad: experts in order, in an expert the token tile runs
// fastest, so neighbouring CTAs share the weight rows; kWgrad: (expert, row
// tile, column tile).
template <int kMode>
__device__ __forceinline__ Tile get_tile(const Params& p, const int32_t* offs, const int32_t* mt, int64_t t) {
  Tile T;
  const int rt = (p.rows + Cfg::BM - 1) / Cfg::BM;
  if constexpr (kMode == kWgrad) {
    const int ct = (p.cols + Cfg::BN - 1) / Cfg::BN;
    const int64_t per = int64_t(rt) * ct;
    T.e = int(t / per);
    const int w = int(t - T.e * per);
    T.r0 = (w / ct) * Cfg::BM;
    T.c0 = (w % ct) * Cfg::BN;
    T.n = min(Cfg::BN, p.cols - T.c0);
    T.t0 = offs[T.e];
    T.len = offs[T.e + 1] - offs[T.e];
    T.nk = (T.len + kBK - 1) / kBK;
  } else {
    int lo = 0, hi = p.E;                      // last expert whose first tile is at or before t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (int64_t(mt[mid]) * rt <= t) lo = mid; else hi = mid;
    }
    T.e = lo;
    const int w = int(t - int64_t(mt[lo]) * rt);
    const int tiles = mt[lo + 1] - mt[lo];
    T.r0 = (w / tiles) * Cfg::BM;
    T.t0 = offs[lo] + int64_t(w % tiles) * Cfg::BN;
    T.n = int(min(int64_t(Cfg::BN), int64_t(offs[lo + 1]) - T.t0));
    T.nk = (p.kext + kBK - 1) / kBK;
    T.c0 = 0;
    T.len = 0;
  }
  return T;
}

// Bounded wait of the MMA issuer: one thread, in kWgrad the warp as one.
template <int kMode>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  if constexpr (kMode == kWgrad) return __all_sync(0xffffffffu, mbar_wait(bar, parity));
  return mbar_wait(bar, parity);
}

template <int kMode, int kDt>
__global__ void __launch_bounds__(384, 1)
ragged_gemm_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                   const __grid_constant__ CUtensorMap tmap_o, const Params p) {
  using C = Cfg;
  constexpr bool kAMn = kMode != kFwd, kBMn = kMode == kWgrad;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  auto full_bar = [&](int s) { return smem_u32(&bars[s]); };
  auto empty_bar = [&](int s) { return smem_u32(&bars[C::kStages + s]); };
  auto tfull_bar = [&](int a) { return smem_u32(&bars[2 * C::kStages + a]); };
  auto tempty_bar = [&](int a) { return smem_u32(&bars[2 * C::kStages + 2 + a]); };
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC);
  int32_t* offs = reinterpret_cast<int32_t*>(smem + C::OFF_TAB);
  int32_t* mt = offs + (kMaxE + 1);

  // ---- the offsets table, checked by every CTA
  for (int i = threadIdx.x; i <= p.E; i += blockDim.x) offs[i] = p.offsets[i];
  __syncthreads();
  bool bad = false;
  for (int i = threadIdx.x; i <= p.E; i += blockDim.x) {
    const int32_t o = offs[i];
    if (o < 0 || int64_t(o) > p.M || (i == 0 && o != 0) || (i < p.E && offs[i + 1] < o)) bad = true;
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0 && blockIdx.x == 0) raise_device_error(kErrOffsets);
    return;
  }
  // first token tile of each expert: warp 3 scans 32 experts at a time
  if (kMode != kWgrad && warp == 3) {
    int run = 0;
    for (int b = 0; b < p.E; b += 32) {
      const int e = b + lane;
      const int c = e < p.E ? (offs[e + 1] - offs[e] + C::BN - 1) / C::BN : 0;
      int s = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += v;
      }
      if (e < p.E) mt[e] = run + s - c;
      run += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) mt[p.E] = run;
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmap_a);
    prefetch_tmap(&tmap_b);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 8);
    }
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(const_cast<uint32_t*>(misc)), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = misc[0];
  const int rt = (p.rows + C::BM - 1) / C::BM;
  const int64_t ntiles = kMode == kWgrad ? int64_t(p.E) * rt * ((p.cols + C::BN - 1) / C::BN) : int64_t(mt[p.E]) * rt;

  if (warp == 0) {
    // ================= producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; t < ntiles && ok; t += gridDim.x) {
        const Tile T = get_tile<kMode>(p, offs, mt, t);
        const int boxes = (T.n + 63) >> 6;                       // 64 tokens (kWgrad: 64 columns) each
        for (int kb = 0; kb < T.nk; ++kb) {
          if (!mbar_wait(empty_bar(stage), phase ^ 1)) { ok = false; break; }
          const uint32_t fb = full_bar(stage);
          const uint32_t as = sbase + C::OFF_A + stage * C::A_BYTES, bs = sbase + C::OFF_B + stage * C::B_BYTES;
          mbar_arrive_expect_tx(fb, C::A_BYTES + boxes * 8192);
          if constexpr (kMode == kFwd) {
            tma_load_3d(as, &tmap_a, fb, kb * kBK, T.r0, T.e);
          } else if constexpr (kMode == kDgrad) {
            tma_load_3d(as, &tmap_a, fb, T.r0, kb * kBK, T.e);
            tma_load_3d(as + 8192, &tmap_a, fb, T.r0 + 64, kb * kBK, T.e);
          } else {
            tma_load_2d(as, &tmap_a, fb, T.r0, int(T.t0) + kb * kBK);
            tma_load_2d(as + 8192, &tmap_a, fb, T.r0 + 64, int(T.t0) + kb * kBK);
          }
          for (int b = 0; b < boxes; ++b) {
            if constexpr (kMode == kWgrad)
              tma_load_2d(bs + b * 8192, &tmap_b, fb, T.c0 + 64 * b, int(T.t0) + kb * kBK);
            else
              tma_load_2d(bs + b * 8192, &tmap_b, fb, kb * kBK, int(T.t0) + 64 * b);
          }
          if (++stage == C::kStages) { stage = 0; phase ^= 1; }
        }
      }
      if (!ok) raise_device_error(kErrTimeout);
    }
  } else if (warp == 1) {
    // ================= MMA issuer (lane 0; in kWgrad the whole warp goes along
    // and clears the rows past a segment's end before the block's MMAs)
    if (kMode == kWgrad || lane == 0) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; t < ntiles && ok; t += gridDim.x) {
        const Tile T = get_tile<kMode>(p, offs, mt, t);
        if (T.nk == 0) continue;
        if (!warp_wait<kMode>(tempty_bar(acc), acc_phase ^ 1)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d = tmem_base + acc * C::BN;
        const uint32_t idesc = f16_idesc(kDt == kBF16 ? 1 : 0, kAMn, kBMn, C::BM, uint32_t((T.n + 15) & ~15));
        for (int kb = 0; kb < T.nk; ++kb) {
          if (!warp_wait<kMode>(full_bar(stage), phase)) { ok = false; break; }
          tc_fence_after();
          int steps = kBK / 16;
          if constexpr (kMode == kWgrad) {
            const int rem = T.len - kb * kBK;
            if (rem < kBK) {
              steps = (rem + 15) >> 4;
              // a K row is one 128-byte line of each box: the swizzle stays inside the line
              const int boxes = (T.n + 63) >> 6;
              for (int r = rem; r < steps * 16; ++r) {
                for (int b = 0; b < 2; ++b)
                  *reinterpret_cast<uint32_t*>(smem + C::OFF_A + stage * C::A_BYTES + b * 8192 + r * 128 + lane * 4) = 0;
                for (int b = 0; b < boxes; ++b)
                  *reinterpret_cast<uint32_t*>(smem + C::OFF_B + stage * C::B_BYTES + b * 8192 + r * 128 + lane * 4) = 0;
              }
              fence_proxy_async();
              __syncwarp();
            }
          }
          if (lane == 0) {
            const uint32_t as = sbase + C::OFF_A + stage * C::A_BYTES, bs = sbase + C::OFF_B + stage * C::B_BYTES;
            // K-major: 32 bytes a step inside the 128-byte rows, 1024 between 8-row groups.
            // MN-major: 16 rows of 128 bytes a step, 1024 between 8-row groups, 8192 between 64-value boxes.
            for (int k = 0; k < steps; ++k) {
              const uint64_t ad = kAMn ? smem_desc(as + k * 2048, 8192, 1024, 2) : smem_desc(as + k * 32, 0, 1024, 2);
              const uint64_t bd = kBMn ? smem_desc(bs + k * 2048, 8192, 1024, 2) : smem_desc(bs + k * 32, 0, 1024, 2);
              mma_f16(d, ad, bd, idesc, (kb | k) != 0);
            }
            mma_commit(empty_bar(stage));
          }
          if (++stage == C::kStages) { stage = 0; phase ^= 1; }
        }
        if (!ok) break;
        if (lane == 0) mma_commit(tfull_bar(acc));
        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
      }
      if (!ok && lane == 0) raise_device_error(kErrTimeout);
    }
  } else if (warp >= 4) {
    // ================= epilogue
    const int q = warp & 3, h = (warp - 4) >> 2;
    uint8_t* sbuf = smem + C::OFF_EPI + (warp - 4) * C::EPI_WARP_BYTES;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int64_t t = blockIdx.x; t < ntiles; t += gridDim.x) {
      const Tile T = get_tile<kMode>(p, offs, mt, t);
      const int row = T.r0 + q * 32;                             // this warp's 32 M-side rows
      const int chunks = (T.n + 31) >> 5;
      const bool any = T.nk != 0;                                // kWgrad: an expert without rows has a zero gradient
      if (any) {
        if (!__all_sync(0xffffffffu, mbar_wait(tfull_bar(acc), acc_phase))) {
          if (lane == 0) raise_device_error(kErrTimeout);
          break;
        }
        tc_fence_after();
      }
      for (int c = h; c < chunks; c += 2) {
        uint32_t r[32];
        if (any) {
          tmem_ld_32x32b_x32(tmem_base + (uint32_t(q * 32) << 16) + acc * C::BN + 32 * c, r);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = 0u;
        }
        if constexpr (kMode == kWgrad) {
          // one row of 32 columns per lane: staged in the store map's 64-byte
          // swizzle (16-byte piece j of row r at j ^ ((r >> 1) & 3)); the map
          // clips the box at the matrix's edges
          if (row < p.rows) {
            if (lane == 0) bulk_wait_read_all();
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                w[i] = pack16x2<kDt>(__uint_as_float(r[8 * j + 2 * i]), __uint_as_float(r[8 * j + 2 * i + 1]));
              *reinterpret_cast<uint4*>(sbuf + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
              tma_store_3d(&tmap_o, smem_u32(sbuf), T.c0 + 32 * c, row, T.e);
              bulk_commit();
            }
          }
        } else {
          // lane = output column, register = token: transposed through shared
          // memory (a token's 32 columns are one 64-byte line, written two
          // bytes a lane without conflicts), then 16-byte stores of four
          // lanes a token
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const uint32_t w = pack16x2<kDt>(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
            *reinterpret_cast<uint16_t*>(sbuf + (2 * j) * 64 + lane * 2) = uint16_t(w & 0xFFFFu);
            *reinterpret_cast<uint16_t*>(sbuf + (2 * j + 1) * 64 + lane * 2) = uint16_t(w >> 16);
          }
          __syncwarp();
          const int col = row + (lane & 3) * 8;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int tok = 8 * i + (lane >> 2);
            const uint4 v = *reinterpret_cast<const uint4*>(sbuf + tok * 64 + (lane & 3) * 16);
            if (32 * c + tok < T.n && col < p.rows)
              *reinterpret_cast<uint4*>(p.out + (T.t0 + 32 * c + tok) * p.rows + col) = v;
          }
          __syncwarp();
        }
      }
      if (any) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty_bar(acc));
        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
      }
    }
    if (kMode == kWgrad && lane == 0) bulk_wait_all();
  }
  // ---- teardown: every role has left its loop (all waits are bounded)
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

}  // namespace mxmoe::ragged
