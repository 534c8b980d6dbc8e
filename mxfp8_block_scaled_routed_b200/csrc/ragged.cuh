// Grouped 16-bit products over ragged expert segments on the sm_100a tensor
// cores (tcgen05 kind::f16, fp32 accumulators in TMEM, TMA-fed tiles).
//
//   kFwd    out[m, n] = sum_k a[m, k] W[e, n, k]   for the rows m of expert e
//   kDgrad  out[m, k] = sum_n g[m, n] W[e, n, k]
//   kWgrad  dW[e, n, k] = sum_m g[m, n] a[m, k]    over the rows m of expert e
//
// Segments have any length (no padding) and start at any row.  TMA boxes may
// start at any row, so a tile simply reads from its first token on:
//  * kFwd / kDgrad put the weights on the MMA's M side and the tokens on its N
//    side, whose width is the instruction's and not the kernel's: a segment's
//    last tile runs an MMA of its own rows rounded up to 16, so a ragged tail
//    costs its own columns only.  A tile's columns past the segment hold the
//    next expert's tokens; they are not stored.
//  * kWgrad contracts over the tokens.  A segment's last K block is cut at the
//    next multiple of 16 tokens, and a warp clears the up to 15 rows past the
//    end in both operands first (they may hold NaN: a product with zero would
//    not do).
// Operands are read as they lie: W for kFwd and the token matrices are K-major
// (128-byte swizzled rows of 64 values); W for kDgrad and both operands of
// kWgrad are MN-major (boxes of 64 values of the M or N extent by 64 of K).
//
// A CTA pair (cluster of 2, cta_group::2) computes a tile of 256 M-side rows by
// up to 256 columns: each CTA holds 128 rows of A, half of the columns of B and
// its own 128 x 256 accumulator, so a K block of 64 costs each SM 32 KB of
// loads for 512 cycles of MMA where a single CTA's 128 x 256 tile would need
// 48 KB.
//
// CTA = 12 warps: warp 0 works out each tile's place and issues TMA, warp 1 of
// the even CTA issues the pair's MMAs, warp 2 owns TMEM, warp 3 clears kWgrad
// tails, warps 4..11 are the epilogue (warp 4 + q and 8 + q read TMEM lanes
// 32 q.., alternating 32-column chunks).  Two accumulators of 256 columns: a
// tile's epilogue runs beside the next tile's MMAs.
//
// Bound by the MMAs (512 cycles a full K block) from about ten K blocks a tile
// on, and in a long loop by the power limit (49152 rows, 64 x 2816 x 2048: 412 to
// 440 us in a short loop, 1.29 to 1.38 PFLOP/s; 505 to 523 in a long one).  Shorter tiles wait for their stores: a chunk's staging buffer
// is free 300 to 490 cycles late while the tiles' loads and stores together move
// 11 TB/s through L2 (32768 rows, 8 x 4096 x 256: 73 us, ~3,700 cycles a tile of
// 2,048 of MMAs; long contractions load 13 TB/s).  Few tiles with a long
// contraction are split along it and joined (join_kernel).
#pragma once
#include <cuda.h>
#include "half16.cuh"
#include "quant.cuh"
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
  uint16_t* out;             // kFwd / kDgrad: [M, rows]; kWgrad (for join_kernel): [E, rows, cols]
  // Few tiles with a long contraction: a tile's K blocks go to `splits` units,
  // which leave fp32 sums for join_kernel.
  int splits;                // 1: no split
  int* ok;                   // set when the offsets are good, for join_kernel
  float* sums;               // [splits][M, rows] (kWgrad: [splits][E, rows, cols])
};

// Units that share a tile of nk K blocks: at least kMinBlocks each.
constexpr int kMinBlocks = 4;
__host__ __device__ inline int parts_of(int nk, int splits) { return max(1, min(splits, nk / kMinBlocks)); }

struct Cfg {
  static constexpr int BM = 256, BN = 256;                            // of the pair
  static constexpr int A_BYTES = 128 * kBK * 2, B_BYTES = 128 * kBK * 2;   // per CTA and stage
  static constexpr int kBox = 64;                                     // token rows per TMA box (kFwd, kDgrad)
  static constexpr int kStages = 6;
  static constexpr int OFF_A = 0, OFF_B = kStages * A_BYTES;
  static_assert(A_BYTES == B_BYTES, "one stage offset for both operands");
  static constexpr int OFF_EPI = OFF_B + kStages * B_BYTES;
  static constexpr int EPI_WARP_BYTES = 2048;  // a 32 x 32 block of 16-bit outputs per epilogue warp
  static constexpr int OFF_BAR = OFF_EPI + 8 * EPI_WARP_BYTES;
  static constexpr int kInfo = 16;             // tiles that the producer may announce ahead
  static constexpr int NUM_BARS = 3 * kStages + 4 + 2 * kInfo;
  static constexpr int OFF_MISC = (OFF_BAR + NUM_BARS * 8 + 15) & ~15;
  // offsets [E + 1]; first token tile of each expert [E + 1] (kWgrad: its rows); kWgrad's schedule order [E]
  static constexpr int TAB = (kMaxE + 4) * 4;
  static constexpr int OFF_INFO = OFF_MISC + 16, INFO = 32;
  static constexpr int OFF_TAB = OFF_INFO + kInfo * INFO;
  static constexpr int SMEM_BYTES = OFF_TAB + 2 * TAB + kMaxE * 2 + 1024;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
  static_assert(OFF_TAB % 16 == 0 && TAB % 16 == 0, "the tables are read 16 bytes at a time");
};

// Instruction descriptor, kind::f16: fp32 accumulator (bit 4), A and B type at
// 7 and 10 (0 f16, 1 bf16), MN-major A / B at 15 / 16, N >> 3 at 17, M >> 4 at 24.
__device__ __forceinline__ uint32_t f16_idesc(int dt_bits, bool a_mn, bool b_mn, uint32_t M, uint32_t N) {
  return (1u << 4) | (uint32_t(dt_bits) << 7) | (uint32_t(dt_bits) << 10) | (uint32_t(a_mn) << 15) |
         (uint32_t(b_mn) << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
__device__ __forceinline__ void mma_f16_pair(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const void* tmap, uint32_t bar_cluster, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar_cluster)
      : "memory");
}
__device__ __forceinline__ void tma_store_3d(const void* tmap, uint32_t src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(tmap), "r"(x),
               "r"(y), "r"(z), "r"(src)
               : "memory");
}

// One lane of a converged warp (the same one each time).  The TMA and MMA
// roles run their loops with the whole warp (each wait's outcome is the
// warp's) and issue under this: inside an
// `if (lane == 0)` role a tcgen05.mma took its thread ~120 cycles to issue,
// and a K block ~580 cycles however narrow its tile.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(ok));
  return ok != 0;
}

// A barrier of two warps: whether both say yes.
__device__ __forceinline__ bool pair_all(int id, bool yes) {
  uint32_t r;
  asm volatile(
      "{ .reg .pred p, q; setp.ne.u32 p, %1, 0;\n"
      "barrier.cta.red.and.pred q, %2, 64, p; selp.u32 %0, 1, 0, q; }"
      : "=r"(r)
      : "r"(uint32_t(yes)), "r"(id)
      : "memory");
  return r != 0;
}

// The tiles of one pair, a round over all pairs at a time; kWgrad's odd rounds
// run back over the pairs.
template <int kMode>
struct Walk {
  uint32_t unit, units, base, back;
  __device__ __forceinline__ Walk(uint32_t u, uint32_t n) : unit(u), units(n), base(0), back(0) {}
  __device__ __forceinline__ uint32_t at(uint32_t rev) const { return kMode == kWgrad && rev ? units - 1 - unit : unit; }
  __device__ __forceinline__ uint32_t tile() const { return base + at(back); }
  __device__ __forceinline__ void next() { base += units; back ^= 1; }
};

struct Tile {
  int e, part;
  int kb0, kb1; // this unit's K blocks
  int r0;       // first M-side row (of the expert's matrix)
  int n;        // N-side columns (tokens; kWgrad: columns of K)
  int t0;       // first token (kFwd / kDgrad: of the tile; kWgrad: of the segment)
  int c0;       // kWgrad: first N-side column
  int len;      // kWgrad: tokens of the segment
};

// Token columns of a segment's tiles: equal, up to 256, a multiple of 16.
__device__ __forceinline__ int tile_width(int len) {
  const int tiles = max(1, (len + Cfg::BN - 1) / Cfg::BN);
  return ((len + tiles - 1) / tiles + 15) & ~15;
}

// Tile t: experts in order; kWgrad: (expert in schedule order, row tile, column tile).
// The host keeps tile numbers below 2^31.
template <int kMode>
__device__ __forceinline__ Tile get_tile(const Params& p, const int32_t* offs, const int32_t* tab, const uint16_t* ord,
                                         uint32_t t) {
  Tile T;
  int nk;       // of the whole tile
  T.part = 0;
  if (p.splits > 1) {
    T.part = int(t % uint32_t(p.splits));
    t /= uint32_t(p.splits);
  }
  const uint32_t rt = uint32_t(p.rows + Cfg::BM - 1) / Cfg::BM;
  if constexpr (kMode == kWgrad) {
    const uint32_t ct = uint32_t(p.cols + Cfg::BN - 1) / Cfg::BN;
    const uint32_t row = t / ct;
    const uint32_t i = row / rt;
    T.e = ord[i];
    T.r0 = int(row - i * rt) * Cfg::BM;
    T.c0 = int(t - row * ct) * Cfg::BN;
    T.n = min(Cfg::BN, p.cols - T.c0);
    T.t0 = offs[T.e];
    T.len = offs[T.e + 1] - offs[T.e];
    nk = (T.len + kBK - 1) / kBK;
  } else {
    int lo = 0, hi = p.E;                      // last expert whose first tile is at or before t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (uint32_t(tab[mid]) * rt <= t) lo = mid; else hi = mid;
    }
    T.e = lo;
    // blocks of 8 row tiles, inside one the row tile runs fastest: the pairs at
    // work at one time share 8 row tiles of the weights and a few token tiles
    constexpr uint32_t kRows = 8;
    const uint32_t w = t - uint32_t(tab[lo]) * rt, tiles = uint32_t(tab[lo + 1] - tab[lo]);
    const uint32_t blk = w / (kRows * tiles), in = w - blk * kRows * tiles, br = min(kRows, rt - blk * kRows), j = in / br;
    const int len = offs[T.e + 1] - offs[T.e], per = tile_width(len);
    T.r0 = int(blk * kRows + in - j * br) * Cfg::BM;
    T.t0 = offs[T.e] + int(j) * per;
    T.n = min(per, len - int(j) * per);
    nk = (p.kext + kBK - 1) / kBK;
    T.c0 = 0;
    T.len = 0;
  }
  T.kb0 = 0;
  T.kb1 = nk;
  if (p.splits > 1) {
    const int parts = parts_of(nk, p.splits);
    T.kb0 = T.part < parts ? int(int64_t(nk) * T.part / parts) : 0;
    T.kb1 = T.part < parts ? int(int64_t(nk) * (T.part + 1) / parts) : 0;
  }
  return T;
}

// kPair: store boxes of 64 values instead of 32 (kFwd and kDgrad: always).
template <int kMode, int kDt, bool kPair>
__global__ void __launch_bounds__(384, 1)
ragged_gemm_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                   const __grid_constant__ CUtensorMap tmap_o, const Params p) {
  using C = Cfg;
  constexpr bool kAMn = kMode != kFwd, kBMn = kMode == kWgrad;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = int(cluster_ctarank());                           // the cluster is (2, 1, 1)
  const uint32_t unit = blockIdx.x >> 1, units = gridDim.x >> 1;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  auto full_bar = [&](int s) { return smem_u32(&bars[s]); };
  auto empty_bar = [&](int s) { return smem_u32(&bars[C::kStages + s]); };
  auto tail_bar = [&](int s) { return smem_u32(&bars[2 * C::kStages + s]); };
  auto tfull_bar = [&](int a) { return smem_u32(&bars[3 * C::kStages + a]); };
  auto tempty_bar = [&](int a) { return smem_u32(&bars[3 * C::kStages + 2 + a]); };
  auto info_bar = [&](int s) { return smem_u32(&bars[3 * C::kStages + 4 + s]); };
  auto seen_bar = [&](int s) { return smem_u32(&bars[3 * C::kStages + 4 + C::kInfo + s]); };
  // Some waits last as long as a tile: the epilogue's and warp 3's for its last
  // block, the producer's for a slot of the places when tiles without blocks follow
  // it.  A block takes ~430 cycles, so an unsplit contraction of ten million of them
  // is longer than the usual two seconds.
  const long long whole = (1ll << 32) + 4096ll * (kMode == kWgrad ? (p.M + kBK - 1) / kBK : (p.kext + kBK - 1) / kBK);
  // A tile's place takes several hundred cycles to work out (a search, divisions).
  // The producer does it, tiles ahead, and the other roles of its CTA read it
  // (their i-th tile; ok: announced in time): 32768 rows x 8 x 4096 x 256 88 -> 82
  // us against every role on its own, 64 weight gradients of 2048 x 2048 from 6000
  // rows 119 -> 117.
  auto read_tile = [&](uint32_t i, bool& ok) {
    const int s = i % C::kInfo;
    ok = __all_sync(0xffffffffu, mbar_wait(info_bar(s), (i / C::kInfo) & 1, whole));
    const uint4 a = lds128(sbase + C::OFF_INFO + s * C::INFO), b = lds128(sbase + C::OFF_INFO + s * C::INFO + 16);
    __syncwarp();
    if (lane == 0) mbar_arrive(seen_bar(s));
    Tile T;
    T.e = int(a.x & 0xFFFFu);
    T.part = int(a.x >> 16);
    T.kb0 = int(a.y);
    T.kb1 = int(a.z);
    T.r0 = int(a.w);
    T.n = int(b.x);
    T.t0 = int(b.y);
    T.c0 = int(b.z);
    T.len = int(b.w);
    return T;
  };
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC);
  int32_t* offs = reinterpret_cast<int32_t*>(smem + C::OFF_TAB);
  int32_t* tab = offs + C::TAB / 4;
  uint16_t* ord = reinterpret_cast<uint16_t*>(tab + C::TAB / 4);

  // ---- the offsets table, checked by every CTA (both of a pair see the same)
  for (int i = threadIdx.x; i <= p.E; i += blockDim.x) offs[i] = p.offsets[i];
  __syncthreads();
  bool bad = false;
  for (int i = threadIdx.x; i <= p.E; i += blockDim.x) {
    const int32_t o = offs[i];
    if (o < 0 || int64_t(o) > p.M || (i == 0 && o != 0) || (i < p.E && offs[i + 1] < o)) bad = true;
  }
  bad = __syncthreads_or(bad);
  if (p.splits > 1) {
    launch_dependents();
    if (threadIdx.x == 0 && blockIdx.x == 0) *p.ok = !bad;
  }
  if (bad) {
    if (threadIdx.x == 0 && blockIdx.x == 0) raise_device_error(kErrOffsets);
    return;
  }
  if constexpr (kMode == kWgrad) {
    // ---- schedule order: experts by rows, most first, ties in expert order.
    // A tile's time is its expert's rows; with the rounds of tiles going forth
    // and back over the pairs, every pair comes to nearly the same sum.  (24
    // experts by Zipf's law: the longest pair 6 % over the mean, 22 % in expert
    // order; 94.8 -> 90.3 us.  Token tiles are alike in time: kFwd and kDgrad
    // gain nothing and keep the experts' order.)
    for (int i = threadIdx.x; i < ((p.E + 3) & ~3); i += blockDim.x) tab[i] = i < p.E ? offs[i + 1] - offs[i] : -1;
    __syncthreads();
    for (int i = threadIdx.x; i < p.E; i += blockDim.x) {
      const int key = tab[i];
      int r = 0;
      for (int j = 0; j < p.E; j += 4) {
        const int4 k = *reinterpret_cast<const int4*>(tab + j);
        r += (k.x > key || (k.x == key && j < i)) + (k.y > key || (k.y == key && j + 1 < i)) +
             (k.z > key || (k.z == key && j + 2 < i)) + (k.w > key || (k.w == key && j + 3 < i));
      }
      ord[r] = uint16_t(i);
    }
  } else if (warp == 3) {
    // ---- first token tile of each expert, 32 experts at a time
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
      if (e < p.E) tab[e] = run + s - c;
      run += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) tab[p.E] = run;
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmap_a);
    prefetch_tmap(&tmap_b);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full_bar(s), kMode == kWgrad ? 2 : 1);               // kWgrad: one arrival from each CTA
      mbar_init(empty_bar(s), 1);
      mbar_init(tail_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 16);                                  // the epilogue warps of both CTAs
    }
    for (int i = 0; i < C::kInfo; ++i) {
      mbar_init(info_bar(i), 1);
      mbar_init(seen_bar(i), 8 + (rank == 0) + (kMode == kWgrad));   // epilogue warps, MMA issuer, kWgrad's warp 3
    }
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc_pair(smem_u32(const_cast<uint32_t*>(misc)), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = misc[0];
  const int rt = (p.rows + C::BM - 1) / C::BM;
  const uint32_t ntiles = uint32_t(kMode == kWgrad ? p.E * ((p.cols + C::BN - 1) / C::BN) : tab[p.E]) * rt * p.splits;

  if (warp == 0) {
    // ================= producer (each CTA loads its own operand halves; the
    // bytes of both are credited to the even CTA's full barrier)
    int stage = 0;
    uint32_t phase = 0, at = 0;
    bool ok = true;
    for (Walk<kMode> w(unit, units); w.tile() < ntiles && ok; w.next(), ++at) {
      const Tile T = get_tile<kMode>(p, offs, tab, ord, w.tile());
      const int slot = at % C::kInfo;
      if (!__all_sync(0xffffffffu, mbar_wait(seen_bar(slot), ((at / C::kInfo) & 1) ^ 1, whole))) { ok = false; break; }
      if (elect_one()) {
        const uint32_t to = sbase + C::OFF_INFO + slot * C::INFO;
        sts128(to, make_uint4(T.e | T.part << 16, T.kb0, T.kb1, T.r0));
        sts128(to + 16, make_uint4(T.n, T.t0, T.c0, T.len));
        mbar_arrive(info_bar(slot));
      }
      __syncwarp();
      const int half = ((T.n + 15) & ~15) >> 1;                      // columns of B per CTA
      constexpr int kCols = kMode == kWgrad ? 64 : C::kBox;          // per box
      const int boxes = (half + kCols - 1) / kCols;
      const uint32_t bytes = C::A_BYTES + boxes * kCols * 128;       // per CTA
      const int r0 = T.r0 + rank * 128, b0 = rank * half;
      for (int kb = T.kb0; kb < T.kb1; ++kb) {
        if (!__all_sync(0xffffffffu, mbar_wait(empty_bar(stage), phase ^ 1))) { ok = false; break; }
        if (elect_one()) {
          const uint32_t as = sbase + C::OFF_A + stage * C::A_BYTES, bs = sbase + C::OFF_B + stage * C::B_BYTES;
          uint32_t fb = mapa_cluster(full_bar(stage), 0);
          if constexpr (kMode == kWgrad) {
            const int row = T.t0 + kb * kBK, rem = T.len - kb * kBK;
            if (rem < kBK && (rem & 15)) {
              // a tail to clear: this CTA's bytes go to its own tail barrier,
              // and warp 3 arrives on the full one when the rows are clear
              mbar_arrive_expect_tx(tail_bar(stage), bytes);
              fb = mapa_cluster(tail_bar(stage), rank);
            } else if (rank == 0) {
              mbar_arrive_expect_tx(full_bar(stage), 2 * bytes);
            } else {
              mbar_arrive_remote(full_bar(stage), 0);
            }
            tma_load_2d_pair(as, &tmap_a, fb, r0, row);
            tma_load_2d_pair(as + 8192, &tmap_a, fb, r0 + 64, row);
            for (int b = 0; b < boxes; ++b) tma_load_2d_pair(bs + b * 8192, &tmap_b, fb, T.c0 + b0 + 64 * b, row);
          } else {
            if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), 2 * bytes);
            if constexpr (kMode == kFwd) {
              tma_load_3d_pair(as, &tmap_a, fb, kb * kBK, r0, T.e);
            } else {
              tma_load_3d_pair(as, &tmap_a, fb, r0, kb * kBK, T.e);
              tma_load_3d_pair(as + 8192, &tmap_a, fb, r0 + 64, kb * kBK, T.e);
            }
            for (int b = 0; b < boxes; ++b)
              tma_load_2d_pair(bs + b * (C::kBox * 128), &tmap_b, fb, kb * kBK, T.t0 + b0 + C::kBox * b);
          }
        }
        __syncwarp();
        if (++stage == C::kStages) { stage = 0; phase ^= 1; }
      }
    }
    if (!ok && lane == 0) raise_device_error(kErrTimeout);
  } else if (warp == 1) {
    // ================= MMA issuer (the even CTA's, for both)
    if (rank == 0) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      // K-major: 32 bytes a step inside the 128-byte rows, 1024 between 8-row groups.
      // MN-major: 16 rows of 128 bytes a step, 1024 between 8-row groups, 8192 between 64-value boxes.
      const uint64_t a_desc = smem_desc(sbase + C::OFF_A, kAMn ? 8192 : 0, 1024, 2);
      const uint64_t b_desc = smem_desc(sbase + C::OFF_B, kBMn ? 8192 : 0, 1024, 2);
      constexpr uint64_t a_step = (kAMn ? 2048 : 32) >> 4, b_step = (kBMn ? 2048 : 32) >> 4;
      uint32_t at = 0;
      for (Walk<kMode> w(unit, units); w.tile() < ntiles && ok; w.next(), ++at) {
        const Tile T = read_tile(at, ok);
        if (!ok) break;
        if (T.kb1 == T.kb0) continue;
        if (!__all_sync(0xffffffffu, mbar_wait_cluster(tempty_bar(acc), acc_phase ^ 1))) { ok = false; break; }
        tc_fence_after();
        const uint32_t d = tmem_base + acc * C::BN;
        const uint32_t idesc = f16_idesc(kDt == kBF16 ? 1 : 0, kAMn, kBMn, C::BM, uint32_t((T.n + 15) & ~15));
        for (int kb = T.kb0; kb < T.kb1; ++kb) {
          if (!__all_sync(0xffffffffu, mbar_wait_cluster(full_bar(stage), phase))) { ok = false; break; }
          tc_fence_after();
          if (elect_one()) {
            const uint64_t ad = a_desc + stage * (C::A_BYTES >> 4), bd = b_desc + stage * (C::B_BYTES >> 4);
            const int steps = kMode == kWgrad ? min(kBK / 16, (T.len - kb * kBK + 15) >> 4) : kBK / 16;
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k)
              if (kMode != kWgrad || k < steps) mma_f16_pair(d, ad + k * a_step, bd + k * b_step, idesc, kb != T.kb0 || k != 0);
            mma_commit_pair(empty_bar(stage));
            if (kb == T.kb1 - 1) mma_commit_pair(tfull_bar(acc));
          }
          __syncwarp();
          if (++stage == C::kStages) { stage = 0; phase ^= 1; }
        }
        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
      }
      if (!ok && lane == 0) raise_device_error(kErrTimeout);
    }
  } else if (warp == 3) {
    // ================= kWgrad: clear this CTA's rows past a segment's end
    if constexpr (kMode == kWgrad) {
      int stage = 0;
      uint32_t used = 0, at = 0;                                     // used: phase of each stage's tail barrier, one bit each
      bool ok = true;
      for (Walk<kMode> w(unit, units); w.tile() < ntiles && ok; w.next(), ++at) {
        const Tile T = read_tile(at, ok);
        if (!ok) break;
        if (T.kb1 == T.kb0) continue;
        stage = (stage + T.kb1 - T.kb0 - 1) % C::kStages;            // this unit's last block
        const int rem = T.len - (T.kb1 - 1) * kBK;
        if (rem < kBK && (rem & 15)) {
          ok = __all_sync(0xffffffffu, mbar_wait(tail_bar(stage), (used >> stage) & 1, whole));
          if (!ok) break;
          used ^= 1u << stage;
          // a K row is one 128-byte line of each box (the swizzle stays inside
          // the line): the rows to clear are one piece per box
          const int bytes = (((rem + 15) & ~15) - rem) * 128, boxes = (((T.n + 15) & ~15) / 2 + 63) >> 6;
          const uint32_t first = stage * C::A_BYTES + rem * 128 + lane * 16;
          for (int i = lane * 16; i < bytes; i += 512) {
            const uint32_t o = sbase + first + (i - lane * 16);
            sts128(o + C::OFF_A, make_uint4(0, 0, 0, 0));
            sts128(o + C::OFF_A + 8192, make_uint4(0, 0, 0, 0));
            sts128(o + C::OFF_B, make_uint4(0, 0, 0, 0));
            if (boxes > 1) sts128(o + C::OFF_B + 8192, make_uint4(0, 0, 0, 0));
          }
          // the issuer of the MMAs that read these rows is a thread of the even
          // CTA: every lane's stores are fenced to the async proxy, the warp sync
          // orders them before lane 0's release, and that one has to be of cluster
          // scope to pair with the issuer's acquire.  Only shared memory is
          // published: a release of all state spaces waits for the stores under way
          // (64 experts of 760 rows x 2816 x 2048 463 us against 412)
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive_release_shared(full_bar(stage), 0);
        }
        stage = (stage + 1) % C::kStages;
      }
      if (!ok && lane == 0) raise_device_error(kErrTimeout);
    }
  } else if (warp >= 4) {
    // ================= epilogue
    const int q = warp & 3, h = (warp - 4) >> 2;
    constexpr bool kW = kMode == kWgrad;
    static_assert(kW || kPair, "kFwd and kDgrad store boxes of 64 columns");
    // Two warps may share a buffer, so that a store box has whole 128-byte lines:
    // the warps of neighbouring lanes in kFwd / kDgrad (64 features of 32 tokens;
    // 36204 rows x 3784 x 40 111 -> 98 us, 8 experts x 2048 x 512 63 -> 60), the two
    // of the same lanes in kWgrad where the host chose that (64 columns of 32 rows)
    const int pair = kW ? q : (warp - 4) >> 1, side = kPair ? (kW ? h : q & 1) : 0;
    uint8_t* sbuf = smem + C::OFF_EPI + (kPair ? pair * 2 : warp - 4) * C::EPI_WARP_BYTES;
    auto sync = [&]() {
      if constexpr (kPair) named_bar_sync(1 + pair, 64);
      else __syncwarp();
    };
    int acc = 0;
    uint32_t acc_phase = 0;
    uint32_t at = 0;
    for (Walk<kMode> w(unit, units); w.tile() < ntiles; w.next(), ++at) {
      bool ok;
      const Tile T = read_tile(at, ok);
      const int row = T.r0 + rank * 128 + q * 32;                // this warp's 32 M-side rows
      const int chunks = (T.n + 31) >> 5;
      const bool any = T.kb1 != T.kb0;                           // kWgrad: an expert without rows has a zero gradient
      if (ok && any) ok = __all_sync(0xffffffffu, mbar_wait(tfull_bar(acc), acc_phase, whole));
      if (!(kPair ? pair_all(1 + pair, ok) : ok)) {             // (two that share a buffer leave together)
        if (lane == 0) raise_device_error(kErrTimeout);
        break;
      }
      if (!any && p.splits > 1) continue;                        // (join_kernel writes it)
      tc_fence_after();
      const uint32_t from = tmem_base + (uint32_t(q * 32) << 16) + acc * C::BN;
      uint32_t r[32];
      if (p.splits > 1) {
        // fp32 sums as they lie: kWgrad 32 columns of a row per lane, else a
        // column per lane
        for (int c = h; c < chunks; c += 2) {
          tmem_ld_32x32b_x32(from + 32 * c, r);
          tmem_wait_ld(r);
          if (row + lane < p.rows) {
            if constexpr (kMode == kWgrad) {
              float* dst = p.sums + ((int64_t(T.part) * p.E + T.e) * p.rows + row + lane) * p.cols + T.c0 + 32 * c;
#pragma unroll
              for (int j = 0; j < 32; j += 4)
                if (32 * c + j < T.n)                              // (columns are a multiple of 8)
                  *reinterpret_cast<uint4*>(dst + j) = make_uint4(r[j], r[j + 1], r[j + 2], r[j + 3]);
            } else {
              float* dst = p.sums + (int64_t(T.part) * p.M + T.t0 + 32 * c) * p.rows + row + lane;
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (32 * c + j < T.n) dst[int64_t(j) * p.rows] = __uint_as_float(r[j]);
            }
          }
        }
      } else {
        // kWgrad: 32 columns of a row per lane; else fragments for a transposed
        // store, lanes 0..15 and 16..31
        auto load = [&](int c) {
          if constexpr (kMode == kWgrad) {
            tmem_ld_32x32b_x32(from + 32 * c, r);
          } else {
            tmem_ld_16x256b_x4(from + 32 * c, r);
            tmem_ld_16x256b_x4(from + 32 * c + (16u << 16), r + 16);
          }
        };
        // (kWgrad: where an odd number of chunks leaves the second of two warps that
        // share a buffer without a last one, it stages what it finds: that half of
        // the box lies past the matrix)
        const int last = kW && kPair ? (chunks + 1) & ~1 : chunks;
        if (any && h < last) load(h);
        for (int c = h; c < last; c += 2) {
          uint32_t w[16];
          if (any) {
            tmem_wait_ld(r);
#pragma unroll
            for (int j = 0; j < 16; ++j) w[j] = pack16x2<kDt>(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
            if (c + 2 < last) load(c + 2);                         // on its way while this chunk is stored
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) w[j] = 0u;
          }
          if constexpr (kMode == kWgrad) {
            // staged in the store map's swizzle: 16-byte piece j of row r at j ^
            // (r & 7) of 128-byte lines, at j ^ ((r >> 1) & 3) of 64-byte ones; the
            // map clips the box at the matrix's edges
            if (row < p.rows) {
              if (side == 0 && lane == 0) bulk_wait_read_all();
              sync();
              const int line = lane * (kPair ? 128 : 64), turn = kPair ? lane & 7 : (lane >> 1) & 3;
#pragma unroll
              for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint4*>(sbuf + line + (((4 * side + j) ^ turn) << 4)) =
                    make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
              fence_proxy_async();
              sync();
              if (side == 0 && lane == 0) {
                tma_store_3d(&tmap_o, smem_u32(sbuf), T.c0 + 32 * c, row, T.e);
                bulk_commit();
              }
            }
          } else {
            // w[2 g + (0, 1)]: tokens 8 g.. of lanes 0..7 and 8..15; w[8 + ..] of
            // lanes 16..31.  A token's 64 columns become one line (piece j of line
            // t at j ^ (t & 7)).  A chunk of 32 tokens leaves by TMA (the map
            // clips the columns), the segment's last tokens by 16-byte stores of
            // four lanes a token
            if (side == 0 && lane == 0) bulk_wait_read_all();
            sync();
            const uint32_t to = smem_u32(sbuf) + (lane & 7) * 128 + (((4 * side + (lane >> 3)) ^ (lane & 7)) << 4);
#pragma unroll
            for (int g = 0; g < 4; ++g) stmatrix_x4_trans(to + g * 1024, w[2 * g], w[2 * g + 1], w[8 + 2 * g], w[9 + 2 * g]);
            if (32 * c + 32 <= T.n) {
              fence_proxy_async();
              sync();
              if (side == 0 && lane == 0 && row < p.rows) {
                tma_store_2d(&tmap_o, smem_u32(sbuf), row, T.t0 + 32 * c);
                bulk_commit();
              }
            } else {
              __syncwarp();
              const int col = row + (lane & 3) * 8;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int tok = 8 * i + (lane >> 2);
                const uint4 v =
                    *reinterpret_cast<const uint4*>(sbuf + tok * 128 + (((4 * side + (lane & 3)) ^ (tok & 7)) << 4));
                if (32 * c + tok < T.n && col < p.rows)
                  *reinterpret_cast<uint4*>(p.out + int64_t(T.t0 + 32 * c + tok) * p.rows + col) = v;
              }
              __syncwarp();
            }
          }
        }
      }
      if (any) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(tempty_bar(acc), 0);
        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
      }
    }
    if (lane == 0) bulk_wait_all();
  }
  // ---- teardown: every role has left its loop (all waits are bounded); neither
  // CTA frees its TMEM or leaves while the other may still arrive on its
  // barriers or run MMAs into its TMEM
  tc_fence_before();
  cluster_sync_all();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// The units' sums of a split product, added in order and rounded once.
// kWgrad: parts by the expert's rows, zeros for an expert without; else rows
// below offsets[E].  Eight neighbouring values a thread.
template <bool kW, int kDt>
__global__ void __launch_bounds__(256) join_kernel(const Params p) {
  wait_dependency();
  if (!*p.ok) return;
  const int64_t each = int64_t(p.rows) * (kW ? p.cols : 1);          // values of an expert's matrix, of a row
  const int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 8, total = each * (kW ? int64_t(p.E) : p.M);
  const int64_t live = kW ? total : each * p.offsets[p.E];
  if (i >= live) return;
  int parts;
  if constexpr (kW) {
    const int e = int(i / each), len = p.offsets[e + 1] - p.offsets[e];
    parts = len == 0 ? 0 : parts_of((len + kBK - 1) / kBK, p.splits);
  } else {
    parts = parts_of((p.kext + kBK - 1) / kBK, p.splits);
  }
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.0f;
#pragma unroll 4
  for (int q = 0; q < parts; ++q) {
    const float4* s = reinterpret_cast<const float4*>(p.sums + q * total + i);
    const float4 a = s[0], b = s[1];
    v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
    v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
  }
  *reinterpret_cast<uint4*>(p.out + i) = make_uint4(pack16x2<kDt>(v[0], v[1]), pack16x2<kDt>(v[2], v[3]),
                                                    pack16x2<kDt>(v[4], v[5]), pack16x2<kDt>(v[6], v[7]));
}

}  // namespace mxmoe::ragged
