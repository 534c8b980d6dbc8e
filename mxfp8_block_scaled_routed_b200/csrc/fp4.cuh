// MXFP4 expert weights: E2M1 codes (sign, two exponent bits, one mantissa bit:
// 0, 0.5, 1, 1.5, 2, 3, 4, 6) with one E8M0 byte per 32 columns.
//
//   cast      byte = clamp(floor(log2(amax)) - 2 + 127, 0, 254), code = E2M1 of
//             x / 2^(byte - 127), nearest even, saturated at +-6; a block that
//             holds NaN or infinity gets byte 0xFF (its values decode to NaN)
//   matvec    y[s, n] = sum_k W[e_s, n, k] x[row_s, k] for a few slots s
//
// Layouts of a weight [E, R, K]:
//   PLAIN     codes [E, R, K/2], the even column in the low four bits; scales
//             [E, R, K/32]
//   TILE      for the matvec: tiles of 16 rows x 128 columns, tile t, column
//             group kq at (t * K/128 + kq) * 1024 bytes of the expert's codes.
//             In it the four bytes (eight codes) of row 8 h + g, block j (32
//             columns) and quarter q of it sit at h * 512 + g * 64 + q * 16 + 4 j:
//             lane 4 g + q of a warp reads one 16-byte word per half h, and
//             holds in it what the m16n8k16 product wants of rows g and g + 8.
//             Scales: (t * K/128 + kq) * 64 + row * 4 + j.
//   TILE_GATED  the same for W13 [E, 2F, K]: tile t takes gate rows 8t..8t+7 as
//             its half 0 and up rows F + 8t.. as its half 1, so that a lane
//             holds the gate and the up value of the same f.
#pragma once
#include "half16.cuh"
#include "quant.cuh"
#include "sm100.cuh"

namespace mxmoe {

constexpr int kFp4Plain = 0, kFp4Tile = 1, kFp4TileGated = 2;

// Two fp32 -> two E2M1 codes (nearest even, saturating), a in the low bits.
__device__ __forceinline__ uint32_t e2m1x2(float a, float b) {
  uint32_t r;
  asm("{ .reg .b8 c; cvt.rn.satfinite.e2m1x2.f32 c, %2, %1; cvt.u32.u8 %0, c; }" : "=r"(r) : "f"(a), "f"(b));
  return r;
}

// Eight E2M1 codes -> eight f16 (exact), pairs in column order.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{ .reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d; }"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Byte offset of the codes (and of the scale) of row r, columns 8 c8.. in one
// expert's matrix of R rows and K columns.
__device__ __forceinline__ void fp4_place(int layout, int64_t r, uint32_t c8, int64_t R, int64_t K, int64_t& code,
                                          int64_t& scale) {
  if (layout == kFp4Plain) {
    code = r * (K >> 1) + 4 * int64_t(c8);
    scale = r * (K >> 5) + (c8 >> 2);
    return;
  }
  int64_t t = r >> 4;
  uint32_t row = uint32_t(r & 15);
  if (layout == kFp4TileGated) {
    const int64_t F = R >> 1;
    const uint32_t half = r >= F ? 1u : 0u;
    const int64_t f = r - half * F;
    t = f >> 3;
    row = half * 8 + uint32_t(f & 7);
  }
  const int64_t cell = t * (K >> 7) + (c8 >> 4);
  const uint32_t q = c8 & 3, j = (c8 >> 2) & 3;
  code = cell * 1024 + (row >> 3) * 512 + (row & 7) * 64 + q * 16 + j * 4;
  scale = cell * 64 + row * 4 + j;
}

// One thread per eight columns, a 32-block on four neighbouring lanes.  Bound
// by HBM: 2 + 17/32 bytes a value.
template <int kDt>
__global__ void __launch_bounds__(256)
fp4_quantize_kernel(const uint16_t* __restrict__ x, int64_t batch, int64_t R, int64_t K, int layout,
                    uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const uint32_t upr = uint32_t(K >> 3);                      // eight-column units per row, a multiple of 4
  const int64_t first = int64_t(blockIdx.x) * 256;
  const int64_t r0 = first / upr;
  const uint32_t u = uint32_t(first - r0 * upr) + threadIdx.x;
  const uint32_t dr = u / upr;
  const int64_t row = r0 + dr;                                // of the [batch * R, K] matrix
  const uint32_t c8 = u - dr * upr;
  const bool live = row < batch * R;                          // whole 32-blocks: uniform in each group of four lanes
  uint4 v = make_uint4(0, 0, 0, 0);
  if (live) v = __ldcs(reinterpret_cast<const uint4*>(x + row * K) + c8);
  uint32_t m = absmax_f32bits8<kDt>(v);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  if (!live) return;
  uint32_t byte = 0xFFu, w = 0;
  const uint32_t in[4] = {v.x, v.y, v.z, v.w};
  if (m < 0x7F800000u) {
    const int e = int(m >> 23) - 2;
    byte = uint32_t(e < 0 ? 0 : e);
    const float inv = inv_scale_from_byte(byte);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack16x2<kDt>(in[i]);
      w |= e2m1x2(f.x * inv, f.y * inv) << (8 * i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)                               // magnitude 6 and the sign; the byte makes it NaN
      w |= (0x77u | ((in[i] >> 12) & 8u) | ((in[i] >> 24) & 0x80u)) << (8 * i);
  }
  const int64_t e = layout == kFp4Plain ? 0 : row / R;
  int64_t oc, os;
  fp4_place(layout, row - e * R, c8, R, K, oc, os);
  *reinterpret_cast<uint32_t*>(codes + e * R * (K >> 1) + oc) = w;
  if ((c8 & 3) == 0) scales[e * R * (K >> 5) + os] = uint8_t(byte);
}

// PLAIN -> 16-bit values, one thread per eight columns: code * 2^(byte - 127)
// is exact in fp32 and rounded once (bf16: never, but below 2^-133).
template <int kDt>
__global__ void __launch_bounds__(256)
fp4_dequantize_kernel(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t units,
                      uint4* __restrict__ out) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= units) return;
  const uint32_t w = __ldcs(codes + i);
  const float s = e8m0_to_f32(scales[i >> 2]);
  uint32_t h[4], o[4];
  e2m1x8_to_f16(w, h);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
    o[j] = pack16x2<kDt>(f.x * s, f.y * s);
  }
  out[i] = make_uint4(o[0], o[1], o[2], o[3]);
}

// ---------------------------------------------------------------- matvec
// A warp's product is mma.m16n8k16 with the weights as the 16-row operand and
// up to eight slots of one expert as the columns: each weight is read and
// decoded once for all of them.  The codes become f16 exactly; a block's 32
// products are summed by two MMAs from zero and then scaled by the block's
// 2^(byte - 127) into the fp32 sum, so no scale meets a 16-bit value.
//
// The activations become f16 after a division by a power of two per slot that
// puts the row's largest magnitude at 2^12: bf16 and fp16 inputs keep every
// bit down to 2^-36 of the row's largest value (an absolute error of at most
// 2^-37 of it beyond); the fp32 h between the two products is rounded to f16's
// 11 bits, an eighth of the bf16 rounding of the result.
//
// Bound by HBM: (1/2 + 1/32) N K bytes per expert that has a slot.  A block of
// 16 warps per SM walks a contiguous range of (slot group, row tile) units;
// each warp takes every 16th 128-column cell of the tile through its own ring
// of bulk copies, so the loads of later tiles are in flight while this one is
// multiplied, and the warps' partial sums meet in shared memory in a fixed
// order.
constexpr int kMvThreads = 512, kMvWarps = 16;
constexpr int kMvCell = 1024 + 64;          // codes and scales of a 16 x 128 cell
constexpr int kMvRing = 4;                  // cells in flight per warp
constexpr int kMvMaxSlots = 2048, kMvMaxE = 1024;

struct MvArgs {
  const void* x;            // [*, K]
  const int32_t* ids;       // [S] expert of each slot
  int S;
  int x_div;                // slot s reads row s / x_div of x
  int E;
  int64_t tiles;            // row tiles per expert
  int K;
  int group;                // slots per group, 1..8 (shared memory holds group * K f16)
  const uint8_t* codes;
  const uint8_t* scales;
  void* out;                // gated: fp32 h [S, 8 * tiles]; else y [S, 16 * tiles]
};

__host__ __device__ constexpr int mv_smem(int64_t K, int group, int E, int S) {
  // ring, partial sums (two tiles), f16 activations, then counts, slot order, groups
  return int(kMvWarps * kMvRing * kMvCell + 2 * kMvWarps * 512 + int64_t(group) * K * 2 + (kMvWarps * kMvRing) * 8 +
             64 + (E + 1) * 8 + S * 8 + 256);
}

template <int kDt>   // kBF16, kFP16, or 2 for fp32
__device__ __forceinline__ void mv_load8(const void* x, int64_t i, float (&f)[8]) {
  if constexpr (kDt == 2) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x) + i);
    const float4 a = p[0], b = p[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 t = unpack16x2<kDt>(w[j]);
      f[2 * j] = t.x;
      f[2 * j + 1] = t.y;
    }
  }
}

__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int kDt, bool kGated, int kOut>   // kOut: type of a non-gated result (kBF16, kFP16, 2 = fp32)
__global__ void __launch_bounds__(kMvThreads, 1) fp4_matvec_kernel(const MvArgs p) {
  extern __shared__ __align__(128) uint8_t mv_smem_raw[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  uint8_t* ring = mv_smem_raw;                                                    // [warp][slot][cell]
  float4* red = reinterpret_cast<float4*>(ring + kMvWarps * kMvRing * kMvCell);   // [2][warp][lane]
  uint8_t* xs = reinterpret_cast<uint8_t*>(red + 2 * kMvWarps * 32);              // f16 [K/32][group][4 quarters][8]
  uint64_t* bars = reinterpret_cast<uint64_t*>(xs + int64_t(p.group) * p.K * 2);
  uint32_t* xmax = reinterpret_cast<uint32_t*>(bars + kMvWarps * kMvRing);        // [8] largest magnitude, fp32 bits
  int* first = reinterpret_cast<int*>(xmax + 16);                                 // [E + 1] first slot of each expert
  int* gfirst = first + (p.E + 1);                                                // [E + 1] first group
  int* order = gfirst + (p.E + 1);                                                // [S] slots by expert
  int* pos = order + p.S;                                                         // [S] expert and rank among its slots
  __shared__ int wsum[2][kMvWarps];

  // ---- slots grouped by expert, in slot order: every block has to come to the
  // same groups, since the tiles of one group are spread over blocks
  for (int e = tid; e <= p.E; e += kMvThreads) first[e] = 0;
  for (int s = tid; s < p.S; s += kMvThreads) {
    const int e = p.ids[s];
    const bool ok = e >= 0 && e < p.E;
    pos[s] = ok ? e : -1;
    if (!ok && blockIdx.x == 0) raise_device_error(9);
  }
  for (int s = lane; s < kMvRing; s += 32) sm100::mbar_init(sm100::smem_u32(&bars[warp * kMvRing + s]), 1);
  sm100::fence_mbar_init();
  __syncthreads();
  if (warp == 0) {
    // rank among the expert's slots, 32 slots at a time: those before in the
    // batch and those of the batches before (expert in the low ten bits of pos)
    for (int b = 0; b < p.S; b += 32) {
      const int e = b + lane < p.S ? pos[b + lane] : -1;
      const unsigned peers = __match_any_sync(0xffffffffu, e);
      if (e >= 0) pos[b + lane] = e | ((first[e] + __popc(peers & ((1u << lane) - 1u))) << 10);
      __syncwarp();
      if (e >= 0 && lane == __ffs(peers) - 1) first[e] += __popc(peers);
      __syncwarp();
    }
  }
  __syncthreads();
  {  // exclusive sums over the experts of slots and groups, kMvMaxE / kMvThreads = 2 experts a thread
    int n[2], gr[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = 2 * tid + i;
      n[i] = e < p.E ? first[e] : 0;
      gr[i] = (n[i] + p.group - 1) / p.group;
    }
    int sn = n[0] + n[1], sg = gr[0] + gr[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, sn, o), b = __shfl_up_sync(0xffffffffu, sg, o);
      if (lane >= o) { sn += a; sg += b; }
    }
    if (lane == 31) { wsum[0][warp] = sn; wsum[1][warp] = sg; }
    __syncthreads();
    int bn = 0, bg = 0;
    for (int w = 0; w < warp; ++w) { bn += wsum[0][w]; bg += wsum[1][w]; }
    bn += sn - n[0] - n[1];
    bg += sg - gr[0] - gr[1];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = 2 * tid + i;
      if (e < p.E) { first[e] = bn; gfirst[e] = bg; }
      bn += n[i];
      bg += gr[i];
    }
    if (tid == kMvThreads - 1) { first[p.E] = bn; gfirst[p.E] = bg; }   // the totals, E = 1024 included
  }
  __syncthreads();
  for (int s = tid; s < p.S; s += kMvThreads)
    if (pos[s] >= 0) order[first[pos[s] & 1023] + (pos[s] >> 10)] = s;
  __syncthreads();

  const int64_t units = int64_t(gfirst[p.E]) * p.tiles;
  const int64_t u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;
  const int cells = p.K >> 7;                                  // 128-column cells of a tile
  const int mine = warp < cells ? (cells - warp + kMvWarps - 1) / kMvWarps : 0;
  const int64_t ecodes = p.tiles * cells * 1024, escales = p.tiles * cells * 64;
  auto expert_of = [&](int64_t grp) {                          // last expert whose first group is at or before grp
    int lo = 0, hi = p.E;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (gfirst[mid] <= grp) lo = mid; else hi = mid;
    }
    return lo;
  };
  // producer side of this warp's ring (lane 0): the next cell to load
  int64_t lu = u0;
  int li = 0, ls = 0, le = -1;
  int64_t lgrp = -1;
  auto load_next = [&]() {
    if (mine == 0 || lu >= u1) return;
    const int64_t grp = lu / p.tiles;
    if (grp != lgrp) { le = expert_of(grp); lgrp = grp; }
    const int64_t cell = (lu - grp * p.tiles) * cells + warp + li * kMvWarps;
    const uint32_t bar = sm100::smem_u32(&bars[warp * kMvRing + ls]);
    const uint32_t dst = sm100::smem_u32(ring + (warp * kMvRing + ls) * kMvCell);
    sm100::mbar_arrive_expect_tx(bar, kMvCell);
    sm100::bulk_load(dst, p.codes + le * ecodes + cell * 1024, 1024, bar);
    sm100::bulk_load(dst + 1024, p.scales + le * escales + cell * 64, 64, bar);
    if (++ls == kMvRing) ls = 0;
    if (++li == mine) { li = 0; ++lu; }
  };
  if (lane == 0)
    for (int i = 0; i < kMvRing; ++i) load_next();

  int slot = 0;
  uint32_t phase = 0;
  bool alive = true;
  int n = 0, o0 = 0;                                           // slots of the current group and their place in `order`
  int64_t cur = -1;
  float xscale[2] = {0.0f, 0.0f};                              // 2^exponent of columns 2q, 2q + 1
  for (int64_t u = u0; u < u1; ++u) {
    const int64_t grp = u / p.tiles, tile = u - grp * p.tiles;
    if (grp != cur) {
      // ---- this group's activations: row maxima, then f16 into shared memory
      cur = grp;
      const int e = expert_of(grp);
      o0 = first[e] + int(grp - gfirst[e]) * p.group;
      n = min(p.group, first[e + 1] - o0);
      __syncthreads();                                         // the previous group's activations are done with
      if (tid < 8) xmax[tid] = 0;
      __syncthreads();
      const int c8 = p.K >> 3;
      for (int r = 0; r < n; ++r) {
        const int64_t base = int64_t(order[o0 + r] / p.x_div) * p.K;
        uint32_t m = 0;
        for (int c = tid; c < c8; c += kMvThreads) {
          float f[8];
          mv_load8<kDt>(p.x, base + 8 * c, f);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t b = __float_as_uint(f[j]) & 0x7FFFFFFFu;
            if (b < 0x7F800000u) m = max(m, b);                // infinities and NaN stay what they are below
          }
        }
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0 && m) atomicMax(&xmax[r], m);
      }
      __syncthreads();
      // power of two that takes the largest magnitude to [2^12, 2^13): exponent field of its inverse
      auto inv_exp = [&](int r) { const int ef = int(xmax[r] >> 23); return ef == 0 ? 127 : min(254, max(1, 127 + 12 - (ef - 127))); };
      for (int r = 0; r < n; ++r) {
        const int64_t base = int64_t(order[o0 + r] / p.x_div) * p.K;
        const float inv = __uint_as_float(uint32_t(inv_exp(r)) << 23);
        for (int c = tid; c < c8; c += kMvThreads) {
          float f[8];
          mv_load8<kDt>(p.x, base + 8 * c, f);
          uint32_t h[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) h[j] = pack16x2<kFP16>(f[2 * j] * inv, f[2 * j + 1] * inv);
          *reinterpret_cast<uint4*>(xs + ((int64_t(c >> 2) * p.group + r) * 4 + (c & 3)) * 16) = make_uint4(h[0], h[1], h[2], h[3]);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 2 * q + i;
        xscale[i] = r < n ? __uint_as_float(uint32_t(254 - inv_exp(r)) << 23) : 0.0f;
        if (r < n && inv_exp(r) == 254) xscale[i] = __uint_as_float(0x00400000u);   // 2^-127
      }
      __syncthreads();
    }
    // ---- this warp's cells of the tile
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i = 0; i < mine; ++i) {
      const uint32_t bar = sm100::smem_u32(&bars[warp * kMvRing + slot]);
      if (alive && !sm100::mbar_wait(bar, phase)) alive = false;
      alive = __all_sync(0xffffffffu, alive);
      if (alive) {
        const uint8_t* cell = ring + (warp * kMvRing + slot) * kMvCell;
        const uint4 wg = *reinterpret_cast<const uint4*>(cell + lane * 16);
        const uint4 wu = *reinterpret_cast<const uint4*>(cell + 512 + lane * 16);
        const uint32_t sg = *reinterpret_cast<const uint32_t*>(cell + 1024 + g * 4);
        const uint32_t su = *reinterpret_cast<const uint32_t*>(cell + 1024 + 32 + g * 4);
        __syncwarp();
        if (lane == 0) load_next();
        const int kb = (warp + i * kMvWarps) * 4;              // first 32-block of the cell
        const uint32_t a[4] = {wg.x, wg.y, wg.z, wg.w}, b[4] = {wu.x, wu.y, wu.z, wu.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint4 xv = make_uint4(0, 0, 0, 0);
          if (g < n) xv = *reinterpret_cast<const uint4*>(xs + ((int64_t(kb + j) * p.group + g) * 4 + q) * 16);
          uint32_t ha[4], hb[4];
          e2m1x8_to_f16(a[j], ha);
          e2m1x8_to_f16(b[j], hb);
          float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          mma_f16_16816(c, ha[0], hb[0], ha[1], hb[1], xv.x, xv.y);
          mma_f16_16816(c, ha[2], hb[2], ha[3], hb[3], xv.z, xv.w);
          const float s0 = e8m0_to_f32((sg >> (8 * j)) & 0xFFu), s1 = e8m0_to_f32((su >> (8 * j)) & 0xFFu);
          acc[0] = fmaf(c[0], s0, acc[0]);
          acc[1] = fmaf(c[1], s0, acc[1]);
          acc[2] = fmaf(c[2], s1, acc[2]);
          acc[3] = fmaf(c[3], s1, acc[3]);
        }
      }
      if (++slot == kMvRing) { slot = 0; phase ^= 1; }
    }
    const int buf = int(u & 1);
    red[(buf * kMvWarps + warp) * 32 + lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    __syncthreads();
    // ---- one warp adds the partial sums in warp order and writes the tile;
    // the others go on (the other half of `red` is theirs until the next barrier)
    if (warp == int(tile % kMvWarps)) {
      float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kMvWarps; ++w) {
        const float4 v = red[(buf * kMvWarps + w) * 32 + lane];
        t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 2 * q + i;
        if (r >= n) continue;
        const int64_t s = order[o0 + r];
        const float lo = (i ? t.y : t.x) * xscale[i], hi = (i ? t.w : t.z) * xscale[i];
        if constexpr (kGated) {
          static_cast<float*>(p.out)[s * p.tiles * 8 + tile * 8 + g] = silu_mul(lo, hi);
        } else if constexpr (kOut == 2) {
          float* y = static_cast<float*>(p.out) + s * p.tiles * 16 + tile * 16 + g;
          y[0] = lo;
          y[8] = hi;
        } else {
          uint16_t* y = static_cast<uint16_t*>(p.out) + s * p.tiles * 16 + tile * 16 + g;
          const uint32_t w = pack16x2<kOut>(lo, hi);
          y[0] = uint16_t(w & 0xFFFFu);
          y[8] = uint16_t(w >> 16);
        }
      }
    }
  }
  if (!alive && lane == 0) raise_device_error(7);
}

// out[t] = sum_j w[t, j] y[t * k + j] in fp32, j order, rounded once; a slot
// whose expert id is out of range adds nothing.
template <int kDt>
__global__ void __launch_bounds__(128)
fp4_combine_kernel(const float* __restrict__ y, const int32_t* __restrict__ ids, const float* __restrict__ w, int k,
                   int E, int D, uint16_t* __restrict__ out) {
  const int64_t t = blockIdx.y;
  const int c = (blockIdx.x * 128 + threadIdx.x) * 4;
  if (c >= D) return;
  float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j = 0; j < k; ++j) {
    const int e = ids[t * k + j];
    if (e < 0 || e >= E) continue;
    const float wj = w[t * k + j];
    const float4 v = *reinterpret_cast<const float4*>(y + (t * k + j) * D + c);
    a[0] = fmaf(wj, v.x, a[0]);
    a[1] = fmaf(wj, v.y, a[1]);
    a[2] = fmaf(wj, v.z, a[2]);
    a[3] = fmaf(wj, v.w, a[3]);
  }
  *reinterpret_cast<uint2*>(out + t * D + c) = make_uint2(pack16x2<kDt>(a[0], a[1]), pack16x2<kDt>(a[2], a[3]));
}

}  // namespace mxmoe
