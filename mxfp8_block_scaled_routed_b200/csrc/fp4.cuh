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
#include <type_traits>
#include "half16.cuh"
#include "quant.cuh"
#include "sm100.cuh"

namespace mxmoe {

using sm100::launch_dependents;
using sm100::wait_dependency;

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

// Four E8M0 bytes -> fp32, exact (0 is 2^-127, 0xFF NaN): two conversions to
// bf16 pairs, whose bits are the upper half of the fp32 ones.
__device__ __forceinline__ void e8m0x4_to_f32(uint32_t w, float (&f)[4]) {
  uint32_t lo, hi;
  asm("{ .reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.bf16x2.ue8m0x2 %0, a; cvt.rn.bf16x2.ue8m0x2 %1, b; }"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
  f[0] = bf16lo_to_f32(lo);
  f[1] = bf16hi_to_f32(lo);
  f[2] = bf16lo_to_f32(hi);
  f[3] = bf16hi_to_f32(hi);
}

// Byte offset of the codes (and of the scale) of row r, columns 8 c8.. in the
// tile layout of one expert's matrix of R rows and K columns.
__device__ __forceinline__ void fp4_place(int layout, int64_t r, uint32_t c8, int64_t R, int64_t K, int64_t& code,
                                          int64_t& scale) {
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

// Eight columns a unit, a 32-block on four neighbouring lanes, kFp4Units units
// a thread (a block's width apart) with their loads issued first.  Bound by
// HBM: 2 + 17/32 bytes a value either way.
constexpr int kFp4Units = 4;

template <int kDt>
__global__ void __launch_bounds__(256)
fp4_quantize_kernel(const uint16_t* __restrict__ x, int64_t batch, int64_t R, int64_t K, int layout,
                    uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const uint32_t upr = uint32_t(K >> 3);                      // units per row, a multiple of 4
  const int64_t first = int64_t(blockIdx.x) * (256 * kFp4Units), total = batch * R * upr;
  uint4 v[kFp4Units];
#pragma unroll
  for (int i = 0; i < kFp4Units; ++i) {
    const int64_t u = first + i * 256 + threadIdx.x;
    v[i] = make_uint4(0, 0, 0, 0);
    if (u < total) v[i] = __ldcs(reinterpret_cast<const uint4*>(x) + u);
  }
  const int64_t r0 = first / upr;                             // row of the [batch * R, K] matrix
  const uint32_t c0 = uint32_t(first - r0 * upr);
#pragma unroll
  for (int i = 0; i < kFp4Units; ++i) {
    uint32_t m = absmax_f32bits8<kDt>(v[i]);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const int64_t u = first + i * 256 + threadIdx.x;
    if (u >= total) continue;                                 // whole 32-blocks: uniform in each group of four lanes
    uint32_t byte = 0xFFu, w = 0;
    const uint32_t in[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    if (m < 0x7F800000u) {
      const int e = int(m >> 23) - 2;
      byte = uint32_t(e < 0 ? 0 : e);
      const float inv = inv_scale_from_byte(byte);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = unpack16x2<kDt>(in[j]);
        w |= e2m1x2(f.x * inv, f.y * inv) << (8 * j);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)                             // magnitude 6 and the sign; the byte makes it NaN
        w |= (0x77u | ((in[j] >> 12) & 8u) | ((in[j] >> 24) & 0x80u)) << (8 * j);
    }
    if (layout == kFp4Plain) {
      reinterpret_cast<uint32_t*>(codes)[u] = w;
      if ((u & 3) == 0) scales[u >> 2] = uint8_t(byte);
    } else {
      const uint32_t at = c0 + i * 256 + threadIdx.x, dr = at / upr, c8 = at - dr * upr;
      const int64_t row = r0 + dr, e = row / R;
      int64_t oc, os;
      fp4_place(layout, row - e * R, c8, R, K, oc, os);
      *reinterpret_cast<uint32_t*>(codes + e * R * (K >> 1) + oc) = w;
      if ((c8 & 3) == 0) scales[e * R * (K >> 5) + os] = uint8_t(byte);
    }
  }
}

// PLAIN -> 16-bit values: code * 2^(byte - 127) is exact in fp32 and rounded
// once (bf16: never, but below 2^-133).
template <int kDt>
__global__ void __launch_bounds__(256)
fp4_dequantize_kernel(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t units,
                      uint4* __restrict__ out) {
  const int64_t first = int64_t(blockIdx.x) * (256 * kFp4Units) + threadIdx.x;
  uint32_t w[kFp4Units], b[kFp4Units];
#pragma unroll
  for (int i = 0; i < kFp4Units; ++i) {
    const int64_t u = first + i * 256;
    w[i] = b[i] = 0;
    if (u < units) {
      w[i] = __ldcs(codes + u);
      b[i] = scales[u >> 2];
    }
  }
#pragma unroll
  for (int i = 0; i < kFp4Units; ++i) {
    const int64_t u = first + i * 256;
    if (u >= units) continue;
    const float s = e8m0_to_f32(b[i]);
    uint32_t h[4], o[4];
    e2m1x8_to_f16(w[i], h);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
      o[j] = pack16x2<kDt>(f.x * s, f.y * s);
    }
    __stcs(out + u, make_uint4(o[0], o[1], o[2], o[3]));
  }
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
// 2^-37 of it beyond).  The fp32 h between the two products of a layer becomes
// two f16 pieces (22 bits).  Up to four slots have eight columns to themselves:
// the second pieces are columns 4..7 of the same MMAs, and the two sums meet at
// the tile's end; more slots take twice the MMAs.  Against one piece (11 bits):
// one token of 64 x 2048 x 1408 18.0 us for 17.3, eight of 64 x 7168 x 2048 199.9
// for 195.1, 32 of those (half of the experts with five slots or more) 322 for 292.
//
// Bound by HBM: (1/2 + 1/32) N K bytes per expert that has a slot.  A block of
// 16 warps per SM walks a contiguous range of (slot group, row tile) units;
// each warp takes its share of a tile's 128-column cells through its own ring
// of cp.async loads (every lane reads back the codes it loaded itself), so the
// loads of later tiles are in flight while this one is multiplied, and the
// warps' partial sums meet in shared memory in a fixed order.
// Measured on 46 of 64 experts of 7168 x 2048 (1.08 GB of weights, both
// products and the combine): 200 us, 5.4 TB/s of weights; the loop without its
// products 175 us.  What is left is issue (115 instructions a cell, of which 32
// conversions, 8 MMAs, 16 FMAs).  12 warps with a ring of three 205 us; bulk
// copies instead of cp.async 8 % more (about 75 cycles of the issuing warp a
// copy; all of them from one feeding warp 60 % more); one cell a load 6 % more.
constexpr int kMvWarps = 16, kMvThreads = 32 * kMvWarps;
constexpr int kMvCells = 2;                 // neighbouring cells (16 x 128) that a warp loads together
constexpr int kMvRing = 2;                  // such loads in flight per warp
constexpr int kMvSlot = kMvCells * (1024 + 64);
constexpr int kMvMaxSlots = 2048, kMvMaxE = 1024;

struct MvArgs {
  const void* x;            // [*, K]
  const int32_t* ids;       // [S] expert of each slot
  int S;
  int x_div;                // slot s reads row s / x_div of x
  int E;
  int tiles;                // row tiles per expert (S * tiles < 2^31)
  int K;
  int team_log2;            // warps that share a tile's cells: 1, 2 or 4 as a power of two (no divisions in a
                            // block's first instructions, which come from L2)
  int group;                // slots per group, 1..8 (shared memory holds group * K f16, of fp32 rows `pieces` times)
  int pieces;               // fp32 rows: f16 pieces of a value; else 1
  const uint8_t* codes;
  const uint8_t* scales;
  void* out;                // gated: fp32 h [S, 8 * tiles]; else y [S, 16 * tiles]
};

// Types of the activations and of the result: kBF16, kFP16, and fp32.
constexpr int kF32 = 2;

__host__ __device__ constexpr int mv_smem(int64_t K, int group, int E, int S, int pieces) {
  // ring, partial sums (two tiles), f16 activations, then counts, slot order, groups
  return int(kMvWarps * kMvRing * kMvSlot + 2 * kMvWarps * 512 + int64_t(group) * K * 2 * pieces + 64 + (E + 1) * 4 + (4 * S + 1) * 4 + 256);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

template <int kDt>
__device__ __forceinline__ void mv_load8(const void* x, int64_t i, float (&f)[8]) {
  if constexpr (kDt == kF32) {
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

__device__ __forceinline__ void mma_f16_16816_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                   uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

template <int kDt, bool kGated, int kOut>   // kOut: type of a non-gated result (kBF16, kFP16, kF32)
__global__ void __launch_bounds__(kMvThreads, 1) fp4_matvec_kernel(const MvArgs p) {
  extern __shared__ __align__(128) uint8_t mv_smem_raw[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  uint8_t* ring = mv_smem_raw;                                                    // [warp][slot]: codes, then scales
  float4* red = reinterpret_cast<float4*>(ring + kMvWarps * kMvRing * kMvSlot);   // [2][warp][lane]
  uint8_t* xs = reinterpret_cast<uint8_t*>(red + 2 * kMvWarps * 32);              // f16 [K/32][group][4 quarters][8]
  const int plane = p.group * p.K * 2;                                            // bytes of one f16 piece of the group
  const bool two = kDt == kF32 && p.pieces == 2;
  uint32_t* xmax = reinterpret_cast<uint32_t*>(xs + (two ? 2 * plane : plane));   // [8] largest magnitude, fp32 bits
  int* order = reinterpret_cast<int*>(xmax + 16);                                 // [S] slots, group after group
  int* gexp = order + p.S;                                                        // [S] expert of each group
  int* gstart = gexp + p.S;                                                       // [S + 1] its first place in `order`
  int* pos = gstart + (p.S + 1);                                                  // [S] expert and rank among its slots
  int* first = pos + p.S;                                                         // [E + 1] first slot of each expert
  __shared__ int wsum[2][kMvWarps];
  __shared__ uint4 zero;
  if (tid == 0) zero = make_uint4(0, 0, 0, 0);
  launch_dependents();

  // ---- slots grouped by expert, in slot order: every block has to come to the
  // same groups, since the tiles of one group are spread over blocks
  __shared__ int ngroups;
  if (p.S <= 32) {
    // one warp, no counters: a group starts at every slot whose rank among its
    // expert's slots is a multiple of the group size
    if (warp == 0) {
      int e = lane < p.S ? p.ids[lane] : -1;
      if (lane < p.S && (e < 0 || e >= p.E)) {
        e = -1;
        if (blockIdx.x == 0) raise_device_error(9);
      }
      const unsigned peers = __match_any_sync(0xffffffffu, e), lt = (1u << lane) - 1u;
      const int rank = __popc(peers & lt), part = rank / p.group, in = rank - part * p.group;
      const unsigned heads = __ballot_sync(0xffffffffu, e >= 0 && in == 0);
      const int g0 = __popc(heads & lt);                       // of a head: its group
      const int size = min(p.group, __popc(peers) - rank);     // of a head: its slots
      int at = e >= 0 && in == 0 ? size : 0;                   // exclusive sum over the heads
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += v;
      }
      at -= e >= 0 && in == 0 ? size : 0;
      // a member's head: the slot of its expert with rank part * group
      unsigned rest = peers;
      for (int i = 0; i < part * p.group; ++i) rest &= rest - 1;
      const int base = __shfl_sync(0xffffffffu, at, __ffs(rest) - 1);
      if (e >= 0) {
        order[base + in] = lane;
        if (in == 0) { gexp[g0] = e; gstart[g0] = at; }
      }
      const int live = __popc(__ballot_sync(0xffffffffu, e >= 0));
      if (lane == 0) { ngroups = __popc(heads); gstart[__popc(heads)] = live; }
    }
    __syncthreads();
  } else {
    for (int e = tid; e <= p.E; e += kMvThreads) first[e] = 0;
    for (int s = tid; s < p.S; s += kMvThreads) {
      const int e = p.ids[s];
      const bool ok = e >= 0 && e < p.E;
      pos[s] = ok ? e : -1;
      if (!ok && blockIdx.x == 0) raise_device_error(9);
    }
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
    {  // exclusive sums over the experts of slots and groups, a few experts a thread
      constexpr int kPer = (kMvMaxE + kMvThreads - 1) / kMvThreads;
      int n[kPer], sn = 0, sg = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int e = kPer * tid + i;
        n[i] = e < p.E ? first[e] : 0;
        sn += n[i];
        sg += (n[i] + p.group - 1) / p.group;
      }
      const int own_n = sn, own_g = sg;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, sn, o), b = __shfl_up_sync(0xffffffffu, sg, o);
        if (lane >= o) { sn += a; sg += b; }
      }
      if (lane == 31) { wsum[0][warp] = sn; wsum[1][warp] = sg; }
      __syncthreads();
      int bn = 0, bg = 0;
      for (int w = 0; w < warp; ++w) { bn += wsum[0][w]; bg += wsum[1][w]; }
      bn += sn - own_n;
      bg += sg - own_g;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int e = kPer * tid + i;
        if (e < p.E) first[e] = bn;
        for (int o = 0; o < n[i]; o += p.group) { gexp[bg] = e; gstart[bg++] = bn + o; }
        bn += n[i];
      }
      if (tid == kMvThreads - 1) { ngroups = bg; gstart[bg] = bn; }
    }
    __syncthreads();
    for (int s = tid; s < p.S; s += kMvThreads)
      if (pos[s] >= 0) order[first[pos[s] & 1023] + (pos[s] >> 10)] = s;
    __syncthreads();
  }

  // ---- units (group, tile), a contiguous range of them per block, cut into
  // one segment per group; a segment's units go round the teams of warps, a
  // unit's cells are shared out to the warps of a team
  const int units = ngroups * p.tiles, share = units / int(gridDim.x), over = units - share * int(gridDim.x);
  const int u0 = share * int(blockIdx.x) + min(int(blockIdx.x), over), total = share + (int(blockIdx.x) < over);
  const int cells = p.K >> 7;                                  // 128-column cells of a tile
  const int W = 1 << p.team_log2, teams = kMvWarps >> p.team_log2, team = warp >> p.team_log2, member = warp & (W - 1);
  // this warp's cells of a tile, [cell0, cell0 + mine)
  const int cell0 = (member * cells) >> p.team_log2, mine = (((member + 1) * cells) >> p.team_log2) - cell0;
  const uint32_t ring_at = sm100::smem_u32(ring) + warp * kMvRing * kMvSlot;
  const int grp0 = u0 / p.tiles, first_tile = u0 - grp0 * p.tiles;
  // (segment i of this block: group grp0 + i, tiles [tile0, tile1))

  // ---- the warp's next cell to load: `left` units from the start of its
  // segment on, (ld_grp, ld_tile, ld_i) its place
  int left = mine > 0 ? total : 0, ld_tile0 = first_tile, ld_tile = 0, ld_tile1 = 0, ld_grp = grp0, ld_i = 0, ld_slot = 0;
  const uint8_t *ld_codes = nullptr, *ld_scales = nullptr;
  const int jump = teams * cells - mine;          // from behind a unit's last cell to the next unit's first
  auto to_segment = [&]() {                                    // to the team's first unit at or after the segment's start
    ld_tile = ld_tile0 + team;
    ld_tile1 = min(p.tiles, ld_tile0 + left);
    while (ld_tile >= ld_tile1 && left > 0) {
      left -= ld_tile1 - ld_tile0;
      ld_tile0 = 0;
      ++ld_grp;
      ld_tile = team;
      ld_tile1 = min(p.tiles, left);
    }
    if (left > 0) {
      const int64_t cell = (int64_t(gexp[ld_grp]) * p.tiles + ld_tile) * cells + cell0;
      ld_codes = p.codes + cell * 1024 + lane * 16;
      ld_scales = p.scales + cell * 64 + (lane & 7) * 16;
    }
  };
  auto load_next = [&]() {
    if (left > 0) {
      const uint32_t dst = ring_at + ld_slot * kMvSlot + lane * 16;
      const int nc = min(kMvCells, mine - ld_i);
      cp_async16(dst, ld_codes);
      cp_async16(dst + 512, ld_codes + 512);
      if (nc > 1) {
        cp_async16(dst + 1024, ld_codes + 1024);
        cp_async16(dst + 1536, ld_codes + 1536);
      }
      if (lane < 4 * nc) cp_async16(dst + kMvCells * 1024, ld_scales);
      ld_i += nc;
      int step = nc;
      if (ld_i == mine) {
        ld_i = 0;
        step += jump;
        ld_tile += teams;
      }
      ld_codes += int64_t(step) * 1024;
      ld_scales += int64_t(step) * 64;
      if (ld_tile >= ld_tile1) {                               // on to the next group's segment
        left -= ld_tile1 - ld_tile0;
        ld_tile0 = 0;
        ++ld_grp;
        to_segment();
      }
    }
    cp_async_commit();                                         // (empty at the end: the waits count groups)
    if (++ld_slot == kMvRing) ld_slot = 0;
  };
  if (left > 0) to_segment();
#pragma unroll 1   // (one copy: a block's first instructions come from L2)
  for (int i = 0; i < kMvRing; ++i) load_next();
  // up to here only the ids and the weights were read; x may be the result of
  // the launch before this one
  wait_dependency();

  int done = 0;                                                // units of the segments before the current one
  int slot = 0;
  float4* tred = red + team * 2 * W * 32;                      // this team's partial sums, two units deep
  for (int grp = grp0; done < total; ++grp) {
    const int tile0 = grp == grp0 ? first_tile : 0, tile1 = min(p.tiles, tile0 + (total - done));
    done += tile1 - tile0;
    // ---- this group's activations: row maxima, then f16 into shared memory
    const int o0 = gstart[grp], n = gstart[grp + 1] - o0;      // the group's slots in `order`
    __syncthreads();                                           // the previous group's activations are done with
    if (tid < 8) xmax[tid] = 0;
    __syncthreads();
    const int c8 = p.K >> 3;                                   // eight-column pieces of a row: a multiple of 16
    auto piece_max = [&](const float (&f)[8]) {                // largest finite magnitude; infinities and NaN stay what they are below
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t b = __float_as_uint(f[j]) & 0x7FFFFFFFu;
        if (b < 0x7F800000u) m = max(m, b);
      }
      return m;
    };
    // power of two that takes the largest magnitude to [2^12, 2^13), 2^127 at most
    // (rows below 2^-114: what f16 holds then goes down to 2^-151, beyond the inputs'
    // own last bits): its exponent field, 12 .. 254
    auto inv_exp = [&](int r) { return min(254, 127 + 12 + 127 - int(xmax[r] >> 23)); };
    auto put = [&](int r, int c, const float (&f)[8]) {
      const float inv = __uint_as_float(uint32_t(inv_exp(r)) << 23);
      uint8_t* at = xs + ((int64_t(c >> 2) * p.group + r) * 4 + (c & 3)) * 16;
      uint32_t h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = pack16x2<kFP16>(f[2 * j] * inv, f[2 * j + 1] * inv);
      *reinterpret_cast<uint4*>(at) = make_uint4(h[0], h[1], h[2], h[3]);
      if (two) {
        // what the first piece left (of an infinity: nothing)
        uint32_t l[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 v = unpack16x2<kFP16>(h[j]);
          const float a = f[2 * j] * inv, b = f[2 * j + 1] * inv;
          l[j] = pack16x2<kFP16>(isinf(a) ? 0.0f : a - v.x, isinf(b) ? 0.0f : b - v.y);
        }
        *reinterpret_cast<uint4*>(at + plane) = make_uint4(l[0], l[1], l[2], l[3]);
      }
    };
    if (n * c8 <= 2 * kMvThreads) {
      // a piece or two a thread: held in registers between the two steps
      float f[2][8];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int at = tid + i * kMvThreads, r = at / c8, c = at - r * c8;
        if (at < n * c8) mv_load8<kDt>(p.x, int64_t(order[o0 + r] / p.x_div) * p.K + 8 * c, f[i]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int at = tid + i * kMvThreads;
        uint32_t m = at < n * c8 ? piece_max(f[i]) : 0;        // (sixteen lanes share a row)
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        if ((lane & 15) == 0 && m) atomicMax(&xmax[at / c8], m);
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int at = tid + i * kMvThreads, r = at / c8;
        if (at < n * c8) put(r, at - r * c8, f[i]);
      }
    } else {
      for (int r = 0; r < n; ++r) {
        const int64_t base = int64_t(order[o0 + r] / p.x_div) * p.K;
        uint32_t m = 0;
        for (int c = tid; c < c8; c += kMvThreads) {
          float f[8];
          mv_load8<kDt>(p.x, base + 8 * c, f);
          m = max(m, piece_max(f));
        }
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0 && m) atomicMax(&xmax[r], m);
      }
      __syncthreads();
      for (int r = 0; r < n; ++r) {
        const int64_t base = int64_t(order[o0 + r] / p.x_div) * p.K;
        for (int c = tid; c < c8; c += kMvThreads) {
          float f[8];
          mv_load8<kDt>(p.x, base + 8 * c, f);
          put(r, c, f);
        }
      }
    }
    // its inverse as two factors, of exponents -124 .. 100 and -3 .. 15
    auto down1 = [&](int r) { return max(-124, min(100, 127 - inv_exp(r))); };
    auto pow2 = [](int e) { return __uint_as_float(uint32_t(127 + e) << 23); };
    // second pieces: in columns 4..7 (packed), or by MMAs of their own
    const bool packed = two && n <= 4, more = two && n > 4;
    const int cols = packed ? 3 : 7;                                           // column & cols: slot of a column
    const float xs1[2] = {pow2(down1(2 * q & cols)), pow2(down1((2 * q + 1) & cols))};   // (of no slot: its sums are zero)
    __syncthreads();
    // this lane's column of a 32-block; columns past the group's slots read one zero piece
    const bool live = (g & cols) < n;
    const uint32_t xlane = live ? sm100::smem_u32(xs) + ((g & cols) * 4 + q) * 16 + (g > cols ? plane : 0) : sm100::smem_u32(&zero);
    const int xstep = live ? p.group * 64 : 0, xplane = live ? plane : 0;
    int buf = 0;
    for (int tile = tile0 + team; tile < tile1; tile += teams) {
      // ---- this warp's cells of the tile
      float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      auto multiply = [&](uint4 wa, uint4 wb, uint32_t sa, uint32_t sb, uint32_t xat, auto down, auto pieces) {   // a cell's products
        float fa[4], fb[4];
        e8m0x4_to_f32(sa, fa);
        e8m0x4_to_f32(sb, fb);
        const uint32_t a[4] = {wa.x, wa.y, wa.z, wa.w}, b[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 xv = lds128(xat + j * xstep);
          uint32_t ha[4], hb[4];
          e2m1x8_to_f16(a[j], ha);
          e2m1x8_to_f16(b[j], hb);
          float d[4];
          mma_f16_16816_zero(d, ha[0], hb[0], ha[1], hb[1], xv.x, xv.y);
          mma_f16_16816(d, ha[2], hb[2], ha[3], hb[3], xv.z, xv.w);
          if constexpr (decltype(pieces)::value) {
            const uint4 xl = lds128(xat + j * xstep + xplane);
            mma_f16_16816(d, ha[0], hb[0], ha[1], hb[1], xl.x, xl.y);
            mma_f16_16816(d, ha[2], hb[2], ha[3], hb[3], xl.z, xl.w);
          }
          if constexpr (decltype(down)::value) {
#pragma unroll
            for (int k = 0; k < 4; ++k) d[k] *= xs1[k & 1];
          }
          acc[0] = fmaf(d[0], fa[j], acc[0]);
          acc[1] = fmaf(d[1], fa[j], acc[1]);
          acc[2] = fmaf(d[2], fb[j], acc[2]);
          acc[3] = fmaf(d[3], fb[j], acc[3]);
        }
      };
      for (int i = 0; i < mine; i += kMvCells) {
        // the oldest load has come: into registers, and its slot takes the
        // next one before the products (a missing second cell: stale bytes,
        // not used)
        cp_async_wait<kMvRing - 1>();
        __syncwarp();
        const uint32_t at = ring_at + slot * kMvSlot;
        uint4 wa[kMvCells], wb[kMvCells];
        uint32_t sa[kMvCells], sb[kMvCells];
#pragma unroll
        for (int c = 0; c < kMvCells; ++c) {
          wa[c] = lds128(at + c * 1024 + lane * 16);
          wb[c] = lds128(at + c * 1024 + 512 + lane * 16);
          sa[c] = lds32(at + kMvCells * 1024 + c * 64 + g * 4);
          sb[c] = lds32(at + kMvCells * 1024 + c * 64 + 32 + g * 4);
        }
        __syncwarp();
        load_next();
        if (++slot == kMvRing) slot = 0;
        const uint32_t xb = xlane + (cell0 + i) * 4 * xstep;
        auto both = [&](auto pieces) {
#pragma unroll
          for (int c = 0; c < kMvCells; ++c) {
            if (c > 0 && i + c >= mine) break;
            multiply(wa[c], wb[c], sa[c], sb[c], xb + 4 * c * xstep, std::false_type{}, pieces);
          }
        };
        if constexpr (kDt == kF32) {
          if (more) both(std::true_type{}); else both(std::false_type{});
        } else {
          both(std::false_type{});
        }
      }
      // ---- the sums lose the row's power of two.  Lifted by it they may have
      // overflowed where the result does not (scales far above 1): then the tile is
      // taken again, each block's sum brought down before its scale meets it.  (A
      // block's sum is a multiple of 2^-25 below 2^21, which the first factor neither
      // rounds nor overflows.  On eight tokens 199.6 us, without the second look 197;
      // every block that way 213; chosen by the scales on the way 205.)
      const bool finite = isfinite(acc[0]) && isfinite(acc[1]) && isfinite(acc[2]) && isfinite(acc[3]);
      if (__all_sync(0xffffffffu, finite)) {
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] *= xs1[k & 1];
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] = 0.0f;
        const int64_t cell = (int64_t(gexp[grp]) * p.tiles + tile) * cells + cell0;
#pragma unroll 1
        for (int i = 0; i < mine; ++i) {
          const uint4* wp = reinterpret_cast<const uint4*>(p.codes + (cell + i) * 1024) + lane;
          const uint32_t* sp = reinterpret_cast<const uint32_t*>(p.scales + (cell + i) * 64) + g;
          const uint4 wa = __ldg(wp), wb = __ldg(wp + 32);
          const uint32_t sa = __ldg(sp), sb = __ldg(sp + 8), xb = xlane + (cell0 + i) * 4 * xstep;
          if (more) multiply(wa, wb, sa, sb, xb, std::true_type{}, std::true_type{});
          else multiply(wa, wb, sa, sb, xb, std::true_type{}, std::false_type{});
        }
      }
      // ---- one warp of the team adds the partial sums in warp order and
      // writes the tile; the others go on (the other half of the team's buffer
      // is theirs until the next barrier)
      float4 t = make_float4(acc[0], acc[1], acc[2], acc[3]);
      if (W > 1) {
        tred[(buf * W + member) * 32 + lane] = t;
        sm100::named_bar_sync(1 + team, W * 32);
        if (member != (tile & (W - 1))) { buf ^= 1; continue; }
        t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int w = 0; w < W; ++w) {
          const float4 v = tred[(buf * W + w) * 32 + lane];
          t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
        }
        buf ^= 1;
      }
      if (packed) {                                            // columns c and c + 4: lanes q and q + 2
        t.x += __shfl_xor_sync(0xffffffffu, t.x, 2);
        t.y += __shfl_xor_sync(0xffffffffu, t.y, 2);
        t.z += __shfl_xor_sync(0xffffffffu, t.z, 2);
        t.w += __shfl_xor_sync(0xffffffffu, t.w, 2);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 2 * q + i;
        if (r >= n) continue;
        const int64_t s = order[o0 + r];
        const float xs2 = pow2(127 - inv_exp(r) - down1(r)), lo = (i ? t.y : t.x) * xs2, hi = (i ? t.w : t.z) * xs2;
        if constexpr (kGated) {
          static_cast<float*>(p.out)[s * p.tiles * 8 + tile * 8 + g] = silu_mul(lo, hi);
        } else if constexpr (kOut == kF32) {
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
}

// out[t] = sum_j w[t, j] y[t * k + j] in fp32, j order, rounded once; a slot
// whose expert id is out of range adds nothing.
template <int kDt>
__global__ void __launch_bounds__(128)
fp4_combine_kernel(const float* y, const int32_t* __restrict__ ids, const float* __restrict__ w, int k,
                   int E, int D, uint16_t* __restrict__ out) {
  const int64_t t = blockIdx.y;
  const int c = (blockIdx.x * 128 + threadIdx.x) * 4;
  wait_dependency();
  if (c >= D) return;
  float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int j = 0; j < k; ++j) {
    const int e = ids[t * k + j];
    const float wj = w[t * k + j];
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const bool ok = e >= 0 && e < E;
    if (ok) v = *reinterpret_cast<const float4*>(y + (t * k + j) * D + c);
    if (!ok) continue;
    a[0] = fmaf(wj, v.x, a[0]);
    a[1] = fmaf(wj, v.y, a[1]);
    a[2] = fmaf(wj, v.z, a[2]);
    a[3] = fmaf(wj, v.w, a[3]);
  }
  *reinterpret_cast<uint2*>(out + t * D + c) = make_uint2(pack16x2<kDt>(a[0], a[1]), pack16x2<kDt>(a[2], a[3]));
}

}  // namespace mxmoe
