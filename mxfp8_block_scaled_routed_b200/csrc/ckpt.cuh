// SwiGLU with an 8-bit copy of its input for the backward pass.
//
//   forward   h = silu(a) * b of h13 = [a | b]; the input is kept as MXFP8:
//             blocks of 32 along each half, E4M3 codes and one E8M0 byte
//   backward  with a~, b~ the kept values and s = 1 / (1 + e^-a~):
//             h  = a~ s b~                       (FC2's weight-gradient operand)
//             da = dh b~ s (1 + a~ (1 - s)),  db = dh a~ s
//
// The copy takes 1 + 1/32 bytes a value where the 16-bit h13 takes two, and h
// is not kept at all.  All arithmetic is fp32 with one rounding at each
// output; the codes' rounding is the checkpoint's price and is the only one
// that the gradients see beside it.
//
// Bound by HBM: 8.06 F bytes a row forward, 10.06 F backward.  One thread per
// eight columns f of both halves: 16-byte loads and stores, a 32-block is four
// neighbouring lanes, so its maximum takes two shuffles and nothing is staged.
// A block's first unit (row, column) costs one 64-bit division, its other 255
// a 32-bit one.
#pragma once
#include "half16.cuh"
#include "quant.cuh"

namespace mxmoe {

struct CkptArgs {
  int64_t rows;
  const int32_t* rows_dev;   // optional: rows at or past *rows_dev are neither read nor written
  uint32_t F;
  uint32_t units;            // 8-column units per row, whole 32-blocks: 4 * ceil(F / 32)
  const uint16_t* in;        // h13 [rows, 2F] (forward), dh [rows, F] (backward)
  uint8_t* codes;            // [rows, 2F]
  uint8_t* scales;           // [rows, 2, ceil(F / 32)]
  uint16_t* h;               // [rows, F] (backward: may be null)
  uint16_t* dh13;            // [rows, 2F] (backward)
};

__device__ __forceinline__ uint2 e4m3_encode8(const float (&x)[8], uint32_t byte) {
  uint2 o;
  if (byte == 0xFFu) {
    uint32_t s[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i >> 2] |= (__float_as_uint(x[i]) >> 31) << (7 + 8 * (i & 3));
    o = make_uint2(s[0] | 0x7F7F7F7Fu, s[1] | 0x7F7F7F7Fu);
  } else {
    const float inv = inv_scale_from_byte(byte);
    o.x = e4m3x2(x[0] * inv, x[1] * inv) | (e4m3x2(x[2] * inv, x[3] * inv) << 16);
    o.y = e4m3x2(x[4] * inv, x[5] * inv) | (e4m3x2(x[6] * inv, x[7] * inv) << 16);
  }
  return o;
}

__device__ __forceinline__ void e4m3_decode8(uint2 c, float s, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = i < 2 ? c.x : c.y;
    const uint32_t h = fp8x2_to_f16x2<0>((w >> (16 * (i & 1))) & 0xFFFFu);   // exact; NaN codes stay NaN
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    x[2 * i] = f.x * s;
    x[2 * i + 1] = f.y * s;
  }
}

template <int kDt>
__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack16x2<kDt>(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <int kDt>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack16x2<kDt>(x[0], x[1]), pack16x2<kDt>(x[2], x[3]), pack16x2<kDt>(x[4], x[5]),
                    pack16x2<kDt>(x[6], x[7]));
}

// Row and unit of this thread's i-th unit (kCkptUnits of them, a block's width
// apart); false past the last row or the last column.
constexpr int kCkptUnits = 2;

__device__ __forceinline__ bool ckpt_place(const CkptArgs& p, int64_t r0, uint32_t u0, int64_t limit, int i, int64_t& row,
                                           uint32_t& unit) {
  const uint32_t u = u0 + i * 256 + threadIdx.x, dr = u / p.units;
  row = r0 + dr;
  unit = u - dr * p.units;
  return row < limit && unit * 8 < p.F;
}

__device__ __forceinline__ uint32_t ckpt_byte(uint32_t m) {
  if (m >= 0x7F800000u) return 0xFFu;
  const int e = int(m >> 23) - 8;
  return uint32_t(e < 0 ? 0 : e);
}

template <int kDt>
__global__ void __launch_bounds__(256) swiglu_ckpt_kernel(const CkptArgs p) {
  const int64_t first = int64_t(blockIdx.x) * (256 * kCkptUnits), r0 = first / p.units;
  const uint32_t u0 = uint32_t(first - r0 * p.units);
  const int64_t limit = p.rows_dev ? min(p.rows, int64_t(*p.rows_dev)) : p.rows;
  uint4 va[kCkptUnits], vb[kCkptUnits];
#pragma unroll
  for (int i = 0; i < kCkptUnits; ++i) {
    int64_t row;
    uint32_t unit;
    va[i] = vb[i] = make_uint4(0, 0, 0, 0);
    if (ckpt_place(p, r0, u0, limit, i, row, unit)) {
      const uint16_t* src = p.in + row * 2 * p.F + unit * 8;
      va[i] = __ldcs(reinterpret_cast<const uint4*>(src));
      vb[i] = __ldcs(reinterpret_cast<const uint4*>(src + p.F));
    }
  }
#pragma unroll
  for (int i = 0; i < kCkptUnits; ++i) {
    uint32_t ma = absmax_f32bits8<kDt>(va[i]), mb = absmax_f32bits8<kDt>(vb[i]);
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
      ma = max(ma, __shfl_xor_sync(0xffffffffu, ma, o));
      mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, o));
    }
    int64_t row;
    uint32_t unit;
    if (!ckpt_place(p, r0, u0, limit, i, row, unit)) continue;
    const uint32_t ba = ckpt_byte(ma), bb = ckpt_byte(mb), c = unit * 8;
    float a[8], b[8], h[8];
    unpack8<kDt>(va[i], a);
    unpack8<kDt>(vb[i], b);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = silu_mul(a[j], b[j]);
    uint8_t* codes = p.codes + row * 2 * p.F + c;
    *reinterpret_cast<uint2*>(codes) = e4m3_encode8(a, ba);
    *reinterpret_cast<uint2*>(codes + p.F) = e4m3_encode8(b, bb);
    *reinterpret_cast<uint4*>(p.h + row * p.F + c) = pack8<kDt>(h);
    if ((unit & 3) == 0) {
      const uint32_t nb = p.units >> 2;
      uint8_t* s = p.scales + row * 2 * nb + (unit >> 2);
      s[0] = uint8_t(ba);
      s[nb] = uint8_t(bb);
    }
  }
}

template <int kDt>
__global__ void __launch_bounds__(256) swiglu_ckpt_bwd_kernel(const CkptArgs p) {
  const int64_t first = int64_t(blockIdx.x) * (256 * kCkptUnits), r0 = first / p.units;
  const uint32_t u0 = uint32_t(first - r0 * p.units), nb = p.units >> 2;
  const int64_t limit = p.rows_dev ? min(p.rows, int64_t(*p.rows_dev)) : p.rows;
  uint4 vd[kCkptUnits];
  uint2 ca[kCkptUnits], cb[kCkptUnits];
  uint32_t sa[kCkptUnits], sb[kCkptUnits];
#pragma unroll
  for (int i = 0; i < kCkptUnits; ++i) {
    int64_t row;
    uint32_t unit;
    if (!ckpt_place(p, r0, u0, limit, i, row, unit)) continue;
    const uint8_t* codes = p.codes + row * 2 * p.F + unit * 8;
    const uint8_t* sc = p.scales + row * 2 * nb + (unit >> 2);
    vd[i] = __ldcs(reinterpret_cast<const uint4*>(p.in + row * p.F + unit * 8));
    ca[i] = __ldcs(reinterpret_cast<const uint2*>(codes));
    cb[i] = __ldcs(reinterpret_cast<const uint2*>(codes + p.F));
    sa[i] = sc[0];
    sb[i] = sc[nb];
  }
#pragma unroll
  for (int i = 0; i < kCkptUnits; ++i) {
    int64_t row;
    uint32_t unit;
    if (!ckpt_place(p, r0, u0, limit, i, row, unit)) continue;
    const uint32_t c = unit * 8;
    float a[8], b[8], d[8], da[8], db[8], h[8];
    e4m3_decode8(ca[i], e8m0_to_f32(sa[i]), a);
    e4m3_decode8(cb[i], e8m0_to_f32(sb[i]), b);
    unpack8<kDt>(vd[i], d);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // (the factors of the gate first: they lie in [-0.1, 1.1] and [-0.3, a], and
      // dh b or dh a alone could overflow and meet a zero)
      const float s = sigmoid_fast(a[j]), silu = a[j] * s;
      da[j] = d[j] * (s * (1.0f + a[j] * (1.0f - s))) * b[j];
      db[j] = d[j] * silu;
      h[j] = silu * b[j];
    }
    uint16_t* g = p.dh13 + row * 2 * p.F + c;
    *reinterpret_cast<uint4*>(g) = pack8<kDt>(da);
    *reinterpret_cast<uint4*>(g + p.F) = pack8<kDt>(db);
    if (p.h) *reinterpret_cast<uint4*>(p.h + row * p.F + c) = pack8<kDt>(h);
  }
}

}  // namespace mxmoe
