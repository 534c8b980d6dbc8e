// What the ragged, checkpoint and 4-bit operators share: the two 16-bit float
// types as packed pairs (low half first), and dependent launches.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "mx_common.cuh"

namespace mxmoe::sm100 {

// Programmatic dependent launch: the next launch of the stream may start its
// blocks as this grid's leave; it waits for all of this grid's results itself.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_dependency() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace mxmoe::sm100

namespace mxmoe {

constexpr int kBF16 = 0, kFP16 = 1;   // MXMOE_BF16, MXMOE_FP16

template <int kDt>
__device__ __forceinline__ float2 unpack16x2(uint32_t w) {
  if constexpr (kDt == kBF16) {
    return make_float2(bf16lo_to_f32(w), bf16hi_to_f32(w));
  } else {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
}

// Round to nearest even (fp16: beyond 65504 to infinity).
template <int kDt>
__device__ __forceinline__ uint32_t pack16x2(float a, float b) {
  if constexpr (kDt == kBF16) {
    return pack_bf16x2(a, b);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// Largest magnitude pattern of eight packed values, as fp32 bits (for
// non-negative floats the integer order is the numeric one; NaN and infinity
// sort above every finite value).
template <int kDt>
__device__ __forceinline__ uint32_t absmax_f32bits8(uint4 v) {
  if constexpr (kDt == kBF16) {
    return absmax_bits8(v) << 16;
  } else {
    // fp16 patterns order the same way; one conversion of the largest
    const uint32_t m = 0x7FFF7FFFu;
    uint32_t a = __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
    a = max(a & 0xFFFFu, a >> 16);
    return __float_as_uint(__half2float(__ushort_as_half(uint16_t(a))));
  }
}

}  // namespace mxmoe
