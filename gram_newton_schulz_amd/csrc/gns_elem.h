// Element types and streaming accesses shared by the device sources.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gns_kernels.h"

namespace gns {

// ---------------------------------------------------------------------------
// element types
// ---------------------------------------------------------------------------
__device__ __forceinline__ float bf16_to_f32(uint16_t h) {
  return __uint_as_float(static_cast<uint32_t>(h) << 16);
}
// Round to nearest even; NaN stays NaN.  gfx950 converts in hardware
// (v_cvt_pk_bf16_f32, two values per instruction): checked against the
// integer rounding (u + 0x7fff + lsb) >> 16 on every fp32 bit pattern, in
// both halves, on the GPU.
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t f32x2_to_bf16x2(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{lo, hi}), bf16x2_t));
}
__device__ __forceinline__ uint16_t f32_to_bf16(float f) {
  return static_cast<uint16_t>(f32x2_to_bf16x2(f, 0.0f));
}
__device__ __forceinline__ float f16_to_f32(uint16_t h) {
  return static_cast<float>(__builtin_bit_cast(_Float16, h));
}
__device__ __forceinline__ uint16_t f32_to_f16(float f) {
  return __builtin_bit_cast(uint16_t, static_cast<_Float16>(f));
}
__device__ __forceinline__ uint32_t f32x2_to_f16x2(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{lo, hi}), f16x2_t));
}

struct EBF16 {
  using S = uint16_t;
  static constexpr int code = DT_BF16;
  __device__ static float ld(S v) { return bf16_to_f32(v); }
  __device__ static S st(float f) { return f32_to_bf16(f); }
  // two values rounded into one packed pair (lo in bits 0-15)
  __device__ static uint32_t st2(float lo, float hi) { return f32x2_to_bf16x2(lo, hi); }
};
struct EF16 {
  using S = uint16_t;
  static constexpr int code = DT_F16;
  __device__ static float ld(S v) { return f16_to_f32(v); }
  __device__ static S st(float f) { return f32_to_f16(f); }
  __device__ static uint32_t st2(float lo, float hi) { return f32x2_to_f16x2(lo, hi); }
};
struct EF32 {
  using S = float;
  static constexpr int code = DT_F32;
  __device__ static float ld(S v) { return v; }
  __device__ static S st(float f) { return f; }
};

// Streaming passes that read and write every element once give their loads
// and stores the non-temporal hint, which moves these mixed read/write
// streams faster (Dion3 momentum pass 4.7 -> 5.1 TB/s, update 4.7 -> 5.2,
// row sums 4.3 -> 5.4).
__device__ __forceinline__ void st_once(float4 *p, float4 x) {
  typedef float v4f __attribute__((ext_vector_type(4)));
  __builtin_nontemporal_store(v4f{x.x, x.y, x.z, x.w}, reinterpret_cast<v4f *>(p));
}
__device__ __forceinline__ float4 ld_once(const float4 *p) {
  typedef float v4f __attribute__((ext_vector_type(4)));
  const v4f v = __builtin_nontemporal_load(reinterpret_cast<const v4f *>(p));
  return make_float4(v.x, v.y, v.z, v.w);
}
__device__ __forceinline__ uint2 ld_once(const uint2 *p) {
  typedef unsigned v2u __attribute__((ext_vector_type(2)));
  const v2u v = __builtin_nontemporal_load(reinterpret_cast<const v2u *>(p));
  return make_uint2(v.x, v.y);
}

// Streaming passes keep kUnroll 16-byte pieces per lane in flight: all their
// loads are issued before the first use, which one piece at a time (a single
// load round trip per wave) left at about two thirds of HBM bandwidth.
constexpr int kUnroll = 4;

}  // namespace gns
