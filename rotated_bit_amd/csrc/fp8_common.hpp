// Rows of e4m3 codes with one float32 scale per 128 values (the layout of
// harp.h): helpers shared by the kernels that write and read them.
#pragma once

#include "device_common.hpp"

namespace harp {

constexpr int kFp8Run = 128;          // values per scale
constexpr float kFp8Max = 448.0f;     // largest e4m3 value
constexpr float kFp8MinScale = 0x1p-126f;   // keeps 1 / s finite

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__host__ __device__ constexpr int fp8_runs(int n) { return (n + kFp8Run - 1) / kFp8Run; }

template <int CTRL>
__device__ __forceinline__ float row_rotated(float v) {
  return __int_as_float(
      __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, false));
}

// Maximum over the 16 lanes of a row of lanes (every lane gets it).  fmaxf
// passes over a NaN.
__device__ __forceinline__ float row16_max(float v) {
  v = fmaxf(v, row_rotated<0x128>(v));
  v = fmaxf(v, row_rotated<0x124>(v));
  v = fmaxf(v, row_rotated<0x122>(v));
  return fmaxf(v, row_rotated<0x121>(v));
}

// Eight values as e4m3 codes, round to nearest even.  |v inv| <= 448 up to
// rounding, far from the 464 from which e4m3 would overflow.
__device__ __forceinline__ u32x2 fp8_pack8(const float (&v)[8], float inv) {
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inv, v[1] * inv, lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inv, v[3] * inv, lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] * inv, v[5] * inv, hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6] * inv, v[7] * inv, hi, true);
  return u32x2{static_cast<uint32_t>(lo), static_cast<uint32_t>(hi)};
}

// The scale of a run with maximum magnitude amax.
__device__ __forceinline__ float fp8_scale(float amax) {
  return fmaxf(amax * (1.0f / kFp8Max), kFp8MinScale);
}

// Eight consecutive values at p (16-byte aligned) as float32.
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const floatx4 a = *reinterpret_cast<const floatx4*>(p);
  const floatx4 b = *reinterpret_cast<const floatx4*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  const u32x4 a = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(a[i] << 16);
    v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<floatx4*>(p) = floatx4{v[0], v[1], v[2], v[3]};
  *reinterpret_cast<floatx4*>(p + 4) = floatx4{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<u32x4*>(p) = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                       pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}

__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(uint16_t v) { return bf16_to_f32(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = f32_to_bf16(v); }

}  // namespace harp
