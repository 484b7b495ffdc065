// 8-bit activations on the device: e4m3 values (4 significant bits, |q| <= 448,
// steps of 2^-9 below 2^-6) in blocks of 32 along a row; a block's scale is a
// power of two, kept as its biased exponent, the least with no finite value of
// the block above 448 of it and not below 2^-117, so that what a value stands
// for is a normal number of fp32 and an exact one of bf16 (2^128 from 1.9375 2^127
// on, the nearest e4m3 has: infinity).  A power of two
// loses nothing against a finer scale: e4m3's steps are relative.
#pragma once
#include "act.h"
#include "common.h"

namespace muonh {
namespace {

typedef u32x2_t __attribute__((aligned(1))) u32x2_b;
typedef u32x4_t __attribute__((aligned(1))) u32x4_b;

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true));
}
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppHalfMirror = 0x141, kDppMirror = 0x140;

__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, dpp<kDppXor1>(v));
  return fmaxf(v, dpp<kDppXor2>(v));
}

// Largest finite magnitude of 8 values (0 if none is).
__device__ __forceinline__ float finite_max(const float (&v)[8]) {
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float a = fabsf(v[k]);
    m = fmaxf(m, a < INFINITY ? a : 0.f);
  }
  return m;
}

// Biased exponent of the scale for a largest magnitude: 448 = 1.75 * 2^8, so the
// exponent less 8, one more where the significand is above 1.75.
__device__ __forceinline__ uint32_t mx_scale(float top) {
  return (uint32_t)max((int)((__float_as_uint(top) + 0x1fffffu) >> 23) - 8, 10);
}
__device__ __forceinline__ float mx_inverse(uint32_t scale) { return __uint_as_float((254u - scale) << 23); }
// Any scale byte: 2^(scale - 127), 255 stands for NaN.
__device__ __forceinline__ float mx_factor(uint32_t scale) {
  return __uint_as_float(scale == 0 ? 0x00400000u : scale == 255 ? 0x7fc00000u : scale << 23);
}

// 8 values times inv (at most 448 each where finite) as e4m3, nearest even; what is
// not finite becomes NaN.
__device__ __forceinline__ u32x2_t to_e4m3(const float (&v)[8], float inv) {
  u32x2_t q;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * k] * inv, v[4 * k + 1] * inv, 0, false);
    q[k] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * k + 2] * inv, v[4 * k + 3] * inv, w, true);
  }
  return q;
}
__device__ __forceinline__ void from_e4m3(const u32x2_t q, float factor, float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(q[k], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(q[k], true);
    v[4 * k] = lo[0] * factor;
    v[4 * k + 1] = lo[1] * factor;
    v[4 * k + 2] = hi[0] * factor;
    v[4 * k + 3] = hi[1] * factor;
  }
}

// The same, rounded to bf16 (exact but for scales that this library does not write);
// one conversion for two values.
__device__ __forceinline__ u32x4_t e4m3_to_bf16(const u32x2_t q, uint32_t scale) {
  const float f = __uint_as_float(scale << 23);
  u32x4_t w;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    w[2 * k] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[k], f, false));
    w[2 * k + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[k], f, true));
  }
  return w;
}

// 8 bytes at any address, or the first m of them (the others 0).
__device__ __forceinline__ u32x2_t load_q8(const uint8_t* p) { return *reinterpret_cast<const MUONH_GLOBAL u32x2_b*>(gmem(p)); }
__device__ __forceinline__ u32x2_t load_q8(const uint8_t* p, int m) {
  u32x2_t q = {0u, 0u};
  for (int k = 0; k < m; ++k) {
    const uint32_t b = (uint32_t)gmem(p)[k] << (8 * (k & 3));
    q[0] |= k < 4 ? b : 0u;
    q[1] |= k < 4 ? 0u : b;
  }
  return q;
}
__device__ __forceinline__ void store_q8(uint8_t* p, u32x2_t q) { *reinterpret_cast<MUONH_GLOBAL u32x2_b*>(gmem(p)) = q; }
__device__ __forceinline__ void store_q8(uint8_t* p, u32x2_t q, int m) {
  for (int k = 0; k < m; ++k) gmem(p)[k] = (uint8_t)((k < 4 ? q[0] : q[1]) >> (8 * (k & 3)));
}

// The first m of 8 values, the others 0.
template <typename T>
__device__ __forceinline__ void load_first(const T* p, int64_t i, int m, float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = k < m ? St<T>::ld(p, i + k) : 0.f;
}
template <typename T>
__device__ __forceinline__ void store_first(T* p, int64_t i, int m, const float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k < m) St<T>::st(p, i + k, v[k]);
}

}  // namespace
}  // namespace muonh
