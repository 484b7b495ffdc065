// What the norm's kernels share: sums over a row's waves, and which waves those are.
#pragma once
#include <algorithm>
#include <type_traits>

#include "act.h"
#include "common.h"
#include "mx.h"

namespace muonh {
namespace {

// Sum over the wave's 64 lanes, in every lane; no LDS.
__device__ __forceinline__ float lanes_sum(float v) {
  v += dpp<kDppXor1>(v);
  v += dpp<kDppXor2>(v);
  v += dpp<kDppHalfMirror>(v);
  v += dpp<kDppMirror>(v);
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const long long b = __double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)b, CTRL, 0xf, 0xf, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(b >> 32), CTRL, 0xf, 0xf, true);
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
__device__ __forceinline__ double join64(uint32_t lo, uint32_t hi) {
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
__device__ __forceinline__ double lanes_sum(double v) {
  v += dpp<kDppXor1>(v);
  v += dpp<kDppXor2>(v);
  v += dpp<kDppHalfMirror>(v);
  v += dpp<kDppMirror>(v);
  uint64_t b = (uint64_t)__double_as_longlong(v);
  auto l = __builtin_amdgcn_permlane16_swap((uint32_t)b, (uint32_t)b, false, false);
  auto h = __builtin_amdgcn_permlane16_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false);
  v = join64(l[0], h[0]) + join64(l[1], h[1]);
  b = (uint64_t)__double_as_longlong(v);
  l = __builtin_amdgcn_permlane32_swap((uint32_t)b, (uint32_t)b, false, false);
  h = __builtin_amdgcn_permlane32_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false);
  return join64(l[0], h[0]) + join64(l[1], h[1]);
}

// Sum over the NW waves of a row.  red: 2 x NW values; `turn` alternates between
// the calls of a workgroup, so that one barrier a call is enough (a wave writes
// a slot again only behind the next call's barrier, which its readers have passed).
template <int NW, typename T>
__device__ __forceinline__ T row_sum(T v, T (*red)[NW], int turn) {
  v = lanes_sum(v);
  if constexpr (NW == 1) return v;
  if ((threadIdx.x & 63) == 0) red[turn][threadIdx.x >> 6] = v;
  __syncthreads();
  T s = red[turn][0];
#pragma unroll
  for (int k = 1; k < NW; ++k) s += red[turn][k];
  return s;
}

template <bool ONCE, typename T>
__device__ __forceinline__ void load_chunk(Raw8<T>& r, const T* p, int64_t i) {
  if constexpr (ONCE) r.load_once(p, i);
  else r.load_any(p, i);
}
template <bool ONCE, typename T>
__device__ __forceinline__ void store_chunk(T* p, int64_t i, const float (&v)[8]) {
  if constexpr (ONCE) store8_once(p, i, v);
  else store8_any(p, i, v);
}

constexpr int norm_threads(int nw) { return nw == 1 ? 256 : 64 * nw; }

// Waves of a row and chunks of 8 a lane, by the row's length.
struct NormShape {
  int nw, ch;
};
NormShape norm_shape(int64_t width) {
  if (width <= 512) return {1, 1};
  if (width <= 1024) return {2, 1};
  if (width <= 2048) return {4, 1};
  if (width <= 4096) return {8, 1};
  return {16, width <= 8192 ? 1 : 2};
}

// f of the row's kind (not ending with a whole chunk of 8; moved past the caches, for
// whole chunks alone) and its shape.
template <typename F>
hipError_t with_shape(int64_t width, bool once, F&& f) {
  const NormShape p = norm_shape(width);
  using std::integral_constant;
  const integral_constant<int, 1> one;
  auto shaped = [&](auto tail, auto past) {
    if (p.nw == 1) return f(tail, past, one, one);
    if (p.nw == 2) return f(tail, past, integral_constant<int, 2>{}, one);
    if (p.nw == 4) return f(tail, past, integral_constant<int, 4>{}, one);
    if (p.nw == 8) return f(tail, past, integral_constant<int, 8>{}, one);
    const integral_constant<int, 16> most;
    return p.ch == 1 ? f(tail, past, most, one) : f(tail, past, most, integral_constant<int, 2>{});
  };
  const std::true_type yes;
  const std::false_type no;
  return width % 8 ? shaped(yes, no) : once ? shaped(no, yes) : shaped(no, no);
}

}  // namespace
}  // namespace muonh
