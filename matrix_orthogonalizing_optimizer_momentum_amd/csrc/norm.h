// What the norm's kernels share: sums over a row's threads, and which threads those are.
#pragma once
#include <algorithm>
#include <type_traits>

#include "act.h"
#include "common.h"
#include "mx.h"

namespace muonh {
namespace {

// Sum over each L consecutive lanes (8 to 64, a power of two), in every one of them; no LDS.
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  v += dpp<kDppXor1>(v);
  v += dpp<kDppXor2>(v);
  v += dpp<kDppHalfMirror>(v);
  if constexpr (L >= 16) v += dpp<kDppMirror>(v);
  if constexpr (L >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (L == 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}
__device__ __forceinline__ double join64(uint32_t lo, uint32_t hi) {
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const long long b = __double_as_longlong(v);
  return join64((uint32_t)__builtin_amdgcn_mov_dpp((int)b, CTRL, 0xf, 0xf, true),
                (uint32_t)__builtin_amdgcn_mov_dpp((int)(b >> 32), CTRL, 0xf, 0xf, true));
}
template <int L>
__device__ __forceinline__ double lanes_sum(double v) {
  v += dpp<kDppXor1>(v);
  v += dpp<kDppXor2>(v);
  v += dpp<kDppHalfMirror>(v);
  if constexpr (L >= 16) v += dpp<kDppMirror>(v);
  if constexpr (L >= 32) {
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    const auto l = __builtin_amdgcn_permlane16_swap((uint32_t)b, (uint32_t)b, false, false);
    const auto h = __builtin_amdgcn_permlane16_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false);
    v = join64(l[0], h[0]) + join64(l[1], h[1]);
  }
  if constexpr (L == 64) {
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    const auto l = __builtin_amdgcn_permlane32_swap((uint32_t)b, (uint32_t)b, false, false);
    const auto h = __builtin_amdgcn_permlane32_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false);
    v = join64(l[0], h[0]) + join64(l[1], h[1]);
  }
  return v;
}

// Waves that a row of L threads needs an exchange between.
constexpr int row_waves(int l) { return l > 64 ? l / 64 : 1; }

// Sum over the L threads of a row.  red: 2 x row_waves(L) values; `turn` alternates between
// the calls of a workgroup, so that one barrier a call is enough (a wave writes
// a slot again only behind the next call's barrier, which its readers have passed).
template <int L, typename T>
__device__ __forceinline__ T row_sum(T v, T (*red)[row_waves(L)], int turn) {
  v = lanes_sum<L < 64 ? L : 64>(v);
  if constexpr (L <= 64) return v;
  if ((threadIdx.x & 63) == 0) red[turn][threadIdx.x >> 6] = v;
  __syncthreads();
  T s = red[turn][0];
#pragma unroll
  for (int k = 1; k < row_waves(L); ++k) s += red[turn][k];
  return s;
}

// fp32 chunks are two accesses of every other 16 bytes of a line, past the caches as well (norm of
// 16384 x 4096 bf16 into an fp32 stream, with 8 bits: 157 us, the bytes alone 128).
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

// Threads of a workgroup for rows of l threads: several rows where no barrier is
// needed between their lanes.
constexpr int norm_threads(int l) { return l <= 64 ? 256 : l; }

// Threads of a row and chunks of 8 a thread, by the row's length.
struct NormShape {
  int lanes, ch;
};
NormShape norm_shape(int64_t width) {
  int l = 8;
  while (l < 1024 && 8 * (int64_t)l < width) l *= 2;
  return {l, 8 * (int64_t)l < width ? 2 : 1};
}

// f of the row's kind (not ending with a whole chunk of 8; moved past the caches, for
// whole chunks alone) and its shape.
template <typename F>
hipError_t with_shape(int64_t width, bool once, F&& f) {
  const NormShape p = norm_shape(width);
  using std::integral_constant;
  const integral_constant<int, 1> one;
  auto shaped = [&](auto tail, auto past) {
    switch (p.lanes) {
      case 8: return f(tail, past, integral_constant<int, 8>{}, one);
      case 16: return f(tail, past, integral_constant<int, 16>{}, one);
      case 32: return f(tail, past, integral_constant<int, 32>{}, one);
      case 64: return f(tail, past, integral_constant<int, 64>{}, one);
      case 128: return f(tail, past, integral_constant<int, 128>{}, one);
      case 256: return f(tail, past, integral_constant<int, 256>{}, one);
      case 512: return f(tail, past, integral_constant<int, 512>{}, one);
    }
    const integral_constant<int, 1024> most;
    return p.ch == 1 ? f(tail, past, most, one) : f(tail, past, most, integral_constant<int, 2>{});
  };
  const std::true_type yes;
  const std::false_type no;
  return width % 8 ? shaped(yes, no) : once ? shaped(no, yes) : shaped(no, no);
}

}  // namespace
}  // namespace muonh
