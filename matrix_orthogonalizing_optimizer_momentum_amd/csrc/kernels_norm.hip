// Root-mean-square norm with the residual's addition (gfx950).
//
//   h  = round(x + r)          (r: the residual stream; h = x without it)
//   s  = (mean_j h_j^2 + eps)^-1/2,   xn = s h,   y = xn g
//
// One pass: a row is read once, held in registers over its sum, and what comes of
// it is written.  The row in 8 bits (mx.h) leaves in the same pass, so that
// the backward pass reads 1.03 bytes a value instead of h and y.
//
// A row belongs to 8 to 1024 threads by its length (norm_shape), a thread to the same
// columns of every row of its workgroup, in chunks of 8.  Squares are summed in
// fp64: h^2 may leave fp32's range, and the sum's rounding would reach every value
// of the row.
#include "norm.h"

namespace muonh {

namespace {

// a^-1/2: the hardware's estimate and one Newton step, some 2^-50 off.
__device__ __forceinline__ double rsqrt64(double a) {
  const double r = __builtin_amdgcn_rsq(a);
  const double e = fma(-a * r, r, 1.0);
  return a < (double)INFINITY ? fma(0.5 * r, e, r) : a > 0.0 ? 0.0 : a;
}

// What becomes 8 bits is rounded to 4 significant ones.  Its fp32 value, a few roundings
// off, decides as the exact one does unless it is within them of where two e4m3
// values meet, whose last 19 bits are zeros: near_border tells (8 values: 1 wave in a
// hundred, and each that has a 0 in its row), and such values are formed anew in fp64 and moved
// off the border to the side where they lie.
__device__ __forceinline__ bool near_border(const float (&v)[8]) {
  uint32_t low = ~0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) low = min(low, (__float_as_uint(v[j]) + 4) & 0x7ffffu);
  return low < 9;
}
// Those roundings are relative ones of normal numbers alone.  Below them are rstd where the row's
// values are some 2^126 and more, and the product of rstd with a value other than 0 below 2^-126 / rstd,
// which a gain may bring back: the bits of the values up to which a row is formed anew.
__device__ __forceinline__ uint32_t anew_below(float rstd, bool gained) {
  return rstd < 0x1p-126f ? 0x7f800000u : gained ? __float_as_uint(0x1p-125f * __builtin_amdgcn_rcpf(rstd)) : 0u;
}
__device__ __forceinline__ bool any_below(const float (&v)[8], uint32_t bits) {
  uint32_t low = ~0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) low = min(low, (__float_as_uint(v[j]) & 0x7fffffffu) - 1);
  return low < bits;
}
__device__ __forceinline__ float settle(double t) {
  const float f = (float)t;
  uint32_t u = __float_as_uint(f);
  if ((u & 0x7ffffu) == 0 && fabsf(f) < INFINITY && (double)f != t) u += fabs(t) > fabs((double)f) ? 1 : -1;
  return __uint_as_float(u);
}

// TAIL: rows that do not end with a whole chunk of 8 (the others' code is free of the
// values taken one by one).  ONCE: past the caches.
template <typename XT, typename RT, bool RES, bool TAIL, bool ONCE, int L, int CH>
__global__ __launch_bounds__(norm_threads(L)) void k_rms_norm(const NormArgs a) {
  constexpr int G = norm_threads(L) / L;  // rows at a time
  __shared__ double red[2][row_waves(L)];
  const int lt = L <= 64 ? threadIdx.x & (L - 1) : threadIdx.x;
  const int64_t width = a.width, nblk = mx_blocks(width);
  const int nfull = (int)(width / 8), tail = (int)(width % 8);
  const XT* const x = static_cast<const XT*>(a.x);
  const RT* const res = static_cast<const RT*>(a.res);
  float g[CH][8];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = lt + L * k;
#pragma unroll
    for (int j = 0; j < 8; ++j) g[k][j] = 1.f;
    if (a.gain != nullptr) {
      if (c < nfull) load8_any(a.gain, 8 * c, g[k]);
      else if (TAIL && c == nfull) load_first(a.gain, 8 * (int64_t)c, tail, g[k]);
    }
  }
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * G + (G == 1 ? 0 : threadIdx.x / L); row < a.n; row += (int64_t)gridDim.x * G) {
    const int64_t at = row * width;
    Raw8<XT> rx[CH];
    Raw8<RT> rr[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = lt + L * k;
      if (c < nfull) {
        load_chunk<ONCE>(rx[k], x, at + 8 * c);
        if constexpr (RES) load_chunk<ONCE>(rr[k], res, at + 8 * c);
      }
    }
    float v[CH][8];
    double s = 0.0;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = lt + L * k;
      if (c < nfull) {
        rx[k].unpack(v[k]);
        if constexpr (RES) {
          float r[8];
          rr[k].unpack(r);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[k][j] = St<RT>::round(v[k][j] + r[j]);
          store_chunk<ONCE>(static_cast<RT*>(a.h), at + 8 * c, v[k]);
        }
      } else if constexpr (!TAIL) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] = 0.f;
      } else {
        const int m = c == nfull ? tail : 0;
        load_first(x, at + 8 * (int64_t)c, m, v[k]);
        if constexpr (RES) {
          float r[8];
          load_first(res, at + 8 * (int64_t)c, m, r);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[k][j] = St<RT>::round(v[k][j] + r[j]);
          store_first(static_cast<RT*>(a.h), at + 8 * (int64_t)c, m, v[k]);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) s = fma((double)v[k][j], (double)v[k][j], s);
    }
    s = row_sum<L>(s, red, turn);
    turn ^= 1;
    const double rstd64 = rsqrt64(s / (double)width + a.eps);
    const float rstd = (float)rstd64;
    if (lt == 0 && a.rstd != nullptr) gmem(a.rstd)[row] = rstd;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = lt + L * k;
      const int m = c < nfull ? 8 : TAIL && c == nfull ? tail : 0;
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = v[k][j] * rstd * g[k][j];
      if (a.y != nullptr) {
        if (a.y_dt == DT_BF16) {
          bf16_t* const o = static_cast<bf16_t*>(a.y);
          if (m == 8) store_chunk<ONCE>(o, at + 8 * (int64_t)c, y);
          else if (TAIL) store_first(o, at + 8 * (int64_t)c, m, y);
        } else {
          float* const o = static_cast<float*>(a.y);
          if (m == 8) store_chunk<ONCE>(o, at + 8 * (int64_t)c, y);
          else if (TAIL) store_first(o, at + 8 * (int64_t)c, m, y);
        }
      }
      if (a.q != nullptr) {
        if (!a.packs_output) {
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = v[k][j] * rstd;
        }
        // lanes behind the row's end hold zeros
        if (m > 0 && (near_border(y) || any_below(v[k], anew_below(rstd, a.packs_output != 0)))) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            // copies that the compiler does not see through: it would keep fp64 values of the
            // whole chunk in registers for this (90 and not 60: a norm of 268 MB 46 -> 56 us)
            float h = v[k][j], f = a.packs_output ? g[k][j] : 1.f;
            asm volatile("" : "+v"(h), "+v"(f));
            y[j] = settle((double)h * rstd64 * (double)f);
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = (TAIL ? j < m : m > 0) ? y[j] : 0.f;  // 0 times a NaN behind the row's end
        const uint32_t sc = mx_scale(quad_max(finite_max(y)));
        const u32x2_t q = to_e4m3(y, mx_inverse(sc));
        if (m == 8) store_q8(a.q + at + 8 * (int64_t)c, q);
        else if (TAIL) store_q8(a.q + at + 8 * (int64_t)c, q, m);
        if (c % 4 == 0 && m > 0) gmem(a.scales)[row * nblk + c / 4] = (uint8_t)sc;
      }
    }
  }
}

template <typename XT, typename RT, bool RES>
hipError_t norm(const NormArgs& a, hipStream_t s) {
  const int64_t each = sizeof(XT) + (RES ? 2 * sizeof(RT) : 0) + (a.y ? (a.y_dt == DT_BF16 ? 2 : 4) : 0) + (a.q ? 1 : 0);
  return with_shape(a.width, a.n * a.width * each > kActOnceBytes, [&](auto tail, auto once, auto lanes, auto ch) {
    constexpr int L = decltype(lanes)::value, CH = decltype(ch)::value, NT = norm_threads(L), G = NT / L;
    // a row of 1024 threads is worth its workgroup's start less often (at most 1024, 2048 and 8192
    // workgroups: 4096 x 16384 105, 108 and 114 us, 16384 x 4096 100, 99 and 97, 8000 x 1999 fp32
    // 53, 60 and 54, 8192 x 768 18, 16.0 and 15.8)
    const int64_t blocks = std::min<int64_t>((a.n + G - 1) / G, L == 1024 ? 1024 : 8192);
    k_rms_norm<XT, RT, RES, decltype(tail)::value, decltype(once)::value, L, CH><<<dim3((uint32_t)blocks), NT, 0, s>>>(a);
    return hipGetLastError();
  });
}

}  // namespace

hipError_t launch_rms_norm(int x_dt, int res_dt, const NormArgs& a, hipStream_t s) {
  if (x_dt == DT_BF16) {
    if (res_dt < 0) return norm<bf16_t, bf16_t, false>(a, s);
    return res_dt == DT_BF16 ? norm<bf16_t, bf16_t, true>(a, s) : norm<bf16_t, float, true>(a, s);
  }
  if (res_dt < 0) return norm<float, float, false>(a, s);
  return res_dt == DT_BF16 ? norm<float, bf16_t, true>(a, s) : norm<float, float, true>(a, s);
}

}  // namespace muonh
