// Root-mean-square norm with the residual's addition, and its gradient (gfx950).
//
//   h  = round(x + r)          (r: the residual stream; h = x without it)
//   s  = (mean_j h_j^2 + eps)^-1/2,   xn = s h,   y = xn g
//   c  = mean_j g_j dy_j xn_j
//   dx = dres + s (g dy - xn c),      dg = sum over the rows of dy xn
//
// Both stream: a row is read once, held in registers over its sum, and what
// comes of it is written.  The row in 8 bits (mx.h) leaves in the same pass, so
// that the backward pass reads 1.03 bytes a value instead of h and y: the
// gradient takes xn from it as it stands, no statistics but s are kept.
//
// A row belongs to 1 to 16 waves by its length (norm_shape), a lane to the
// same columns of every row of its workgroup, in chunks of 8: the gain is read
// once a lane, and the gain's gradient is summed in the lane's registers over the
// workgroup's rows, written as one row of partial sums a workgroup and added up
// by a second launch, in a fixed order.  Squares are summed in fp64: h^2 may leave
// fp32's range, and the sum's rounding would reach every value of the row.
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

// a^-1/2: the hardware's estimate and one Newton step, some 2^-50 off.
__device__ __forceinline__ float rsqrt64(double a) {
  const double r = __builtin_amdgcn_rsq(a);
  const double e = fma(-a * r, r, 1.0);
  return a < (double)INFINITY ? (float)fma(0.5 * r, e, r) : a > 0.0 ? 0.f : (float)a;
}

constexpr int norm_threads(int nw) { return nw == 1 ? 256 : 64 * nw; }

template <typename XT, typename RT, bool RES, int NW, int CH>
__global__ __launch_bounds__(norm_threads(NW)) void k_rms_norm(const NormArgs a) {
  constexpr int G = norm_threads(NW) / (64 * NW);  // rows at a time
  __shared__ double red[2][NW];
  const int lt = NW == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int64_t width = a.width, nblk = mx_blocks(width);
  const int nfull = (int)(width / 8), tail = (int)(width % 8);
  const XT* const x = static_cast<const XT*>(a.x);
  const RT* const res = static_cast<const RT*>(a.res);
  float g[CH][8];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = lt + 64 * NW * k;
#pragma unroll
    for (int j = 0; j < 8; ++j) g[k][j] = 1.f;
    if (a.gain != nullptr) {
      if (c < nfull) load8_any(a.gain, 8 * c, g[k]);
      else if (c == nfull) load_first(a.gain, 8 * (int64_t)c, tail, g[k]);
    }
  }
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * G + (G == 1 ? 0 : threadIdx.x >> 6); row < a.n; row += (int64_t)gridDim.x * G) {
    const int64_t at = row * width;
    Raw8<XT> rx[CH];
    Raw8<RT> rr[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = lt + 64 * NW * k;
      if (c < nfull) {
        rx[k].load_any(x, at + 8 * c);
        if constexpr (RES) rr[k].load_any(res, at + 8 * c);
      }
    }
    float v[CH][8];
    double s = 0.0;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = lt + 64 * NW * k;
      if (c < nfull) {
        rx[k].unpack(v[k]);
        if constexpr (RES) {
          float r[8];
          rr[k].unpack(r);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[k][j] = St<RT>::round(v[k][j] + r[j]);
          store8_any(static_cast<RT*>(a.h), at + 8 * c, v[k]);
        }
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
    s = row_sum<NW>(s, red, turn);
    turn ^= 1;
    const float rstd = rsqrt64(s / (double)width + a.eps);
    if (lt == 0 && a.rstd != nullptr) gmem(a.rstd)[row] = rstd;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = lt + 64 * NW * k;
      const int m = c < nfull ? 8 : c == nfull ? tail : 0;
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[k][j] *= rstd;
        y[j] = v[k][j] * g[k][j];
      }
      if (a.y != nullptr) {
        if (a.y_dt == DT_BF16) {
          bf16_t* const o = static_cast<bf16_t*>(a.y);
          if (m == 8) store8_any(o, at + 8 * (int64_t)c, y);
          else store_first(o, at + 8 * (int64_t)c, m, y);
        } else {
          float* const o = static_cast<float*>(a.y);
          if (m == 8) store8_any(o, at + 8 * (int64_t)c, y);
          else store_first(o, at + 8 * (int64_t)c, m, y);
        }
      }
      if (a.q != nullptr) {
        if (!a.packs_output) {
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = v[k][j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = j < m ? y[j] : 0.f;  // 0 times a NaN behind the row's end
        const uint32_t sc = mx_scale(quad_max(finite_max(y)));
        const u32x2_t q = to_e4m3(y, mx_inverse(sc));
        if (m == 8) store_q8(a.q + at + 8 * (int64_t)c, q);
        else store_q8(a.q + at + 8 * (int64_t)c, q, m);
        if (c % 4 == 0 && m > 0) gmem(a.scales)[row * nblk + c / 4] = (uint8_t)sc;
      }
    }
  }
}

// RT: type of dx, dres and x (x: the norm's input; PACKED: xn in 8 bits instead).
template <typename YT, typename RT, bool PACKED, int NW, int CH>
__global__ __launch_bounds__(norm_threads(NW)) void k_rms_norm_grad(const NormGradArgs a) {
  constexpr int NT = norm_threads(NW), G = NT / (64 * NW);
  __shared__ float red[2][NW];
  __shared__ float lsum[G == 1 ? 1 : (G - 1) * 64 * CH * 8];
  const int lt = NW == 1 ? threadIdx.x & 63 : threadIdx.x, grp = NW == 1 ? threadIdx.x >> 6 : 0;
  const int64_t width = a.width, nblk = mx_blocks(width);
  const int nfull = (int)(width / 8), tail = (int)(width % 8);
  const YT* const dy = static_cast<const YT*>(a.dy);
  const RT* const x = static_cast<const RT*>(a.x);
  const RT* const dres = static_cast<const RT*>(a.dres);
  float g[CH][8], acc[CH][8];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = lt + 64 * NW * k;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      g[k][j] = 1.f;
      acc[k][j] = 0.f;
    }
    if (a.gain != nullptr) {
      if (c < nfull) load8_any(a.gain, 8 * c, g[k]);
      else if (c == nfull) load_first(a.gain, 8 * (int64_t)c, tail, g[k]);
    }
  }
  const float inv = 1.f / (float)width;
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * G + grp; row < a.n; row += (int64_t)gridDim.x * G) {
    const int64_t at = row * width;
    const float rstd = gmem(a.rstd)[row];
    Raw8<YT> ry[CH];
    Raw8<RT> rx[CH], rd[CH];
    u32x2_t rq[CH];
    uint32_t rs[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = lt + 64 * NW * k;
      if (c < nfull) {
        ry[k].load_any(dy, at + 8 * c);
        if constexpr (PACKED) {
          rq[k] = load_q8(a.q + at + 8 * c);
          rs[k] = gmem(a.scales)[row * nblk + c / 4];
        } else {
          rx[k].load_any(x, at + 8 * c);
        }
        if (dres != nullptr) rd[k].load_any(dres, at + 8 * c);
      }
    }
    float u[CH][8], xn[CH][8];
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = lt + 64 * NW * k;
      const int m = c == nfull ? tail : 0;
      if (c < nfull) ry[k].unpack(u[k]);
      else load_first(dy, at + 8 * (int64_t)c, m, u[k]);
      if constexpr (PACKED) {
        if (c < nfull) from_e4m3(rq[k], mx_factor(rs[k]), xn[k]);
        else from_e4m3(load_q8(a.q + at + 8 * (int64_t)c, m), m ? mx_factor(gmem(a.scales)[row * nblk + c / 4]) : 0.f, xn[k]);
      } else {
        if (c < nfull) rx[k].unpack(xn[k]);
        else load_first(x, at + 8 * (int64_t)c, m, xn[k]);
#pragma unroll
        for (int j = 0; j < 8; ++j) xn[k][j] *= rstd;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        acc[k][j] = fmaf(u[k][j], xn[k][j], acc[k][j]);
        u[k][j] *= g[k][j];
        s = fmaf(u[k][j], xn[k][j], s);
      }
    }
    s = row_sum<NW>(s, red, turn) * inv;
    turn ^= 1;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = lt + 64 * NW * k;
      const int m = c < nfull ? 8 : c == nfull ? tail : 0;
      float d[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = 0.f;
      if (dres != nullptr) {
        if (m == 8) rd[k].unpack(d);
        else load_first(dres, at + 8 * (int64_t)c, m, d);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = fmaf(rstd, fmaf(-xn[k][j], s, u[k][j]), d[j]);
      if (m == 8) store8_any(static_cast<RT*>(a.dx), at + 8 * (int64_t)c, d);
      else store_first(static_cast<RT*>(a.dx), at + 8 * (int64_t)c, m, d);
    }
  }
  if (a.part == nullptr) return;
  if constexpr (G > 1) {  // the workgroup's rows of lanes in order
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (grp > 0) lsum[(((grp - 1) * CH + k) * 8 + j) * 64 + lt] = acc[k][j];
    __syncthreads();
    if (grp > 0) return;
#pragma unroll
    for (int w = 0; w < G - 1; ++w)
#pragma unroll
      for (int k = 0; k < CH; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[k][j] += lsum[((w * CH + k) * 8 + j) * 64 + lt];
  }
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = lt + 64 * NW * k;
    const int64_t at = (int64_t)blockIdx.x * width + 8 * (int64_t)c;
    if (c < nfull) store8_any(a.part, at, acc[k]);
    else if (c == nfull) store_first(a.part, at, tail, acc[k]);
  }
}

// dgain from the workgroups' partial rows: 32 columns a workgroup, 32 threads a
// column, each a fixed stride of rows.
__global__ __launch_bounds__(1024) void k_norm_gain_sum(const float* __restrict__ part, int rows, int64_t width,
                                                        float* __restrict__ dgain, int accumulate) {
  __shared__ float red[32][33];
  const int cl = threadIdx.x & 31, gr = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + cl;
  float s = 0.f;
  if (c < width)
    for (int r = gr; r < rows; r += 32) s += gmem(part)[r * width + c];
  red[gr][cl] = s;
  __syncthreads();
  if (gr == 0 && c < width) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) t += red[k][cl];
    gmem(dgain)[c] = accumulate ? gmem(dgain)[c] + t : t;
  }
}

// Waves of a row and chunks of 8 a lane, by the row's length.
struct NormShape {
  int nw, ch;
};
NormShape norm_shape(int64_t width) {
  if (width <= 512) return {1, 1};
  if (width <= 1024) return {1, 2};
  if (width <= 2048) return {4, 1};
  if (width <= 4096) return {4, 2};
  if (width <= 8192) return {8, 2};
  return {16, 2};
}

template <typename F>
hipError_t with_shape(int64_t width, F&& f) {
  const NormShape p = norm_shape(width);
  using std::integral_constant;
  const integral_constant<int, 1> one;
  const integral_constant<int, 2> two;
  if (p.nw == 1) return p.ch == 1 ? f(one, one) : f(one, two);
  if (p.nw == 4) return p.ch == 1 ? f(integral_constant<int, 4>{}, one) : f(integral_constant<int, 4>{}, two);
  if (p.nw == 8) return f(integral_constant<int, 8>{}, two);
  return f(integral_constant<int, 16>{}, two);
}

template <typename XT, typename RT, bool RES>
hipError_t norm(const NormArgs& a, hipStream_t s) {
  return with_shape(a.width, [&](auto nw, auto ch) {
    constexpr int NW = decltype(nw)::value, CH = decltype(ch)::value, NT = norm_threads(NW), G = NT / (64 * NW);
    const int64_t blocks = std::min<int64_t>((a.n + G - 1) / G, 2048);
    k_rms_norm<XT, RT, RES, NW, CH><<<dim3((uint32_t)blocks), NT, 0, s>>>(a);
    return hipGetLastError();
  });
}

template <typename YT, typename RT, bool PACKED>
hipError_t norm_grad(const NormGradArgs& a, hipStream_t s) {
  const int blocks = norm_grad_blocks(a.n, a.width);
  const hipError_t e = with_shape(a.width, [&](auto nw, auto ch) {
    constexpr int NW = decltype(nw)::value, CH = decltype(ch)::value;
    k_rms_norm_grad<YT, RT, PACKED, NW, CH><<<dim3(blocks), norm_threads(NW), 0, s>>>(a);
    return hipGetLastError();
  });
  if (e != hipSuccess || a.dgain == nullptr) return e;
  k_norm_gain_sum<<<dim3((uint32_t)((a.width + 31) / 32)), 1024, 0, s>>>(a.part, blocks, a.width, a.dgain, a.accumulate);
  return hipGetLastError();
}

}  // namespace

int norm_grad_blocks(int64_t n, int64_t width) {
  const NormShape p = norm_shape(width);
  const int64_t per = norm_threads(p.nw) / (64 * p.nw), most = p.nw == 16 ? 256 : 512;
  return (int)std::max<int64_t>(1, std::min<int64_t>((n + per - 1) / per, most));
}

hipError_t launch_rms_norm(int x_dt, int res_dt, const NormArgs& a, hipStream_t s) {
  if (x_dt == DT_BF16) {
    if (res_dt < 0) return norm<bf16_t, bf16_t, false>(a, s);
    return res_dt == DT_BF16 ? norm<bf16_t, bf16_t, true>(a, s) : norm<bf16_t, float, true>(a, s);
  }
  if (res_dt < 0) return norm<float, float, false>(a, s);
  return res_dt == DT_BF16 ? norm<float, bf16_t, true>(a, s) : norm<float, float, true>(a, s);
}

hipError_t launch_rms_norm_grad(int dy_dt, int dx_dt, const NormGradArgs& a, hipStream_t s) {
  const bool packed = a.x == nullptr;
  if (dy_dt == DT_BF16) {
    if (dx_dt == DT_BF16) return packed ? norm_grad<bf16_t, bf16_t, true>(a, s) : norm_grad<bf16_t, bf16_t, false>(a, s);
    return packed ? norm_grad<bf16_t, float, true>(a, s) : norm_grad<bf16_t, float, false>(a, s);
  }
  if (dx_dt == DT_BF16) return packed ? norm_grad<float, bf16_t, true>(a, s) : norm_grad<float, bf16_t, false>(a, s);
  return packed ? norm_grad<float, float, true>(a, s) : norm_grad<float, float, false>(a, s);
}

}  // namespace muonh
