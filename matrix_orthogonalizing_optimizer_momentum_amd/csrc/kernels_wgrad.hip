// Gradient of a weight from activations kept in 8 bits (gfx950):
//
//   dW[o][i] = c g_i sum_t dz[t][o] x[t][i],   x = q 2^e (mx.h)
//
// Both operands lie along their columns, the sum runs over the tokens.  x is
// brought to bf16 along the tokens once (exact: e4m3 times a power of two), a
// pass of 3 bytes a value beside the product's 2 rows flop; dz is read as it is
// through the transposing LDS read of the main loop (product.h), sums in fp32.
// The gain is a factor of the result's columns.  Weights of few tiles have their
// tokens cut into parts, one product each, that a second launch adds in order.
#include <algorithm>

#include "common.h"
#include "mx.h"
#include "product.h"
#include "wgrad.h"

namespace muonh {

namespace {

// 64 tokens x 64 columns of q a workgroup (x < xtiles), transposed; behind them
// 64 rows x 256 columns of dz's copy.
__global__ __launch_bounds__(256) void k_wgrad_prepare(const WgradArgs a, int xtiles, int xcols, int dcols) {
  __shared__ uint16_t t[64][72];
  if ((int)blockIdx.x < xtiles) {
    const int64_t r0 = (int64_t)(blockIdx.x / xcols) * 64, c0 = (int64_t)(blockIdx.x % xcols) * 64;
    const int r = threadIdx.x >> 3, c = (threadIdx.x & 7) * 8;
    const int64_t nblk = mx_blocks(a.width);
    const int m = (int)min<int64_t>(max<int64_t>(a.width - c0 - c, 0), 8);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int64_t row = r0 + r + 32 * k;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.f;
      if (row < a.n && m > 0) {
        const uint8_t* const p = a.q + row * a.width + c0 + c;
        const float f = mx_factor(gmem(a.scales)[row * nblk + (c0 + c) / kMxBlock]);
        from_e4m3(m == 8 ? load_q8(p) : load_q8(p, m), f, v);
      }
      u32x4_t w;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
      *reinterpret_cast<u32x4_t*>(&t[r + 32 * k][c]) = w;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      u32x4_t w;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = (uint32_t)t[c + 2 * e][r + 32 * k] | (uint32_t)t[c + 2 * e + 1][r + 32 * k] << 16;
      *reinterpret_cast<MUONH_GLOBAL u32x4_t*>(gmem(a.xt + (c0 + r + 32 * k) * a.ldxt + r0 + c)) = w;
    }
    return;
  }
  const int b = (int)blockIdx.x - xtiles;
  const int64_t r0 = a.dfull + (int64_t)(b / dcols) * 64, c = (int64_t)(b % dcols) * 256 + (threadIdx.x & 31) * 8;
  if (c >= a.lddz) return;
  const int m = (int)min<int64_t>(max<int64_t>(a.rows - c, 0), 8);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int64_t row = r0 + (threadIdx.x >> 5) + 8 * k;
    u32x4_t w = {0u, 0u, 0u, 0u};
    if (row < a.n) {
      const uint16_t* const p = a.dz + row * a.rows + c;
      if (m == 8) {
        w = *reinterpret_cast<const MUONH_GLOBAL u32x4_u*>(gmem(p));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < m) w[j / 2] |= (uint32_t)gmem(p)[j] << (16 * (j & 1));
      }
    }
    *reinterpret_cast<MUONH_GLOBAL u32x4_t*>(gmem(a.dzc + (row - a.dfull) * a.lddz + c)) = w;
  }
}

// One 256 x 256 tile over one part of the tokens.
template <typename WT>
__global__ __launch_bounds__(kXThreads) __attribute__((amdgpu_waves_per_eu(2))) void k_wgrad(const WgradArgs a, int ni,
                                                                                             int no) {
  __shared__ __attribute__((aligned(16))) char smem[kXSmem];
  constexpr int MI = 4, NI = 2, WM = Waves<MI, NI>::WM, WN = Waves<MI, NI>::WN;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, hi = lane >> 5;
  const int wm = wave / Waves<MI, NI>::GN, wn = wave % Waves<MI, NI>::GN;
  const int job = xcd_job(blockIdx.x, gridDim.x), per = ni * no, split = job / per;
  int to, ti;
  block_order(job - split * per, ni, no, ti, to);
  const int64_t i0 = (int64_t)ti * kXTile, o0 = (int64_t)to * kXTile;
  const int64_t all = a.npad / kXStage;
  const int64_t s0 = all * split / a.splits, s1 = all * (split + 1) / a.splits;
  const uint16_t* const xt = a.xt + i0 * a.ldxt + s0 * kXStage;
  const uint16_t *const dz = a.dz + o0, *const dzc = a.dzc + o0;
  const int64_t full = a.dfull, ld = a.lddz;
  f32x16_t acc[MI][NI];
  product<false, true, MI, NI>(
      smem, (int)(s1 - s0), [=](int s) { return xt + (int64_t)s * kXStage; }, a.ldxt, 0,
      [=](int s) {
        const int64_t t = (s0 + s) * kXStage;
        return t < full ? dz + t * ld : dzc + (t - full) * ld;
      },
      ld, ld - o0, acc);
  if (a.splits > 1) {
    float* const out = a.part + (int64_t)split * a.rows * a.ldp;
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int64_t o = o0 + wn * WN + j * 32 + (lane & 31);
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int64_t d = i0 + wm * WM + i * 32 + 8 * q + 4 * hi;
          if (d >= a.ldp || o >= a.rows) continue;
          *reinterpret_cast<MUONH_GLOBAL f32x4_t*>(gmem(out + o * a.ldp + d)) =
              f32x4_t{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        }
    }
    return;
  }
  WT* const dw = static_cast<WT*>(a.dw);
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int pq = 0; pq < 2; ++pq) {
      const int64_t d = i0 + wm * WM + i * 32 + 16 * pq + 8 * hi;
      const int m = (int)min<int64_t>(max<int64_t>(a.width - d, 0), 8);
      float f[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = a.scale;
      if (a.gain != nullptr) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < m) f[k] *= gmem(a.gain)[d + k];
      }
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const int64_t o = o0 + wn * WN + j * 32 + (lane & 31);
        float e[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(acc[i][j][8 * pq + k]),
                                                           __float_as_uint(acc[i][j][8 * pq + 4 + k]), false, false);
          e[k] = __uint_as_float(sw[0]);
          e[4 + k] = __uint_as_float(sw[1]);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) e[k] *= f[k];
        if (o >= a.rows || m == 0) continue;
        const int64_t at = o * a.width + d;
        if (a.accumulate) {
          float old[8];
          if (m == 8) load8_any(dw, at, old);
          else load_first(dw, at, m, old);
#pragma unroll
          for (int k = 0; k < 8; ++k) e[k] += old[k];
        }
        if (m == 8) store8_any(dw, at, e);
        else store_first(dw, at, m, e);
      }
    }
}

// dw from the parts: 8 columns a thread.
template <typename WT>
__global__ __launch_bounds__(256) void k_wgrad_join(const WgradArgs a) {
  const int64_t per = a.ldp / 8, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= per * a.rows) return;
  const int64_t o = id / per, d = (id - o * per) * 8;
  const int m = (int)min<int64_t>(a.width - d, 8);
  if (m <= 0) return;
  float e[8], p[8], f[8];
  load8(a.part, o * a.ldp + d, e);
  for (int k = 1; k < a.splits; ++k) {
    load8(a.part, ((int64_t)k * a.rows + o) * a.ldp + d, p);
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] += p[j];
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = 1.f;
  if (a.gain != nullptr) load_first(a.gain, d, m, f);
#pragma unroll
  for (int j = 0; j < 8; ++j) e[j] *= a.scale * f[j];
  WT* const dw = static_cast<WT*>(a.dw);
  const int64_t at = o * a.width + d;
  if (a.accumulate) {
    load_first(dw, at, m, p);
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] += p[j];
  }
  if (m == 8) store8_any(dw, at, e);
  else store_first(dw, at, m, e);
}

}  // namespace

hipError_t launch_wgrad_prepare(const WgradArgs& a, hipStream_t s) {
  const int64_t xcols = (a.width + 63) / 64, xtiles = a.npad / 64 * xcols;
  const int64_t dcols = (a.lddz + 255) / 256, dtiles = (a.npad - a.dfull) / 64 * dcols;
  if (xtiles + dtiles == 0) return hipSuccess;
  k_wgrad_prepare<<<dim3((uint32_t)(xtiles + dtiles)), 256, 0, s>>>(a, (int)xtiles, (int)xcols, (int)dcols);
  return hipGetLastError();
}

hipError_t launch_wgrad(const WgradArgs& a, hipStream_t s) {
  const int ni = (int)((a.width + kXTile - 1) / kXTile), no = (int)((a.rows + kXTile - 1) / kXTile);
  const dim3 g((uint32_t)((int64_t)ni * no * a.splits));
  if (a.dw_dt == DT_BF16) k_wgrad<bf16_t><<<g, kXThreads, 0, s>>>(a, ni, no);
  else k_wgrad<float><<<g, kXThreads, 0, s>>>(a, ni, no);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  const dim3 j((uint32_t)((a.rows * (a.ldp / 8) + 255) / 256));
  if (a.dw_dt == DT_BF16) k_wgrad_join<bf16_t><<<j, 256, 0, s>>>(a);
  else k_wgrad_join<float><<<j, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace muonh
