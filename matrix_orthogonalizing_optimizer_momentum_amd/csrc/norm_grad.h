// Gradient of the root-mean-square norm (gfx950):
//
//   c  = mean_j g_j dy_j xn_j
//   dx = dres + s (g dy - xn c),      dg = sum over the rows of dy xn
//
// with xn = s h from the norm's input, or as the norm kept it in 8 bits (no
// statistics but s are kept then).  One pass over the rows, as in the norm.  The
// gain's gradient is summed in the lanes' registers over the workgroup's rows,
// written as one row of partial sums a workgroup and added up by a second launch, in
// a fixed order.  Few rows take one launch, in which further workgroups read them
// again by columns.
//
// A header: the types of dy are compiled in files of their own.
#pragma once
#include "norm.h"

namespace muonh {
namespace {

// Lanes along a row below, for rows of l threads: 4, and 2 where 32 columns a workgroup
// would leave few workgroups (2 lanes against 4: 512 x 768 5.8 us and 7.9, 256 x 2048 5.7
// and 5.2, 512 x 4096 11.0 and 9.1).
constexpr int gain_lanes(int l) { return l <= 128 ? 2 : 4; }

// The gain's gradient of 8 columns a lane over all rows, by one workgroup: GL lanes
// along a row, the others down the rows.
template <typename YT, typename RT, bool PACKED, int L>
__device__ __forceinline__ void gain_columns(const NormGradArgs& a, int block) {
  constexpr int NT = norm_threads(L), GL = gain_lanes(L), C = 8 * GL;
  constexpr int RG = NT / GL, F = 8;                          // rows side by side; rows in flight
  __shared__ float part[NT / 64][C];
  const int64_t width = a.width, nblk = mx_blocks(width), c = (int64_t)block * C + (threadIdx.x & (GL - 1)) * 8;
  const int m = (int)min<int64_t>(max<int64_t>(width - c, 0), 8);
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const YT* const dy = static_cast<const YT*>(a.dy);
  const RT* const x = static_cast<const RT*>(a.x);
  for (int64_t r0 = threadIdx.x / GL; r0 < a.n; r0 += F * RG) {
    Raw8<YT> ry[F];
    Raw8<RT> rx[F];
    u32x2_t rq[F];
    float f[F];
#pragma unroll
    for (int u = 0; u < F; ++u) {
      const int64_t r = min(r0 + u * RG, a.n - 1);
      if (m == 8) {
        ry[u].load_any(dy, r * width + c);
        if constexpr (PACKED) rq[u] = load_q8(a.q + r * width + c);
        else rx[u].load_any(x, r * width + c);
      }
      if constexpr (PACKED) f[u] = m > 0 ? mx_factor(gmem(a.scales)[r * nblk + c / kMxBlock]) : 0.f;
      else f[u] = gmem(a.rstd)[r];
    }
#pragma unroll
    for (int u = 0; u < F; ++u) {
      const int64_t r = r0 + u * RG;
      if (r >= a.n) break;
      float y[8], xn[8];
      if (m == 8) ry[u].unpack(y);
      else load_first(dy, r * width + c, m, y);
      if constexpr (PACKED) {
        from_e4m3(m == 8 ? rq[u] : load_q8(a.q + r * width + c, m), f[u], xn);
      } else {
        if (m == 8) rx[u].unpack(xn);
        else load_first(x, r * width + c, m, xn);
#pragma unroll
        for (int j = 0; j < 8; ++j) xn[j] *= f[u];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = fmaf(y[j], xn[j], acc[j]);
    }
  }
#pragma unroll
  for (int o = GL; o < 64; o *= 2)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] += __shfl_xor(acc[j], o, 64);
  if ((threadIdx.x & 63) < GL) {
#pragma unroll
    for (int j = 0; j < 8; ++j) part[threadIdx.x >> 6][(threadIdx.x & (GL - 1)) * 8 + j] = acc[j];
  }
  __syncthreads();
  const int64_t at = (int64_t)block * C + threadIdx.x;
  if (threadIdx.x < C && at < width) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < NT / 64; ++k) t += part[k][threadIdx.x];
    gmem(a.dgain)[at] = a.accumulate ? gmem(a.dgain)[at] + t : t;
  }
}

// RT: type of dx, dres and x (x: the norm's input; PACKED: xn in 8 bits instead).
// COLS: workgroups behind the first `blocks` sum the gain's gradient by columns
// (an instance of its own: the others need fewer registers).
// A workgroup has one row in flight: the next one's loads wait for its sum and stores
// (8192 x 768, 768 workgroups of 2 waves: 4.7 TB/s; 16384 x 4096, 512 of 8: 6.9).  Rows of 1024 threads have
// 128 registers a lane, which two chunks of 8 columns (widths above 8192: gain, sums and three
// operands of 16 columns) exceed by 10 to 87 (4096 x 16384 bf16 119 us, the bytes alone 69), and the
// 8 rows in flight of gain_columns by 24 to 178 but for bf16 dy and x in 8 bits (256 x 5120 from
// bf16 x 13 us, from fp32 x 23).
template <typename YT, typename RT, bool PACKED, bool TAIL, bool ONCE, bool COLS, int L, int CH>
__global__ __launch_bounds__(norm_threads(L)) void k_rms_norm_grad(const NormGradArgs a, int blocks) {
  constexpr int NT = norm_threads(L), G = NT / L;
  if constexpr (COLS) {
    if ((int)blockIdx.x >= blocks) {
      gain_columns<YT, RT, PACKED, L>(a, (int)blockIdx.x - blocks);
      return;
    }
  }
  __shared__ float red[2][row_waves(L)];
  __shared__ float lsum[G == 1 || COLS ? 1 : (G - 1) * L * CH * 8];
  const int lt = L <= 64 ? threadIdx.x & (L - 1) : threadIdx.x, grp = G == 1 ? 0 : threadIdx.x / L;
  const int64_t width = a.width, nblk = mx_blocks(width);
  const int nfull = (int)(width / 8), tail = (int)(width % 8);
  const YT* const dy = static_cast<const YT*>(a.dy);
  const RT* const x = static_cast<const RT*>(a.x);
  const RT* const dres = static_cast<const RT*>(a.dres);
  float g[CH][8], acc[CH][8];
  auto load_gain = [&](int k) {
    const int c = lt + L * k;
#pragma unroll
    for (int j = 0; j < 8; ++j) g[k][j] = 1.f;
    if (a.gain != nullptr) {
      if (c < nfull) load8_any(a.gain, 8 * c, g[k]);
      else if (TAIL && c == nfull) load_first(a.gain, 8 * (int64_t)c, tail, g[k]);
    }
  };
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    load_gain(k);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[k][j] = 0.f;
  }
  const float inv = 1.f / (float)width;
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * G + grp; row < a.n; row += (int64_t)blocks * G) {
    const int64_t at = row * width;
    const float rstd = gmem(a.rstd)[row];
    Raw8<YT> ry[CH];
    Raw8<RT> rx[CH], rd[CH];
    u32x2_t rq[CH];
    uint32_t rs[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = lt + L * k;
      if (c < nfull) {
        load_chunk<ONCE>(ry[k], dy, at + 8 * c);
        if constexpr (PACKED) {
          rq[k] = load_q8(a.q + at + 8 * c);
          rs[k] = gmem(a.scales)[row * nblk + c / 4];
        } else {
          load_chunk<ONCE>(rx[k], x, at + 8 * c);
        }
        if (dres != nullptr) load_chunk<ONCE>(rd[k], dres, at + 8 * c);
      }
    }
    float u[CH][8], xn[CH][8];
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = lt + L * k;
      const int m = TAIL && c == nfull ? tail : 0;
      if (!TAIL || c < nfull) ry[k].unpack(u[k]);
      else load_first(dy, at + 8 * (int64_t)c, m, u[k]);
      if constexpr (PACKED) {
        if (!TAIL || c < nfull) from_e4m3(rq[k], mx_factor(rs[k]), xn[k]);
        else from_e4m3(load_q8(a.q + at + 8 * (int64_t)c, m), m ? mx_factor(gmem(a.scales)[row * nblk + c / 4]) : 0.f, xn[k]);
      } else {
        if (!TAIL || c < nfull) rx[k].unpack(xn[k]);
        else load_first(x, at + 8 * (int64_t)c, m, xn[k]);
#pragma unroll
        for (int j = 0; j < 8; ++j) xn[k][j] *= rstd;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (!TAIL && c >= nfull) u[k][j] = xn[k][j] = 0.f;  // no chunk of the row: nothing was loaded
        if constexpr (!COLS) acc[k][j] = fmaf(u[k][j], xn[k][j], acc[k][j]);
        u[k][j] *= g[k][j];
        s = fmaf(u[k][j], xn[k][j], s);
      }
    }
    s = row_sum<L>(s, red, turn) * inv;
    turn ^= 1;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = lt + L * k;
      const int m = c < nfull ? 8 : TAIL && c == nfull ? tail : 0;
      float d[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = 0.f;
      if (dres != nullptr) {
        if (m == 8) rd[k].unpack(d);
        else if (TAIL) load_first(dres, at + 8 * (int64_t)c, m, d);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = fmaf(rstd, fmaf(-xn[k][j], s, u[k][j]), d[j]);
      if (m == 8) store_chunk<ONCE>(static_cast<RT*>(a.dx), at + 8 * (int64_t)c, d);
      else if (TAIL) store_first(static_cast<RT*>(a.dx), at + 8 * (int64_t)c, m, d);
    }
  }
  if (COLS || a.part == nullptr) return;
  if constexpr (G > 1) {  // the workgroup's rows of lanes in order
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (grp > 0) lsum[(((grp - 1) * CH + k) * 8 + j) * L + lt] = acc[k][j];
    __syncthreads();
    if (grp > 0) return;
#pragma unroll
    for (int w = 0; w < G - 1; ++w)
#pragma unroll
      for (int k = 0; k < CH; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[k][j] += lsum[((w * CH + k) * 8 + j) * L + lt];
  }
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int c = lt + L * k;
    const int64_t at = (int64_t)blockIdx.x * width + 8 * (int64_t)c;
    if (c < nfull) store8_any(a.part, at, acc[k]);
    else if (TAIL && c == nfull) store_first(a.part, at, tail, acc[k]);
  }
}

template <typename YT, typename RT, bool PACKED>
hipError_t norm_grad(const NormGradArgs& a, hipStream_t s) {
  const int blocks = norm_grad_blocks(a.n, a.width);
  const bool columns = a.dgain != nullptr && a.part == nullptr;
  const int64_t each = sizeof(YT) + (a.dres ? 2 : 1) * sizeof(RT) + (PACKED ? 1 : sizeof(RT));
  return with_shape(a.width, a.n * a.width * each > kActOnceBytes, [&](auto tail, auto once, auto lanes, auto ch) {
    constexpr int L = decltype(lanes)::value, CH = decltype(ch)::value, NT = norm_threads(L);
    if (columns) {
      constexpr int C = 8 * gain_lanes(L);
      const int64_t sums = (a.width + C - 1) / C;
      k_rms_norm_grad<YT, RT, PACKED, true, false, true, L, CH><<<dim3((uint32_t)(blocks + sums)), NT, 0, s>>>(a, blocks);
    } else {
      k_rms_norm_grad<YT, RT, PACKED, decltype(tail)::value, decltype(once)::value, false, L, CH>
          <<<dim3(blocks), NT, 0, s>>>(a, blocks);
    }
    return hipGetLastError();
  });
}

// dx and dres of type RT for dy of type YT, by dx's type.
template <typename YT>
hipError_t norm_grad_of(int dx_dt, const NormGradArgs& a, hipStream_t s) {
  if (dx_dt == DT_BF16) return a.x == nullptr ? norm_grad<YT, bf16_t, true>(a, s) : norm_grad<YT, bf16_t, false>(a, s);
  return a.x == nullptr ? norm_grad<YT, float, true>(a, s) : norm_grad<YT, float, false>(a, s);
}

}  // namespace
}  // namespace muonh
