// Gradient of a weight from activations kept in 8 bits (gfx950):
//
//   dW[o][i] = c g_i sum_t dz[t][o] x[t][i],   x = q 2^e (mx.h)
//
// Both operands lie along their columns, the sum runs over the tokens.  x is
// brought to bf16 along the tokens once (exact: e4m3 times a power of two), a
// pass of 3 bytes a value beside the product's 2 rows flop; dz is read as it is
// through the transposing LDS read of the main loop (product.h), or brought along the
// tokens too where x is so wide that the plain reads are worth a pass (api_act.hip);
// sums in fp32.
// The gain is a factor of the result's columns.  Weights of few tiles have their
// tokens cut into parts, one product each, that a second launch adds in order; so
// have the tiles of a large weight that are left over when the others fill the
// compute units.
#include <algorithm>

#include "common.h"
#include "mx.h"
#include "product.h"
#include "wgrad.h"

namespace muonh {

namespace {

// 8 tokens of 8 columns (16 bits each) to 8 runs of 8 tokens.
__device__ __forceinline__ void turn(const u32x4_t (&w)[8], u32x4_t (&run)[8]) {
#pragma unroll
  for (int h = 0; h < 4; ++h)
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      run[2 * h][p] = __builtin_amdgcn_perm(w[2 * p + 1][h], w[2 * p][h], 0x05040100);
      run[2 * h + 1][p] = __builtin_amdgcn_perm(w[2 * p + 1][h], w[2 * p][h], 0x07060302);
    }
}

// 128 tokens x 128 columns along the tokens, zeros behind the last one: x (X), or dz.
// A thread turns 8 x 8 values in registers; LDS brings the runs of a column together
// (16 bytes of chunk c of row r at c ^ swizzle), so that whole lines are read and stored.
template <bool X>
__device__ __forceinline__ void turn_tile(const WgradArgs& a, int64_t t0, int64_t c0, uint16_t (*lds)[128]) {
  const int cg = threadIdx.x & 15, og = threadIdx.x >> 4;
  const int64_t width = X ? a.width : a.rows, c = c0 + 8 * cg, nblk = mx_blocks(a.width);
  const int m = (int)min<int64_t>(max<int64_t>(width - c, 0), 8);
  u32x4_t w[8];
  uint32_t f[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int64_t t = t0 + 8 * og + k;
    w[k] = u32x4_t{0u, 0u, 0u, 0u};
    f[k] = 127;
    if (t < a.n && m > 0) {
      if constexpr (X) {
        const uint8_t* const p = a.q + t * width + c;
        f[k] = gmem(a.scales)[t * nblk + c / kMxBlock];
        const u32x2_t q = m == 8 ? load_q8(p) : load_q8(p, m);
        w[k][0] = q[0];
        w[k][1] = q[1];
      } else {
        const uint16_t* const p = a.dz + t * width + c;
        if (m == 8) {
          w[k] = *reinterpret_cast<const MUONH_GLOBAL u32x4_u*>(gmem(p));
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < m) w[k][j / 2] |= (uint32_t)gmem(p)[j] << (16 * (j & 1));
        }
      }
    }
  }
  if constexpr (X) {
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = e4m3_to_bf16(u32x2_t{w[k][0], w[k][1]}, f[k]);
  }
  u32x4_t run[8];
  turn(w, run);
  // rows 8 apart are written at once, consecutive chunks of a row are read
#pragma unroll
  for (int j = 0; j < 8; ++j) *reinterpret_cast<u32x4_t*>(&lds[8 * cg + j][(og ^ cg) * 8]) = run[j];
  __syncthreads();
  uint16_t* const out = X ? a.xt : a.dzt;
  const int64_t rows = min<int64_t>((width + 7) / 8 * 8 - c0, 128);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int r = (threadIdx.x >> 4) + 16 * k, o = threadIdx.x & 15;
    if (r < rows)
      *reinterpret_cast<MUONH_GLOBAL u32x4_t*>(gmem(out + (c0 + r) * a.ldxt + t0 + 8 * o)) =
          *reinterpret_cast<const u32x4_t*>(&lds[r][(o ^ (r >> 3)) * 8]);
  }
}

// What a product of 256 tiles reads: x along the tokens (workgroups below xtiles), and
// dz along them too (TURN), or dz's last, partial stage or all of it as it lies, padded with
// zeros.
template <bool TURN>
__global__ __launch_bounds__(256) void k_wgrad_prepare(const WgradArgs a, int xtiles, int xcols, int dcols) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[128][128];
  if ((int)blockIdx.x < xtiles) {
    turn_tile<true>(a, (int64_t)(blockIdx.x / xcols) * 128, (int64_t)(blockIdx.x % xcols) * 128, lds);
    return;
  }
  const int b = (int)blockIdx.x - xtiles;
  if constexpr (TURN) {
    turn_tile<false>(a, (int64_t)(b / dcols) * 128, (int64_t)(b % dcols) * 128, lds);
  } else {
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
      *reinterpret_cast<MUONH_GLOBAL u32x4_t*>(gmem(a.dzt + (row - a.dfull) * a.lddz + c)) = w;
    }
  }
}

constexpr int kDThreads = 256;

// Puts a wave's NI x NJ blocks at (di, dj) of the tile in LDS: rows of T + 4 values
// along the width.
template <int T, int NI, int NJ>
__device__ __forceinline__ void stage_tile(float* tile, int di, int dj, const f32x16_t (&acc)[NI][NJ]) {
  const int lane = threadIdx.x & 63, hi = lane >> 5;
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<f32x4_t*>(tile + (dj + 32 * j + (lane & 31)) * (T + 4) + di + 32 * i + 8 * q + 4 * hi) =
            f32x4_t{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
}

// Stores ROWS rows of a tile from LDS by whole rows (from the registers a store
// instruction would reach 32 bytes of each of 32 rows): to dw, or as sums of one part of the
// tokens to `part`, rows of ldp.
template <typename WT, int T, int ROWS, int THREADS>
__device__ __forceinline__ void put_rows(const WgradArgs& a, float* part, int64_t ldp, int64_t i0, int64_t o0,
                                         const float* tile) {
  constexpr int C = T / 8, R = THREADS / C;                   // chunks of a row, rows at a time
  const int c = threadIdx.x % C * 8, r0 = threadIdx.x / C;
  const int64_t d = i0 + c;
  auto row = [&](int r, float (&e)[8]) {
    const f32x4_t lo = *reinterpret_cast<const f32x4_t*>(tile + r * (T + 4) + c);
    const f32x4_t up = *reinterpret_cast<const f32x4_t*>(tile + r * (T + 4) + c + 4);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      e[k] = lo[k];
      e[4 + k] = up[k];
    }
  };
  float e[8];
  const int m = (int)min<int64_t>(a.width - d, 8);
  if (m <= 0) return;
  if (part != nullptr) {
#pragma unroll 2
    for (int r = r0; r < ROWS && o0 + r < a.rows; r += R) {
      row(r, e);
      store8(part, r * ldp + c, e);
    }
    return;
  }
  float f[8];
  if (a.gain != nullptr) load_first(a.gain, d, m, f);
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = a.gain != nullptr ? a.scale * f[k] : a.scale;
  WT* const dw = static_cast<WT*>(a.dw);
#pragma unroll 2
  for (int r = r0; r < ROWS && o0 + r < a.rows; r += R) {
    const int64_t at = (o0 + r) * a.width + d;
    row(r, e);
#pragma unroll
    for (int k = 0; k < 8; ++k) e[k] *= f[k];
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

// One 256 x 256 tile; those from a.first on, which would not fill the compute units once
// more, over one part of the tokens.
template <typename WT, bool TURN>
__global__ __launch_bounds__(kXThreads) __attribute__((amdgpu_waves_per_eu(2))) void k_wgrad(const WgradArgs a, int ni,
                                                                                             int no) {
  // the operands' stages; behind the loop half a tile's sums, in rows of 128 + 4
  __shared__ __attribute__((aligned(16))) char smem[kXTile * 132 * 4];
  constexpr int MI = 4, NI = 2, WM = Waves<MI, NI>::WM, WN = Waves<MI, NI>::WN;
  const int wave = threadIdx.x >> 6;
  const int wm = wave / Waves<MI, NI>::GN, wn = wave % Waves<MI, NI>::GN;
  const int all = (int)(a.npad / kXStage), first = a.first;
  int tile_id, s0 = 0, s1 = all;
  float* part = nullptr;
  if ((int)blockIdx.x < first) {
    tile_id = xcd_job(blockIdx.x, first);
  } else {
    const int job = xcd_job(blockIdx.x - first, gridDim.x - first), cut = ni * no - first, split = job / cut;
    tile_id = first + job - split * cut;
    s0 = (int)((uint32_t)(all * split) / (uint32_t)a.splits);
    s1 = (int)((uint32_t)(all * (split + 1)) / (uint32_t)a.splits);
    if (a.splits > 1) part = a.part + (int64_t)job * (kXTile * kXTile);
  }
  int to, ti;
  block_order(tile_id, ni, no, ti, to);
  const int64_t i0 = (int64_t)ti * kXTile, o0 = (int64_t)to * kXTile;
  const uint16_t* const xt = a.xt + i0 * a.ldxt + (int64_t)s0 * kXStage;
  f32x16_t acc[MI][NI];
  if constexpr (TURN) {
    const uint16_t* const dzt = a.dzt + o0 * a.ldxt + (int64_t)s0 * kXStage;
    product<false, false, MI, NI>(
        smem, s1 - s0, [=](int s) { return xt + (int64_t)s * kXStage; }, a.ldxt, 0,
        [=](int s) { return dzt + (int64_t)s * kXStage; }, a.ldxt, 0, acc);
  } else {
    const uint16_t *const dz = a.dz + o0, *const dzc = a.dzt + o0;
    const int64_t full = a.dfull, ld = a.lddz;
    product<false, true, MI, NI>(
        smem, s1 - s0, [=](int s) { return xt + (int64_t)s * kXStage; }, a.ldxt, 0,
        [=](int s) {
          const int64_t t = (int64_t)(s0 + s) * kXStage;
          return t < full ? dz + t * ld : dzc + (t - full) * ld;
        },
        ld, ld - o0, acc);
  }
  // half of the width at a time through LDS
  static_assert(WM == 128 && kXTile * (WM + 4) * 4 <= (int)sizeof(smem), "half a tile's sums fit");
  float* const tile = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    __syncthreads();
    if (wm == h) stage_tile<WM>(tile, 0, wn * WN, acc);
    __syncthreads();
    put_rows<WT, WM, kXTile, kXThreads>(a, part == nullptr ? nullptr : part + h * WM, kXTile, i0 + h * WM, o0, tile);
  }
}

// A T x T tile over one part of the tokens, from the caller's buffers in one
// launch, by 4 waves.  A stage of 64 tokens comes through registers (any
// alignment; x is brought to bf16 there) into LDS as it lies, tokens down, and
// both operands are read transposed.  Rows are padded by 64 bytes, so that the 4
// tokens which a transposing read touches lie in different banks.  A wave multiplies
// 64 x 64: a quarter of a tile of 128, or a whole tile of 64 for a quarter of the
// tokens, with the waves' sums joined at the end.  Two stages are
// in flight in registers and one in LDS beside the one that is multiplied, with
// one barrier a stage.  A 64 tile is bound by its loads (8192 x 2304 x 768: 52 of 62
// us, 14 TB/s), a 128 tile by its loads, stores and products one after the other (0.2,
// 0.2 and 0.25 us of a stage's 0.72); four stages in flight, the stores between the
// products, and operands turned in registers before LDS, with reads of half the
// time, took as long or longer.  What lies behind a row's end is read as it comes
// (the next row) and reaches only results that are not kept; stages whose reads
// would leave a buffer are read value by value, with zeros behind the last token.
template <typename WT, int T>
__global__ __launch_bounds__(kDThreads) __attribute__((amdgpu_waves_per_eu(2))) void k_wgrad_direct(const WgradArgs a, int ni,
                                                                                                    int no) {
  constexpr bool kWhole = T == 64;                            // a wave multiplies the whole tile
  constexpr int P = T + 32, NB = 2;                           // pitch of a row in LDS; 32 x 32 blocks of a wave along a side
  constexpr int XC = T / 16, XU = 64 * XC / kDThreads;        // chunks of 16 x values of a row, of a thread
  constexpr int ZC = T / 8, ZU = 64 * ZC / kDThreads;         // chunks of 8 dz values
  __shared__ __attribute__((aligned(16))) uint16_t smem[4 * 64 * P];
  uint16_t (*const sx)[64 * P] = reinterpret_cast<uint16_t (*)[64 * P]>(smem);
  uint16_t (*const sz)[64 * P] = sx + 2;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int job = xcd_job(blockIdx.x, gridDim.x), per = ni * no, split = job / per;
  int to, ti;
  block_order(job - split * per, ni, no, ti, to);
  const int64_t i0 = (int64_t)ti * T, o0 = (int64_t)to * T, nblk = mx_blocks(a.width);
  const int all = (int)((a.n + 63) / 64);
  const int s0 = (int)((uint32_t)(all * split) / (uint32_t)a.splits), s1 = (int)((uint32_t)(all * (split + 1)) / (uint32_t)a.splits);
  const int sf = max(s0, min(s1, (int)a.whole));
  f32x16_t acc[NB][NB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

  struct Stage {
    u32x4_t x[XU], z[ZU];
    uint32_t f[XU];
  };
  // this thread's chunks, from the first value of the next stage to be loaded
  uint32_t vx[XU], vf[XU], vz[ZU];
#pragma unroll
  for (int u = 0; u < XU; ++u) {
    const int id = tid + u * kDThreads;
    vx[u] = (uint32_t)((id / XC) * a.width + id % XC * 16);
    vf[u] = (uint32_t)((id / XC) * nblk + id % XC / 2);
  }
#pragma unroll
  for (int u = 0; u < ZU; ++u) {
    const int id = tid + u * kDThreads;
    vz[u] = (uint32_t)(((id / ZC) * a.rows + id % ZC * 8) * 2);
  }
  const MUONH_GLOBAL uint8_t* px = gmem(a.q + (int64_t)s0 * 64 * a.width + i0);
  const MUONH_GLOBAL uint8_t* pf = gmem(a.scales + (int64_t)s0 * 64 * nblk + i0 / kMxBlock);
  const MUONH_GLOBAL char* pz = reinterpret_cast<const MUONH_GLOBAL char*>(gmem(a.dz + (int64_t)s0 * 64 * a.rows + o0));
  const int64_t ax = 64 * a.width, af = 64 * nblk, az = 128 * a.rows;
  // the next stage (the last one again behind it)
  auto load = [&](Stage& r, bool more) {
#pragma unroll
    for (int u = 0; u < XU; ++u) {
      r.x[u] = *reinterpret_cast<const MUONH_GLOBAL u32x4_b*>(px + vx[u]);
      r.f[u] = pf[vf[u]];
    }
#pragma unroll
    for (int u = 0; u < ZU; ++u) r.z[u] = *reinterpret_cast<const MUONH_GLOBAL u32x4_u*>(pz + vz[u]);
    px += more ? ax : 0;
    pf += more ? af : 0;
    pz += more ? az : 0;
    __builtin_amdgcn_sched_barrier(0);  // the waits count loads in this order
  };
  // a stage value by value where a chunk is not whole; zeros behind the last token
  auto load_edge = [&](int64_t s, Stage& r) {
#pragma unroll
    for (int u = 0; u < XU; ++u) {
      const int id = tid + u * kDThreads;
      const int64_t t = s * 64 + id / XC, c = i0 + id % XC * 16;
      r.x[u] = u32x4_t{0u, 0u, 0u, 0u};
      r.f[u] = 127;
      if (t < a.n && c < a.width) {
        const uint8_t* const p = a.q + t * a.width + c;
        r.f[u] = gmem(a.scales)[t * nblk + c / kMxBlock];
        if (c + 16 <= a.width) {
          r.x[u] = *reinterpret_cast<const MUONH_GLOBAL u32x4_b*>(gmem(p));
        } else {
          const int m = (int)(a.width - c);
          const u32x2_t lo = load_q8(p, min(m, 8)), up = load_q8(p + 8, max(m - 8, 0));
          r.x[u] = u32x4_t{lo[0], lo[1], up[0], up[1]};
        }
      }
    }
#pragma unroll
    for (int u = 0; u < ZU; ++u) {
      const int id = tid + u * kDThreads;
      const int64_t t = s * 64 + id / ZC, c = o0 + id % ZC * 8;
      r.z[u] = u32x4_t{0u, 0u, 0u, 0u};
      if (t < a.n && c < a.rows) {
        const uint16_t* const p = a.dz + t * a.rows + c;
        if (c + 8 <= a.rows) {
          r.z[u] = *reinterpret_cast<const MUONH_GLOBAL u32x4_u*>(gmem(p));
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (c + k < a.rows) r.z[u][k / 2] |= (uint32_t)gmem(p)[k] << (16 * (k & 1));
        }
      }
    }
  };
  auto store = [&](int buf, const Stage& r) {
#pragma unroll
    for (int u = 0; u < XU; ++u) {
      const int id = tid + u * kDThreads;
      uint16_t* const p = sx[buf] + id / XC * P + id % XC * 16;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<u32x4_t*>(p + 8 * h) = e4m3_to_bf16(u32x2_t{r.x[u][2 * h], r.x[u][2 * h + 1]}, r.f[u]);
    }
#pragma unroll
    for (int u = 0; u < ZU; ++u) {
      const int id = tid + u * kDThreads;
      *reinterpret_cast<u32x4_t*>(sz[buf] + id / ZC * P + id % ZC * 8) = r.z[u];
    }
  };
  const int j16 = lane & 15, g = lane >> 4;
  const int at = (8 * (g >> 1) + (j16 >> 2)) * P + 16 * (g & 1) + 4 * (j16 & 3);
  const int wi = kWhole ? 0 : (wave >> 1) * 64, wo = kWhole ? 0 : (wave & 1) * 64;
  auto fragment = [&](const uint16_t* base, int kk, int col) {
    const uint16_t* p = base + at + kk * 16 * P + col;
    const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4_t*)p);
    const i16x4_t up = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4_t*)(p + 4 * P));
    return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, up, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  auto multiply = [&](int buf) {
    constexpr int K = kWhole ? 1 : 4;                         // steps of 16 tokens that a wave takes of a stage
    bf16x8_t fa[K][NB], fb[K][NB];
#pragma unroll
    for (int q = 0; q < K; ++q) {
      const int kk = kWhole ? wave : q;
#pragma unroll
      for (int i = 0; i < NB; ++i) fa[q][i] = fragment(sx[buf], kk, wi + 32 * i);
#pragma unroll
      for (int j = 0; j < NB; ++j) fb[q][j] = fragment(sz[buf], kk, wo + 32 * j);
      if (q & 1) __builtin_amdgcn_sched_barrier(0);           // half a stage's reads are on their way before any product
    }
#pragma unroll
    for (int q = 0; q < K; ++q)
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[q][i], fb[q][j], acc[i][j], 0, 0, 0);
  };
  // Stage s goes to buffer (s - s0) % 2; that buffer's readers, of stage s - 2, are
  // behind the barrier of stage s - 1.
  auto step = [&](int buf, Stage& r, int next) {
    store(buf, r);
    load(r, next + 1 < sf);
    lds_release();
    barrier();
    lds_acquire();
    multiply(buf);
  };
  if (s0 < sf) {
    Stage even, odd;
    load(even, s0 + 1 < sf);
    load(odd, s0 + 2 < sf);
    int s = s0;
    for (; s + 1 < sf; s += 2) {
      step(0, even, s + 2);
      step(1, odd, s + 3);
    }
    if (s < sf) step(0, even, s + 2);
  }
  for (int s = sf; s < s1; ++s) {
    Stage r;
    load_edge(s, r);
    store((s - s0) & 1, r);
    __syncthreads();
    multiply((s - s0) & 1);
  }
  static_assert(T * (T + 4) * 4 <= 4 * 64 * P * 2, "the tile's sums fit the operands' place");
  float* const tile = reinterpret_cast<float*>(smem);
  if constexpr (!kWhole) {
    __syncthreads();
    stage_tile<T>(tile, wi, wo, acc);
  } else {
    // each wave takes one block of the tile from the others, in the order of the waves
    static_assert(12 * 4096 <= 4 * 64 * P * 2, "three blocks a wave");
    f32x4_t* const sh = reinterpret_cast<f32x4_t*>(smem);
    __syncthreads();
    f32x16_t mine[1][1];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const f32x16_t& v = acc[b >> 1][b & 1];
      if (b == wave) {
        mine[0][0] = v;
      } else {
        f32x4_t* const to_b = sh + (b * 3 + (wave < b ? wave : wave - 1)) * 256 + lane;
#pragma unroll
        for (int q = 0; q < 4; ++q) to_b[64 * q] = f32x4_t{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4_t e = sh[(wave * 3 + k) * 256 + 64 * q + lane];
#pragma unroll
        for (int r = 0; r < 4; ++r) mine[0][0][4 * q + r] += e[r];
      }
    __syncthreads();
    stage_tile<T>(tile, 32 * (wave >> 1), 32 * (wave & 1), mine);
  }
  __syncthreads();
  float* const part = a.splits > 1 ? a.part + ((int64_t)split * a.rows + o0) * a.ldp + i0 : nullptr;
  put_rows<WT, T, T, kDThreads>(a, part, a.ldp, i0, o0, tile);
}

// dw from the parts: 4 columns a thread, 8 parts in flight, added in their order.
// TILES: of the 256 tiles from a.first on, ni x no in all.
template <typename WT, bool TILES>
__global__ __launch_bounds__(256) void k_wgrad_join(const WgradArgs a, int ni, int no) {
  const uint32_t id = blockIdx.x * 256 + threadIdx.x;
  int64_t o, d, step;
  const float* p;
  if constexpr (TILES) {
    const int t = (int)(id / (kXTile * kXTile / 4));
    int to, ti;
    block_order(a.first + t, ni, no, ti, to);
    o = (int64_t)to * kXTile + id / (kXTile / 4) % kXTile;
    d = (int64_t)ti * kXTile + id % (kXTile / 4) * 4;
    step = (int64_t)(ni * no - a.first) * (kXTile * kXTile);
    p = a.part + (int64_t)id * 4;
  } else {
    const uint32_t per = (uint32_t)(a.ldp / 4);
    o = id / per;
    d = (int64_t)(id % per) * 4;
    step = a.rows * a.ldp;
    p = a.part + o * a.ldp + d;
  }
  if (o >= a.rows) return;
  const int m = (int)min<int64_t>(a.width - d, 4);
  if (m <= 0) return;
  f32x4_t e = {0.f, 0.f, 0.f, 0.f};
  for (int k = 0; k < a.splits; k += 8, p += 8 * step) {
    f32x4_t r[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (k + u < a.splits) r[u] = *reinterpret_cast<const MUONH_GLOBAL f32x4_t*>(gmem(p + u * step));
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (k + u < a.splits) e += r[u];
  }
  WT* const dw = static_cast<WT*>(a.dw);
  const int64_t at = o * a.width + d;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < m) {
      e[j] *= a.gain != nullptr ? a.scale * gmem(a.gain)[d + j] : a.scale;
      if (a.accumulate) e[j] += St<WT>::ld(dw, at + j);
    }
  if (m == 4) {
    if constexpr (sizeof(WT) == 4) {
      typedef f32x4_t __attribute__((aligned(4))) f32x4_a;
      *reinterpret_cast<MUONH_GLOBAL f32x4_a*>(gmem(dw + at)) = e;
    } else {
      typedef u32x2_t __attribute__((aligned(2))) u32x2_a;
      *reinterpret_cast<MUONH_GLOBAL u32x2_a*>(gmem(dw + at)) = u32x2_t{pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3])};
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < m) St<WT>::st(dw, at + j, e[j]);
  }
}

}  // namespace

hipError_t launch_wgrad_prepare(const WgradArgs& a, hipStream_t s) {
  const int64_t ttiles = (a.n + 127) / 128, xcols = (a.width + 127) / 128, xtiles = ttiles * xcols;
  const int64_t dcols = a.turn ? (a.rows + 127) / 128 : (a.lddz + 255) / 256;
  const int64_t dtiles = a.turn ? ttiles * dcols : (a.npad - a.dfull) / 64 * dcols;
  if (xtiles + dtiles == 0) return hipSuccess;
  const dim3 g((uint32_t)(xtiles + dtiles));
  if (a.turn) k_wgrad_prepare<true><<<g, 256, 0, s>>>(a, (int)xtiles, (int)xcols, (int)dcols);
  else k_wgrad_prepare<false><<<g, 256, 0, s>>>(a, (int)xtiles, (int)xcols, (int)dcols);
  return hipGetLastError();
}

namespace {
template <typename WT>
hipError_t wgrad(const WgradArgs& a, hipStream_t s) {
  const int ni = (int)((a.width + a.tile - 1) / a.tile), no = (int)((a.rows + a.tile - 1) / a.tile);
  const int64_t cut = (int64_t)ni * no - a.first;  // tiles in parts
  const dim3 g((uint32_t)(a.first + cut * a.splits));
  if (a.tile == kXTile && a.turn) k_wgrad<WT, true><<<g, kXThreads, 0, s>>>(a, ni, no);
  else if (a.tile == kXTile) k_wgrad<WT, false><<<g, kXThreads, 0, s>>>(a, ni, no);
  else if (a.tile == 128) k_wgrad_direct<WT, 128><<<g, kDThreads, 0, s>>>(a, ni, no);
  else k_wgrad_direct<WT, 64><<<g, kDThreads, 0, s>>>(a, ni, no);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  if (a.tile == kXTile)
    k_wgrad_join<WT, true><<<dim3((uint32_t)(cut * (kXTile * kXTile / 4 / 256))), 256, 0, s>>>(a, ni, no);
  else
    k_wgrad_join<WT, false><<<dim3((uint32_t)((a.rows * (a.ldp / 4) + 255) / 256)), 256, 0, s>>>(a, ni, no);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_wgrad(const WgradArgs& a, hipStream_t s) {
  return a.dw_dt == DT_BF16 ? wgrad<bf16_t>(a, s) : wgrad<float>(a, s);
}

}  // namespace muonh
