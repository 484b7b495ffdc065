// Softmax cross entropy of an output layer with its gradient (gfx950).
//
//   l_iv   = <x_i, w_v>,   lse_i = log sum_v exp(l_iv),   loss_i = lse_i - l_i,t_i
//   P_iv   = exp(l_iv - lse_i) - [v = t_i]
//   dx_i   = c sum_v P_iv w_v,     dw_v = c sum_i P_iv x_i
//
// over the counted tokens only (target inside [0, rows) and not ignore_index):
// they are gathered to the front of a padded copy of x, so that ignored tokens
// cost no product and whatever they hold reaches nothing.
//
// The logits are never stored.  A first product over the whole vocabulary
// keeps, per token and tile of 256 words, the maximum and the sum of exponents
// (k_xent_logits, STATS); they give lse and the loss.  The gradient then takes
// the vocabulary in pieces: the same product again, its epilogue turning the
// logits into P in bf16 (off by at most 2^-8 of each value; the operand type of the
// matrix cores) for one piece, and two products that read that P:
// dx += P w_piece (fp32 across pieces) and dw_piece = P^T x.
//
// P's rounding is the one place below 32 bits.  8192 tokens, 50257 x 768: bf16
// results are 0.00168 of their norm from 64 bits, 0.00166 with P in fp32; an fp32
// dw is 2.6e-4 from the one with P in fp32.  A second bf16 part of P for what the
// first leaves would double the two products that read it, half of the call.
//
// All products run on one 256 x 256 main loop of 8 waves, D[m][n] =
// sum_k A[m][k] B[n][k]: v_mfma_f32_32x32x16_bf16, 64-deep operand stages
// double buffered in LDS, brought in by direct global -> LDS loads; the two
// waves of a SIMD alternate between reading fragments and running MFMAs.  An
// operand whose rows run along k is read as it is; one stored [k][m] is read
// through gfx950's transposing LDS read, so that neither P nor w is transposed
// in memory (x is, once: dw needs both its operands along the tokens, and
// transposing reads of both would bound it by LDS).  The side a lane holds four consecutive values of (m)
// is the one the result's rows run along: words for P, width for dx and dw.
#include <type_traits>

#include "common.h"
#include "xent.h"

namespace muonh {

namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef short i16x8_t __attribute__((ext_vector_type(8)));
typedef __attribute__((ext_vector_type(16))) float f32x16_t;

constexpr int kXThreads = 512;
constexpr int kOperand = kXTile * kXStage;        // elements of one operand stage
constexpr int kOperandB = kOperand * 2;           // 32 KiB
constexpr int kXSmem = 4 * kOperandB;             // two stages of two operands
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void wait_loads() { __builtin_amdgcn_s_waitcnt(0x0F70); }   // vmcnt(0)
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(0xC07F); }     // lgkmcnt(0)
__device__ __forceinline__ void barrier() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
}
// barrier() waits for no memory access.  LDS stores that other waves read
// behind one are followed by lds_release(), those reads led by lds_acquire().
__device__ __forceinline__ void lds_release() { __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local"); }
__device__ __forceinline__ void lds_acquire() { __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local"); }
__device__ __forceinline__ void wave_fence() {  // orders a wave's LDS accesses, which execute in order
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Chunk c (16 bytes) of a k-contiguous LDS row r sits at c ^ swz(r): any 16
// consecutive rows of one chunk are spread over all banks.
__device__ __forceinline__ int swz(int r) { return (r >> 1) & 7; }

// A wave's block of the tile: MI x NI blocks of 32 x 32, 8 in all.
template <int MI, int NI>
struct Waves {
  static constexpr int WM = 32 * MI, WN = 32 * NI, GN = kXTile / WN;
  static_assert(MI * NI == 8 && (kXTile / WM) * GN == 8, "8 waves cover the tile");
};
// Transposing reads take twice the LDS time of plain ones (two 8-byte
// accesses for one of 16), so an operand that needs them goes to the side a
// wave has fewer fragments of.

// One operand of the product: TR false, 256 rows of k-contiguous values (row
// stride ld elements); TR true, k rows of 256 values along m.
template <bool TR>
struct Operand {
  uint32_t voff;      // this lane's byte offset of the wave's first 1 KiB run
  uint32_t rstride;   // bytes between its runs
  // ncols (TR): columns of the operand from the tile's first one; chunks past
  // them are read from the last one and only reach results that are not kept
  __device__ __forceinline__ void init(int wv4, int lane, int64_t ld, int64_t ncols) {
    if constexpr (TR) {
      const int k = 2 * wv4 + (lane >> 5), pc = lane & 31;
      const int c = (pc - 4 * (k & 3)) & 31;  // row k is rotated by 4 (k % 4) chunks
      const int64_t col = min((int64_t)c * 8, ncols - 8);
      voff = (uint32_t)((k * ld + col) * 2);
      rstride = (uint32_t)(8 * ld * 2);
    } else {
      const int r = 8 * wv4 + lane / 8, pc = lane % 8;
      voff = (uint32_t)((r * ld + (pc ^ swz(r)) * 8) * 2);
      rstride = (uint32_t)(32 * ld * 2);
    }
  }
};

template <bool TR>
__device__ __forceinline__ int frag_base(int wave_row, int lane) {
  if constexpr (TR) {
    const int j = lane & 15, g = lane >> 4;
    const int k = 8 * (g >> 1) + (j >> 2);
    return k * kXTile + ((wave_row + 16 * (g & 1) + 4 * (j & 3) + 32 * (j >> 2)) & (kXTile - 1));
  } else {
    return (wave_row + (lane & 31)) * kXStage;
  }
}

// Fragment of k-step kk (16 deep): 8 consecutive k of one row per lane.
template <bool TR>
__device__ __forceinline__ bf16x8_t frag(const uint16_t* stage, int base, int xk, int kk) {
  if constexpr (TR) {
    const uint16_t* p = stage + base + kk * 16 * kXTile;
    const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4_t*)p);
    const i16x4_t hi =
        __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4_t*)(p + 4 * kXTile));
    return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  } else {
    return *reinterpret_cast<const bf16x8_t*>(stage + base + xk);
  }
}

// acc = sum over nstage stages.  abase(s) / bbase(s): address of the tile's
// first value of stage s (uniform).  Waves 0-3 load operand A, waves 4-7
// operand B; the groups run one phase apart, each phase (a half stage's
// fragments, or its MFMAs) ending at a barrier of all 8 waves, so that of the
// two waves on a SIMD one always feeds the matrix core.  Stage s + 1
// overwrites the buffer of stage s - 1, whose last fragments were read in
// phase 4 s - 1; its loads ride between the MFMAs of phases 4 s and 4 s + 1
// and are waited for at the end of phase 4 s + 3, before their first use.
template <bool TRA, bool TRB, int MI, int NI, typename FA, typename FB>
__device__ __forceinline__ void product(char* smem, int nstage, FA&& abase, int64_t lda, int64_t acols, FB&& bbase,
                                        int64_t ldb, int64_t bcols, f32x16_t (&acc)[MI][NI]) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  using G = Waves<MI, NI>;
  const int grp = wv >> 2, wm = wv / G::GN, wn = wv % G::GN;
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
  if (nstage <= 0) return;
  uint32_t voff, rstride;
  if (grp == 0) {
    Operand<TRA> o;
    o.init(wv & 3, lane, lda, acols);
    voff = o.voff;
    rstride = o.rstride;
  } else {
    Operand<TRB> o;
    o.init(wv & 3, lane, ldb, bcols);
    voff = o.voff;
    rstride = o.rstride;
  }
  const int half = grp * kOperandB + (wv & 3) * 1024;
  auto stage_base = [&](int s) -> const char* {
    return reinterpret_cast<const char*>(grp == 0 ? abase(s) : bbase(s));
  };
  // run (wave % 4) + 4 p of a stage of this wave's operand
  auto load_run = [&](const char* src, int s, int p) {
    __builtin_amdgcn_global_load_lds(
        (MUONH_GLOBAL void*)(gmem(src + (int64_t)p * rstride) + voff),
        (__attribute__((address_space(3))) void*)(smem + (s & 1) * 2 * kOperandB + half + 4 * p * 1024), 16, 0, 0);
  };
  auto load_stage = [&](int s) {
    const char* src = stage_base(s);
#pragma unroll
    for (int p = 0; p < 8; ++p) load_run(src, s, p);
  };
  int xk[4];
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) xk[kk] = ((2 * kk + (lane >> 5)) ^ swz(lane & 31)) * 8;
  int ab[MI], bb[NI];
#pragma unroll
  for (int i = 0; i < MI; ++i) ab[i] = frag_base<TRA>(wm * G::WM + i * 32, lane);
#pragma unroll
  for (int j = 0; j < NI; ++j) bb[j] = frag_base<TRB>(wn * G::WN + j * 32, lane);
  bf16x8_t fa[2][MI], fb[2][NI];
  auto read_half = [&](int s, int h) {
    const uint16_t* sa = reinterpret_cast<const uint16_t*>(smem + (s & 1) * 2 * kOperandB);
    const uint16_t* sb = sa + kOperand;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int kk = 2 * h + q;
#pragma unroll
      for (int i = 0; i < MI; ++i) fa[q][i] = frag<TRA>(sa, ab[i], xk[kk], kk);
#pragma unroll
      for (int j = 0; j < NI; ++j) fb[q][j] = frag<TRB>(sb, bb[j], xk[kk], kk);
    }
  };
  // a half stage's 16 MFMAs, with this wave's loads of stage ls in between
  auto mma_half = [&](int ls) {
    const char* src = ls >= 0 ? stage_base(ls) : nullptr;
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int t = 0; t < 2 * MI * NI; ++t) {
      const int q = t / (MI * NI), i = (t / NI) % MI, j = t % NI;
      acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[q][i], fb[q][j], acc[i][j], 0, 0, 0);
      if (t & 1) {
        __builtin_amdgcn_sched_barrier(0);
        if (ls >= 0) load_run(src, ls, t / 2);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
  };
  load_stage(0);
  wait_loads();
  barrier();
  if (grp == 0) {
    for (int s = 0; s < nstage; ++s) {
      read_half(s, 0);                           // phase 4 s
      wait_lds();
      barrier();
      mma_half(s + 1 < nstage ? s + 1 : -1);     // phase 4 s + 1
      barrier();
      read_half(s, 1);                           // phase 4 s + 2
      wait_lds();
      barrier();
      mma_half(-1);                              // phase 4 s + 3
      wait_loads();
      barrier();
    }
  } else {
    for (int s = 0; s < nstage; ++s) {
      if (s > 0) mma_half(s + 1 < nstage ? s + 1 : -1);  // phase 4 s
      else if (nstage > 1) load_stage(1);
      barrier();
      read_half(s, 0);                           // phase 4 s + 1
      wait_lds();
      barrier();
      mma_half(-1);                              // phase 4 s + 2
      barrier();
      read_half(s, 1);                           // phase 4 s + 3
      wait_lds();
      wait_loads();
      barrier();
    }
    mma_half(-1);
  }
}

// Job order: hardware deals workgroups round-robin over the 8 XCDs; each XCD
// gets a contiguous run of the job list, whose neighbours share operand panels
// in its L2.
__device__ __forceinline__ int xcd_job(int bid, int njobs) {
  const int q = njobs / 8, rem = njobs % 8, xcd = bid % 8, loc = bid / 8;
  return xcd * q + min(xcd, rem) + loc;
}

// Job -> (row tile, column tile) with 8 row tiles at a time running over all
// columns, so that 32 neighbouring jobs form an 8 x 4 block.
__device__ __forceinline__ void block_order(int job, int nr, int nc, int& r, int& c) {
  const int per = 8 * nc, band = job / per;
  const int h = min(8, nr - band * 8), in = job - band * per;
  c = in / h;
  r = band * 8 + in - c * h;
}

// Address of row v of the weights; rows from full on are in the padded copy.
__device__ __forceinline__ const uint16_t* w_row(const uint16_t* w, const uint16_t* tail, int64_t full, int64_t ld,
                                                 int64_t v) {
  return v < full ? w + v * ld : tail + (v - full) * ld;
}

// ---------------------------------------------------------------------------
// logits of a 256-word x 256-token tile: statistics (first pass) or P
// ---------------------------------------------------------------------------
// Persistent: workgroup b takes every gridDim / 8-th job of its XCD's run.  The
// operand stages of all its tiles form one stream: while the last stage of a
// tile is multiplied, the first one of the next is already on its way, and the
// epilogues run with those loads in flight.  (One tile a workgroup: 8.6 us of
// launch, first load and epilogue beside 17 us of products at width 768.)
template <bool STATS>
__global__ __launch_bounds__(kXThreads) __attribute__((amdgpu_waves_per_eu(2))) void k_xent_logits(
    const XentArgs a, const XentPiece p, int nvoc) {
  constexpr int MI = 2, NI = 4, WM = Waves<MI, NI>::WM, WN = Waves<MI, NI>::WN;
  // operand stages, then (STATS) the maximum and sum of each token per row of
  // waves.  One array: with the latter in an array of its own, which the
  // compiler placed first, the kernel ran 10% longer.
  // For P the rest holds 4 KiB a wave (below).
  __shared__ __attribute__((aligned(16))) char smem[kXSmem + (STATS ? 4 * kXTile * (int)sizeof(float2) : 8 * 4096)];
  float2* const st = reinterpret_cast<float2*>(smem + kXSmem);
  const int count = a.sc->count;
  const int ntok = (count + kXTile - 1) / kXTile;
  const int njobs = ntok * nvoc;
  const int xcd = blockIdx.x % 8, step = gridDim.x / 8;
  const int q = njobs / 8, rem = njobs % 8;
  const int end = xcd * q + min(xcd, rem) + q + (xcd < rem ? 1 : 0);
  int job = xcd * q + min(xcd, rem) + (int)(blockIdx.x / 8);
  if (job >= end) return;

  const int tid = threadIdx.x, lane = tid & 63, hi = lane >> 5;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int grp = wv >> 2, wm = wv / Waves<MI, NI>::GN, wn = wv % Waves<MI, NI>::GN;
  const int nstage = (int)(a.wpad / kXStage);
  const int64_t ldw = a.ldw, ldx = a.wpad, full = a.wfull;
  const uint16_t *const w = a.w, *const tail = a.wtail, *const xp = a.xp;
  uint32_t voff, rstride;
  {
    Operand<false> o;
    o.init(wv & 3, lane, grp == 0 ? ldw : ldx, 0);
    voff = o.voff;
    rstride = __builtin_amdgcn_readfirstlane(o.rstride);
  }
  auto origin = [&](int j, int64_t& tok0, int64_t& v0) {
    int tt, tv;
    block_order(j, ntok, nvoc, tt, tv);
    tok0 = (int64_t)tt * kXTile;
    v0 = p.v0 + (int64_t)tv * kXTile;
  };
  // this wave's operand of a tile: words (waves 0-3) or tokens (4-7)
  auto source = [&](int64_t tok0, int64_t v0) -> const char* {
    return reinterpret_cast<const char*>(grp == 0 ? w_row(w, tail, full, ldw, v0) : xp + tok0 * ldx);
  };
  const int half = grp * kOperandB + (wv & 3) * 1024;
  // run r of a stage; src moves on to the next one
  auto load_run = [&](const char*& src, int buf, int r) {
    __builtin_amdgcn_global_load_lds(
        (MUONH_GLOBAL void*)(gmem(src) + voff),
        (__attribute__((address_space(3))) void*)(smem + buf * 2 * kOperandB + half + 4 * r * 1024), 16, 0, 0);
    src += rstride;
  };
  auto load_stage = [&](const char* src, int buf) {
#pragma unroll
    for (int r = 0; r < 8; ++r) load_run(src, buf, r);
  };
  int xk[4];
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) xk[kk] = ((2 * kk + hi) ^ swz(lane & 31)) * 8;
  int ab[MI], bb[NI];
#pragma unroll
  for (int i = 0; i < MI; ++i) ab[i] = frag_base<false>(wm * WM + i * 32, lane);
#pragma unroll
  for (int j = 0; j < NI; ++j) bb[j] = frag_base<false>(wn * WN + j * 32, lane);
  f32x16_t acc[MI][NI];
  bf16x8_t fa[2][MI], fb[2][NI];
  auto read_half = [&](int buf, int h) {
    const uint16_t* sa = reinterpret_cast<const uint16_t*>(smem + buf * 2 * kOperandB);
    const uint16_t* sb = sa + kOperand;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int i = 0; i < MI; ++i) fa[k][i] = frag<false>(sa, ab[i], xk[2 * h + k], 0);
#pragma unroll
      for (int j = 0; j < NI; ++j) fb[k][j] = frag<false>(sb, bb[j], xk[2 * h + k], 0);
    }
  };
  // a half stage's 16 MFMAs, LOAD: with this wave's loads of the next stage
  // (from src, into buffer buf) in between; FIRST: of a tile, from zero
  auto mma_half = [&](auto load_c, auto first_c, const char* src, int buf) {
    constexpr bool LOAD = decltype(load_c)::value, FIRST = decltype(first_c)::value;
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int t = 0; t < 2 * MI * NI; ++t) {
      const int k = t / (MI * NI), i = (t / NI) % MI, j = t % NI;
      acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[k][i], fb[k][j],
                                                          FIRST && k == 0 ? f32x16_t{} : acc[i][j], 0, 0, 0);
      if (t & 1) {
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (LOAD) load_run(src, buf, t / 2);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
  };

  // What becomes of a finished tile.
  auto epilogue = [&](int64_t tok0, int64_t v0) {
    const int64_t vw = v0 + wm * WM;                       // the wave's first word
    const int words = (int)max<int64_t>(0, min<int64_t>(WM, a.rows - vw));  // of them real
    // word of acc[i][.][v], counted from the lane's first one, vw + 4 hi
    auto word = [](int i, int v) { return i * 32 + 8 * (v >> 2) + (v & 3); };
    // the same count for a word t of the vocabulary; far outside for others
    auto rel = [&](int t) {
      const int64_t r = (int64_t)t - vw;
      return t >= 0 && r >= 0 && r < WM ? (int)r - 4 * hi : -64;
    };
    if (words < WM) {  // the last tile: words that are none get no weight
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int v = 0; v < 16; ++v)
            if (word(i, v) >= words - 4 * hi) acc[i][j][v] = -INFINITY;
    }
    if constexpr (STATS) {
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const int tl = wn * WN + j * 32 + (lane & 31);
        float m = acc[0][j][0];
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int v = 0; v < 16; ++v) m = fmaxf(m, acc[i][j][v]);
        m = fmaxf(m, __shfl_xor(m, 32, 64));
        const float mb = m == -INFINITY ? 0.f : m * kLog2e;  // nothing finite: the sum is 0
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int v = 0; v < 16; ++v) s += __builtin_amdgcn_exp2f(fmaf(acc[i][j][v], kLog2e, -mb));
        s += __shfl_xor(s, 32, 64);
        if (hi == 0) st[wm * kXTile + tl] = make_float2(m, s);
        // the target's logit, where this wave holds it
        const int64_t ci = tok0 + tl;
        const int t = rel(ci < count ? a.tgt[ci] : -1);
        if (__ballot(t != -64)) {
          float l = 0.f;
          bool have = false;
#pragma unroll
          for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int v = 0; v < 16; ++v) {
              l = word(i, v) == t ? acc[i][j][v] : l;
              have |= word(i, v) == t;
            }
          if (have) a.tlogit[ci] = l;
        }
      }
      lds_release();  // join() reads what other waves put into st
    } else {
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const int64_t ci = tok0 + wn * WN + j * 32 + (lane & 31);
        const int left = count - (int)tok0 - wn * WN - j * 32;  // tokens of these 32 rows
        const bool in = (lane & 31) < left;
        const float lb = in ? a.lse[ci] * kLog2e : 0.f;
        const int t = rel(in ? a.tgt[ci] : -1);
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[i][j][v] = __builtin_amdgcn_exp2f(fmaf(acc[i][j][v], kLog2e, -lb));
        // Rows of no token, in the last tile only, have weights of 0, also where
        // an infinite w makes their logits (0 times w) NaN.
        if (left < 32) {
#pragma unroll
          for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = in ? acc[i][j][v] : 0.f;
        }
        // - 1 at the target, where this wave holds any token's
        if (__ballot(t != -64)) {
#pragma unroll
          for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] -= word(i, v) == t ? 1.f : 0.f;
        }
        // Through LDS (chunks of 8 words, swizzled by token against bank
        // conflicts), so that every store covers whole 128-byte lines, and past
        // the caches, which P (up to 512 MiB) would only sweep: at 8192 tokens,
        // 50257 words, width 768 this kernel takes 631 us, with stores of 32
        // bytes a row 682; the products that read P 1183, 1267.  (The same for
        // dw and dx's sums gained nothing.)
        char* const own = smem + kXSmem + wv * 4096;
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int pq = 0; pq < 2; ++pq) {
            const f32x16_t e = acc[i][j];
            const int o = 8 * pq;
            // lanes l and l + 32 trade groups: each then holds 8 consecutive words
            const uint32_t w0 = pack_bf16x2(e[o], e[o + 1]), w1 = pack_bf16x2(e[o + 2], e[o + 3]);
            const uint32_t w2 = pack_bf16x2(e[o + 4], e[o + 5]), w3 = pack_bf16x2(e[o + 6], e[o + 7]);
            const auto s0 = __builtin_amdgcn_permlane32_swap(w0, w2, false, false);
            const auto s1 = __builtin_amdgcn_permlane32_swap(w1, w3, false, false);
            const u32x4_t pk = {s0[0], s1[0], s0[1], s1[1]};
            const int r = lane & 31, c = 4 * i + 2 * pq + hi;
            *reinterpret_cast<u32x4_t*>(own + r * 128 + ((c ^ (r & 7)) * 16)) = pk;
          }
        wave_fence();
        uint16_t* const block = a.prob + (tok0 + wn * WN + j * 32) * p.cols + (vw - p.v0);
        u32x4_t line[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = 8 * q + (lane >> 3), c = lane & 7;
          line[q] = *reinterpret_cast<const u32x4_t*>(own + r * 128 + ((c ^ (r & 7)) * 16));
        }
        wave_fence();  // before the next 32 tokens' values
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = 8 * q + (lane >> 3), c = lane & 7;
          __builtin_nontemporal_store(line[q], reinterpret_cast<MUONH_GLOBAL u32x4_t*>(gmem(block + r * p.cols + c * 8)));
        }
      }
    }
  };
  // Joins the four rows of waves of a tile, a barrier after its epilogue: one
  // token a thread of waves 4-7.
  auto join = [&](int64_t tok0, int64_t v0) {
    if constexpr (STATS) {
      lds_acquire();
      const int t = tid & (kXTile - 1);
      float m = st[t].x;
#pragma unroll
      for (int k = 1; k < 4; ++k) m = fmaxf(m, st[k * kXTile + t].x);
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 r = st[k * kXTile + t];
        s += r.x == -INFINITY ? r.y : r.y * __builtin_amdgcn_exp2f((r.x - m) * kLog2e);
      }
      a.stats[(v0 / kXTile) * a.npad + tok0 + t] = make_float2(m, s);
    }
  };

  int64_t tok0, v0, ntok0 = 0, nv0 = 0;
  origin(job, tok0, v0);
  const char* src = source(tok0, v0);
  // After its last tile a workgroup loads that tile's first stage once more,
  // to no use, which keeps the loop free of branches around the loads.
  const char* nsrc;
  const std::true_type load{}, first{};
  const std::false_type no_load{}, more{};
  load_stage(src, 0);
  wait_loads();
  barrier();
  int buf = 0;
  // phases of a stage as in product(); a barrier ends each
  if (grp == 0) {
    for (;;) {
      const int next = job + step;
      nsrc = src;
      if (next < end) {
        origin(next, ntok0, nv0);
        nsrc = source(ntok0, nv0);
      }
      for (int s = 0; s < nstage; ++s) {
        read_half(buf, 0);
        wait_lds();
        barrier();
        const char* const ld = s + 1 < nstage ? src + (s + 1) * (kXStage * 2) : nsrc;
        if (s == 0) mma_half(load, first, ld, buf ^ 1);
        else mma_half(load, more, ld, buf ^ 1);
        barrier();
        read_half(buf, 1);
        wait_lds();
        barrier();
        mma_half(no_load, more, src, 0);
        wait_loads();
        barrier();
        buf ^= 1;
      }
      epilogue(tok0, v0);
      if (next >= end) break;
      job = next;
      tok0 = ntok0;
      v0 = nv0;
      src = nsrc;
    }
    if constexpr (STATS) __syncthreads();
  } else {
    int64_t ptok0 = -1, pv0 = 0;  // the tile before, whose last MFMAs and epilogue fall into this one's first phase
    for (;;) {
      const int next = job + step;
      nsrc = src;
      if (next < end) {
        origin(next, ntok0, nv0);
        nsrc = source(ntok0, nv0);
      }
      for (int s = 0; s < nstage; ++s) {
        const char* const ld = s + 1 < nstage ? src + (s + 1) * (kXStage * 2) : nsrc;
        if (s > 0 || ptok0 >= 0) mma_half(load, more, ld, buf ^ 1);
        else load_stage(ld, buf ^ 1);
        if (s == 0 && ptok0 >= 0) epilogue(ptok0, pv0);
        barrier();
        if (s == 0 && ptok0 >= 0) join(ptok0, pv0);
        __builtin_amdgcn_sched_barrier(0);
        read_half(buf, 0);
        wait_lds();
        barrier();
        if (s == 0) mma_half(no_load, first, src, 0);
        else mma_half(no_load, more, src, 0);
        barrier();
        read_half(buf, 1);
        wait_lds();
        wait_loads();
        barrier();
        buf ^= 1;
      }
      ptok0 = tok0;
      pv0 = v0;
      if (next >= end) break;
      job = next;
      tok0 = ntok0;
      v0 = nv0;
      src = nsrc;
    }
    mma_half(no_load, more, src, 0);
    epilogue(ptok0, pv0);
    if constexpr (STATS) {
      __syncthreads();
      join(ptok0, pv0);
    }
  }
}

// ---------------------------------------------------------------------------
// gradients of one piece: ndw jobs are dw tiles (256 of width x 256 words,
// depth = tokens), ndx dx tiles (256 of width x 256 tokens, depth = one split
// of the piece's words); the kind with the longer jobs starts
// ---------------------------------------------------------------------------
template <typename WT>
__global__ __launch_bounds__(kXThreads) __attribute__((amdgpu_waves_per_eu(2))) void k_xent_grad(
    const XentArgs a, const XentPiece p, int ndw, int ndx, int nd) {
  __shared__ __attribute__((aligned(16))) char smem[kXSmem];
  const int count = a.sc->count;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int hi = lane >> 5;
  const bool is_dw = p.dx_first ? (int)blockIdx.x >= ndx : (int)blockIdx.x < ndw;
  const int job0 = (int)blockIdx.x - (is_dw == (p.dx_first != 0) ? (is_dw ? ndx : ndw) : 0);
  if (is_dw) {
    constexpr int MI = 4, NI = 2, WM = Waves<MI, NI>::WM, WN = Waves<MI, NI>::WN;
    const int wm = wave / Waves<MI, NI>::GN, wn = wave % Waves<MI, NI>::GN;
    f32x16_t acc[MI][NI];
    int tv, td;
    block_order(xcd_job(job0, ndw), nd, ndw / nd, td, tv);
    const int64_t d0 = (int64_t)td * kXTile, vl = (int64_t)tv * kXTile;  // word in the piece
    const uint16_t* const xt = a.xt + d0 * a.ldxt;
    const uint16_t* const pt = a.prob + vl;
    const int64_t ldp = p.cols;
    product<false, true, MI, NI>(
        smem, (count + kXStage - 1) / kXStage, [=](int s) { return xt + s * kXStage; }, a.ldxt, 0,
        [=](int s) { return pt + (int64_t)s * kXStage * ldp; }, ldp, ldp - vl, acc);
    const float g = a.sc->gscale;
    WT* const dw = reinterpret_cast<WT*>(a.dw);
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int64_t v = p.v0 + vl + wn * WN + j * 32 + (lane & 31);
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int pq = 0; pq < 2; ++pq) {
          float e[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(acc[i][j][8 * pq + k] * g),
                                                             __float_as_uint(acc[i][j][8 * pq + 4 + k] * g), false, false);
            e[k] = __uint_as_float(sw[0]);
            e[4 + k] = __uint_as_float(sw[1]);
          }
          const int64_t d = d0 + wm * WM + i * 32 + 16 * pq + 8 * hi;
          if (v >= a.rows || d >= a.width) continue;
          const int64_t at = v * a.width + d;
          if (d + 8 <= a.width) {
            if (a.accumulate) {
              float old[8];
              load8_any(dw, at, old);
#pragma unroll
              for (int k = 0; k < 8; ++k) e[k] += old[k];
            }
            store8_any(dw, at, e);
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (d + k < a.width) St<WT>::st(dw, at + k, a.accumulate ? e[k] + St<WT>::ld(dw, at + k) : e[k]);
          }
        }
    }
    return;
  }
  constexpr int MI = 2, NI = 4, WM = Waves<MI, NI>::WM, WN = Waves<MI, NI>::WN;
  const int wm = wave / Waves<MI, NI>::GN, wn = wave % Waves<MI, NI>::GN;
  f32x16_t acc[MI][NI];
  const int job = xcd_job(job0, ndx);
  const int per = ndx / p.splits, split = job / per;
  int tt, td;
  block_order(job - split * per, nd, per / nd, td, tt);
  const int64_t tok0 = (int64_t)tt * kXTile, d0 = (int64_t)td * kXTile;
  if (tok0 >= count) return;
  // this split's stages of the piece
  const int64_t all = p.cols / kXStage;
  const int s0 = (int)(all * split / p.splits), s1 = (int)(all * (split + 1) / p.splits);
  const uint16_t* const pt = a.prob + tok0 * p.cols + (int64_t)s0 * kXStage;
  const uint16_t *const w = a.w + d0, *const tail = a.wtail + d0;
  const int64_t ldw = a.ldw, full = a.wfull, vs = p.v0 + (int64_t)s0 * kXStage;
  product<true, false, MI, NI>(
      smem, s1 - s0, [=](int s) { return w_row(w, tail, full, ldw, vs + (int64_t)s * kXStage); }, ldw, a.wpad - d0,
      [=](int s) { return pt + (int64_t)s * kXStage; }, p.cols, 0, acc);
  float* const out = a.dxacc + (int64_t)split * a.npad * a.wpad;
#pragma unroll
  for (int j = 0; j < NI; ++j) {
    const int64_t ci = tok0 + wn * WN + j * 32 + (lane & 31);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t d = d0 + wm * WM + i * 32 + 8 * q + 4 * hi;
        if (d >= a.wpad || ci >= count) continue;  // 64 tokens, 50257 x 768: 134 -> 127 us a call
        f32x4_t e = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        MUONH_GLOBAL f32x4_t* const o = reinterpret_cast<MUONH_GLOBAL f32x4_t*>(gmem(out + ci * a.wpad + d));
        if (!p.first) e += *o;
        *o = e;
      }
  }
}

// ---------------------------------------------------------------------------
// around the products
// ---------------------------------------------------------------------------
__device__ __forceinline__ int64_t target_of(const XentArgs& a, int64_t i) {
  return a.id_bits == 32 ? (int64_t)gmem(reinterpret_cast<const int32_t*>(a.targets))[i]
                         : gmem(reinterpret_cast<const int64_t*>(a.targets))[i];
}
__device__ __forceinline__ bool counted(const XentArgs& a, int64_t t) {
  return t >= 0 && t < a.rows && t != a.ignore_index;
}
__device__ __forceinline__ void put_scalars(const XentArgs& a, int64_t count) {
  const double c = a.mean ? 1.0 / (double)max<int64_t>(count, 1) : 1.0;
  a.sc->count = (int32_t)count;
  a.sc->gscale = (float)(c * (double)a.grad_scale);
}

// One workgroup: the list of counted tokens in batch order, and the factors.
constexpr int kIndexThreads = 1024;
__global__ __launch_bounds__(kIndexThreads) void k_xent_index(const XentArgs a) {
  __shared__ int32_t wsum[kIndexThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int PER = 8;  // 64-token rows of a wave, all its loads in flight together
  int64_t base = 0;
  for (int64_t i0 = 0; i0 < a.n; i0 += kIndexThreads * PER) {
    const int64_t w0 = i0 + wave * (64 * PER) + lane;
    int64_t t[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int64_t i = min(w0 + 64 * k, a.n - 1);
      t[k] = target_of(a, i);
    }
    uint64_t in[PER];
    int mine = 0;  // of the wave
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int64_t i = w0 + 64 * k;
      const bool ok = i < a.n && counted(a, t[k]);
      in[k] = __ballot(ok);
      mine += __popcll(in[k]);
      if (i < a.n && !ok && a.token_loss != nullptr) a.token_loss[i] = 0.f;
    }
    if (lane == 0) wsum[wave] = mine;
    __syncthreads();
    int64_t at = base;
    int total = 0;
#pragma unroll
    for (int w = 0; w < kIndexThreads / 64; ++w) {
      if (w < wave) at += wsum[w];
      total += wsum[w];
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      if ((in[k] >> lane) & 1) {
        const int64_t to = at + __popcll(in[k] & ((1ull << lane) - 1));
        a.perm[to] = (int32_t)(w0 + 64 * k);
        a.tgt[to] = (int32_t)t[k];
      }
      at += __popcll(in[k]);
    }
    base += total;
    __syncthreads();
  }
  if (tid == 0) put_scalars(a, base);
}

// Rows of `width` values copied to rows of `ld`, zero padded: element e of an
// 8-element chunk past the row or its end is 0.
__device__ __forceinline__ void copy_chunk(const uint16_t* src, bool row_ok, int64_t width, int64_t col,
                                           uint16_t* dst) {
  u32x4_t q = {0u, 0u, 0u, 0u};
  if (row_ok) {
    if (col + 8 <= width) {
      q = *reinterpret_cast<const MUONH_GLOBAL u32x4_u*>(gmem(src + col));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t v = col + e < width ? (uint32_t)gmem(src)[col + e] : 0u;
        q[e / 2] |= v << (16 * (e & 1));
      }
    }
  }
  *reinterpret_cast<MUONH_GLOBAL u32x4_t*>(gmem(dst + col)) = q;
}

// Blocks [0, npad): one row of xp each (counted tokens of x, then zeros); the
// others: chunks of the padded copy of the weights, wrows rows from row w0 on.  LIST: up
// to kXListTokens tokens, where every block finds its token itself and the
// first one writes the list, which saves k_xent_index.
constexpr int kCopyPer = 4;
template <bool LIST>
__global__ __launch_bounds__(256) void k_xent_gather(const XentArgs a, const uint16_t* w_in, uint16_t* w_out,
                                                     int64_t w0, int64_t wrows) {
  const int64_t b = blockIdx.x;
  if (b < a.npad) {
    bool ok;
    int64_t token;
    if constexpr (LIST) {
      constexpr int PER = (int)(kXListTokens / 256);
      __shared__ int32_t part[4];
      __shared__ int32_t mine;
      const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
      const int i0 = wave * 64 * PER + lane;
      int64_t t[PER];
      uint64_t in[PER];
      int sum = 0;
#pragma unroll
      for (int k = 0; k < PER; ++k) t[k] = i0 + 64 * k < a.n ? target_of(a, i0 + 64 * k) : -1;
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        in[k] = __ballot(i0 + 64 * k < a.n && counted(a, t[k]));
        sum += __popcll(in[k]);
      }
      if (lane == 0) part[wave] = sum;
      __syncthreads();
      int at = 0, count = 0;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        if (w < wave) at += part[w];
        count += part[w];
      }
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const int i = i0 + 64 * k, to = at + __popcll(in[k] & ((1ull << lane) - 1));
        if ((in[k] >> lane) & 1) {
          if (to == b) mine = i;
          if (b == 0) {
            a.perm[to] = i;
            a.tgt[to] = (int32_t)t[k];
          }
        } else if (b == 0 && i < a.n && a.token_loss != nullptr) {
          a.token_loss[i] = 0.f;
        }
        at += __popcll(in[k]);
      }
      if (b == 0 && threadIdx.x == 0) put_scalars(a, count);
      __syncthreads();
      ok = b < count;
      token = ok ? mine : 0;
    } else {
      ok = b < a.sc->count;
      token = ok ? a.perm[b] : 0;
    }
    const uint16_t* const src = a.x + token * a.width;
    for (int64_t c = threadIdx.x * 8; c < a.wpad; c += 256 * 8) copy_chunk(src, ok, a.width, c, a.xp + b * a.wpad);
    return;
  }
  // kCopyPer chunks of 8 values a thread (a block a row took 63 us for 140788 x
  // 103, this 16); a block's first row comes from one 64-bit division, a thread's
  // from a 32-bit one
  const uint32_t cpr = (uint32_t)(a.wpad / 8);
  for (int64_t i0 = (b - a.npad) * (256 * kCopyPer); i0 < wrows * cpr;
       i0 += (int64_t)(gridDim.x - a.npad) * (256 * kCopyPer)) {
    const int64_t row0 = i0 / cpr;
    const uint32_t off0 = (uint32_t)(i0 - row0 * cpr);
#pragma unroll
    for (int k = 0; k < kCopyPer; ++k) {
      const uint32_t x = off0 + threadIdx.x + 256 * k, q = x / cpr;
      const int64_t r = row0 + q, v = w0 + r;
      if (r < wrows)
        copy_chunk(w_in + min(v, a.rows - 1) * a.width, v < a.rows, a.width, 8 * (int64_t)(x - q * cpr),
                   w_out + r * a.wpad);
    }
  }
}

// xt = xp transposed, 64 x 64 values a block.
__global__ __launch_bounds__(256) void k_xent_transpose(const XentArgs a) {
  __shared__ uint16_t t[64][72];
  const int64_t r0 = (int64_t)blockIdx.x * 64, c0 = (int64_t)blockIdx.y * 64;
  if (r0 >= a.sc->count) return;  // dw reads no further than the counted tokens' last stage
  const int r = threadIdx.x >> 3, c = (threadIdx.x & 7) * 8;
#pragma unroll
  for (int k = 0; k < 2; ++k)
    *reinterpret_cast<u32x4_t*>(&t[r + 32 * k][c]) =
        *reinterpret_cast<const MUONH_GLOBAL u32x4_t*>(gmem(a.xp + (r0 + r + 32 * k) * a.wpad + c0 + c));
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    u32x4_t q;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      q[e] = (uint32_t)t[c + 2 * e][r + 32 * k] | (uint32_t)t[c + 2 * e + 1][r + 32 * k] << 16;
    *reinterpret_cast<MUONH_GLOBAL u32x4_t*>(gmem(a.xt + (c0 + r + 32 * k) * a.ldxt + r0 + c)) = q;
  }
}

// lse and loss of a counted token from its tiles' statistics.  32 tokens by 8
// threads each; every thread of the workgroup calls it (ci may be past the
// tokens).  The thread with part 0 returns the loss.
__device__ __forceinline__ float token_lse(const XentArgs& a, int64_t ci, int count, int part, int tl,
                                           float2 (*sh)[32]) {
  const int64_t tiles = a.rpad / kXTile;
  float m = -INFINITY, s = 0.f;
  constexpr int U = 8;  // tiles in flight
  if (ci < count)
    for (int64_t k0 = part; k0 < tiles; k0 += 8 * U) {
      float2 q[U];
#pragma unroll
      for (int u = 0; u < U; ++u) q[u] = a.stats[min(k0 + 8 * u, tiles - 1) * a.npad + ci];
      float nm = m;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (k0 + 8 * u >= tiles) q[u] = make_float2(-INFINITY, 0.f);
        nm = fmaxf(nm, q[u].x);
      }
      // nothing finite so far: the sums are 0, or a NaN to pass on
      const float b = nm == -INFINITY ? 0.f : nm;
      s *= __builtin_amdgcn_exp2f((m - b) * kLog2e);
#pragma unroll
      for (int u = 0; u < U; ++u)
        s += q[u].x == -INFINITY ? q[u].y : q[u].y * __builtin_amdgcn_exp2f((q[u].x - b) * kLog2e);
      m = nm;
    }
  sh[part][tl] = make_float2(m, s);
  __syncthreads();
  float loss = 0.f;
  if (part == 0 && ci < count) {
    float mm = sh[0][tl].x;
#pragma unroll
    for (int k = 1; k < 8; ++k) mm = fmaxf(mm, sh[k][tl].x);
    double t = 0.0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 q = sh[k][tl];
      t += q.x == -INFINITY ? (double)q.y : (double)q.y * (double)__builtin_amdgcn_exp2f((q.x - mm) * kLog2e);
    }
    const float l = mm + logf((float)t);
    a.lse[ci] = l;
    loss = l - a.tlogit[ci];
    if (a.token_loss != nullptr) a.token_loss[a.perm[ci]] = loss;
  }
  __syncthreads();
  return loss;
}

// The loss from each thread's sum, in a fixed order.
__device__ __forceinline__ void put_loss(const XentArgs& a, double s, int count) {
  __shared__ double red[16];
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double v = 0.0;
#pragma unroll
    for (int k = 0; k < 16; ++k) v += red[k];
    a.loss[0] = (float)(a.mean ? v / (double)max(count, 1) : v);
  }
}

__global__ __launch_bounds__(256) void k_xent_lse(const XentArgs a) {
  __shared__ float2 sh[8][32];
  const int count = a.sc->count;
  if ((int64_t)blockIdx.x * 32 >= count) return;
  const int tl = threadIdx.x & 31, part = threadIdx.x >> 5;
  const int64_t ci = (int64_t)blockIdx.x * 32 + tl;
  const float loss = token_lse(a, ci, count, part, tl, sh);
  if (part == 0 && ci < count) a.tlogit[ci] = loss;  // summed by k_xent_total
}

__global__ __launch_bounds__(1024) void k_xent_total(const XentArgs a) {
  const int count = a.sc->count;
  double s = 0.0;
  for (int i = threadIdx.x; i < count; i += 1024) s += (double)a.tlogit[i];
  put_loss(a, s, count);
}

// Both in one workgroup, 128 tokens at a time, for few statistics (below
// kXSoloStats): one launch instead of two.
__global__ __launch_bounds__(1024) void k_xent_loss(const XentArgs a) {
  __shared__ float2 sh[4][8][32];
  const int count = a.sc->count;
  const int tl = threadIdx.x & 31, part = (threadIdx.x >> 5) & 7, g = threadIdx.x >> 8;
  double s = 0.0;
  for (int64_t c0 = 0; c0 < count; c0 += 128) s += (double)token_lse(a, c0 + 32 * g + tl, count, part, tl, sh[g]);
  put_loss(a, s, count);
}

// dx: the splits' sums in order, scaled and rounded; ignored tokens get zeros.
// Block b < npad handles row b of dxacc; the row of an ignored token is
// written by the blocks after them, one a token.
__global__ __launch_bounds__(256) void k_xent_dx(const XentArgs a, int splits) {
  const int64_t b = blockIdx.x;
  const int count = a.sc->count;
  int64_t token;
  bool zero = false;
  if (b < a.n) {  // rows of dxacc
    if (b >= count) return;
    token = a.perm[b];
  } else {
    token = b - a.n;
    if (counted(a, target_of(a, token))) return;
    zero = true;
  }
  const float g = a.sc->gscale;
  for (int64_t c = threadIdx.x * 8; c < a.width; c += 256 * 8) {
    float e[8] = {};
    if (!zero) {
      constexpr int U = 8;  // parts in flight
      int k = 0;
      for (; k + U <= splits; k += U) {
        float q[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) load8(a.dxacc, ((int64_t)(k + u) * a.npad + b) * a.wpad + c, q[u]);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int x = 0; x < 8; ++x) e[x] += q[u][x];
      }
      for (; k < splits; ++k) {
        float q[8];
        load8(a.dxacc, ((int64_t)k * a.npad + b) * a.wpad + c, q);
#pragma unroll
        for (int x = 0; x < 8; ++x) e[x] += q[x];
      }
#pragma unroll
      for (int x = 0; x < 8; ++x) e[x] *= g;
    }
    const int64_t at = token * a.width + c;
    if (c + 8 <= a.width) store8_any(a.dx, at, e);
    else
      for (int x = 0; x < 8; ++x)
        if (c + x < a.width) St<bf16_t>::st(a.dx, at + x, e[x]);
  }
}

// ---------------------------------------------------------------------------
// few tokens, loss only: up to kXFewTokens
// ---------------------------------------------------------------------------
// Tiles of 256 tokens would be nearly empty, and the time is that of reading w
// once.  Here a wave is a workgroup and takes 64 words and 32 NT tokens at a
// time.  It reads whole 128-byte runs of rows, at any alignment (w needs no
// padded copy), two stages of 64 values ahead into registers, and passes them through
// its own LDS to the fragments' layout: nothing waits for another wave.  Bound
// by HBM: 17 us for 50257 x 768 (4.6 TB/s).  Reads straight into the fragments'
// layout (32 rows an instruction), the depth split over four waves: 32 tokens 34
// us a call against 25, at 151936 x 2048 234 against 140.
// A token stands in its own column, so what an uncounted one holds stays there.
// What a sum of exponents is multiplied by when its maximum m becomes nm >= m:
// exactly 1 where it stays, so that the rounds of a long vocabulary add up no
// error.  (With the rounded nm log2(e) subtracted from the exact m log2(e), each
// round lost up to 1.3e-6 at logits below 44: 1.5e-4 of a loss over 64 rounds.)
// Nothing finite so far: the sum is 0, or a NaN to pass on.
__device__ __forceinline__ float rescale(float m, float nm) {
  return __builtin_amdgcn_exp2f((m - (nm == -INFINITY ? 0.f : nm)) * kLog2e);
}

template <int NT>
__global__ __launch_bounds__(64) __attribute__((amdgpu_waves_per_eu(2))) void k_xent_few(const XentArgs a,
                                                                                         int blocks) {
  constexpr int MW = kXFewWords / 32, RW = kXFewWords / 8, RT = 4 * NT;  // runs of 8 rows of a stage
  __shared__ __attribute__((aligned(16))) uint16_t tile[(kXFewWords + 32 * NT) * kXStage];
  const int lane = threadIdx.x, hi = lane >> 5;
  const int64_t units = (a.width + kXStage - 1) / kXStage;
  const int64_t tiles = (a.rows + kXFewWords - 1) / kXFewWords;
  const int64_t mine = (tiles - (int64_t)blockIdx.x + blocks - 1) / blocks;
  const int64_t stages = mine * units;
  // 8 lanes a row; a lane's chunk of 8 values, as swizzled in LDS
  const int r8 = lane >> 3;
  int col[2];  // chunks of even and odd runs differ: swz of rows 8 apart
#pragma unroll
  for (int e = 0; e < 2; ++e) col[e] = 8 * ((lane & 7) ^ swz(8 * e + r8));
  uint32_t offw[RW], offt[RT];  // of the rows, from their tile's first one, in elements
#pragma unroll
  for (int p = 0; p < RT; ++p) offt[p] = (uint32_t)(min<int64_t>(8 * p + r8, a.n - 1) * a.width);
  // the next stage to load
  int64_t lv = (int64_t)blockIdx.x * kXFewWords, lu = 0;
  auto rows_of = [&]() {
#pragma unroll
    for (int p = 0; p < RW; ++p) offw[p] = (uint32_t)((min<int64_t>(lv + 8 * p + r8, a.rows - 1) - lv) * a.width);
  };
  rows_of();
  struct Stage {
    u32x4_t w[RW], t[RT];
  };
  // A lane's chunk that ends behind its row is read from the row's end, and
  // moved into place before it is used.
  auto fetch = [&](Stage& q) {
    const int64_t c = lu * kXStage;
    const int last = (int)min<int64_t>(a.width - c, kXStage) - 8;  // may be below 0: widths are 8 at least
    const uint16_t* const bw = a.w + lv * a.width + c;
    const uint16_t* const bt = a.x + c;
    const int c0 = min(col[0], last), c1 = min(col[1], last);
#pragma unroll
    for (int p = 0; p < RW; ++p)
      q.w[p] = *reinterpret_cast<const MUONH_GLOBAL u32x4_u*>(gmem(bw) + ((int64_t)offw[p] + (p & 1 ? c1 : c0)));
#pragma unroll
    for (int p = 0; p < RT; ++p)
      q.t[p] = *reinterpret_cast<const MUONH_GLOBAL u32x4_u*>(gmem(bt) + ((int64_t)offt[p] + (p & 1 ? c1 : c0)));
    // on to the next; after the last one the first of this tile again, to no use
    if (++lu == units) {
      lu = 0;
      if (lv + (int64_t)blocks * kXFewWords < a.rows) {
        lv += (int64_t)blocks * kXFewWords;
        rows_of();
      }
    }
  };
  int64_t t[NT];
  float m[NT], s[NT];  // running maximum and sum of this lane's words, by token
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int token = 32 * j + (lane & 31);
    t[j] = token < a.n ? target_of(a, token) : -1;
    m[j] = -INFINITY;
    s[j] = 0.f;
  }
  f32x16_t acc[NT][MW];
  int64_t v0 = lv, u = 0;  // the stage in hand
  const int short_last = (int)(a.width - (units - 1) * kXStage) - 8;  // of the last stage
  auto shift = [](u32x4_t& q, int by) {  // by values down, zeros from above; by = 8: all zeros
    uint64_t lo = (uint64_t)q[1] << 32 | q[0], up = (uint64_t)q[3] << 32 | q[2];
    const int b = 16 * (by & 3);
    if (by >= 4) {
      lo = by >= 8 ? 0 : up >> b;
      up = 0;
    } else if (by > 0) {
      lo = lo >> b | up << (64 - b);
      up >>= b;
    }
    q = u32x4_t{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)up, (uint32_t)(up >> 32)};
  };
  auto work = [&](Stage& q, bool ahead) {
    if (u == units - 1 && short_last < kXStage - 8) {
      const int by0 = min(max(col[0] - short_last, 0), 8), by1 = min(max(col[1] - short_last, 0), 8);
#pragma unroll
      for (int p = 0; p < RW; ++p) shift(q.w[p], p & 1 ? by1 : by0);
#pragma unroll
      for (int p = 0; p < RT; ++p) shift(q.t[p], p & 1 ? by1 : by0);
    }
    wave_fence();
#pragma unroll
    for (int p = 0; p < RW; ++p) *reinterpret_cast<u32x4_t*>(tile + p * 512 + lane * 8) = q.w[p];
#pragma unroll
    for (int p = 0; p < RT; ++p) *reinterpret_cast<u32x4_t*>(tile + (RW + p) * 512 + lane * 8) = q.t[p];
    wave_fence();
    if (ahead) fetch(q);
    if (u == 0) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < MW; ++i) acc[j][i] = f32x16_t{};
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int xk = ((2 * k + hi) ^ swz(lane & 31)) * 8;
      bf16x8_t fa[MW], fb[NT];
#pragma unroll
      for (int i = 0; i < MW; ++i) fa[i] = frag<false>(tile, frag_base<false>(32 * i, lane), xk, 0);
#pragma unroll
      for (int j = 0; j < NT; ++j) fb[j] = frag<false>(tile, frag_base<false>(kXFewWords + 32 * j, lane), xk, 0);
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < MW; ++i)
          acc[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[i], fb[j], acc[j][i], 0, 0, 0);
    }
    if (++u < units) return;
    // the tile's logits are complete
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int token = 32 * j + (lane & 31);
      const int64_t tr = t[j] - v0 - 4 * hi;  // the target, counted as below
      const int own = tr >= 0 && tr < kXFewWords ? (int)tr : -1;
      const int words = (int)min<int64_t>(a.rows - v0, kXFewWords) - 4 * hi;
      float nm = m[j];
#pragma unroll
      for (int i = 0; i < MW; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int word = 32 * i + 8 * (v >> 2) + (v & 3);
          if (word >= words) acc[j][i][v] = -INFINITY;
          if (word == own) a.tlogit[token] = acc[j][i][v];
          nm = fmaxf(nm, acc[j][i][v]);
        }
      // nothing finite so far: the sums are 0, or a NaN to pass on
      const float b = nm == -INFINITY ? 0.f : nm * kLog2e;
      float part = 0.f;  // of this tile: small terms are not lost one by one in the running sum
#pragma unroll
      for (int i = 0; i < MW; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) part += __builtin_amdgcn_exp2f(fmaf(acc[j][i][v], kLog2e, -b));
      s[j] = fmaf(s[j], rescale(m[j], nm), part);
      m[j] = nm;
    }
    u = 0;
    v0 += (int64_t)blocks * kXFewWords;
  };
  Stage q0;
  fetch(q0);
  if constexpr (NT == 1) {
    Stage q1;
    fetch(q1);
    for (int64_t g = 0; g < stages; g += 2) {
      work(q0, g + 2 < stages);
      if (g + 1 < stages) work(q1, g + 3 < stages);
    }
  } else {  // registers for one stage ahead
    for (int64_t g = 0; g < stages; ++g) work(q0, g + 1 < stages);
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int token = 32 * j + (lane & 31);
    const float m1 = __shfl_xor(m[j], 32, 64), s1 = __shfl_xor(s[j], 32, 64);
    const float mm = fmaxf(m[j], m1), sum = s[j] * rescale(m[j], mm) + s1 * rescale(m1, mm);
    if (hi == 0 && token < a.n) a.stats[(int64_t)token * blocks + blockIdx.x] = make_float2(mm, sum);
  }
}

// Their losses, a wave a token.
__global__ __launch_bounds__(1024) void k_xent_few_loss(const XentArgs a, int blocks) {
  __shared__ double red[16];
  __shared__ int cnt[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double sum = 0.0;
  int count = 0;
  for (int token = wave; token < a.n; token += 16) {
    if (!counted(a, target_of(a, token))) {
      if (lane == 0 && a.token_loss != nullptr) a.token_loss[token] = 0.f;
      continue;
    }
    const float tl = a.tlogit[token];
    float m = -INFINITY, s = 0.f;
    constexpr int U = 8;  // statistics in flight, a lane
    for (int b0 = lane; b0 - lane < blocks; b0 += 64 * U) {
      float2 q[U];
#pragma unroll
      for (int u = 0; u < U; ++u) q[u] = a.stats[(int64_t)token * blocks + min(b0 + 64 * u, blocks - 1)];
      float nm = m;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (b0 + 64 * u >= blocks) q[u] = make_float2(-INFINITY, 0.f);
        nm = fmaxf(nm, q[u].x);
      }
      s *= rescale(m, nm);
#pragma unroll
      for (int u = 0; u < U; ++u) s += q[u].y * rescale(q[u].x, nm);
      m = nm;
    }
    float top = m;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    s *= rescale(m, top);
    m = top;
    const double all = wave_sum((double)s);
    const float loss = m + logf((float)all) - tl;
    if (lane == 0 && a.token_loss != nullptr) a.token_loss[token] = loss;
    sum += (double)loss;
    ++count;
  }
  if (lane == 0) {
    red[wave] = sum;
    cnt[wave] = count;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    double v = 0.0;
    int c = 0;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      v += red[k];
      c += cnt[k];
    }
    a.loss[0] = (float)(a.mean ? v / (double)max(c, 1) : v);
  }
}

}  // namespace

hipError_t launch_xent_prepare(const XentArgs& a, bool copy_w, const uint16_t* w_in, hipStream_t s) {
  const bool list = a.n <= kXListTokens;
  if (!list) hipLaunchKernelGGL(k_xent_index, dim3(1), dim3(kIndexThreads), 0, s, a);
  // the whole of w where its rows are no operand as they stand, else its last tile
  const int64_t w0 = copy_w ? 0 : a.wfull;
  uint16_t* const w_out = const_cast<uint16_t*>(copy_w ? a.w : a.wtail);
  const int64_t wrows = copy_w ? a.rpad : a.rpad - a.wfull;
  const int64_t copies = (wrows * (a.wpad / 8) + 256 * kCopyPer - 1) / (256 * kCopyPer);
  const dim3 grid(a.npad + (copies < (1 << 20) ? copies : 1 << 20));
  if (list) hipLaunchKernelGGL(k_xent_gather<true>, grid, dim3(256), 0, s, a, w_in, w_out, w0, wrows);
  else hipLaunchKernelGGL(k_xent_gather<false>, grid, dim3(256), 0, s, a, w_in, w_out, w0, wrows);
  if (a.dw != nullptr)
    hipLaunchKernelGGL(k_xent_transpose, dim3(a.npad / 64, a.wpad / 64), dim3(256), 0, s, a);
  return hipGetLastError();
}

// Persistent workgroups of the logits kernels: one a CU, whole rounds over the
// XCDs.
static int logit_blocks(const XentArgs& a, int nvoc) {
  const int64_t jobs = a.npad / kXTile * nvoc;
  return (int)(jobs < kXCus ? (jobs + 7) / 8 * 8 : kXCus);
}

hipError_t launch_xent_few(const XentArgs& a, hipStream_t s) {
  const int blocks = xent_few_blocks(a.rows);
  if (a.n > 32) hipLaunchKernelGGL(k_xent_few<2>, dim3(blocks), dim3(64), 0, s, a, blocks);
  else if (a.n > 0) hipLaunchKernelGGL(k_xent_few<1>, dim3(blocks), dim3(64), 0, s, a, blocks);
  hipLaunchKernelGGL(k_xent_few_loss, dim3(1), dim3(1024), 0, s, a, blocks);
  return hipGetLastError();
}

hipError_t launch_xent_stats(const XentArgs& a, hipStream_t s) {
  const int nvoc = (int)(a.rpad / kXTile);
  const XentPiece p{0, a.rpad, 1, 1, 0};
  hipLaunchKernelGGL((k_xent_logits<true>), dim3(logit_blocks(a, nvoc)), dim3(kXThreads), 0, s, a, p, nvoc);
  return hipGetLastError();
}

hipError_t launch_xent_loss(const XentArgs& a, hipStream_t s) {
  if (a.n * (a.rpad / kXTile) <= kXSoloStats) {
    hipLaunchKernelGGL(k_xent_loss, dim3(1), dim3(1024), 0, s, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(k_xent_lse, dim3(a.npad / 32), dim3(256), 0, s, a);
  hipLaunchKernelGGL(k_xent_total, dim3(1), dim3(1024), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_xent_prob(const XentArgs& a, const XentPiece& p, hipStream_t s) {
  const int nvoc = (int)(p.cols / kXTile);
  hipLaunchKernelGGL((k_xent_logits<false>), dim3(logit_blocks(a, nvoc)), dim3(kXThreads), 0, s, a, p, nvoc);
  return hipGetLastError();
}

hipError_t launch_xent_grad(const XentArgs& a, const XentPiece& p, hipStream_t s) {
  const int nd = (int)((a.wpad + kXTile - 1) / kXTile);
  const int ndw = a.dw ? (int)(p.cols / kXTile) * nd : 0;
  const int ndx = a.dx ? (int)(a.npad / kXTile) * nd * p.splits : 0;
  if (a.dw_dt == DT_BF16)
    hipLaunchKernelGGL((k_xent_grad<bf16_t>), dim3(ndw + ndx), dim3(kXThreads), 0, s, a, p, ndw, ndx, nd);
  else
    hipLaunchKernelGGL((k_xent_grad<float>), dim3(ndw + ndx), dim3(kXThreads), 0, s, a, p, ndw, ndx, nd);
  return hipGetLastError();
}

hipError_t launch_xent_dx(const XentArgs& a, int splits, hipStream_t s) {
  hipLaunchKernelGGL(k_xent_dx, dim3(2 * a.n), dim3(256), 0, s, a, splits);
  return hipGetLastError();
}

}  // namespace muonh
