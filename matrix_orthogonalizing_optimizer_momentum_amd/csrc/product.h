// The 256 x 256 main loop that the products around the optimizer step run on
// (gfx950): D[m][n] = sum_k A[m][k] B[n][k] by 8 waves,
// v_mfma_f32_32x32x16_bf16, 64-deep operand stages double buffered in LDS.
#pragma once
#include "common.h"

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

}  // namespace
}  // namespace muonh
