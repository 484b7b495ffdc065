// Layout and launchers of the cross-entropy kernels, shared by the kernels
// and the entry point.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "desc.h"

namespace muonh {

constexpr int64_t kXListTokens = 1024; // up to these, the list of counted tokens needs no launch of its own
constexpr int64_t kXSoloStats = 16384; // statistics (128 KiB) that one workgroup turns into the loss
// Parts that dx is summed in: many at few tokens, where dx has few tiles and
// each is as deep as a piece (256 tokens, 50257 words, width 768: 224 us with up
// to 8 parts, 151 with up to 64), within a bound on their size.
constexpr int kXMaxSplits = 64;
constexpr int64_t kXSplitBytes = (int64_t)256 << 20;
constexpr int64_t kXMaxWidth = 65536, kXMaxTokens = (int64_t)1 << 22, kXMaxRows = (int64_t)1 << 23;

// The loss of up to kXFewTokens tokens without gradients (rows of w of 8 values
// at least) has kernels of its own, that take 64 words at a time in at most
// kXFewBlocks workgroups.  Against tiles of 256 tokens: 17 tokens, 50257 x 768
// 33 -> 23 us, 64 tokens 34 -> 33; 151936 x 2048, 8 tokens 195 -> 136, 64 tokens
// 194 -> 157; 3 tokens, 141353 x 221, where the tiles need a copy of w, 101 -> 24.
constexpr int64_t kXFewTokens = 64;
constexpr int kXFewWords = 64, kXFewBlocks = 2048;
// Workgroups (of one wave, all resident at once), with the same number of
// rounds each.
inline int xent_few_blocks(int64_t rows) {
  const int64_t tiles = (rows + kXFewWords - 1) / kXFewWords;
  const int64_t rounds = (tiles + kXFewBlocks - 1) / kXFewBlocks;
  return (int)((tiles + rounds - 1) / rounds);
}

// Device scalars of one call.
struct XentScalars {
  int32_t count;                     // counted tokens
  float gscale;                      // factor of both gradients
};

struct XentArgs {
  const uint16_t* x;                 // n x width, the caller's
  const uint16_t* w;                 // rows x width (ldw), or its padded copy
  const uint16_t* wtail;             // rows [wfull, rows) padded to a whole tile, ldw
  const void* targets;
  uint16_t* xp;                      // counted tokens of x, npad x wpad, zero padded
  uint16_t* xt;                      // xp transposed (for dw): width rounded up to a tile rows of ldxt
  int32_t* perm;                     // xp row -> token
  int32_t* tgt;                      // xp row -> target
  float* lse;                        // per xp row
  float* tlogit;                     // per xp row (few tokens: per token): the target's logit
  float2* stats;                     // [rows / kXTile][npad]: maximum and sum of exp per tile (few tokens: [n][blocks])
  uint16_t* prob;                    // npad x piece
  float* dxacc;                      // [splits][npad][wpad]
  XentScalars* sc;
  float* loss;
  float* token_loss;                 // per token, or nullptr
  uint16_t* dx;                      // n x width or nullptr
  void* dw;                          // rows x width or nullptr
  int64_t n, npad, rows, rpad, wfull, width, wpad, ldw, ldxt;
  int64_t ignore_index;
  float grad_scale;
  int32_t id_bits, mean, dw_dt, accumulate;
};

// One piece of the vocabulary: rows [v0, v0 + cols) of w, cols a multiple of
// kXTile (rows past the last one count as zero).
struct XentPiece {
  int64_t v0, cols;
  int32_t splits;                    // parts of cols that dx is summed over separately
  int32_t first;                     // the first piece: dxacc is written, not added to
  int32_t dx_first;                  // order of the jobs of one launch
};

hipError_t launch_xent_prepare(const XentArgs& a, bool copy_w, const uint16_t* w_in, hipStream_t s);
hipError_t launch_xent_few(const XentArgs& a, hipStream_t s);  // the whole call
hipError_t launch_xent_stats(const XentArgs& a, hipStream_t s);
hipError_t launch_xent_loss(const XentArgs& a, hipStream_t s);
hipError_t launch_xent_prob(const XentArgs& a, const XentPiece& p, hipStream_t s);
hipError_t launch_xent_grad(const XentArgs& a, const XentPiece& p, hipStream_t s);
hipError_t launch_xent_dx(const XentArgs& a, int splits, hipStream_t s);

}  // namespace muonh
