// Layout and launchers of the cross-entropy kernels, shared by the kernels
// and the entry point.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace muonh {

constexpr int kXTile = 256;          // output tile side of the products
constexpr int kXStage = 64;          // depth of one operand stage
constexpr int64_t kXListTokens = 1024; // up to these, the list of counted tokens needs no launch of its own
constexpr int64_t kXSoloStats = 16384; // statistics (128 KiB) that one workgroup turns into the loss
constexpr int kXCus = 256;            // compute units, a multiple of the 8 XCDs
// Parts that dx is summed in: many at few tokens, where dx has few tiles and
// each is as deep as a piece (256 tokens, 50257 words, width 768: 224 us with up
// to 8 parts, 151 with up to 64), within a bound on their size.
constexpr int kXMaxSplits = 64;
constexpr int64_t kXSplitBytes = (int64_t)256 << 20;
constexpr int64_t kXMaxWidth = 65536, kXMaxTokens = (int64_t)1 << 22, kXMaxRows = (int64_t)1 << 23;

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
  float* tlogit;                     // per xp row: the target's logit
  float2* stats;                     // [rows / kXTile][npad]: maximum and sum of exp per tile
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
hipError_t launch_xent_stats(const XentArgs& a, hipStream_t s);
hipError_t launch_xent_loss(const XentArgs& a, hipStream_t s);
hipError_t launch_xent_prob(const XentArgs& a, const XentPiece& p, hipStream_t s);
hipError_t launch_xent_grad(const XentArgs& a, const XentPiece& p, hipStream_t s);
hipError_t launch_xent_dx(const XentArgs& a, int splits, hipStream_t s);

}  // namespace muonh
