// Layout and launchers of the weight gradient from 8-bit activations, shared by
// the kernels and the entry point.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act.h"

namespace muonh {

constexpr int64_t kWgMaxTokens = (int64_t)1 << 22, kWgMaxSide = (int64_t)1 << 20, kWgMaxValues = (int64_t)1 << 37;

struct WgradArgs {
  const uint16_t* dz;                // n x rows
  const uint8_t* q;                  // n x width e4m3
  const uint8_t* scales;             // n x mx_blocks(width)
  const float* gain;                 // width, or nullptr
  void* dw;                          // rows x width
  uint16_t* xt;                      // width up to a tile rows of ldxt: q's values in bf16 along the tokens
  uint16_t* dzt;                     // turn: dz along the tokens, rows up to a tile of ldxt; else dz's rows [dfull, n),
                                     // padded with zeros to a whole stage, of lddz
  float* part;                       // with splits > 1: [splits][rows][ldp], or [splits][256 tiles from first on][256][256]
  int64_t n, npad, rows, width, ldxt, lddz, dfull, ldp;
  int64_t whole;                     // stages that the 64 and 128 tiles read whole, over the rows' ends
  int32_t first;                     // 256 tiles before this one (in the order of the jobs) are not cut into parts
  float scale;
  int32_t dw_dt, accumulate, splits, turn, tile;  // tile: 256 (from xt and dz or dzt), or 128 or 64 from q and dz
};

hipError_t launch_wgrad_prepare(const WgradArgs& a, hipStream_t s);
hipError_t launch_wgrad(const WgradArgs& a, hipStream_t s);

}  // namespace muonh
