// Tables and launchers of the gradient norm / clipping kernels, shared by the
// kernels and the entry points.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace muonh {

constexpr int kGradThreads = 256;
constexpr int kTabTensors = 128;  // tensors per launch: the tables stay below 4 KiB of kernel arguments

struct GradTab {
  const void* in[kTabTensors];
  int64_t numel[kTabTensors];
  int32_t first[kTabTensors];      // first block of each tensor (every tensor has at least one)
  uint32_t bf16[kTabTensors / 32]; // bit t: tensor t is bf16, else fp32
  int64_t chunk;                   // bytes per block, a multiple of 32
  int32_t n;                       // tensors in this table
  int32_t tensor0;                 // index of its first tensor in the call's list
  int32_t part0;                   // index of its first block among the call's partials
};

struct ScaleTab {
  GradTab g;
  void* out[kTabTensors];
};
static_assert(sizeof(ScaleTab) <= 4000, "kernel argument size");

// once: the gradients are read past the caches
hipError_t launch_grad_sumsq(const GradTab& tab, int nblocks, bool once, double* partials, int32_t* bounds,
                             hipStream_t s);
hipError_t launch_grad_finish(const double* partials, const int32_t* bounds, int n, int nparts, float max_norm,
                              float* total, float* coef, float* norms, hipStream_t s);
hipError_t launch_grad_scale(const ScaleTab& tab, int nblocks, const float* coef, hipStream_t s);

}  // namespace muonh
