// Arguments and launchers of the activation kernels (norm, 8-bit activations),
// shared by the kernels and the entry points.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "desc.h"

namespace muonh {

// Values that share one scale: the block of the OCP microscaling formats, which
// gfx950's scaled matrix instructions take too.
constexpr int64_t kMxBlock = 32;
__host__ __device__ inline int64_t mx_blocks(int64_t width) { return (width + kMxBlock - 1) / kMxBlock; }

// A row is held in registers: at most 1024 threads of 2 chunks of 8 values.
constexpr int64_t kNormMaxWidth = 16384, kActMaxTokens = (int64_t)1 << 26, kActMaxWidth = (int64_t)1 << 20;

// What moves more bytes than this is read and written past the caches, as no cache
// holds it for the next kernel (603 MB of a norm 113 -> 100 us, 470 MB of its
// gradient 89 -> 74, 350 MB to 8 bits 75 -> 66; 268 MB 45.5 -> 48, 82 MB 15 -> 18).
constexpr int64_t kActOnceBytes = (int64_t)320 << 20;

struct NormArgs {
  const void* x;                     // n x width
  const void* res;                   // n x width of h's type, or nullptr
  const float* gain;                 // width, or nullptr
  void* h;                           // n x width (with res)
  void* y;                           // n x width, or nullptr
  float* rstd;                       // n, or nullptr
  uint8_t* q;                        // n x width e4m3, or nullptr
  uint8_t* scales;                   // n x mx_blocks(width)
  int64_t n, width;
  double eps;
  int32_t y_dt;
  int32_t packs_output;              // q holds y, else the row before the gain
};

struct NormGradArgs {
  const void* dy;                    // n x width
  const void* x;                     // n x width of dx's type, or nullptr: q and scales
  const uint8_t* q;
  const uint8_t* scales;
  const float* rstd;                 // n
  const float* gain;                 // width, or nullptr
  const void* dres;                  // n x width of dx's type, or nullptr
  void* dx;
  float* part;                       // [blocks][width]: sums of dy * xn; nullptr: no dgain, or by columns
  float* dgain;                      // width, or nullptr
  int64_t n, width;
  int32_t accumulate;
};

struct MxArgs {
  const void* in;                    // pack: values; unpack: nullptr
  uint8_t* q;
  uint8_t* scales;
  void* out;                         // unpack: values
  int64_t n, width;
};

// Workgroups of the norm's gradient, and so partial sums of the gain's (8192 x 2048:
// 256 take 41.9 us, 512 28.0, 768 25.3, 1536 31.0; 8192 x 8192, 1024 threads a
// row: 256 90.7, 512 93.0).
int norm_grad_blocks(int64_t n, int64_t width);
// Rows few enough to be read again by columns in the same launch, which the host
// takes 6 us for, two 10 (on the GPU 64 x 2048 4.5 us against 5.5, 512 x 2048 8.2 and 7.2,
// 777 x 1999 fp32 15.0 and 12.8).
inline bool norm_grad_columns(int64_t n, int64_t width) { return n <= 512 && n * width <= (int64_t)3 << 19; }

hipError_t launch_rms_norm(int x_dt, int res_dt, const NormArgs& a, hipStream_t s);  // res_dt: -1 without res
hipError_t launch_rms_norm_grad(int dy_dt, int dx_dt, const NormGradArgs& a, hipStream_t s);
hipError_t launch_mx_pack(int dt, const MxArgs& a, hipStream_t s);
hipError_t launch_mx_unpack(int dt, const MxArgs& a, hipStream_t s);

}  // namespace muonh
