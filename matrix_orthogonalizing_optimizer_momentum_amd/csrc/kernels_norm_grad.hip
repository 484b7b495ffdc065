// The norm's gradient: bf16 dy, the sum of the gain's parts, and the launcher.
#include "norm_grad.h"

namespace muonh {

namespace {

// dgain from the workgroups' partial rows: 32 columns a workgroup, 32 threads a
// column, each a fixed stride of rows.
__global__ __launch_bounds__(1024) void k_norm_gain_sum(const float* __restrict__ part, int rows, int64_t width,
                                                        float* __restrict__ dgain, int accumulate) {
  __shared__ float red[32][33];
  const int cl = threadIdx.x & 31, gr = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + cl;
  float s = 0.f;
  if (c < width)
    for (int r = gr; r < rows; r += 32 * 8) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = r + 32 * u < rows ? gmem(part)[(int64_t)(r + 32 * u) * width + c] : 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u) s += v[u];
    }
  red[gr][cl] = s;
  __syncthreads();
  if (gr == 0 && c < width) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) t += red[k][cl];
    gmem(dgain)[c] = accumulate ? gmem(dgain)[c] + t : t;
  }
}

}  // namespace

// Some 4 rows each in turn, at least a workgroup a compute unit, at most what runs at once
// (777 x 1999 and 2000 x 768 fp32: 256 and 512 workgroups 12.7 and 10.2 us, 768 15.2 and 10.9).
int norm_grad_blocks(int64_t n, int64_t width) {
  const int l = norm_shape(width).lanes;
  const int64_t rows = std::max<int64_t>(1, (n + norm_threads(l) / l - 1) / (norm_threads(l) / l));
  const int64_t most = l == 1024 ? 256 : l == 512 ? 512 : 768;
  return (int)std::min(rows, std::min(most, std::max<int64_t>(256, (rows + 3) / 4)));
}

hipError_t launch_rms_norm_grad_f32(int dx_dt, const NormGradArgs& a, hipStream_t s);  // kernels_norm_grad_f32.hip

hipError_t launch_rms_norm_grad(int dy_dt, int dx_dt, const NormGradArgs& a, hipStream_t s) {
  const hipError_t e = dy_dt == DT_BF16 ? norm_grad_of<bf16_t>(dx_dt, a, s) : launch_rms_norm_grad_f32(dx_dt, a, s);
  if (e != hipSuccess || a.part == nullptr) return e;
  k_norm_gain_sum<<<dim3((uint32_t)((a.width + 31) / 32)), 1024, 0, s>>>(a.part, norm_grad_blocks(a.n, a.width), a.width,
                                                                        a.dgain, a.accumulate);
  return hipGetLastError();
}

}  // namespace muonh
