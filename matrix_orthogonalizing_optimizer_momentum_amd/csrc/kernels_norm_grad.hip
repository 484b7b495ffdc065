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

int norm_grad_blocks(int64_t n, int64_t width) {
  const NormShape p = norm_shape(width);
  const int64_t per = norm_threads(p.nw) / (64 * p.nw), most = p.nw == 16 ? 256 : p.nw == 8 ? 512 : 768;
  return (int)std::max<int64_t>(1, std::min<int64_t>((n + per - 1) / per, most));
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
