// The norm's gradient: fp32 dy.
#include "norm_grad.h"

namespace muonh {

hipError_t launch_rms_norm_grad_f32(int dx_dt, const NormGradArgs& a, hipStream_t s);
hipError_t launch_rms_norm_grad_f32(int dx_dt, const NormGradArgs& a, hipStream_t s) { return norm_grad_of<float>(dx_dt, a, s); }

}  // namespace muonh
