// What the entry-point files share: error text and per-kernel timing.
#pragma once
#include <hip/hip_runtime.h>

#include "muonh.h"

namespace muonh {

// Kernel classes of muonh_profile_read.
enum {
  PC_MOM = 0, PC_G1, PC_G2, PC_G3, PC_HR, PC_HW, PC_SQ, PC_FIN, PC_TILE, PC_AM, PC_AW, PC_T256,
  PC_GNORM, PC_GSCALE, PC_EMB, PC_EMBSORT, PC_EMBGRAD, PC_XPREP, PC_XLOGIT, PC_XPROB, PC_XGRAD, PC_N
};

// Records e as this thread's last HIP failure and returns MUONH_EHIP.
int hip_fail(hipError_t e, const char* what);

#define MUONH_TRY_HIP(x)                                  \
  do {                                                    \
    const hipError_t e_ = (x);                            \
    if (e_ != hipSuccess) return hip_fail(e_, #x);        \
  } while (0)

// Event pair around the launches of its scope while muonh_profile_begin is in
// effect; nothing otherwise.  Takes the library's lock to hand in a finished
// pair: for entry points that do not hold it, which wait for nobody while
// nothing is profiled (a call that holds the lock may wait for the device).
class ProfScope {
 public:
  ProfScope(hipStream_t s, int cls, double flops, double bytes);
  ~ProfScope();
  ProfScope(const ProfScope&) = delete;
  ProfScope& operator=(const ProfScope&) = delete;

 private:
  hipStream_t s_;
  int cls_;
  double flops_, bytes_;
  hipEvent_t e0_{};
};

}  // namespace muonh
