// Activations to 8 bits and back (gfx950); the format is mx.h's.
//
// One pass each at the rate of memory: a thread takes 8 values of a row, the 4
// threads of a block of 32 find its largest magnitude by lane exchanges, and
// the values leave as 8 bytes with one scale byte a block.  A row belongs to a power of two of
// threads, so that short rows share a workgroup and nothing is divided; a
// thread has kRows rows in flight.  A workgroup's rows are neighbours and those
// side by side over a row follow each other, so that what is in flight at a time is one
// stretch of memory (rows of a workgroup as far apart as the grid is long: 8192 x 14336
// to bf16 71 us and not 61, 16384 x 4096 fp32 to 8 bits 76 and not 67).  Matrices
// beyond the last-level cache are read and written past the caches (ONCE).  16
// values a thread, two stores of every other 16 bytes of a line, took longer: 8192 x
// 14336 to bf16 by 7% (ONCE: 76%), 1021 x 331 fp32 to 8 bits 7.1 us against 4.4.  An fp32 result
// is 32 bytes a thread and stored so all the same: 16384 x 4096 76 us, the bytes alone 49 at the
// rate of a fill (from fp32 65).
#include <algorithm>
#include <type_traits>

#include "act.h"
#include "common.h"
#include "mx.h"

namespace muonh {

namespace {

constexpr int kRows = 4;

// Threads of a row (their logarithm): whole blocks, at most the workgroup's 256.
int row_log(int64_t width) {
  int l = 2;
  while (l < 8 && ((int64_t)8 << l) < width) ++l;
  return l;
}

template <typename T, bool ONCE>
__global__ __launch_bounds__(256) void k_mx_pack(const MxArgs a, int lg, uint32_t side) {
  const int64_t width = a.width, nblk = mx_blocks(width);
  const T* const in = static_cast<const T*>(a.in);
  const uint32_t down = blockIdx.x / side;
  const int64_t c = ((int64_t)(blockIdx.x - down * side) << lg) + (threadIdx.x & ((1 << lg) - 1));
  const int m = (int)min<int64_t>(max<int64_t>(width - 8 * c, 0), 8);
  const int64_t per = 256 >> lg, all = per * (gridDim.x / side);
  for (int64_t r0 = (int64_t)down * per * kRows + (threadIdx.x >> lg); r0 < a.n; r0 += kRows * all) {
    Raw8<T> raw[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u)
      if (m == 8 && r0 + u * per < a.n) {
        const int64_t at = (r0 + u * per) * width + 8 * c;
        if constexpr (ONCE) raw[u].load_once(in, at);
        else raw[u].load_any(in, at);
      }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int64_t r = r0 + u * per;
      if (r >= a.n) break;  // the same for the 4 lanes of a block
      float v[8];
      if (m == 8) raw[u].unpack(v);
      else load_first(in, r * width + 8 * c, m, v);
      const uint32_t sc = mx_scale(quad_max(finite_max(v)));
      const u32x2_t q = to_e4m3(v, mx_inverse(sc));
      if (m == 8) store_q8(a.q + r * width + 8 * c, q);
      else store_q8(a.q + r * width + 8 * c, q, m);
      if (c % 4 == 0 && m > 0) gmem(a.scales)[r * nblk + c / 4] = (uint8_t)sc;
    }
  }
}

template <typename T, bool ONCE>
__global__ __launch_bounds__(256) void k_mx_unpack(const MxArgs a, int lg, uint32_t side) {
  const int64_t width = a.width, nblk = mx_blocks(width);
  T* const out = static_cast<T*>(a.out);
  const uint32_t down = blockIdx.x / side;
  const int64_t c = ((int64_t)(blockIdx.x - down * side) << lg) + (threadIdx.x & ((1 << lg) - 1));
  const int m = (int)min<int64_t>(max<int64_t>(width - 8 * c, 0), 8);
  if (m == 0) return;
  const int64_t per = 256 >> lg, all = per * (gridDim.x / side);
  for (int64_t r0 = (int64_t)down * per * kRows + (threadIdx.x >> lg); r0 < a.n; r0 += kRows * all) {
    u32x2_t q[kRows];
    uint32_t sc[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int64_t r = r0 + u * per;
      if (r < a.n) {
        sc[u] = gmem(a.scales)[r * nblk + c / 4];
        q[u] = m == 8 ? load_q8(a.q + r * width + 8 * c) : load_q8(a.q + r * width + 8 * c, m);
      }
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int64_t r = r0 + u * per;
      if (r >= a.n) break;
      float v[8];
      from_e4m3(q[u], mx_factor(sc[u]), v);
      if (m == 8 && ONCE) store8_once(out, r * width + 8 * c, v);
      else if (m == 8) store8_any(out, r * width + 8 * c, v);
      else store_first(out, r * width + 8 * c, m, v);
    }
  }
}

// Workgroups side by side over a row.
uint32_t across(int64_t width, int lg) { return (uint32_t)((width + ((int64_t)8 << lg) - 1) / ((int64_t)8 << lg)); }
// Those over all rows.
dim3 grid(const MxArgs& a, int lg) {
  const int64_t side = across(a.width, lg), per = 256 >> lg;
  const int64_t down = std::min<int64_t>((a.n + per * kRows - 1) / (per * kRows), std::max<int64_t>(1, 65536 / side));
  return dim3((uint32_t)(down * side));
}

// f with std::true_type where `bytes` are moved that no cache holds.
template <typename F>
void past_caches(int64_t bytes, F&& f) {
  if (bytes > kActOnceBytes) f(std::true_type{});
  else f(std::false_type{});
}

}  // namespace

hipError_t launch_mx_pack(int dt, const MxArgs& a, hipStream_t s) {
  const int lg = row_log(a.width);
  past_caches(a.n * a.width * (dt == DT_BF16 ? 3 : 5), [&](auto once) {
    if (dt == DT_BF16) k_mx_pack<bf16_t, decltype(once)::value><<<grid(a, lg), 256, 0, s>>>(a, lg, across(a.width, lg));
    else k_mx_pack<float, decltype(once)::value><<<grid(a, lg), 256, 0, s>>>(a, lg, across(a.width, lg));
  });
  return hipGetLastError();
}

hipError_t launch_mx_unpack(int dt, const MxArgs& a, hipStream_t s) {
  const int lg = row_log(a.width);
  past_caches(a.n * a.width * (dt == DT_BF16 ? 3 : 5), [&](auto once) {
    if (dt == DT_BF16) k_mx_unpack<bf16_t, decltype(once)::value><<<grid(a, lg), 256, 0, s>>>(a, lg, across(a.width, lg));
    else k_mx_unpack<float, decltype(once)::value><<<grid(a, lg), 256, 0, s>>>(a, lg, across(a.width, lg));
  });
  return hipGetLastError();
}

}  // namespace muonh
