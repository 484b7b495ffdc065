// Global gradient norm over many tensors, and clipping (gfx950).
//
//   total   = sqrt(sum_t sum_e g_t[e]^2),  norms[t] = sqrt(sum_e g_t[e]^2)
//   coef    = min(1, max_norm / (total + 1e-6))
//   out_t   = coef * g_t
//
// Both passes stream: the norm reads every gradient once, clipping reads it
// again and writes it.  What the norm read stays in the last-level cache as far
// as it fits; clipping reads and writes past the caches (non-temporal), so that
// its results do not push out what it has yet to read (85 million bf16 values:
// 110 -> 85 us with its norm).  Tensors' 16-byte grids are used for loads;
// stores go to any alignment.  The list of tensors travels in the kernel arguments
// (kTabTensors a launch), so a call uploads no table, keeps nothing between
// calls and can be captured into a graph as it is.
//
// Work split: every tensor is cut into blocks of `chunk` bytes, one for the
// whole call and chosen so that the blocks of all tensors together fill the
// chip about once; a block sums its squares in fp64 (squares of bf16 and fp32
// values neither overflow nor underflow there, and no order of the values
// changes the result by more than a few units of fp64's last place) and stores
// one partial.  k_grad_finish adds the partials in a fixed order.
#include "common.h"
#include "grad.h"

namespace muonh {

namespace {

// Index of the tensor that block b belongs to: the last t < n with
// first[t] <= b.  One load per lane and a count instead of a dependent chain.
__device__ __forceinline__ int tensor_of(const int32_t* first, int n, int b) {
  int t = -1;
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int k = 0; k < kTabTensors / 64; ++k) {
    const int i = 64 * k + lane;
    const bool below = i < n && first[i] <= b;
    t += __popcll(__ballot(below));
  }
  return __builtin_amdgcn_readfirstlane(t);
}

// Elements before the first 16-byte boundary of p.
template <typename T>
__device__ __forceinline__ int head_of(const void* p) {
  return (int)(((16 - (uintptr_t)p % 16) % 16) / sizeof(T));
}

constexpr int kVec = 8;  // elements a thread takes at a time
constexpr int kDepth = 4;  // such groups in flight

template <bool ONCE, typename T>
__device__ __forceinline__ double sumsq_block(const T* __restrict__ p, int64_t lo, int64_t hi) {
  const int t = threadIdx.x;
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  // [lo, v0) and [v1, hi) are at most 7 elements each
  const int64_t v0 = min(lo + head_of<T>(p), hi);
  const int64_t v1 = v0 + (hi - v0) / kVec * kVec;
  auto one = [&](int64_t i) {
    const double x = (double)St<T>::ld(p, i);
    s[0] = fma(x, x, s[0]);
  };
  if (t < 7 && lo + t < v0) one(lo + t);
  if (t >= 8 && t < 15 && v1 + (t - 8) < hi) one(v1 + (t - 8));
  auto add = [&](const Raw8<T>& r) {
    float v[8];
    r.unpack(v);
#pragma unroll
    for (int k = 0; k < 8; ++k) s[k & 3] = fma((double)v[k], (double)v[k], s[k & 3]);
  };
  constexpr int64_t kStep = (int64_t)kGradThreads * kVec;
  int64_t i = v0 + (int64_t)t * kVec;
  for (; i + (kDepth - 1) * kStep < v1; i += kDepth * kStep) {
    Raw8<T> r[kDepth];
#pragma unroll
    for (int k = 0; k < kDepth; ++k) {
      if constexpr (ONCE) r[k].load_once(p, i + k * kStep);
      else r[k].load(p, i + k * kStep);
    }
#pragma unroll
    for (int k = 0; k < kDepth; ++k) add(r[k]);
  }
  for (; i < v1; i += kStep) {
    Raw8<T> r;
    r.load(p, i);
    add(r);
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

template <bool ONCE>
__global__ __launch_bounds__(kGradThreads) void k_grad_sumsq(const GradTab tab, double* __restrict__ partials,
                                                             int32_t* __restrict__ bounds) {
  __shared__ double red[kGradThreads / 64];
  const int b = blockIdx.x;
  const int t = tensor_of(tab.first, tab.n, b);
  const int64_t n = tab.numel[t];
  const bool half = (tab.bf16[t >> 5] >> (t & 31)) & 1;
  const int64_t per = tab.chunk >> (half ? 1 : 2);
  const int64_t lo = (int64_t)(b - tab.first[t]) * per;
  const int64_t hi = min(n, lo + per);
  double s;
  if (half) s = sumsq_block<ONCE>(reinterpret_cast<const bf16_t*>(tab.in[t]), lo, hi);
  else s = sumsq_block<ONCE>(reinterpret_cast<const float*>(tab.in[t]), lo, hi);
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double v = 0.0;
#pragma unroll
    for (int k = 0; k < kGradThreads / 64; ++k) v += red[k];
    gmem(partials)[tab.part0 + b] = v;
    // where this tensor's partials begin, for k_grad_finish
    if (lo == 0) gmem(bounds)[tab.tensor0 + t] = tab.part0 + b;
  }
}

// One workgroup: group g of 16 lanes sums the partials of tensors g, g + 64, ...
// (each lane a fixed stride of them), then the groups' totals are added in
// order.  Lists of ordinary length are staged in LDS first, with one trip to
// memory for all.
constexpr int kStagePartials = 4096, kStageTensors = 2047;
__global__ __launch_bounds__(1024) void k_grad_finish(const double* __restrict__ partials,
                                                      const int32_t* __restrict__ bounds, int n, int nparts,
                                                      float max_norm, float* __restrict__ total,
                                                      float* __restrict__ coef, float* __restrict__ norms) {
  constexpr int NW = 16, NG = 64, GL = 16;  // waves; groups and lanes of one
  __shared__ double red[NG];
  __shared__ double part[kStagePartials];
  __shared__ int32_t first[kStageTensors + 1];
  const int g = threadIdx.x / GL, l = threadIdx.x % GL;
  const bool staged = nparts <= kStagePartials && n <= kStageTensors;
  if (staged) {
    for (int i = threadIdx.x; i < nparts; i += 64 * NW) part[i] = gmem(partials)[i];
    for (int i = threadIdx.x; i < n; i += 64 * NW) first[i] = gmem(bounds)[i];
    __syncthreads();
  }
  auto bound = [&](int t) { return t >= n ? nparts : staged ? first[t] : gmem(bounds)[t]; };
  auto value = [&](int p) { return staged ? part[p] : gmem(partials)[p]; };
  double mine = 0.0;
  for (int t = g; t < n; t += NG) {
    const int p0 = bound(t), p1 = bound(t + 1);
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    int p = p0 + l;
    for (; p + 3 * GL < p1; p += 4 * GL) {
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k] += value(p + GL * k);
    }
    for (; p < p1; p += GL) s[0] += value(p);
    double v = (s[0] + s[1]) + (s[2] + s[3]);
#pragma unroll
    for (int o = GL / 2; o > 0; o >>= 1) v += __shfl_xor(v, o, GL);
    mine += v;
    if (l == 0 && norms != nullptr) gmem(norms)[t] = (float)sqrt(v);
  }
  if (l == 0) red[g] = mine;
  __syncthreads();
  if (threadIdx.x < NG) {
    const double tot = sqrt(wave_sum(red[threadIdx.x]));
    if (threadIdx.x > 0) return;
    gmem(total)[0] = (float)tot;
    if (coef != nullptr) {
      const double c = (double)max_norm / (tot + 1e-6);
      gmem(coef)[0] = c >= 1.0 ? 1.f : (float)c;  // a NaN norm stays NaN
    }
  }
}

template <typename T>
__device__ __forceinline__ void scale_block(const T* p, T* o, int64_t lo, int64_t hi, float c) {
  const int t = threadIdx.x;
  const int64_t v0 = min(lo + head_of<T>(p), hi);
  const int64_t v1 = v0 + (hi - v0) / kVec * kVec;
  if (t < 7 && lo + t < v0) St<T>::st(o, lo + t, c * St<T>::ld(p, lo + t));
  if (t >= 8 && t < 15 && v1 + (t - 8) < hi) St<T>::st(o, v1 + (t - 8), c * St<T>::ld(p, v1 + (t - 8)));
  auto put = [&](const Raw8<T>& r, int64_t i) {
    float v[8];
    r.unpack(v);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= c;
    store8_once(o, i, v);
  };
  constexpr int64_t kStep = (int64_t)kGradThreads * kVec;
  int64_t i = v0 + (int64_t)t * kVec;
  for (; i + (kDepth - 1) * kStep < v1; i += kDepth * kStep) {
    Raw8<T> r[kDepth];
#pragma unroll
    for (int k = 0; k < kDepth; ++k) r[k].load_once(p, i + k * kStep);
#pragma unroll
    for (int k = 0; k < kDepth; ++k) put(r[k], i + k * kStep);
  }
  for (; i < v1; i += kStep) {
    Raw8<T> r;
    r.load(p, i);
    put(r, i);
  }
}

__global__ __launch_bounds__(kGradThreads) void k_grad_scale(const ScaleTab tab, const float* __restrict__ coef) {
  const int b = blockIdx.x;
  const int t = tensor_of(tab.g.first, tab.g.n, b);
  const float c = gmem(coef)[0];
  const void* const in = tab.g.in[t];
  void* const out = tab.out[t];
  if (c == 1.f && in == out) return;  // nothing to change in place
  const int64_t n = tab.g.numel[t];
  const bool half = (tab.g.bf16[t >> 5] >> (t & 31)) & 1;
  const int64_t per = tab.g.chunk >> (half ? 1 : 2);
  const int64_t lo = (int64_t)(b - tab.g.first[t]) * per;
  const int64_t hi = min(n, lo + per);
  if (half)
    scale_block(reinterpret_cast<const bf16_t*>(in), reinterpret_cast<bf16_t*>(out), lo, hi, c);
  else
    scale_block(reinterpret_cast<const float*>(in), reinterpret_cast<float*>(out), lo, hi, c);
}

}  // namespace

hipError_t launch_grad_sumsq(const GradTab& tab, int nblocks, bool once, double* partials, int32_t* bounds,
                             hipStream_t s) {
  if (once) hipLaunchKernelGGL(k_grad_sumsq<true>, dim3(nblocks), dim3(kGradThreads), 0, s, tab, partials, bounds);
  else hipLaunchKernelGGL(k_grad_sumsq<false>, dim3(nblocks), dim3(kGradThreads), 0, s, tab, partials, bounds);
  return hipGetLastError();
}

hipError_t launch_grad_finish(const double* partials, const int32_t* bounds, int n, int nparts, float max_norm,
                              float* total, float* coef, float* norms, hipStream_t s) {
  hipLaunchKernelGGL(k_grad_finish, dim3(1), dim3(1024), 0, s, partials, bounds, n, nparts, max_norm, total, coef,
                     norms);
  return hipGetLastError();
}

hipError_t launch_grad_scale(const ScaleTab& tab, int nblocks, const float* coef, hipStream_t s) {
  hipLaunchKernelGGL(k_grad_scale, dim3(nblocks), dim3(kGradThreads), 0, s, tab, coef);
  return hipGetLastError();
}

}  // namespace muonh
