// Entry points between the embedding and the output layer: the root-mean-square
// norm and its gradient, activations in 8 bits, the weight gradient from them.
// They hold no state: each call validates, computes its layout on the host and
// queues kernels on the caller's stream, with scratch memory from the caller.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "act.h"
#include "checks.h"
#include "desc.h"
#include "muonh.h"
#include "runtime.h"
#include "wgrad.h"

namespace muonh {
namespace {

int check_rows(int64_t n, int64_t width, int64_t max_width) {
  if (n < 0 || width < 1) return MUONH_EINVAL;
  return n > kActMaxTokens || width > max_width || n * up(width, 8) > ((int64_t)1 << 40) ? MUONH_ENOTIMPL : MUONH_OK;
}

// A buffer of `bytes` aligned to `a`: given, unless it has none.
bool bad_buffer(const void* p, int64_t bytes, int64_t a) { return bytes > 0 && (!p || misaligned(p, a)); }

// Outputs, scratch memory among them, apart from the inputs and from each other.
// same[k]: the one input that output k may be, value for value.
bool bad_outputs(const Span* outs, int no, const Span* ins, int ni, const Span* const* same) {
  for (int k = 0; k < no; ++k) {
    for (int i = 0; i < ni; ++i)
      if (overlap(outs[k], ins[i]) && !(same[k] == &ins[i] && outs[k].lo == ins[i].lo && outs[k].hi == ins[i].hi)) return true;
    for (int j = 0; j < k; ++j)
      if (overlap(outs[k], outs[j])) return true;
  }
  return false;
}

// ------------------------------------------------------------ weight gradient
struct WgradPlan {
  bool copy_dz, turn;
  int64_t npad, ldxt, lddz, dfull, ldp, whole, xt, dzt, part, bytes;
  int splits, first, tile;
};

int check_wgrad(const void* dz, int64_t n, int64_t rows, int64_t width) {
  if (n < 0 || rows < 1 || width < 1 || (dz && misaligned(dz, 2))) return MUONH_EINVAL;
  if (n > kWgMaxTokens || rows > kWgMaxSide || width > kWgMaxSide) return MUONH_ENOTIMPL;
  // what the kernels' grids hold (below 2^32 threads a launch)
  const int64_t side = std::max(rows, width);
  return up(rows, kXTile) * up(width, kXTile) > kWgMaxValues || up(n, kXTile) * up(side, kXTile) > ((int64_t)1 << 35)
             ? MUONH_ENOTIMPL
             : MUONH_OK;
}

// Tile and parts of the tokens, by an estimate of the call's time in microseconds,
// within some 15% of what these took (8192 x 2304 x 768: 256 tiles in 9 parts 60, 128
// in 4 parts 56, 64 whole 63; 2048 x 2304 x 768: 40, 28 and 20; 512 x 4096 x 4096: 37
// and 32; 16384 x 2048 x 2048: 157 in 4 parts, 175; 8192 x 9000 x 2100: 319, 416).  A stage
// of 64 tokens of a 256 tile takes 1.55 on its own compute unit, with x brought to bf16
// by a launch before it (3 bytes a value); of a 128 tile 0.72, or 1.25 of the two that
// share a unit; of a 64 tile 0.28.  Each tile has an epilogue, the result is stored at
// 5 GB/ms (2.5 for 256 tiles), and parts cost a launch and are written and read.
//
// 256 tiles that fill the compute units once or more are whole, and those left over are cut
// by themselves, against a round in which units are idle and the others run some 15%
// faster (8192 x 14336 x 4096, 3 rounds and 128 tiles: whole 930, those in 2 parts 863; 8192 x 4352 x
// 4096, 1 round and 16 tiles: whole 407, in 8 parts 274; 8192 x 5120 x 5120, 1 round and
// 144 tiles: whole 420, in 3 parts 451).
struct WgradChoice {
  int tile, splits, first;
};
WgradChoice wgrad_choice(int64_t n, int64_t rows, int64_t width) {
  const int64_t stages = up(n, kXStage) / kXStage;
  const double values = (double)rows * (double)width;
  WgradChoice best{kXTile, 1, 0};
  double least = 0;
  for (const int tile : {256, 128, 64}) {
    const int64_t tiles = up(rows, tile) / tile * (up(width, tile) / tile);
    if (tile != kXTile && tiles > 64 * kXCus) continue;
    const int64_t first = tile == kXTile ? tiles / kXCus * kXCus : 0, cut = tiles - first;
    for (int64_t k = 1; k <= 32 && k <= std::max<int64_t>(stages, 1); ++k) {
      if (k > 1 && (cut == 0 || cut * k > 4 * kXCus)) break;
      const double each = (double)((stages + k - 1) / k);
      // tiles of the busiest unit; many tiles even out
      const double c = cut * k > 4 * kXCus ? (double)(cut * k) / kXCus : (double)((cut * k + kXCus - 1) / kXCus);
      double t;
      if (tile == kXTile)
        t = 8.0 + 3.0 * (double)n * (double)width / 3.5e6 + (double)(first / kXCus) * (1.55 * (double)stages + 5.0) +
            c * ((first && k == 1 ? 1.32 : 1.55) * each + 5.0) + 2.0 * values / 2.5e6;
      else if (tile == 128)
        t = 3.5 + (c > 4 ? 0.64 * c : c == 1 ? 0.72 : c == 2 ? 1.25 : c == 3 ? 1.82 : 2.5) * each + 0.8 * (c + 1) +
            2.0 * values / 5e6;
      else
        t = 3.2 + c * (0.28 * each + 0.6) + 2.0 * values / 5e6;
      if (k > 1) t += 3.0 + 8.0 * (double)k * (tile == kXTile ? (double)cut * (kXTile * kXTile) : values) / 6e6;
      if (least == 0 || t < least) {
        least = t;
        best = {tile, (int)k, (int)(k > 1 ? first : 0)};
      }
    }
  }
  return best;
}

// Whether dz is brought along the tokens too.  The pass costs its 4 bytes a value of dz, and the
// product's plain reads of it save some 5% of a time that grows with the width
// (8192 x 4096, with and without: width 4096 258 and 241 us, 8192 493 and 503,
// 14336 965 and 1056; 4096 x 4096, width 6144 237 and 237; 8192 x 14336 x 4096 927
// and 914, 8192 x 28672 x 8192 3129 and 3281).
bool wgrad_turns(int64_t width) { return width >= 8192; }

WgradPlan wgrad_plan(const void* dz, int64_t n, int64_t rows, int64_t width) {
  WgradPlan p{};
  const WgradChoice c = wgrad_choice(n, rows, width);
  p.tile = c.tile;
  p.splits = c.splits;
  p.first = c.first;
  // The smaller tiles' reads run over a row's end by less than a tile: the last
  // rows that this leaves the buffers from are in stages read value by value.
  auto behind = [&](int64_t row, int64_t over) { return (over + row - 1) / row; };
  const int64_t tail = std::max({behind(width, up(width, c.tile) - width), behind(rows, up(rows, c.tile) - rows),
                                 behind(mx_blocks(width), up(width, c.tile) / kMxBlock - mx_blocks(width))});
  p.whole = std::max<int64_t>(0, n - tail) / kXStage;
  // dz is an operand as it stands when its rows are on a 16-byte grid, but for
  // the rows of its last, partial stage; else the call works on a padded copy
  p.copy_dz = rows % 8 != 0 || misaligned(dz, 16);
  p.npad = up(n, kXStage);
  p.ldxt = up(n, 128) + 64;  // off the powers of two, so that rows fall on different memory channels
  p.lddz = up(rows, 8);
  p.dfull = p.copy_dz ? 0 : n / kXStage * kXStage;
  p.ldp = up(width, 8);
  const bool large = p.tile == kXTile;  // the others read the caller's buffers
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += up(bytes, 256);
    return o;
  };
  p.xt = take(large && n ? 2 * up(width, kXTile) * p.ldxt : 0);
  p.turn = large && wgrad_turns(width);
  p.dzt = take(!large || n == 0 ? 0 : p.turn ? 2 * up(rows, kXTile) * p.ldxt : 2 * (p.npad - p.dfull) * p.lddz);
  const int64_t cut = up(width, kXTile) / kXTile * (up(rows, kXTile) / kXTile) - p.first;
  p.part = take(p.splits == 1 ? 0 : large ? 4 * p.splits * cut * (kXTile * kXTile) : 4 * p.splits * rows * p.ldp);
  p.bytes = std::max<int64_t>(at, 256);
  return p;
}

}  // namespace
}  // namespace muonh

using namespace muonh;

extern "C" {

int muonh_rms_norm(const void* x, int x_dtype, const void* residual, int h_dtype, const float* gain, float eps, int64_t n,
                   int64_t width, void* h, void* y, int y_dtype, float* rstd, void* q, void* scales, int packs,
                   void* stream) {
  const int rc = check_rows(n, width, kNormMaxWidth);
  if (rc != MUONH_OK) return rc;
  if (bad_dtype(x_dtype) || bad_dtype(y_dtype) || (residual && bad_dtype(h_dtype))) return MUONH_EINVAL;
  if (!std::isfinite(eps) || eps <= 0.f) return MUONH_EINVAL;
  if (packs != MUONH_PACK_NORMALIZED && packs != MUONH_PACK_OUTPUT) return MUONH_EINVAL;
  if ((residual == nullptr) != (h == nullptr) || (q == nullptr) != (scales == nullptr)) return MUONH_EINVAL;
  if (misaligned(gain, 4) || misaligned(rstd, 4) || misaligned(y, dtype_size(y_dtype))) return MUONH_EINVAL;
  if (residual && (misaligned(residual, dtype_size(h_dtype)) || misaligned(h, dtype_size(h_dtype)))) return MUONH_EINVAL;
  if (bad_buffer(x, n, dtype_size(x_dtype))) return MUONH_EINVAL;
  if (n == 0) return MUONH_OK;
  const int64_t all = n * width;
  const Span ins[] = {span_of(x, all * dtype_size(x_dtype)), span_of(residual, all * dtype_size(h_dtype)),
                      span_of(gain, 4 * width)};
  const Span outs[] = {span_of(h, all * dtype_size(h_dtype)), span_of(y, all * dtype_size(y_dtype)), span_of(rstd, 4 * n),
                       span_of(q, all), span_of(scales, n * mx_blocks(width))};
  const Span* const same[] = {&ins[1], nullptr, nullptr, nullptr, nullptr};
  if (bad_outputs(outs, 5, ins, 3, same)) return MUONH_EINVAL;
  NormArgs a{};
  a.x = x;
  a.res = residual;
  a.gain = gain;
  a.h = h;
  a.y = y;
  a.rstd = rstd;
  a.q = static_cast<uint8_t*>(q);
  a.scales = static_cast<uint8_t*>(scales);
  a.n = n;
  a.width = width;
  a.eps = (double)eps;
  a.y_dt = internal_dtype(y_dtype);
  a.packs_output = packs == MUONH_PACK_OUTPUT ? 1 : 0;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const double per = (double)(dtype_size(x_dtype) + (h ? 2 * dtype_size(h_dtype) : 0) + (y ? dtype_size(y_dtype) : 0)) +
                     (q ? 33.0 / 32 : 0.0);
  ProfScope pf(s, PC_NORM, 0, (double)all * per);
  MUONH_TRY_HIP(launch_rms_norm(internal_dtype(x_dtype), residual ? internal_dtype(h_dtype) : -1, a, s));
  return MUONH_OK;
}

size_t muonh_rms_norm_grad_workspace(int64_t n, int64_t width) {
  if (check_rows(n, width, kNormMaxWidth) != MUONH_OK) return 0;
  return (size_t)up(4 * width * norm_grad_blocks(n, width), 256);
}

int muonh_rms_norm_grad(const void* dy, int dy_dtype, const void* x, const void* q, const void* scales, const float* rstd,
                        const float* gain, const void* dres, int dx_dtype, int64_t n, int64_t width, void* dx,
                        float* dgain, int accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  const int rc = check_rows(n, width, kNormMaxWidth);
  if (rc != MUONH_OK) return rc;
  if (bad_dtype(dy_dtype) || bad_dtype(dx_dtype) || (accumulate != 0 && accumulate != 1)) return MUONH_EINVAL;
  if ((x == nullptr) == (q == nullptr) && n > 0) return MUONH_EINVAL;
  if ((q == nullptr) != (scales == nullptr)) return MUONH_EINVAL;
  const int64_t sx = dtype_size(dx_dtype);
  if (bad_buffer(dy, n, dtype_size(dy_dtype)) || bad_buffer(rstd, n, 4) || bad_buffer(dx, n, sx)) return MUONH_EINVAL;
  if (misaligned(x, sx) || misaligned(dres, sx) || misaligned(gain, 4) || misaligned(dgain, 4)) return MUONH_EINVAL;
  const size_t scratch = dgain ? muonh_rms_norm_grad_workspace(n, width) : 0;
  if (dgain) {
    if (!workspace || misaligned(workspace, 256)) return MUONH_EINVAL;
    if (workspace_bytes < scratch) return MUONH_ENOMEM;
  }
  const int64_t all = n * width;
  const Span ins[] = {span_of(dy, all * dtype_size(dy_dtype)), span_of(x, all * sx), span_of(q, all),
                      span_of(scales, n * mx_blocks(width)), span_of(rstd, 4 * n), span_of(gain, 4 * width),
                      span_of(dres, all * sx)};
  const Span outs[] = {span_of(dx, all * sx), span_of(dgain, 4 * width), span_of(workspace, (int64_t)scratch)};
  const Span* const same[] = {&ins[6], nullptr, nullptr};
  if (bad_outputs(outs, 3, ins, 7, same)) return MUONH_EINVAL;
  if (n == 0 && (!dgain || accumulate)) return MUONH_OK;
  NormGradArgs a{};
  a.dy = dy;
  a.x = x;
  a.q = static_cast<const uint8_t*>(q);
  a.scales = static_cast<const uint8_t*>(scales);
  a.rstd = rstd;
  a.gain = gain;
  a.dres = dres;
  a.dx = dx;
  a.part = dgain && !norm_grad_columns(n, width) ? static_cast<float*>(workspace) : nullptr;
  a.dgain = dgain;
  a.n = n;
  a.width = width;
  a.accumulate = accumulate;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const double per = (double)(dtype_size(dy_dtype) + (dres ? 2 : 1) * sx) + (x ? (double)sx : 33.0 / 32);
  ProfScope pf(s, PC_NORMGRAD, 0, (double)all * per);
  MUONH_TRY_HIP(launch_rms_norm_grad(internal_dtype(dy_dtype), internal_dtype(dx_dtype), a, s));
  return MUONH_OK;
}

int muonh_mx_pack(const void* x, int x_dtype, int64_t n, int64_t width, void* q, void* scales, void* stream) {
  const int rc = check_rows(n, width, kActMaxWidth);
  if (rc != MUONH_OK) return rc;
  if (bad_dtype(x_dtype)) return MUONH_EINVAL;
  if (bad_buffer(x, n, dtype_size(x_dtype)) || bad_buffer(q, n, 1) || bad_buffer(scales, n, 1)) return MUONH_EINVAL;
  if (n == 0) return MUONH_OK;
  const Span ins[] = {span_of(x, n * width * dtype_size(x_dtype))};
  const Span outs[] = {span_of(q, n * width), span_of(scales, n * mx_blocks(width))};
  const Span* const same[] = {nullptr, nullptr};
  if (bad_outputs(outs, 2, ins, 1, same)) return MUONH_EINVAL;
  const MxArgs a{x, static_cast<uint8_t*>(q), static_cast<uint8_t*>(scales), nullptr, n, width};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  ProfScope pf(s, PC_MX, 0, (double)n * (double)width * ((double)dtype_size(x_dtype) + 33.0 / 32));
  MUONH_TRY_HIP(launch_mx_pack(internal_dtype(x_dtype), a, s));
  return MUONH_OK;
}

int muonh_mx_unpack(const void* q, const void* scales, int64_t n, int64_t width, void* out, int out_dtype, void* stream) {
  const int rc = check_rows(n, width, kActMaxWidth);
  if (rc != MUONH_OK) return rc;
  if (bad_dtype(out_dtype)) return MUONH_EINVAL;
  if (bad_buffer(out, n, dtype_size(out_dtype)) || bad_buffer(q, n, 1) || bad_buffer(scales, n, 1)) return MUONH_EINVAL;
  if (n == 0) return MUONH_OK;
  const Span ins[] = {span_of(q, n * width), span_of(scales, n * mx_blocks(width))};
  const Span outs[] = {span_of(out, n * width * dtype_size(out_dtype))};
  const Span* const same[] = {nullptr};
  if (bad_outputs(outs, 1, ins, 2, same)) return MUONH_EINVAL;
  const MxArgs a{nullptr, const_cast<uint8_t*>(static_cast<const uint8_t*>(q)),
                 const_cast<uint8_t*>(static_cast<const uint8_t*>(scales)), out, n, width};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  ProfScope pf(s, PC_MX, 0, (double)n * (double)width * ((double)dtype_size(out_dtype) + 33.0 / 32));
  MUONH_TRY_HIP(launch_mx_unpack(internal_dtype(out_dtype), a, s));
  return MUONH_OK;
}

size_t muonh_weight_grad_workspace(const void* dz, int64_t n, int64_t rows, int64_t width) {
  if (check_wgrad(dz, n, rows, width) != MUONH_OK) return 0;
  return (size_t)wgrad_plan(dz, n, rows, width).bytes;
}

int muonh_weight_grad(const void* dz, const void* q, const void* scales, const float* gain, float scale, int64_t n,
                      int64_t rows, int64_t width, void* dw, int dw_dtype, int accumulate, void* workspace,
                      size_t workspace_bytes, void* stream) {
  const int rc = check_wgrad(dz, n, rows, width);
  if (rc != MUONH_OK) return rc;
  if (bad_dtype(dw_dtype) || (accumulate != 0 && accumulate != 1) || !std::isfinite(scale)) return MUONH_EINVAL;
  if (bad_buffer(dz, n, 2) || bad_buffer(q, n, 1) || bad_buffer(scales, n, 1)) return MUONH_EINVAL;
  if (!dw || misaligned(dw, dtype_size(dw_dtype)) || misaligned(gain, 4)) return MUONH_EINVAL;
  if (!workspace || misaligned(workspace, 256)) return MUONH_EINVAL;
  const WgradPlan p = wgrad_plan(dz, n, rows, width);
  if (workspace_bytes < (size_t)p.bytes) return MUONH_ENOMEM;
  const Span ins[] = {span_of(dz, 2 * n * rows), span_of(q, n * width), span_of(scales, n * mx_blocks(width)),
                      span_of(gain, 4 * width)};
  const Span outs[] = {span_of(dw, rows * width * dtype_size(dw_dtype)), span_of(workspace, p.bytes)};
  const Span* const same[] = {nullptr, nullptr};
  if (bad_outputs(outs, 2, ins, 4, same)) return MUONH_EINVAL;
  if (n == 0 && accumulate) return MUONH_OK;
  char* const ws = static_cast<char*>(workspace);
  WgradArgs a{};
  a.dz = static_cast<const uint16_t*>(dz);
  a.q = static_cast<const uint8_t*>(q);
  a.scales = static_cast<const uint8_t*>(scales);
  a.gain = n > 0 ? gain : nullptr;  // of no tokens the sums stay 0, whatever the factors are
  a.dw = dw;
  a.xt = reinterpret_cast<uint16_t*>(ws + p.xt);
  a.dzt = reinterpret_cast<uint16_t*>(ws + p.dzt);
  a.part = reinterpret_cast<float*>(ws + p.part);
  a.n = n;
  a.npad = p.npad;
  a.rows = rows;
  a.width = width;
  a.ldxt = p.ldxt;
  a.lddz = p.lddz;
  a.dfull = p.dfull;
  a.ldp = p.ldp;
  a.whole = p.whole;
  a.scale = n > 0 ? scale : 1.f;
  a.dw_dt = internal_dtype(dw_dtype);
  a.accumulate = accumulate;
  a.splits = p.splits;
  a.first = p.first;
  a.tile = p.tile;
  a.turn = p.turn ? 1 : 0;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (p.tile == kXTile) {
    ProfScope pf(s, PC_WPREP, 0, 3.0 * (double)n * (double)width);
    MUONH_TRY_HIP(launch_wgrad_prepare(a, s));
  }
  ProfScope pf(s, PC_WGRAD, 2.0 * (double)n * (double)rows * (double)width, 0);
  MUONH_TRY_HIP(launch_wgrad(a, s));
  return MUONH_OK;
}

}  // extern "C"
