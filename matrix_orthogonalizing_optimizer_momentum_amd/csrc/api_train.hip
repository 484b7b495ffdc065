// Entry points around the optimizer step: gradient norm and clipping, the
// embedding and its gradient, the output layer's cross entropy.  They hold no
// state: each call validates, computes its layout on the host and queues
// kernels on the caller's stream, with scratch memory from the caller.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <memory>
#include <new>

#include "checks.h"
#include "desc.h"
#include "embed.h"
#include "grad.h"
#include "muonh.h"
#include "runtime.h"
#include "xent.h"

namespace muonh {
namespace {

// ------------------------------------------------------------ gradient norm
// Blocks of all tensors together: about 8 for each of the 256 CUs (all
// resident at once), at least kMinChunk bytes each.
constexpr int64_t kGradBlocks = 2048;
constexpr int64_t kMinChunk = 32768;
// Gradients above this size (the last-level cache) are read past the caches:
// 3.5 GB of bf16 600 -> 534 us.  Smaller ones stay there for the step that
// reads them next, as does what is left of larger ones for clipping's second
// pass (470 MB: 232 us, 252 past the caches).
constexpr int64_t kGradOnceBytes = (int64_t)256 << 20;

int64_t grad_bytes(int64_t numel, int dtype) { return numel * (dtype == MUONH_BF16 ? 2 : 4); }

// Bytes per block: with it the blocks of n tensors are at most
// kGradBlocks + n.
int64_t grad_chunk(int64_t bytes) {
  return std::max(kMinChunk, up((bytes + kGradBlocks - 1) / kGradBlocks, 8192));
}

// total: bytes of all gradients.
int check_grads(const void* const* grads, const int64_t* numel, const int* dtypes, int n, int64_t& total) {
  if (!grads || !numel || !dtypes || n <= 0) return MUONH_EINVAL;
  if (n > (1 << 24)) return MUONH_ENOTIMPL;
  total = 0;
  for (int i = 0; i < n; ++i) {
    if (numel[i] < 0 || numel[i] > ((int64_t)1 << 46)) return MUONH_EINVAL;
    if (dtypes[i] != MUONH_F32 && dtypes[i] != MUONH_BF16) return MUONH_EINVAL;
    if (numel[i] > 0 && !grads[i]) return MUONH_EINVAL;
    if (numel[i] > 0 && (uintptr_t)grads[i] % (dtypes[i] == MUONH_F32 ? 4 : 2) != 0) return MUONH_EINVAL;
    total += grad_bytes(numel[i], dtypes[i]);
  }
  return total > ((int64_t)1 << 50) ? MUONH_EINVAL : MUONH_OK;
}

// Clipping writes outs[i] while it reads grads: outs must not overlap each
// other, nor a gradient other than their own, in place.
int check_outs(const void* const* grads, void* const* outs, const int64_t* numel, const int* dtypes, int n) {
  std::unique_ptr<Span[]> v(new (std::nothrow) Span[n]);
  if (!v) return MUONH_ENOMEM;
  auto span = [&](const void* p, int i) { return span_of(p, grad_bytes(numel[i], dtypes[i])); };
  int m = 0;
  for (int i = 0; i < n; ++i)
    if (numel[i] > 0) v[m++] = span(outs[i], i);
  Span* const end = v.get() + m;
  std::sort(v.get(), end, [](const Span& x, const Span& y) { return x.lo < y.lo; });
  for (int k = 1; k < m; ++k)
    if (v[k].lo < v[k - 1].hi) return MUONH_EINVAL;
  for (int i = 0; i < n; ++i) {
    if (numel[i] == 0 || grads[i] == outs[i]) continue;
    const Span g = span(grads[i], i);
    const Span* const o = std::partition_point(v.get(), end, [&](const Span& x) { return x.hi <= g.lo; });
    if (o != end && o->lo < g.hi) return MUONH_EINVAL;
  }
  return MUONH_OK;
}

// Its scalars are written before the gradients are read again, and read beside
// the writing of outs.
int check_clip_scalars(const float* total, const float* coef, const void* const* grads, void* const* outs,
                       const int64_t* numel, const int* dtypes, int n) {
  const Span t = span_of(total, 4), c = span_of(coef, 4);
  if (overlap(t, c)) return MUONH_EINVAL;
  for (int i = 0; i < n; ++i)
    for (const void* p : {grads[i], (const void*)outs[i]}) {
      const Span s = span_of(p, grad_bytes(numel[i], dtypes[i]));
      if (overlap(s, t) || overlap(s, c)) return MUONH_EINVAL;
    }
  return MUONH_OK;
}

// The table of tensors [i0, i0 + t.n) and its number of blocks.
int fill_table(GradTab& t, const void* const* grads, const int64_t* numel, const int* dtypes, int i0, int n,
               int64_t chunk) {
  t.n = std::min(n - i0, kTabTensors);
  t.tensor0 = i0;
  t.chunk = chunk;
  std::fill(t.bf16, t.bf16 + kTabTensors / 32, 0u);
  int64_t b = 0;
  for (int k = 0; k < t.n; ++k) {
    t.in[k] = grads[i0 + k];
    t.numel[k] = numel[i0 + k];
    t.first[k] = (int32_t)b;
    if (dtypes[i0 + k] == MUONH_BF16) t.bf16[k / 32] |= 1u << (k % 32);
    b += std::max<int64_t>(1, (grad_bytes(numel[i0 + k], dtypes[i0 + k]) + chunk - 1) / chunk);
  }
  return (int)b;
}

int queue_norm(const void* const* grads, const int64_t* numel, const int* dtypes, int n, int64_t bytes,
               bool once, float max_norm, float* total, float* coef, float* norms, void* ws, hipStream_t s) {
  const int64_t chunk = grad_chunk(bytes);
  int32_t* const bounds = reinterpret_cast<int32_t*>(ws);
  double* const partials = reinterpret_cast<double*>(reinterpret_cast<char*>(ws) + up(4 * (int64_t)n, 256));
  ProfScope pf(s, PC_GNORM, 0, (double)bytes);
  int part = 0;
  for (int i0 = 0; i0 < n; i0 += kTabTensors) {
    GradTab t;
    const int nb = fill_table(t, grads, numel, dtypes, i0, n, chunk);
    t.part0 = part;
    part += nb;
    MUONH_TRY_HIP(launch_grad_sumsq(t, nb, once, partials, bounds, s));
  }
  MUONH_TRY_HIP(launch_grad_finish(partials, bounds, n, part, max_norm, total, coef, norms, s));
  return MUONH_OK;
}

// ------------------------------------------------------------------ embedding
// n tokens, a table of rows x width; n = 0 is allowed.
int check_embedding(const void* ids, int id_bits, int64_t n, int64_t rows, int64_t width) {
  if (n < 0 || rows < 1 || rows >= INT32_MAX || width < 1) return MUONH_EINVAL;
  if (id_bits != 32 && id_bits != 64) return MUONH_EINVAL;
  if (n > 0 && (!ids || misaligned(ids, id_bits / 8))) return MUONH_EINVAL;
  // what the kernels' grids hold (below 2^32 threads a launch)
  return width > kEmbMaxWidth || n > kEmbMaxTokens || n * up(width, 8) > ((int64_t)1 << 36) ? MUONH_ENOTIMPL
                                                                                              : MUONH_OK;
}

// Scratch of the embedding gradient.
struct EmbedPlan {
  bool solo;
  int need, bits, passes, tile, blocks, run;
  int64_t key[2], pos[2], hist, part, bytes;
};

EmbedPlan embed_plan(int64_t n, int64_t rows, int64_t width) {
  EmbedPlan p{};
  int need = 1;  // bits of the largest key, rows itself (the ignored tokens)
  while (((int64_t)1 << need) <= rows) ++need;
  p.need = need;
  p.solo = n <= kSoloTokens;
  p.passes = (need + kSortBits - 1) / kSortBits;
  p.bits = (need + p.passes - 1) / p.passes;
  // tiles of at least 1024 tokens (256 a wave), at most kSortMaxBlocks of them:
  // every block reads the counts of all
  p.tile = (int)std::max<int64_t>(1024, up((n + kSortMaxBlocks - 1) / kSortMaxBlocks, 256));
  p.blocks = (int)((n + p.tile - 1) / p.tile);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += up(bytes, 256);
    return o;
  };
  for (int k = 0; k < 2; ++k) {
    p.key[k] = take(4 * n);
    p.pos[k] = take(4 * n);
  }
  p.hist = take(4 * ((int64_t)p.blocks << p.bits));
  // Pieces as long as leave 8 waves a CU (a wave takes 512 columns of a piece):
  // long ones save partial rows, short ones fill the chip at few tokens.
  p.run = kRunMax;
  while (p.run > kRunMin && (n + p.run - 1) / p.run * ((width + 511) / 512) < 2048) p.run /= 2;
  p.part = take(8 * ((n + p.run - 1) / p.run) * up(width, 8));
  p.bytes = std::max<int64_t>(at, 256);
  return p;
}

// ------------------------------------------------------------ cross entropy
// Scratch of one call: what every call needs, then what the gradients need.
struct XentPlan {
  bool few, copy_w;
  int64_t npad, rpad, wpad, wfull, ldxt, cols, splits;
  int64_t sc, xp, xt, perm, tgt, lse, tlogit, wcopy, area, dxacc, bytes;
};

// P of one piece, in bytes, unless the caller sets a workspace limit.  Larger
// pieces leave fewer passes over dx's sums and fuller rounds: at 8192 tokens,
// 50257 words, width 768 128 MiB take 2.76 ms, 256 2.69, 512 2.62, 1024 2.66.
constexpr int64_t kXentPieceBytes = (int64_t)512 << 20;

int check_xent(const void* w, int64_t n, int64_t rows, int64_t width) {
  if (n < 0 || rows < 1 || width < 1 || (w && misaligned(w, 2))) return MUONH_EINVAL;
  // what the kernels' grids hold (below 2^32 threads a launch)
  if (n > kXMaxTokens || rows > kXMaxRows || width > kXMaxWidth) return MUONH_ENOTIMPL;
  return up(n, kXTile) * up(width, kXTile) > ((int64_t)1 << 34) ? MUONH_ENOTIMPL : MUONH_OK;
}

// Time of a launch in units of one operand stage: n1 jobs of c1, then n2 of c2,
// each taken by the first compute unit that is free.
int64_t makespan(int64_t n1, int64_t c1, int64_t n2, int64_t c2) {
  const int64_t late = n1 % kXCus, early = kXCus - late;  // units that end the first kind a round later
  int64_t te = n1 / kXCus * c1, tl = te + c1, end = late ? tl : te;
  while (n2 > 0) {
    if (te <= tl || late == 0) {
      n2 -= early;
      end = std::max(end, te += c2);
    } else {
      n2 -= late;
      end = std::max(end, tl += c2);
    }
  }
  return end;
}

// Estimated time of both gradients with pieces of `tiles` tiles and dx in
// `splits` parts (also where only one is asked for, so that dx is the same
// sum of parts with and without dw).  Beside its stages a job costs the time of
// a few more: a stage takes 1.6 us, a tile of P 3 us beside its own, one of dw
// 9, one of dx 16 (256 KiB of sums, stored by all compute units at once), or 28
// where it adds to the sums of the pieces before.
int64_t xent_cost(int64_t ntok, int64_t nvoc, int64_t wpad, int64_t tiles, int64_t splits) {
  constexpr int64_t kProbExtra = 2, kDwExtra = 6, kDxExtra = 10, kDxAddExtra = 18;
  const int64_t nd = up(wpad, kXTile) / kXTile, per = kXTile / kXStage;
  auto piece = [&](int64_t k, bool first) {
    const int64_t cw = ntok * per + kDwExtra;
    const int64_t cx = (k * per + splits - 1) / splits + (first ? kDxExtra : kDxAddExtra);
    const int64_t nw = k * nd, nx = ntok * nd * splits;
    return makespan(ntok * k, wpad / kXStage + kProbExtra, 0, 0) +
           (cx > cw ? makespan(nx, cx, nw, cw) : makespan(nw, cw, nx, cx));
  };
  const int64_t whole = nvoc / tiles;
  int64_t t = piece(tiles, true) + (whole - 1) * piece(tiles, false);
  if (nvoc % tiles) t += piece(nvoc % tiles, false);
  return t;
}

// Layout for a piece of `cols` words (0: no gradient).
XentPlan xent_layout(const void* w, int64_t n, int64_t rows, int64_t width, bool dx, bool dw, int64_t cols,
                     int64_t splits) {
  XentPlan p{};
  // w's rows are an operand as they stand when they are whole stages on a
  // 16-byte grid; else the call works on a padded copy
  p.copy_w = width % kXStage != 0 || misaligned(w, 16);
  p.npad = up(std::max<int64_t>(n, 1), kXTile);
  p.rpad = up(rows, kXTile);
  p.wpad = up(width, kXStage);
  p.wfull = p.copy_w ? p.rpad : rows / kXTile * kXTile;
  p.cols = cols;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += up(bytes, 256);
    return o;
  };
  p.sc = take(sizeof(XentScalars));
  p.xp = take(2 * p.npad * p.wpad);
  p.ldxt = p.npad + 128;  // off the powers of two, so that rows fall on different memory channels
  p.xt = take(dw ? 2 * up(p.wpad, kXTile) * p.ldxt : 0);
  p.perm = take(4 * p.npad);
  p.tgt = take(4 * p.npad);
  p.lse = take(4 * p.npad);
  p.tlogit = take(4 * p.npad);
  p.wcopy = take(2 * (p.copy_w ? p.rpad : p.rpad - p.wfull) * p.wpad);
  // the statistics are read before the first piece's P is written
  p.area = take(std::max<int64_t>(8 * (p.rpad / kXTile) * p.npad, 2 * p.npad * cols));
  if (cols > 0) {
    p.splits = splits;
    if (dx) p.dxacc = take(4 * p.splits * p.npad * p.wpad);
  }
  p.bytes = at;
  return p;
}

// The piece and split, among those whose layout fits `limit`, that fill the
// rounds of the chip best (by xent_cost): pieces of the largest size down to
// half of it, smaller ones only where the limit asks for them.
int xent_plan(const void* w, int64_t n, int64_t rows, int64_t width, bool dx, bool dw, int64_t limit, XentPlan& p) {
  const int64_t npad = up(std::max<int64_t>(n, 1), kXTile), rpad = up(rows, kXTile);
  if (!dx && !dw) {
    if (n <= kXFewTokens && width >= 8) {
      p = XentPlan{};
      p.few = true;
      p.area = up(4 * kXFewTokens, 256);  // behind the targets' logits
      p.bytes = p.area + up(8 * n * xent_few_blocks(rows), 256);
      return p.bytes <= limit ? MUONH_OK : MUONH_ENOMEM;
    }
    p = xent_layout(w, n, rows, width, false, false, 0, 1);
    return p.bytes <= limit ? MUONH_OK : MUONH_ENOMEM;
  }
  const int64_t ntok = npad / kXTile, nvoc = rpad / kXTile, wpad = up(width, kXStage);
  int64_t top = std::max<int64_t>(1, std::min(rpad, kXentPieceBytes / (2 * npad)) / kXTile);
  for (;; top = std::max<int64_t>(1, top / 2)) {
    int64_t best = 0, best_tiles = 0, best_splits = 0;
    const int64_t step = std::max<int64_t>(1, top / 32);
    for (int64_t tiles = top; tiles > top / 2; tiles -= step)
      for (int64_t splits = 1; splits <= kXMaxSplits && splits <= tiles; splits *= 2) {
        if (splits > 1 && 4 * splits * npad * wpad > kXSplitBytes) break;
        if (xent_layout(w, n, rows, width, dx, dw, tiles * kXTile, splits).bytes > limit) continue;
        const int64_t t = xent_cost(ntok, nvoc, wpad, tiles, splits);
        if (best_tiles == 0 || t < best) {
          best = t;
          best_tiles = tiles;
          best_splits = splits;
        }
      }
    if (best_tiles) {
      p = xent_layout(w, n, rows, width, dx, dw, best_tiles * kXTile, best_splits);
      return MUONH_OK;
    }
    if (top == 1) return MUONH_ENOMEM;
  }
}

}  // namespace
}  // namespace muonh

using namespace muonh;

extern "C" {

size_t muonh_grad_norm_workspace(int n) {
  if (n <= 0) return 0;
  return (size_t)(up(4 * (int64_t)n, 256) + 8 * (kGradBlocks + (int64_t)n));
}

int muonh_grad_norm(const void* const grads[], const int64_t numel[], const int dtypes[], int n, float max_norm,
                    float* total, float* coef, float* norms, void* workspace, size_t workspace_bytes, void* stream) {
  int64_t bytes = 0;
  const int rc = check_grads(grads, numel, dtypes, n, bytes);
  if (rc != MUONH_OK) return rc;
  if (!total || !workspace || (uintptr_t)workspace % 256 != 0) return MUONH_EINVAL;
  if (coef && (!std::isfinite(max_norm) || max_norm < 0.f)) return MUONH_EINVAL;
  if (workspace_bytes < muonh_grad_norm_workspace(n)) return MUONH_ENOMEM;
  return queue_norm(grads, numel, dtypes, n, bytes, bytes > kGradOnceBytes, max_norm, total, coef, norms, workspace,
                    reinterpret_cast<hipStream_t>(stream));
}

int muonh_clip_grads(const void* const grads[], void* const outs[], const int64_t numel[], const int dtypes[], int n,
                     float max_norm, float* total, float* coef, void* workspace, size_t workspace_bytes,
                     void* stream) {
  int64_t bytes = 0;
  const int rc = check_grads(grads, numel, dtypes, n, bytes);
  if (rc != MUONH_OK) return rc;
  if (!outs || !total || !coef || !workspace || (uintptr_t)workspace % 256 != 0) return MUONH_EINVAL;
  for (int i = 0; i < n; ++i)
    if (numel[i] > 0 && (!outs[i] || (uintptr_t)outs[i] % (dtypes[i] == MUONH_F32 ? 4 : 2) != 0)) return MUONH_EINVAL;
  if (!std::isfinite(max_norm) || max_norm < 0.f) return MUONH_EINVAL;
  const int rd = check_outs(grads, outs, numel, dtypes, n);
  if (rd != MUONH_OK) return rd;
  if (workspace_bytes < muonh_grad_norm_workspace(n)) return MUONH_ENOMEM;
  const int rs = check_clip_scalars(total, coef, grads, outs, numel, dtypes, n);
  if (rs != MUONH_OK) return rs;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const int rq = queue_norm(grads, numel, dtypes, n, bytes, false, max_norm, total, coef, nullptr, workspace, s);
  if (rq != MUONH_OK) return rq;
  ProfScope pf(s, PC_GSCALE, 0, 2.0 * (double)bytes);
  const int64_t chunk = grad_chunk(bytes);
  for (int i0 = 0; i0 < n; i0 += kTabTensors) {
    ScaleTab t;
    const int nb = fill_table(t.g, grads, numel, dtypes, i0, n, chunk);
    for (int k = 0; k < t.g.n; ++k) t.out[k] = outs[i0 + k];
    MUONH_TRY_HIP(launch_grad_scale(t, nb, coef, s));
  }
  return MUONH_OK;
}

int muonh_embedding(const void* table, int table_dtype, int64_t rows, int64_t width, const void* ids, int id_bits,
                    int64_t n, float scale, void* out, int out_dtype, void* stream) {
  int rc = check_embedding(ids, id_bits, n, rows, width);
  if (rc != MUONH_OK) return rc;
  if (bad_dtype(table_dtype) || bad_dtype(out_dtype) || !std::isfinite(scale)) return MUONH_EINVAL;
  if (!table || misaligned(table, dtype_size(table_dtype))) return MUONH_EINVAL;
  if (n > 0 && (!out || misaligned(out, dtype_size(out_dtype)))) return MUONH_EINVAL;
  if (n == 0) return MUONH_OK;
  const Span o = span_of(out, n * width * dtype_size(out_dtype));
  if (overlap(o, span_of(table, rows * width * dtype_size(table_dtype))) || overlap(o, span_of(ids, n * (id_bits / 8))))
    return MUONH_EINVAL;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  ProfScope pf(s, PC_EMB, 0, (double)n * (double)width * (double)(dtype_size(table_dtype) + dtype_size(out_dtype)));
  const EmbedArgs a{table, ids, out, n, rows, width, scale, id_bits,
                    n * width * dtype_size(out_dtype) > kEmbOnceBytes ? 1 : 0};
  MUONH_TRY_HIP(launch_embedding(internal_dtype(table_dtype), internal_dtype(out_dtype), a, s));
  return MUONH_OK;
}

size_t muonh_embedding_grad_workspace(int64_t n, int64_t rows, int64_t width) {
  alignas(4) static const char any[4] = {};  // a pointer that passes for the ids
  if (check_embedding(any, 32, n, rows, width) != MUONH_OK) return 0;
  return (size_t)embed_plan(n, rows, width).bytes;
}

int muonh_embedding_grad(const void* ids, int id_bits, int64_t n, const void* dout, int dout_dtype, float scale,
                         int accumulate, void* dtable, int dtable_dtype, int64_t rows, int64_t width, void* workspace,
                         size_t workspace_bytes, void* stream) {
  int rc = check_embedding(ids, id_bits, n, rows, width);
  if (rc != MUONH_OK) return rc;
  if (bad_dtype(dout_dtype) || bad_dtype(dtable_dtype) || !std::isfinite(scale)) return MUONH_EINVAL;
  if (accumulate != 0 && accumulate != 1) return MUONH_EINVAL;
  if (!dtable || misaligned(dtable, dtype_size(dtable_dtype))) return MUONH_EINVAL;
  if (n > 0 && (!dout || misaligned(dout, dtype_size(dout_dtype)))) return MUONH_EINVAL;
  if (!workspace || misaligned(workspace, 256)) return MUONH_EINVAL;
  const EmbedPlan p = embed_plan(n, rows, width);
  if (workspace_bytes < (size_t)p.bytes) return MUONH_ENOMEM;
  const Span o = span_of(dtable, rows * width * dtype_size(dtable_dtype));
  if (overlap(o, span_of(dout, n * width * dtype_size(dout_dtype))) || overlap(o, span_of(ids, n * (id_bits / 8))))
    return MUONH_EINVAL;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  char* const ws = reinterpret_cast<char*>(workspace);
  auto u32 = [&](int64_t off) { return reinterpret_cast<uint32_t*>(ws + off); };
  int cur = 0;
  ZeroSlice z{static_cast<uint16_t*>(dtable), rows * width * dtype_size(dtable_dtype) / 2, 0, 0};
  if (n == 0) {
    z.count = accumulate ? 0 : 1;
    MUONH_TRY_HIP(launch_zero(z, s));
    return MUONH_OK;
  }
  if (p.solo) {
    ProfScope pf(s, PC_EMBSORT, 0, (double)n * (id_bits / 8 + 8.0) + (accumulate ? 0.0 : 2.0 * (double)z.halves));
    SortPass sp{};
    sp.ids = ids;
    sp.key_out = u32(p.key[0]);
    sp.pos_out = u32(p.pos[0]);
    sp.n = n;
    sp.rows = (uint32_t)rows;
    sp.id_bits = id_bits;
    sp.bits = p.need;
    z.count = accumulate ? 0 : 1;
    MUONH_TRY_HIP(launch_sort_solo(sp, z, s));
  } else {
    ProfScope pf(s, PC_EMBSORT, 0, (double)n * (id_bits / 8 + 16.0 * p.passes - 8.0) + (accumulate ? 0.0 : 2.0 * (double)z.halves));
    for (int k = 0; k < p.passes; ++k) {
      SortPass sp{};
      sp.ids = k == 0 ? ids : nullptr;
      sp.key_in = u32(p.key[cur]);
      sp.pos_in = u32(p.pos[cur]);
      sp.key_out = u32(p.key[cur ^ 1]);
      sp.pos_out = u32(p.pos[cur ^ 1]);
      sp.hist = u32(p.hist);
      sp.n = n;
      sp.rows = (uint32_t)rows;
      sp.id_bits = id_bits;
      sp.shift = k * p.bits;
      sp.bits = p.bits;
      sp.tile = p.tile;
      sp.blocks = p.blocks;
      ZeroSlice z0 = z, z1 = z;
      z0.count = z1.count = accumulate ? 0 : 2 * p.passes;
      z0.index = 2 * k;
      z1.index = 2 * k + 1;
      MUONH_TRY_HIP(launch_sort_pass(sp, z0, z1, s));
      cur ^= 1;
    }
  }
  ProfScope pf(s, PC_EMBGRAD, 0,
               (double)n * (double)width * (double)(dtype_size(dout_dtype) + dtype_size(dtable_dtype)));
  const EmbedGradArgs a{u32(p.key[cur]), u32(p.pos[cur]), dout, dtable, reinterpret_cast<float*>(ws + p.part),
                        n, rows, width, scale, accumulate, p.run};
  MUONH_TRY_HIP(launch_embedding_grad(internal_dtype(dout_dtype), internal_dtype(dtable_dtype), a, s));
  return MUONH_OK;
}

size_t muonh_cross_entropy_workspace(const void* w, int64_t n, int64_t rows, int64_t width, int grads, size_t limit) {
  if (check_xent(w, n, rows, width) != MUONH_OK || grads < 0 || grads > 3) return 0;
  XentPlan p;
  const int64_t lim = limit ? (int64_t)std::min<size_t>(limit, (size_t)INT64_MAX) : INT64_MAX;
  return xent_plan(w, n, rows, width, grads & 1, grads & 2, lim, p) == MUONH_OK ? (size_t)p.bytes : 0;
}

int muonh_cross_entropy(const void* x, const void* w, const void* targets, int id_bits, int64_t n, int64_t rows,
                        int64_t width, int64_t ignore_index, int reduction, float grad_scale, float* loss,
                        float* token_loss, void* dx, void* dw, int dw_dtype, int accumulate, void* workspace,
                        size_t workspace_bytes, void* stream) {
  int rc = check_xent(w, n, rows, width);
  if (rc != MUONH_OK) return rc;
  if (id_bits != 32 && id_bits != 64) return MUONH_EINVAL;
  if (reduction != MUONH_REDUCE_MEAN && reduction != MUONH_REDUCE_SUM) return MUONH_EINVAL;
  if (!std::isfinite(grad_scale) || bad_dtype(dw_dtype) || (accumulate != 0 && accumulate != 1)) return MUONH_EINVAL;
  if (!w || !loss || misaligned(loss, 4) || misaligned(token_loss, 4)) return MUONH_EINVAL;
  if (n > 0 && (!x || !targets || misaligned(x, 2) || misaligned(targets, id_bits / 8))) return MUONH_EINVAL;
  if (misaligned(dx, 2) || misaligned(dw, dtype_size(dw_dtype))) return MUONH_EINVAL;
  if (!workspace || misaligned(workspace, 256)) return MUONH_EINVAL;
  XentPlan p;
  rc = xent_plan(w, n, rows, width, dx != nullptr, dw != nullptr,
                 (int64_t)std::min<size_t>(workspace_bytes, (size_t)INT64_MAX), p);
  if (rc != MUONH_OK) return rc;
  // x is copied before anything but token_loss is written
  const Span outs[] = {span_of(loss, 4), span_of(token_loss, 4 * n), span_of(dx, 2 * n * width),
                       span_of(dw, rows * width * dtype_size(dw_dtype))};
  for (const Span& o : outs) {
    if (overlap(o, span_of(w, 2 * rows * width)) || overlap(o, span_of(targets, n * (id_bits / 8)))) return MUONH_EINVAL;
    for (const Span* other = outs; other != &o; ++other)
      if (overlap(*other, o)) return MUONH_EINVAL;
  }
  if (overlap(outs[1], span_of(x, 2 * n * width))) return MUONH_EINVAL;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  char* const ws = reinterpret_cast<char*>(workspace);
  auto u16 = [&](int64_t off) { return reinterpret_cast<uint16_t*>(ws + off); };
  auto f32 = [&](int64_t off) { return reinterpret_cast<float*>(ws + off); };
  XentArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.w = p.copy_w ? u16(p.wcopy) : static_cast<const uint16_t*>(w);
  a.wtail = u16(p.wcopy);
  a.targets = targets;
  a.xp = u16(p.xp);
  a.xt = u16(p.xt);
  a.perm = reinterpret_cast<int32_t*>(ws + p.perm);
  a.tgt = reinterpret_cast<int32_t*>(ws + p.tgt);
  a.lse = f32(p.lse);
  a.tlogit = f32(p.tlogit);
  a.stats = reinterpret_cast<float2*>(ws + p.area);
  a.prob = u16(p.area);
  a.dxacc = f32(p.dxacc);
  a.sc = reinterpret_cast<XentScalars*>(ws + p.sc);
  a.loss = loss;
  a.token_loss = token_loss;
  a.dx = static_cast<uint16_t*>(dx);
  a.dw = dw;
  a.n = n;
  a.npad = p.npad;
  a.rows = rows;
  a.rpad = p.rpad;
  a.wfull = p.wfull;
  a.width = width;
  a.wpad = p.wpad;
  a.ldxt = p.ldxt;
  a.ldw = p.copy_w ? p.wpad : width;
  a.ignore_index = ignore_index;
  a.grad_scale = grad_scale;
  a.id_bits = id_bits;
  a.mean = reduction == MUONH_REDUCE_MEAN ? 1 : 0;
  a.dw_dt = internal_dtype(dw_dtype);
  a.accumulate = accumulate;
  const double mac = 2.0 * (double)n * (double)rows * (double)width;
  if (p.few) {
    ProfScope pf(s, PC_XLOGIT, mac, 0);
    MUONH_TRY_HIP(launch_xent_few(a, s));
    return MUONH_OK;
  }
  {
    ProfScope pf(s, PC_XPREP, 0, 4.0 * (double)p.npad * (double)p.wpad);
    MUONH_TRY_HIP(launch_xent_prepare(a, p.copy_w, static_cast<const uint16_t*>(w), s));
  }
  {
    ProfScope pf(s, PC_XLOGIT, mac, 0);
    MUONH_TRY_HIP(launch_xent_stats(a, s));
  }
  MUONH_TRY_HIP(launch_xent_loss(a, s));
  if (!dx && !dw) return MUONH_OK;
  for (int64_t v0 = 0; v0 < p.rpad; v0 += p.cols) {
    XentPiece pc{v0, std::min(p.cols, p.rpad - v0), (int32_t)p.splits, v0 == 0 ? 1 : 0, 0};
    pc.dx_first = pc.cols / pc.splits > p.npad ? 1 : 0;  // the longer jobs first
    const double share = (double)pc.cols / (double)p.rpad;
    {
      ProfScope pf(s, PC_XPROB, mac * share, 0);
      MUONH_TRY_HIP(launch_xent_prob(a, pc, s));
    }
    ProfScope pf(s, PC_XGRAD, ((dx ? 1 : 0) + (dw ? 1 : 0)) * mac * share, 0);
    MUONH_TRY_HIP(launch_xent_grad(a, pc, s));
  }
  if (dx && n > 0) MUONH_TRY_HIP(launch_xent_dx(a, (int)p.splits, s));
  return MUONH_OK;
}

}  // extern "C"
