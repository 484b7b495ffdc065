// Embedding lookup and its gradient (gfx950).
//
//   out[i]    = scale * table[id_i]                     (0 for an id outside [0, rows))
//   dtable[v] = scale * sum over { i : id_i = v } of dout[i]
//
// The gradient sorts the tokens by id (stable: tokens of one id stay in batch
// order), so that every row of the table is summed in a fixed order without
// atomics.  Sorted tokens are cut into pieces of kRun; a piece sums its runs of
// equal ids in fp32 and writes the rows whose run lies inside it.  Runs that
// cross pieces (frequent tokens) leave one partial row per piece, which
// k_embed_join adds in order.  All of it is bound by HBM: dout is read once and
// the table's gradient is written once, the rows without a token included.
#include "common.h"
#include "embed.h"

namespace muonh {

namespace {

__device__ __forceinline__ uint32_t token_key(const void* ids, int id_bits, int64_t i, uint32_t rows) {
  if (id_bits == 32) {
    const uint32_t v = gmem(reinterpret_cast<const uint32_t*>(ids))[i];
    return v < rows ? v : rows;  // a negative id is a large unsigned one (rows < 2^31)
  }
  const uint64_t v = gmem(reinterpret_cast<const uint64_t*>(ids))[i];
  return v < rows ? (uint32_t)v : rows;
}

// ---------------------------------------------------------------------------
// lookup
// ---------------------------------------------------------------------------
// Flat over the V-element chunks of the output; a block's first row and chunk
// come from one 64-bit division, a thread's from a 32-bit one.
constexpr int kEmbThreads = 256;
constexpr int kEmbPer = 4;  // chunks per thread, all loads in flight together

template <typename TT, typename OT, int V>
__global__ __launch_bounds__(kEmbThreads) void k_embedding(const EmbedArgs a, uint32_t cpr) {
  const int64_t c0 = (int64_t)blockIdx.x * (kEmbThreads * kEmbPer);
  const int64_t row0 = c0 / cpr;
  const uint32_t off0 = (uint32_t)(c0 - row0 * cpr);
  const TT* const table = reinterpret_cast<const TT*>(a.table);
  OT* const out = reinterpret_cast<OT*>(a.out);
  int64_t row[kEmbPer];
  uint32_t col[kEmbPer], key[kEmbPer];
#pragma unroll
  for (int k = 0; k < kEmbPer; ++k) {
    const uint32_t x = off0 + threadIdx.x + k * kEmbThreads;
    const uint32_t q = x / cpr;
    row[k] = row0 + q;
    col[k] = (x - q * cpr) * V;
    key[k] = row[k] < a.n ? token_key(a.ids, a.id_bits, row[k], (uint32_t)a.rows) : (uint32_t)a.rows;
  }
  if constexpr (V == 8) {
    Raw8<TT> r[kEmbPer];
#pragma unroll
    for (int k = 0; k < kEmbPer; ++k)
      if (key[k] < a.rows) r[k].load(table, (int64_t)key[k] * a.width + col[k]);
#pragma unroll
    for (int k = 0; k < kEmbPer; ++k) {
      if (row[k] >= a.n) continue;
      float v[8];
      r[k].unpack(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = key[k] < a.rows ? a.scale * v[e] : 0.f;
      store8(out, row[k] * a.width + col[k], v);
    }
  } else {
#pragma unroll
    for (int k = 0; k < kEmbPer; ++k) {
      if (row[k] >= a.n) continue;
      const float v = key[k] < a.rows ? a.scale * St<TT>::ld(table, (int64_t)key[k] * a.width + col[k]) : 0.f;
      St<OT>::st(out, row[k] * a.width + col[k], v);
    }
  }
}

// ---------------------------------------------------------------------------
// stable sort of the tokens by id: counting passes over digits of the id, the
// lowest first.  A block owns a contiguous tile of tokens, a wave of it a
// contiguous quarter.
// ---------------------------------------------------------------------------
constexpr int kSortWaves = kSortThreads / 64;

__device__ __forceinline__ uint32_t pass_key(const SortPass& p, int64_t i) {
  return p.ids != nullptr ? token_key(p.ids, p.id_bits, i, p.rows) : gmem(p.key_in)[i];
}

__global__ __launch_bounds__(kSortThreads) void k_sort_count(const SortPass p) {
  __shared__ uint32_t cnt[1 << kSortBits];
  const uint32_t bins = 1u << p.bits;
  for (uint32_t d = threadIdx.x; d < bins; d += kSortThreads) cnt[d] = 0;
  __syncthreads();
  const int64_t lo = (int64_t)blockIdx.x * p.tile, hi = min(p.n, lo + p.tile);
  for (int64_t i = lo + threadIdx.x; i < hi; i += kSortThreads)
    atomicAdd(&cnt[(pass_key(p, i) >> p.shift) & (bins - 1)], 1u);
  __syncthreads();
  for (uint32_t d = threadIdx.x; d < bins; d += kSortThreads) gmem(p.hist)[(int64_t)blockIdx.x * bins + d] = cnt[d];
}

__global__ __launch_bounds__(kSortThreads) void k_sort_scatter(const SortPass p) {
  // next free place of each digit, one table per wave
  __shared__ uint32_t next[kSortWaves][1 << kSortBits];
  __shared__ uint32_t sums[kSortWaves];
  const uint32_t bins = 1u << p.bits;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t lo = (int64_t)blockIdx.x * p.tile;
  const int quarter = p.tile / kSortWaves;
  const int64_t wlo = min(p.n, lo + (int64_t)wave * quarter), whi = min(p.n, wlo + quarter);
  for (uint32_t d = tid; d < kSortWaves * bins; d += kSortThreads) next[d / bins][d % bins] = 0;
  __syncthreads();
  for (int64_t i = wlo + lane; i < whi; i += 64) atomicAdd(&next[wave][(pass_key(p, i) >> p.shift) & (bins - 1)], 1u);
  __syncthreads();
  // Thread t owns the digits [t * per, (t + 1) * per): the place of a digit's
  // first token in this block is the number of tokens with smaller digits
  // plus those with this digit in the blocks before.
  const uint32_t per = max(1u, bins / kSortThreads);
  uint32_t tot[(1 << kSortBits) / kSortThreads], before[(1 << kSortBits) / kSortThreads];
  uint32_t mine = 0;
  const bool owner = tid * per < bins;
#pragma unroll
  for (uint32_t k = 0; k < (1 << kSortBits) / kSortThreads; ++k) {
    tot[k] = before[k] = 0;
    if (k < per && owner) {
      const uint32_t d = tid * per + k;
      for (int b = 0; b < p.blocks; ++b) {
        const uint32_t c = gmem(p.hist)[(int64_t)b * bins + d];
        tot[k] += c;
        if (b < (int)blockIdx.x) before[k] += c;
      }
      mine += tot[k];
    }
  }
  uint32_t incl = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t v = __shfl_up(incl, o, 64);
    if (lane >= o) incl += v;
  }
  if (lane == 63) sums[wave] = incl;
  __syncthreads();
  uint32_t base = incl - mine;
  for (int w = 0; w < wave; ++w) base += sums[w];
#pragma unroll
  for (uint32_t k = 0; k < (1 << kSortBits) / kSortThreads; ++k) {
    if (k < per && owner) {
      const uint32_t d = tid * per + k;
      uint32_t at = base + before[k];
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) {
        const uint32_t c = next[w][d];
        next[w][d] = at;
        at += c;
      }
      base += tot[k];
    }
  }
  __syncthreads();
  // 64 tokens at a time, in order: a token's rank among the wave's equal
  // digits is the number of lower lanes that hold the same one.
  for (int64_t i0 = wlo; i0 < whi; i0 += 64) {
    const int64_t i = i0 + lane;
    const bool in = i < whi;
    const uint32_t key = in ? pass_key(p, i) : 0u;
    const uint32_t pos = in ? (p.ids != nullptr ? (uint32_t)i : gmem(p.pos_in)[i]) : 0u;
    const uint32_t d = (key >> p.shift) & (bins - 1);
    uint64_t same = __ballot(in);
    for (int b = 0; b < p.bits; ++b) {
      const uint64_t m = __ballot((d >> b) & 1);
      same &= ((d >> b) & 1) ? m : ~m;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    const int lead = in ? __ffsll((unsigned long long)same) - 1 : lane;
    uint32_t first = 0;
    if (in && rank == 0) first = atomicAdd(&next[wave][d], (uint32_t)__popcll(same));
    first = __shfl(first, lead, 64);
    if (in) {
      gmem(p.key_out)[first + rank] = key;
      gmem(p.pos_out)[first + rank] = pos;
    }
  }
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------
constexpr int kEgThreads = 256;
constexpr int kZeroRows = 64;  // rows per block of the pass over rows without tokens

template <typename GT, int V> struct Chunk;
template <typename GT> struct Chunk<GT, 8> {
  Raw8<GT> r;
  __device__ __forceinline__ void load(const GT* p, int64_t i) { r.load(p, i); }
  __device__ __forceinline__ void add(float (&acc)[8]) const {
    float v[8];
    r.unpack(v);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += v[e];
  }
};
template <typename GT> struct Chunk<GT, 1> {
  float v;
  __device__ __forceinline__ void load(const GT* p, int64_t i) { v = St<GT>::ld(p, i); }
  __device__ __forceinline__ void add(float (&acc)[1]) const { acc[0] += v; }
};

template <typename OT>
__device__ __forceinline__ void put_row(const EmbedGradArgs& a, uint32_t key, int64_t col, const float (&acc)[8]) {
  OT* const o = reinterpret_cast<OT*>(a.dtable);
  const int64_t at = (int64_t)key * a.width + col;
  float v[8];
  if (a.accumulate) load8(o, at, v);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = a.accumulate ? fmaf(a.scale, acc[e], v[e]) : a.scale * acc[e];
  store8(o, at, v);
}
template <typename OT>
__device__ __forceinline__ void put_row(const EmbedGradArgs& a, uint32_t key, int64_t col, const float (&acc)[1]) {
  OT* const o = reinterpret_cast<OT*>(a.dtable);
  const int64_t at = (int64_t)key * a.width + col;
  St<OT>::st(o, at, a.accumulate ? fmaf(a.scale, acc[0], St<OT>::ld(o, at)) : a.scale * acc[0]);
}
__device__ __forceinline__ void put_part(float* p, int64_t i, const float (&acc)[8]) { store8(p, i, acc); }
__device__ __forceinline__ void put_part(float* p, int64_t i, const float (&acc)[1]) { gmem(p)[i] = acc[0]; }
__device__ __forceinline__ void add_part(const float* p, int64_t i, float (&acc)[8]) {
  float v[8];
  load8(p, i, v);
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] += v[e];
}
__device__ __forceinline__ void add_part(const float* p, int64_t i, float (&acc)[1]) { acc[0] += gmem(p)[i]; }

// Writes zeros to the rows [row0, row0 + kZeroRows) that hold no token.
template <typename OT, int V>
__device__ void zero_rows(const EmbedGradArgs& a, int64_t row0, uint32_t cpr) {
  __shared__ uint32_t absent[kZeroRows];
  if (threadIdx.x < kZeroRows) {
    const int64_t v = row0 + threadIdx.x;
    // first sorted place with a key >= v
    int64_t lo = 0, hi = a.n;
    while (lo < hi) {
      const int64_t mid = (lo + hi) >> 1;
      if (gmem(a.key)[mid] < v) lo = mid + 1;
      else hi = mid;
    }
    absent[threadIdx.x] = v < a.rows && (lo >= a.n || gmem(a.key)[lo] != v);
  }
  __syncthreads();
  OT* const o = reinterpret_cast<OT*>(a.dtable);
  for (uint32_t x = threadIdx.x; x < kZeroRows * cpr; x += kEgThreads) {
    const uint32_t r = x / cpr;
    if (!absent[r]) continue;
    const int64_t at = (row0 + r) * a.width + (int64_t)(x - r * cpr) * V;
    if constexpr (V == 8) {
      const float z[8] = {};
      store8(o, at, z);
    } else {
      St<OT>::st(o, at, 0.f);
    }
  }
}

// Blocks [0, nsum): sums; the others: rows without tokens.  One launch, so
// that the zeros are written while the sums wait for their gathered rows.
template <typename GT, typename OT, int V>
__global__ __launch_bounds__(kEgThreads) void k_embed_grad(const EmbedGradArgs a, uint32_t cpr, int nsum) {
  if ((int)blockIdx.x >= nsum) {
    zero_rows<OT, V>(a, (int64_t)((int)blockIdx.x - nsum) * kZeroRows, cpr);
    return;
  }
  const int64_t g = (int64_t)blockIdx.x * kEgThreads + threadIdx.x;
  const int64_t piece = g / cpr;
  const int64_t col = (g - piece * cpr) * V;
  const int64_t s = piece * kRun, e = min(a.n, s + kRun);
  if (s >= a.n) return;
  const GT* const dout = reinterpret_cast<const GT*>(a.dout);
  float* const head = a.part + 2 * piece * a.width;
  float* const tail = head + a.width;
  uint32_t cur = gmem(a.key)[s];
  bool before = s > 0 && gmem(a.key)[s - 1] == cur;
  float acc[V] = {};
  auto flush = [&](bool onward) {
    if (cur >= a.rows) return;
    if (before) put_part(head, col, acc);
    else if (onward) put_part(tail, col, acc);
    else put_row<OT>(a, cur, col, acc);
  };
  constexpr int U = 8;
  for (int64_t i0 = s; i0 < e; i0 += U) {
    uint32_t k[U];
    Chunk<GT, V> c[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = min(i0 + u, e - 1);
      k[u] = gmem(a.key)[i];
      c[u].load(dout, (int64_t)gmem(a.pos)[i] * a.width + col);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u >= e) break;
      if (k[u] != cur) {
        flush(false);
        cur = k[u];
        before = false;
#pragma unroll
        for (int x = 0; x < V; ++x) acc[x] = 0.f;
      }
      c[u].add(acc);
    }
  }
  flush(e < a.n && gmem(a.key)[e] == cur);
}

// Rows whose run crosses pieces: the piece where the run starts adds its tail
// and the heads of the pieces that follow.
template <typename OT, int V>
__global__ __launch_bounds__(kEgThreads) void k_embed_join(const EmbedGradArgs a, uint32_t cpr) {
  const int64_t piece = blockIdx.x;
  const int64_t s = piece * kRun, e = s + kRun;
  if (e >= a.n) return;
  const uint32_t k = gmem(a.key)[e - 1];
  if (k >= a.rows || gmem(a.key)[e] != k) return;
  if (s > 0 && gmem(a.key)[s - 1] == k) return;  // the run started in an earlier piece
  const int64_t pieces = (a.n + kRun - 1) / kRun;
  // pieces piece + 1 .. last begin with this key
  __shared__ int64_t last_s;
  if (threadIdx.x < 64) {
    int64_t q = piece + 1;
    for (;;) {
      const int64_t c = q + threadIdx.x;
      const bool same = c < pieces && gmem(a.key)[c * kRun] == k;
      const int run = __popcll(__ballot(same));  // keys are sorted: a prefix of the lanes
      q += run;
      if (run < 64) break;
    }
    if (threadIdx.x == 0) last_s = q;
  }
  __syncthreads();
  const int64_t end = last_s;
  for (uint32_t c = threadIdx.x; c < cpr; c += kEgThreads) {
    const int64_t col = (int64_t)c * V;
    float acc[V] = {};
    add_part(a.part + (2 * piece + 1) * a.width, col, acc);
    for (int64_t q = piece + 1; q < end; ++q) add_part(a.part + 2 * q * a.width, col, acc);
    put_row<OT>(a, k, col, acc);
  }
}

}  // namespace

// 16-byte accesses need rows of whole 8-element chunks on a 16-byte grid.
static bool vec8(int64_t width, const void* p, const void* q) {
  return width % 8 == 0 && ((uintptr_t)p | (uintptr_t)q) % 16 == 0;
}

hipError_t launch_embedding(int table_dt, int out_dt, const EmbedArgs& a, hipStream_t s) {
  const bool v8 = vec8(a.width, a.table, a.out);
  const uint32_t cpr = (uint32_t)(v8 ? a.width / 8 : a.width);
  const int64_t chunks = a.n * cpr, per = kEmbThreads * kEmbPer;
  const int64_t blocks = (chunks + per - 1) / per;
  if (blocks <= 0) return hipSuccess;
  if (blocks > INT32_MAX) return hipErrorInvalidValue;
#define MUONH_EMB(TT, OT)                                                                                   \
  do {                                                                                                      \
    if (v8) hipLaunchKernelGGL((k_embedding<TT, OT, 8>), dim3(blocks), dim3(kEmbThreads), 0, s, a, cpr);    \
    else hipLaunchKernelGGL((k_embedding<TT, OT, 1>), dim3(blocks), dim3(kEmbThreads), 0, s, a, cpr);       \
  } while (0)
  if (table_dt == DT_BF16 && out_dt == DT_BF16) MUONH_EMB(bf16_t, bf16_t);
  else if (table_dt == DT_BF16) MUONH_EMB(bf16_t, float);
  else if (out_dt == DT_BF16) MUONH_EMB(float, bf16_t);
  else MUONH_EMB(float, float);
#undef MUONH_EMB
  return hipGetLastError();
}

hipError_t launch_sort_pass(const SortPass& p, hipStream_t s) {
  hipLaunchKernelGGL(k_sort_count, dim3(p.blocks), dim3(kSortThreads), 0, s, p);
  hipLaunchKernelGGL(k_sort_scatter, dim3(p.blocks), dim3(kSortThreads), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_embedding_grad(int g_dt, int out_dt, const EmbedGradArgs& a, hipStream_t s) {
  const bool v8 = vec8(a.width, a.dout, a.dtable);
  const uint32_t cpr = (uint32_t)(v8 ? a.width / 8 : a.width);
  const int64_t pieces = (a.n + kRun - 1) / kRun;
  const int64_t nsum = (pieces * cpr + kEgThreads - 1) / kEgThreads;
  const int64_t nzero = a.accumulate ? 0 : (a.rows + kZeroRows - 1) / kZeroRows;
  if (nsum + nzero > INT32_MAX) return hipErrorInvalidValue;
#define MUONH_EG(GT, OT, V)                                                                                     \
  do {                                                                                                          \
    if (nsum + nzero > 0)                                                                                       \
      hipLaunchKernelGGL((k_embed_grad<GT, OT, V>), dim3(nsum + nzero), dim3(kEgThreads), 0, s, a, cpr, (int)nsum); \
    if (pieces > 1) hipLaunchKernelGGL((k_embed_join<OT, V>), dim3(pieces), dim3(kEgThreads), 0, s, a, cpr);    \
  } while (0)
#define MUONH_EG_V(GT, OT)       \
  do {                           \
    if (v8) MUONH_EG(GT, OT, 8); \
    else MUONH_EG(GT, OT, 1);    \
  } while (0)
  if (g_dt == DT_BF16 && out_dt == DT_BF16) MUONH_EG_V(bf16_t, bf16_t);
  else if (g_dt == DT_BF16) MUONH_EG_V(bf16_t, float);
  else if (out_dt == DT_BF16) MUONH_EG_V(float, bf16_t);
  else MUONH_EG_V(float, float);
#undef MUONH_EG_V
#undef MUONH_EG
  return hipGetLastError();
}

}  // namespace muonh
