// Embedding lookup and its gradient (gfx950).
//
//   out[i]    = scale * table[id_i]                     (0 for an id outside [0, rows))
//   dtable[v] = scale * sum over { i : id_i = v } of dout[i]
//
// The gradient sorts the tokens by id (stable: tokens of one id stay in batch
// order), so that every row of the table is summed in a fixed order without
// atomics.  Sorted tokens are cut into pieces; a piece sums its runs of equal
// ids in fp32 and writes the rows whose run lies inside it.  Runs that
// cross pieces (frequent tokens) leave one partial row per piece, which
// k_embed_join adds in order.
//
// All of it is bound by HBM: dout is read once, and the whole of the table's
// gradient is written.  The sort is a chain of short steps that leaves the
// chip idle, so its launches carry the clearing of the table in further
// workgroups: the zeros cost no time of their own, at the price of writing the
// rows that have tokens twice (8192 tokens on 50257 x 768 fp32: 25 of 154 MB).
#include "common.h"
#include "embed.h"

namespace muonh {

namespace {

// A row is cut into chunks of V columns: 8, at any alignment, or 1 for rows
// shorter than that.  The last chunk of a row that is no whole number of
// them is moved back to end with the row, and leaves its first `skip` columns
// to the chunk before.
template <int V>
__device__ __forceinline__ int64_t chunk_col(uint32_t chunk, int64_t width, int& skip) {
  if constexpr (V == 1) {
    skip = 0;
    return chunk;
  }
  const int64_t c = (int64_t)chunk * V, last = width - V;
  skip = (int)(c > last ? c - last : 0);
  return c - skip;
}

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
// Flat over the V-column chunks of the output; a block's first row and chunk
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
  int64_t col[kEmbPer];
  uint32_t key[kEmbPer];
  int skip[kEmbPer];
#pragma unroll
  for (int k = 0; k < kEmbPer; ++k) {
    const uint32_t x = off0 + threadIdx.x + k * kEmbThreads;
    const uint32_t q = x / cpr;
    row[k] = row0 + q;
    col[k] = chunk_col<V>(x - q * cpr, a.width, skip[k]);
    key[k] = row[k] < a.n ? token_key(a.ids, a.id_bits, row[k], (uint32_t)a.rows) : (uint32_t)a.rows;
  }
  if constexpr (V == 8) {
    Raw8<TT> r[kEmbPer];
#pragma unroll
    for (int k = 0; k < kEmbPer; ++k)
      if (key[k] < a.rows) r[k].load_any(table, (int64_t)key[k] * a.width + col[k]);
#pragma unroll
    for (int k = 0; k < kEmbPer; ++k) {
      if (row[k] >= a.n) continue;
      float v[8];
      r[k].unpack(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = key[k] < a.rows ? a.scale * v[e] : 0.f;
      const int64_t at = row[k] * a.width + col[k];
      if (skip[k] == 0 && a.once) {
        store8_once(out, at, v);
      } else if (skip[k] == 0) {
        store8_any(out, at, v);
      } else {
#pragma unroll
        for (int e = 1; e < 8; ++e)
          if (e >= skip[k]) St<OT>::st(out, at + e, v[e]);
      }
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
// clearing, as further workgroups (first_block on) of another launch
// ---------------------------------------------------------------------------
template <int NT>
__device__ void zero_slice(const ZeroSlice& z, int64_t block, int64_t blocks) {
  const int64_t head = min<int64_t>(((16 - (uintptr_t)z.p % 16) % 16) / 2, z.halves);
  const int64_t vecs = (z.halves - head) / 8, tail0 = head + vecs * 8;
  if (z.index == 0 && block == 0) {  // what lies before and after the 16-byte grid
    if (threadIdx.x < head) gmem(z.p)[threadIdx.x] = 0;
    if (threadIdx.x >= 64 && tail0 + (threadIdx.x - 64) < z.halves && threadIdx.x < 72)
      gmem(z.p)[tail0 + (threadIdx.x - 64)] = 0;
  }
  const int64_t lo = vecs * z.index / z.count, n = vecs * (z.index + 1) / z.count - lo;
  // a contiguous run a block
  const int64_t b0 = n * block / blocks, b1 = n * (block + 1) / blocks;
  MUONH_GLOBAL u32x4_t* const p = reinterpret_cast<MUONH_GLOBAL u32x4_t*>(gmem(z.p + head)) + lo;
  const u32x4_t zero = {0u, 0u, 0u, 0u};
  for (int64_t i = b0 + threadIdx.x; i < b1; i += NT) p[i] = zero;
}

__global__ __launch_bounds__(256) void k_zero(const ZeroSlice z) { zero_slice<256>(z, blockIdx.x, gridDim.x); }

// ---------------------------------------------------------------------------
// stable sort of the tokens by id: counting passes over digits of the id, the
// lowest first.  A block owns a contiguous tile of tokens, a wave of it a
// contiguous quarter.
// ---------------------------------------------------------------------------
constexpr int kSortWaves = kSortThreads / 64;

__device__ __forceinline__ uint32_t pass_key(const SortPass& p, int64_t i) {
  return p.ids != nullptr ? token_key(p.ids, p.id_bits, i, p.rows) : gmem(p.key_in)[i];
}

// The next place of digit d in a wave's table, for each lane with `in`: a
// token's rank among the wave's equal digits is the number of lower lanes that
// hold the same one, and the lowest of them moves the place on.
__device__ __forceinline__ uint32_t take_place(uint32_t* next, uint32_t d, int bits, bool in) {
  const int lane = threadIdx.x & 63;
  uint64_t same = __ballot(in);
  for (int b = 0; b < bits; ++b) {
    const uint64_t m = __ballot((d >> b) & 1);
    same &= ((d >> b) & 1) ? m : ~m;
  }
  const int rank = __popcll(same & ((1ull << lane) - 1));
  const int lead = in ? __ffsll((unsigned long long)same) - 1 : lane;
  uint32_t first = 0;
  if (in && rank == 0) first = atomicAdd(&next[d], (uint32_t)__popcll(same));
  return __shfl(first, lead, 64) + rank;
}

__global__ __launch_bounds__(kSortThreads) void k_sort_count(const SortPass p, const ZeroSlice z) {
  __shared__ uint32_t cnt[1 << kSortBits];
  if ((int)blockIdx.x >= p.blocks) {
    zero_slice<kSortThreads>(z, blockIdx.x - p.blocks, gridDim.x - p.blocks);
    return;
  }
  const uint32_t bins = 1u << p.bits;
  for (uint32_t d = threadIdx.x; d < bins; d += kSortThreads) cnt[d] = 0;
  __syncthreads();
  const int64_t lo = (int64_t)blockIdx.x * p.tile, hi = min(p.n, lo + p.tile);
  for (int64_t i = lo + threadIdx.x; i < hi; i += kSortThreads)
    atomicAdd(&cnt[(pass_key(p, i) >> p.shift) & (bins - 1)], 1u);
  __syncthreads();
  for (uint32_t d = threadIdx.x; d < bins; d += kSortThreads) gmem(p.hist)[(int64_t)blockIdx.x * bins + d] = cnt[d];
}

__global__ __launch_bounds__(kSortThreads) void k_sort_scatter(const SortPass p, const ZeroSlice z) {
  // next free place of each digit, one table per wave
  __shared__ uint32_t next[kSortWaves][1 << kSortBits];
  __shared__ uint32_t sums[kSortWaves];
  if ((int)blockIdx.x >= p.blocks) {
    zero_slice<kSortThreads>(z, blockIdx.x - p.blocks, gridDim.x - p.blocks);
    return;
  }
  const uint32_t bins = 1u << p.bits;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t lo = (int64_t)blockIdx.x * p.tile;
  const int quarter = p.tile / kSortWaves;
  const int64_t wlo = min(p.n, lo + (int64_t)wave * quarter), whi = min(p.n, wlo + quarter);
  for (uint32_t d = tid; d < kSortWaves * bins; d += kSortThreads) next[d / bins][d % bins] = 0;
  __syncthreads();
  constexpr int R = 4;  // rows of 64 tokens in flight
  for (int64_t i0 = wlo + lane; i0 < whi; i0 += 64 * R) {
    uint32_t k[R];
#pragma unroll
    for (int r = 0; r < R; ++r) k[r] = pass_key(p, min(i0 + 64 * r, whi - 1));
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (i0 + 64 * r < whi) atomicAdd(&next[wave][(k[r] >> p.shift) & (bins - 1)], 1u);
  }
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
      // a batch of blocks' counts in flight at a time
      constexpr int B = 32;
      for (int b0 = 0; b0 < p.blocks; b0 += B) {
        uint32_t c[B];
#pragma unroll
        for (int u = 0; u < B; ++u) c[u] = gmem(p.hist)[(int64_t)min(b0 + u, p.blocks - 1) * bins + d];
#pragma unroll
        for (int u = 0; u < B; ++u) {
          const uint32_t v = b0 + u < p.blocks ? c[u] : 0u;
          tot[k] += v;
          before[k] += b0 + u < (int)blockIdx.x ? v : 0u;
        }
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
  // 64 tokens at a time, in order
  for (int64_t i0 = wlo; i0 < whi; i0 += 64 * R) {
    uint32_t key[R], pos[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t i = min(i0 + 64 * r + lane, whi - 1);
      key[r] = pass_key(p, i);
      pos[r] = p.ids != nullptr ? (uint32_t)i : gmem(p.pos_in)[i];
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool in = i0 + 64 * r + lane < whi;
      const uint32_t at = take_place(next[wave], (key[r] >> p.shift) & (bins - 1), p.bits, in);
      if (in) {
        gmem(p.key_out)[at] = key[r];
        gmem(p.pos_out)[at] = pos[r];
      }
    }
  }
}

// All passes in one workgroup, the tokens in LDS between them: 16 waves, wave
// w owns a contiguous run of tokens.  At 8192 tokens it takes less than the
// launches of the passes above.
__global__ __launch_bounds__(kSoloThreads) void k_sort_solo(const SortPass p, const ZeroSlice z) {
  constexpr int NW = kSoloThreads / 64, BINS = 1 << kSoloBits;
  __shared__ uint32_t skey[kSoloTokens];
  __shared__ uint16_t spos[kSoloTokens];
  __shared__ uint32_t next[NW][BINS];
  __shared__ uint32_t sums[NW];
  if (blockIdx.x > 0) {
    zero_slice<kSoloThreads>(z, blockIdx.x - 1, gridDim.x - 1);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = (int)p.n;
  const int rounds = (n + kSoloThreads - 1) / kSoloThreads;
  const int i0 = wave * rounds * 64 + lane;  // this lane's tokens: i0 + 64 r
  uint32_t key[kSoloItems], pos[kSoloItems], at[kSoloItems];
#pragma unroll
  for (int r = 0; r < kSoloItems; ++r) {
    const int i = i0 + 64 * r;
    pos[r] = i;
    key[r] = r < rounds && i < n ? token_key(p.ids, p.id_bits, i, p.rows) : 0u;
  }
  for (int shift = 0; shift < p.bits; shift += kSoloBits) {
    const int bits = min(kSoloBits, p.bits - shift);
    for (int d = tid; d < NW * BINS; d += kSoloThreads) next[d / BINS][d % BINS] = 0;
    __syncthreads();
    // each token's place among its wave's equal digits; next ends as their counts
#pragma unroll
    for (int r = 0; r < kSoloItems; ++r)
      if (r < rounds) at[r] = take_place(next[wave], (key[r] >> shift) & (BINS - 1), bits, i0 + 64 * r < n);
    __syncthreads();
    // digit tid: where it starts, then where each wave's share of it starts
    uint32_t tot = 0;
    if (tid < BINS) {
#pragma unroll
      for (int w = 0; w < NW; ++w) tot += next[w][tid];
    }
    uint32_t incl = tot;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint32_t v = __shfl_up(incl, o, 64);
      if (lane >= o) incl += v;
    }
    if (lane == 63) sums[wave] = incl;
    __syncthreads();
    if (tid < BINS) {
      uint32_t base = incl - tot;
      for (int w = 0; w < wave; ++w) base += sums[w];
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const uint32_t c = next[w][tid];
        next[w][tid] = base;
        base += c;
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kSoloItems; ++r)
      if (r < rounds && i0 + 64 * r < n) {
        const uint32_t to = next[wave][(key[r] >> shift) & (BINS - 1)] + at[r];
        skey[to] = key[r];
        spos[to] = (uint16_t)pos[r];
      }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kSoloItems; ++r)
      if (r < rounds && i0 + 64 * r < n) {
        key[r] = skey[i0 + 64 * r];
        pos[r] = spos[i0 + 64 * r];
      }
    __syncthreads();
  }
#pragma unroll
  for (int r = 0; r < kSoloItems; ++r)
    if (r < rounds && i0 + 64 * r < n) {
      gmem(p.key_out)[i0 + 64 * r] = key[r];
      gmem(p.pos_out)[i0 + 64 * r] = pos[r];
    }
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------
constexpr int kEgThreads = 256;

template <typename GT, int V> struct Chunk;
template <typename GT> struct Chunk<GT, 8> {
  Raw8<GT> r;
  __device__ __forceinline__ void load(const GT* p, int64_t i) { r.load_once(p, i); }
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
__device__ __forceinline__ void put_row(const EmbedGradArgs& a, uint32_t key, int64_t col, int skip,
                                        const float (&acc)[8]) {
  OT* const o = reinterpret_cast<OT*>(a.dtable);
  const int64_t at = (int64_t)key * a.width + col;
  float v[8];
  if (a.accumulate) load8_any(o, at, v);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = a.accumulate ? fmaf(a.scale, acc[e], v[e]) : a.scale * acc[e];
  if (skip == 0) {
    store8_any(o, at, v);
  } else {
#pragma unroll
    for (int e = 1; e < 8; ++e)
      if (e >= skip) St<OT>::st(o, at + e, v[e]);
  }
}
template <typename OT>
__device__ __forceinline__ void put_row(const EmbedGradArgs& a, uint32_t key, int64_t col, int skip,
                                        const float (&acc)[1]) {
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

// One wave: one piece of sorted tokens, 64 chunks of V columns.  The keys and
// places are the same for all lanes (scalar loads, scalar branches), and the
// rows of 8 tokens are in flight at a time.
template <typename GT, typename OT, int V>
__global__ __launch_bounds__(kEgThreads) void k_embed_grad(const EmbedGradArgs a, uint32_t cpr, uint32_t groups) {
  typedef __attribute__((address_space(4))) const uint32_t ro_t;
  ro_t* const keys = reinterpret_cast<ro_t*>(reinterpret_cast<uintptr_t>(a.key));
  ro_t* const places = reinterpret_cast<ro_t*>(reinterpret_cast<uintptr_t>(a.pos));
  const uint32_t wave = __builtin_amdgcn_readfirstlane(blockIdx.x * (kEgThreads / 64) + (threadIdx.x >> 6));
  const uint32_t piece = wave / groups, chunk = (wave - piece * groups) * 64 + (threadIdx.x & 63);
  const int64_t s = (int64_t)piece * a.run, e = min(a.n, s + a.run);
  if (s >= a.n || chunk >= cpr) return;
  int skip;
  const int64_t col = chunk_col<V>(chunk, a.width, skip), at = (int64_t)chunk * V;
  const GT* const dout = reinterpret_cast<const GT*>(a.dout);
  const int64_t pitch = (int64_t)cpr * V;  // of a partial row
  float* const head = a.part + 2 * (int64_t)piece * pitch;
  float* const tail = head + pitch;
  uint32_t cur = keys[s];
  bool before = s > 0 && keys[s - 1] == cur;
  float acc[V] = {};
  auto flush = [&](bool onward) {
    if (cur >= a.rows) return;
    if (before) put_part(head, at, acc);
    else if (onward) put_part(tail, at, acc);
    else put_row<OT>(a, cur, col, skip, acc);
  };
  auto take = [&](uint32_t k, const Chunk<GT, V>& c) {
    if (k != cur) {
      flush(false);
      cur = k;
      before = false;
#pragma unroll
      for (int x = 0; x < V; ++x) acc[x] = 0.f;
    }
    c.add(acc);
  };
  constexpr int U = 8;
  int64_t i = s;
  for (; i + U <= e; i += U) {
    uint32_t k[U];
    Chunk<GT, V> c[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      k[u] = keys[i + u];
      c[u].load(dout, (int64_t)places[i + u] * a.width + col);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) take(k[u], c[u]);
  }
  for (; i < e; ++i) {
    Chunk<GT, V> c;
    c.load(dout, (int64_t)places[i] * a.width + col);
    take(keys[i], c);
  }
  flush(e < a.n && keys[e] == cur);
}

// Rows whose run crosses pieces: the piece where the run starts adds its tail
// and the heads of the pieces that follow.  A block takes kJoinCols chunks of
// columns; its kJoinParts groups of threads each add a contiguous share of the
// heads (a frequent token has hundreds), and the shares are added in order.
constexpr int kJoinCols = 64, kJoinParts = kEgThreads / kJoinCols;
template <typename OT, int V>
__global__ __launch_bounds__(kEgThreads) void k_embed_join(const EmbedGradArgs a, uint32_t cpr) {
  const int64_t piece = blockIdx.x;
  const int64_t s = piece * a.run, e = s + a.run;
  if (e >= a.n) return;
  const uint32_t k = gmem(a.key)[e - 1];
  if (k >= a.rows || gmem(a.key)[e] != k) return;
  if (s > 0 && gmem(a.key)[s - 1] == k) return;  // the run started in an earlier piece
  const int64_t pieces = (a.n + a.run - 1) / a.run;
  // pieces piece + 1 .. end - 1 begin with this key; every wave finds end itself
  const int lane = threadIdx.x & 63;
  int64_t end = piece + 1;
  for (;;) {
    const int64_t c = end + lane;
    const bool same = c < pieces && gmem(a.key)[c * a.run] == k;
    const int run = __popcll(__ballot(same));  // keys are sorted: a prefix of the lanes
    end += run;
    if (run < 64) break;
  }
  __shared__ float share[kJoinParts][kJoinCols][V];
  const int cl = threadIdx.x % kJoinCols, part = threadIdx.x / kJoinCols;
  const uint32_t chunk = blockIdx.y * kJoinCols + cl;
  const bool in = chunk < cpr;
  int skip;
  const int64_t col = chunk_col<V>(in ? chunk : 0, a.width, skip), at = (int64_t)(in ? chunk : 0) * V;
  const int64_t pitch = (int64_t)cpr * V;
  const int64_t heads = end - (piece + 1);
  const int64_t q0 = piece + 1 + heads * part / kJoinParts, q1 = piece + 1 + heads * (part + 1) / kJoinParts;
  float acc[V] = {};
  if (part == 0) add_part(a.part + (2 * piece + 1) * pitch, at, acc);
  constexpr int U = 8;
  int64_t q = q0;
  for (; q + U <= q1; q += U) {
    float v[U][V] = {};
#pragma unroll
    for (int u = 0; u < U; ++u) add_part(a.part + 2 * (q + u) * pitch, at, v[u]);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int x = 0; x < V; ++x) acc[x] += v[u][x];
  }
  for (; q < q1; ++q) add_part(a.part + 2 * q * pitch, at, acc);
#pragma unroll
  for (int x = 0; x < V; ++x) share[part][cl][x] = acc[x];
  __syncthreads();
  if (part == 0 && in) {
#pragma unroll
    for (int r = 1; r < kJoinParts; ++r)
#pragma unroll
      for (int x = 0; x < V; ++x) acc[x] += share[r][cl][x];
    put_row<OT>(a, k, col, skip, acc);
  }
}

}  // namespace

hipError_t launch_embedding(int table_dt, int out_dt, const EmbedArgs& a, hipStream_t s) {
  const bool v8 = a.width >= 8;
  const uint32_t cpr = (uint32_t)(v8 ? (a.width + 7) / 8 : a.width);
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

// Workgroups that clear a slice: 64 KiB each of 256 threads, at most 8 a CU.
static int zero_blocks(const ZeroSlice& z) {
  if (z.count == 0 || z.halves == 0) return 0;
  const int64_t b = (z.halves / z.count * 2 + 65535) / 65536;
  return (int)(b < 1 ? 1 : b > 2048 ? 2048 : b);
}

hipError_t launch_sort_pass(const SortPass& p, const ZeroSlice& count_z, const ZeroSlice& scatter_z, hipStream_t s) {
  hipLaunchKernelGGL(k_sort_count, dim3(p.blocks + zero_blocks(count_z)), dim3(kSortThreads), 0, s, p, count_z);
  hipLaunchKernelGGL(k_sort_scatter, dim3(p.blocks + zero_blocks(scatter_z)), dim3(kSortThreads), 0, s, p, scatter_z);
  return hipGetLastError();
}

hipError_t launch_sort_solo(const SortPass& p, const ZeroSlice& z, hipStream_t s) {
  const int zb = zero_blocks(z);  // one workgroup a CU fits beside the sort's LDS
  hipLaunchKernelGGL(k_sort_solo, dim3(1 + (zb > 255 ? 255 : zb)), dim3(kSoloThreads), 0, s, p, z);
  return hipGetLastError();
}

hipError_t launch_zero(const ZeroSlice& z, hipStream_t s) {
  const int zb = zero_blocks(z);
  if (zb > 0) hipLaunchKernelGGL(k_zero, dim3(zb), dim3(256), 0, s, z);
  return hipGetLastError();
}

hipError_t launch_embedding_grad(int g_dt, int out_dt, const EmbedGradArgs& a, hipStream_t s) {
  const bool v8 = a.width >= 8;
  const uint32_t cpr = (uint32_t)(v8 ? (a.width + 7) / 8 : a.width);
  const int64_t pieces = (a.n + a.run - 1) / a.run;
  const uint32_t groups = (cpr + 63) / 64;
  const int64_t nsum = (pieces * groups + kEgThreads / 64 - 1) / (kEgThreads / 64);
  if (nsum <= 0) return hipSuccess;
  if (nsum > INT32_MAX || pieces > INT32_MAX) return hipErrorInvalidValue;
#define MUONH_EG(GT, OT, V)                                                                              \
  do {                                                                                                   \
    hipLaunchKernelGGL((k_embed_grad<GT, OT, V>), dim3(nsum), dim3(kEgThreads), 0, s, a, cpr, groups);   \
    if (pieces > 1)                                                                                      \
      hipLaunchKernelGGL((k_embed_join<OT, V>), dim3(pieces, (cpr + kJoinCols - 1) / kJoinCols),         \
                         dim3(kEgThreads), 0, s, a, cpr);                                                \
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
