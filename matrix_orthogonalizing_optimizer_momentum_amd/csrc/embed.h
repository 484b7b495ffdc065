// Layout and launchers of the embedding kernels, shared by the kernels and
// the entry points.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace muonh {

// Outputs above this size (half of the last-level cache) are stored past the
// caches, which leaves them to the table's frequent rows: 65536 x 2048 bf16
// (268 MB) 90 -> 82 us.
constexpr int64_t kEmbOnceBytes = (int64_t)128 << 20;
constexpr int64_t kEmbMaxWidth = (int64_t)1 << 18, kEmbMaxTokens = (int64_t)1 << 26;
constexpr int kSortThreads = 256;
constexpr int kSortBits = 11;      // digit bits of one sort pass, at most
constexpr int kSortMaxBlocks = 256;  // 2^20 tokens of 256 values: 220 us, with 64 blocks 312
constexpr int kSoloThreads = 1024;  // the sort in one workgroup:
// Tokens per thread.  A gradient of 8192 tokens on 50257 x 768 bf16 to fp32: 37 us,
// by passes 50 (into one buffer, which stays in the last-level cache; 47.6 and
// 54.5 where calls take turns with two), of 16384 tokens 60 and 55.
constexpr int kSoloItems = 8;
constexpr int kSoloBits = 9;        // digit bits of one of its passes
constexpr int64_t kSoloTokens = kSoloThreads * kSoloItems;
constexpr int kRunMin = 8, kRunMax = 64;  // sorted tokens per piece of the gradient

// A share of the table's gradient that a launch clears: slice `index` of
// `count` equal ones (count 0: nothing).  p is aligned to 2 bytes.
struct ZeroSlice {
  uint16_t* p;
  int64_t halves;           // of the whole table, in units of 2 bytes
  int32_t index, count;
};

// One stable counting pass of the token sort.
struct SortPass {
  const void* ids;          // first pass: the token ids (id_bits wide); else nullptr
  const uint32_t* key_in;   // later passes
  const uint32_t* pos_in;
  uint32_t* key_out;
  uint32_t* pos_out;
  uint32_t* hist;           // [blocks][1 << bits]
  int64_t n;
  uint32_t rows;            // ids outside [0, rows) get the key rows
  int32_t id_bits, shift, bits, tile, blocks;
};

struct EmbedArgs {
  const void* table;
  const void* ids;
  void* out;
  int64_t n, rows, width;
  float scale;
  int32_t id_bits;
  int32_t once;             // out is too large to be found in the caches later: stored past them
};

struct EmbedGradArgs {
  const uint32_t* key;      // sorted token ids, the ignored ones (= rows) last
  const uint32_t* pos;      // and where each token stands in the batch
  const void* dout;         // n x width
  void* dtable;             // rows x width
  float* part;              // [pieces][2][width]: head and tail sums of runs that cross pieces
  int64_t n, rows, width;
  float scale;
  int32_t accumulate;
  int32_t run;              // tokens per piece, a multiple of 8
};

hipError_t launch_embedding(int table_dt, int out_dt, const EmbedArgs& a, hipStream_t s);
// count and scatter of one pass, with one slice of the clearing each
hipError_t launch_sort_pass(const SortPass& p, const ZeroSlice& count_z, const ZeroSlice& scatter_z, hipStream_t s);
// up to kSoloTokens tokens, all passes; p.bits is the key's width
hipError_t launch_sort_solo(const SortPass& p, const ZeroSlice& z, hipStream_t s);
hipError_t launch_zero(const ZeroSlice& z, hipStream_t s);
hipError_t launch_embedding_grad(int g_dt, int out_dt, const EmbedGradArgs& a, hipStream_t s);

}  // namespace muonh
