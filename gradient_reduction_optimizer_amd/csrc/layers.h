// The layers beside the step -- lookups with their gradient by sorted tokens
// (rows.hip) and experts' products (experts.hip): launch arguments, and the
// rules that host and kernels share.  Internal to the library.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

namespace gro {

// A matrix as a kernel sees it: element (i, j) at at + i * stride + j.
struct Matrix {
  void* at;
  int64_t rows, cols, stride;
  int32_t fp32;             // 1: FP32, 0: BF16
};

// ------------------------------------------------------------- positions by row
// Rows belong to buckets of 2^bits consecutive ones, which one workgroup sorts.
constexpr int64_t kMaxTableRows = int64_t(1) << 20;
constexpr int64_t kMaxIds = (int64_t(1) << 31) - (1 << 16);
constexpr int kMaxBuckets = 1024;
// Positions that one tile of a sorting workgroup holds.  So many ids are sorted in one
// launch, in which every workgroup reads them all: 9.5 us for 8,192 ids, against 15 to
// 16 for three launches of a few more.
constexpr int kSortTile = 8192;

inline int bucket_bits(int64_t n, int64_t n_rows) {
  // One launch, in which every workgroup reads all ids: up to 256 of them (8,192 ids of
  // 16,384 rows in buckets of 64 9.3 us, of 256 10.2).
  if (n <= kSortTile) return n_rows <= int64_t(256) << 6 ? 6 : n_rows <= int64_t(kMaxBuckets) << 8 ? 8 : 10;
  // Few rows: buckets of one row end the sort with the second launch of three, however
  // uneven the rows are (262,144 ids of 64 rows 14 us instead of 410 in one bucket, of
  // 1,024 rows 19 instead of 42).
  if (n_rows <= kMaxBuckets) return 0;
  // More: up to 512 buckets.  The second launch's workgroups all read every chunk's
  // counts of all of them, the third's take about the same time each (262,144 ids of
  // 4,000 rows in 1,000 buckets 27 us, 250 20, 63 23; of 262,144 rows in 1,024 35, 256 22).
  // One workgroup sorts a bucket, so a common id costs its length: 262,144 ids of 32,000
  // rows 22 us, with half of them one id 163, all 305; 2,097,152 54, 1,403 and 2,744.
  int bits = 2;
  while (bits < 10 && n_rows > int64_t(512) << bits) bits += 2;
  return bits;
}

struct RowSortLaunch {
  const void* ids;
  int32_t wide_ids;         // 1: 64-bit ids
  int64_t n;
  int64_t first;
  int64_t n_rows;
  int32_t* order;
  int32_t* starts;
  // Workspace of the sort in several launches (n > kSortTile).
  uint32_t* pairs;          // [n][2]: row, position
  uint32_t* counts;         // [n_chunks][n_buckets]
  uint32_t* bases;          // [n_buckets + 1]
  int32_t n_chunks;
  int32_t n_buckets;
  int64_t chunk;            // ids per chunk, a multiple of kSortChunk
};
constexpr int kSortChunk = 4096;
constexpr int64_t kMaxSortChunks = 256;

inline int64_t sort_chunk(int64_t n) {
  const int64_t tiles = (n + kSortChunk - 1) / kSortChunk;
  return (tiles + kMaxSortChunks - 1) / kMaxSortChunks * kSortChunk;
}

hipError_t launch_row_sort(const RowSortLaunch& a, hipStream_t s);

// ---------------------------------------------------------------------- lookups
struct LookupLaunch {
  Matrix table;
  int64_t first;
  const void* ids;
  int32_t wide_ids;
  float scale;
  Matrix out;
};
hipError_t launch_lookup(const LookupLaunch& a, hipStream_t s);

// Columns of a gradient, 512 to a workgroup across (a grid has fewer than 2^16 that way).
constexpr int64_t kMaxGradCols = int64_t(1) << 24;

constexpr int64_t kShortRun = 16, kMaxRuns = 4096, kRunsFrom = 512;

// Tokens in order are cut into runs of this many; a run within one row is summed
// by the first launch (without it a row that has all of 65,536 tokens is one
// workgroup's work).
inline int64_t run_tokens(int64_t n) {
  int64_t c = kShortRun;
  while (c * kMaxRuns < n) c *= 2;
  return c;
}

// Runs of so many tokens; few tokens do without (the second launch alone takes 5 us
// instead of 7 for both at 37 of them).
inline int64_t whole_runs(int64_t n) { return n < kRunsFrom ? 0 : n / run_tokens(n); }

struct LookupGradLaunch {
  Matrix dy;
  const int32_t* order;
  const int32_t* starts;
  float scale;
  int32_t accumulate;
  Matrix out;
  float* partials;          // [n / run][cols rounded up to 8]
  int64_t run;
  int64_t n_runs;           // whole runs, 0: no first launch
};
hipError_t launch_lookup_grad(const LookupGradLaunch& a, hipStream_t s);

// ------------------------------------------------------------- experts' products
// C = A B^T summed over k, for each expert: rows of A, rows of B or the k of both
// are cut by `starts`.
enum ExpertsMode { kForward = 0, kInputGrad = 1, kWeightGrad = 2 };

struct ExpertsLaunch {
  const uint16_t* a;        // forward x, input gradient dy, weight gradient dy
  const uint16_t* b;        // forward and input gradient W, weight gradient x
  void* c;                  // y, dx, dW
  int64_t a_stride, b_stride, c_stride;
  int64_t b_expert;         // from one expert's matrix to the next: of the weights ...
  int64_t c_expert;         // ... or of their gradients
  const int32_t* starts;
  int32_t n_experts;
  int64_t rows;             // rows that starts may name
  int64_t inner, outer;
  int32_t c_fp32;
  int32_t accumulate;       // weight gradient only
  int32_t n_parts;          // of the sums over k; more than one:
  float* partials;          // [n_parts][C without gaps]
  int64_t c_part;           // elements of one part
};
// Tiles of 128 x 128 that a product takes at most, and may: the kernels number them, and
// some numbers that stand for none, in 32 bits.
int64_t experts_tiles(const ExpertsLaunch& a, ExpertsMode mode);
constexpr int64_t kMaxExpertsTiles = int64_t(1) << 31;
int experts_parts(ExpertsMode mode, int32_t n_experts, int64_t rows, int64_t inner, int64_t outer);
hipError_t launch_experts(const ExpertsLaunch& a, ExpertsMode mode, hipStream_t s);

}  // namespace gro
