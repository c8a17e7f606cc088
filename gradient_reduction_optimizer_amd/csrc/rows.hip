// Embedding lookups with a scale, positions sorted by the row they name, and the
// lookup's gradient as sums over those positions.  gfx950.
#include <hip/hip_runtime.h>

#include "lane.h"
#include "layers.h"

namespace gro {
namespace {

// Accesses at any alignment of their elements, which the hardware takes.
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
typedef u16x8 u16x8_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

struct Eight {
  float v[8];
};

// Elements [col, col + 8) of a row as they lie in memory, those at n and behind as zeros.
template <bool FP32>
struct Raw8 {
  f32x4 a, b;
};
template <>
struct Raw8<false> {
  u16x8 a;
};
template <bool FP32>
__device__ __forceinline__ Raw8<FP32> load_raw(const void* row, int64_t col, int64_t n) {
  Raw8<FP32> x = {};
  if constexpr (FP32) {
    const float* p = static_cast<const float*>(row) + col;
    if (col + 8 <= n) {
      x.a = *reinterpret_cast<const f32x4_any*>(p);
      x.b = *reinterpret_cast<const f32x4_any*>(p + 4);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (col + e < n) x.a[e] = p[e];
        if (col + 4 + e < n) x.b[e] = p[4 + e];
      }
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(row) + col;
    if (col + 8 <= n) {
      x.a = *reinterpret_cast<const u16x8_any*>(p);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (col + e < n) x.a[e] = p[e];
    }
  }
  return x;
}
__device__ __forceinline__ Eight widen8(const Raw8<true>& r) {
  return Eight{r.a[0], r.a[1], r.a[2], r.a[3], r.b[0], r.b[1], r.b[2], r.b[3]};
}
__device__ __forceinline__ Eight widen8(const Raw8<false>& r) {
  Eight x;
#pragma unroll
  for (int e = 0; e < 8; ++e) x.v[e] = widen1(r.a[e]);
  return x;
}
template <bool FP32>
__device__ __forceinline__ Eight load8(const void* row, int64_t col, int64_t n) {
  return widen8(load_raw<FP32>(row, col, n));
}

template <bool FP32, bool NT = false>
__device__ __forceinline__ void store8(void* row, int64_t col, int64_t n, const Eight& x) {
  if (col + 8 <= n) {
    if constexpr (FP32) {
      f32x4_any* p = reinterpret_cast<f32x4_any*>(static_cast<float*>(row) + col);
      const f32x4 lo = {x.v[0], x.v[1], x.v[2], x.v[3]}, hi = {x.v[4], x.v[5], x.v[6], x.v[7]};
      if constexpr (NT) {
        __builtin_nontemporal_store(lo, p);
        __builtin_nontemporal_store(hi, p + 1);
      } else {
        p[0] = lo;
        p[1] = hi;
      }
    } else {
      u16x8 a;
#pragma unroll
      for (int e = 0; e < 8; ++e) a[e] = bf16_bits(x.v[e]);
      u16x8_any* p = reinterpret_cast<u16x8_any*>(static_cast<uint16_t*>(row) + col);
      if constexpr (NT) __builtin_nontemporal_store(a, p);
      else *p = a;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (col + e < n) {
        if constexpr (FP32) static_cast<float*>(row)[col + e] = x.v[e];
        else static_cast<uint16_t*>(row)[col + e] = bf16_bits(x.v[e]);
      }
  }
}

template <bool FP32>
__device__ __forceinline__ char* row_of(const Matrix& m, int64_t i) {
  return static_cast<char*>(m.at) + i * m.stride * (FP32 ? 4 : 2);
}

// The row that id number i names, n_rows or more for none of this table's.
__device__ __forceinline__ uint32_t row_of_id(const void* ids, int wide, int64_t i, int64_t first, int64_t n_rows) {
  const int64_t id = wide ? static_cast<const int64_t*>(ids)[i] : int64_t(static_cast<const int32_t*>(ids)[i]);
  // first >= 0, so the difference of an id from 0 on does not overflow
  return id >= first && id - first < n_rows ? uint32_t(id - first) : 0xffffffffu;
}

// ------------------------------------------------------------------ the lookup
// out[i] = scale * table[id]: HBM-bound copies of whole rows.  `lanes` lanes (a
// power of two) share a row, 8 elements each at a time, four such reads under way.  The
// result is larger than the caches: stored with the non-temporal policy 65,536 rows of
// 2,048 BF16 elements take 58 us, without 78.  They name 13,500 rows of 32,000, 55 MB, of
// which 132 are read, since each XCD has an L2 of its own: with the 269 written 6.9 TB/s,
// and 5.6 of what it cannot do without.
template <bool TF, bool OF>
__global__ __launch_bounds__(256) void k_lookup(const LookupLaunch P, const int lanes) {
  const int group = int(threadIdx.x) / lanes, lane = int(threadIdx.x) & (lanes - 1), groups = 256 / lanes;
  const int64_t n = P.out.cols;
  constexpr int kChunks = 4;
  for (int64_t i = int64_t(blockIdx.x) * groups + group; i < P.out.rows; i += int64_t(gridDim.x) * groups) {
    const uint32_t r = row_of_id(P.ids, P.wide_ids, i, P.first, P.table.rows);
    const char* in = row_of<TF>(P.table, r == 0xffffffffu ? 0 : r);
    char* out = row_of<OF>(P.out, i);
    for (int64_t c0 = 8 * lane; c0 < n; c0 += kChunks * 8 * lanes) {
      Raw8<TF> y[kChunks];
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        const int64_t c = c0 + k * 8 * lanes;
        y[k] = Raw8<TF>{};
        if (c < n && r != 0xffffffffu) y[k] = load_raw<TF>(in, c, n);
      }
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        const int64_t c = c0 + k * 8 * lanes;
        Eight x = widen8(y[k]);
#pragma unroll
        for (int e = 0; e < 8; ++e) x.v[e] = r != 0xffffffffu ? x.v[e] * P.scale : 0.0f;
        if (c < n) store8<OF, true>(out, c, n, x);
      }
    }
  }
}

// ------------------------------------------------------------------- the sort
// A stable counting sort.  Items are numbered wave by wave, 64 * rounds of them to a
// wave, 64 to a round, so ranks within a wave, in this order, and a prefix over waves
// keep equal rows in the order of their positions.  No atomics decide an order.  Bound
// by latency: a few dependent passes over LDS and L2 (one launch of up to 8,192 ids 6 to
// 9 us; 65,536 ids of 32,000 rows 18 us, 2,097,152 ids 56 us in three launches).
constexpr int kSortBlock = 1024;
constexpr int kSortWaves = kSortBlock / 64;

// Lanes of the wave with the same digit as this one, -1 being none.
template <int BITS>
__device__ __forceinline__ uint64_t same_digit(int digit) {
  uint64_t same = __ballot(digit >= 0);
#pragma unroll
  for (int b = 0; b < BITS; ++b) {
    const bool bit = (digit >> b) & 1;
    const uint64_t with = __ballot(bit);
    same &= bit ? with : ~with;
  }
  return same;
}

// The rank of this lane's item among the wave's with the same digit, and one more of
// them in the wave's counts.
template <int BITS>
__device__ __forceinline__ uint32_t rank_in_wave(int digit, uint32_t* counts) {
  const int lane = int(threadIdx.x) & 63;
  const uint64_t same = same_digit<BITS>(digit);
  uint32_t rank = 0;
  if (digit >= 0) {
    rank = counts[digit] + __popcll(same & ((uint64_t(1) << lane) - 1));
    // the last of them stores; the wave's LDS operations keep their order
    if (lane == 63 - __clzll(same)) counts[digit] = rank + 1;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  return rank;
}

// counts[w][d] to the sum over the waves before w; returns digit threadIdx.x's
// total (0 from digit `bins` on).
__device__ __forceinline__ uint32_t prefix_over_waves(uint32_t* counts, int bins) {
  uint32_t total = 0;
  if (int(threadIdx.x) < bins) {
    uint32_t c[kSortWaves];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) c[w] = counts[w * bins + threadIdx.x];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      counts[w * bins + threadIdx.x] = total;
      total += c[w];
    }
  }
  return total;
}

// Exclusive prefix sum over the workgroup's lanes; `all` the sum.  part: 16 words of
// LDS.
__device__ __forceinline__ uint32_t block_prefix(uint32_t x, uint32_t* part, uint32_t& all) {
  const int lane = int(threadIdx.x) & 63, wave = int(threadIdx.x) >> 6;
  uint32_t s = x;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const uint32_t t = __shfl_up(s, m, 64);
    if (lane >= m) s += t;
  }
  __syncthreads();
  if (lane == 63) part[wave] = s;
  __syncthreads();
  uint32_t before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) {
    if (w == wave) before = all;
    all += part[w];
  }
  return before + s - x;
}

// A bucket's items in LDS or memory by row: up to kSortTile of them at a time, each
// read once.  item(k, digit, position) gives number k; `begin`: where the bucket's
// positions lie in the order.
template <int BITS>
struct BucketSort {
  static constexpr int kBins = 1 << BITS, kRounds = kSortTile / kSortBlock;
  uint32_t counts[kSortWaves * kBins];
  uint32_t base[kBins];
  uint32_t part[kSortWaves];

  template <typename Item>
  __device__ __forceinline__ void run(const RowSortLaunch& P, int64_t n, uint32_t begin, int64_t lo, int64_t hi, Item item) {
    const int wave = int(threadIdx.x) >> 6, lane = int(threadIdx.x) & 63;
    uint32_t* mine = counts + wave * kBins;
    int digit[kRounds];
    uint32_t rank[kRounds], position[kRounds];
    const bool whole = n <= kSortTile;
    // several tiles: the rows' totals first.  Many items may be of one row, which would
    // hold the LDS adds up one by one: those of the wave's first item's row go as one.
    if (!whole) {
      for (int i = int(threadIdx.x); i < kBins; i += kSortBlock) base[i] = 0;
      __syncthreads();
      for (int64_t tile = 0; tile < n; tile += kSortTile) {
#pragma unroll
        for (int j = 0; j < kRounds; ++j) {
          const int64_t k = tile + j * kSortBlock + threadIdx.x;
          digit[j] = -1;
          if (k < n) item(k, digit[j], position[j]);
        }
#pragma unroll
        for (int j = 0; j < kRounds; ++j) {
          const int first = __builtin_amdgcn_readfirstlane(digit[j]);
          const uint64_t like = __ballot(digit[j] == first);
          if (digit[j] >= 0 && (digit[j] != first || lane == 0))
            atomicAdd(&base[digit[j]], digit[j] == first ? uint32_t(__popcll(like)) : 1u);
        }
      }
      __syncthreads();
      uint32_t all;
      const uint32_t at = begin + block_prefix(int(threadIdx.x) < kBins ? base[threadIdx.x] : 0, part, all);
      if (int(threadIdx.x) < kBins) base[threadIdx.x] = at;
    }
    for (int64_t tile = 0; tile < n || (tile == 0 && whole); tile += kSortTile) {
      const int here = int(std::min<int64_t>(n - tile, kSortTile)), rounds = (here + kSortBlock - 1) / kSortBlock;
      __syncthreads();
      for (int i = int(threadIdx.x); i < kSortWaves * kBins; i += kSortBlock) counts[i] = 0;
#pragma unroll
      for (int j = 0; j < kRounds; ++j) {
        digit[j] = -1;
        const int k = wave * 64 * rounds + j * 64 + lane;
        if (j < rounds && k < here) item(tile + k, digit[j], position[j]);
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kRounds; ++j)
        if (j < rounds) rank[j] = rank_in_wave<BITS>(digit[j], mine);
      __syncthreads();
      const uint32_t total = prefix_over_waves(counts, kBins);
      if (whole) {
        uint32_t all;
        const uint32_t at = begin + block_prefix(total, part, all);
        if (int(threadIdx.x) < kBins) base[threadIdx.x] = at;
      }
      __syncthreads();
      if (tile == 0) {
        if (int(threadIdx.x) < kBins && lo + int64_t(threadIdx.x) < hi) P.starts[lo + threadIdx.x] = int32_t(base[threadIdx.x]);
        if (threadIdx.x == 0 && hi == P.n_rows) P.starts[hi] = int32_t(begin + n);
      }
#pragma unroll
      for (int j = 0; j < kRounds; ++j)
        if (j < rounds && digit[j] >= 0) P.order[base[digit[j]] + mine[digit[j]] + rank[j]] = int32_t(position[j]);
      __syncthreads();
      if (int(threadIdx.x) < kBins) base[threadIdx.x] += total;
    }
  }
};

// Up to kSortTile ids in one launch: workgroup b reads them all, counts those in
// front of its bucket and sorts those of its bucket.  ROUNDS * kSortBlock ids.
template <int BITS, int ROUNDS>
__global__ __launch_bounds__(kSortBlock) void k_row_sort_few(const RowSortLaunch P) {
  __shared__ BucketSort<BITS> bucket;
  __shared__ uint32_t item[ROUNDS * kSortBlock];
  __shared__ uint16_t row[ROUNDS * kSortBlock];
  const int64_t lo = int64_t(blockIdx.x) << BITS, hi = std::min(lo + (1 << BITS), P.n_rows);
  uint32_t key[ROUNDS], count = 0;
  const int first = int(threadIdx.x) * ROUNDS, n = int(P.n);
#pragma unroll
  for (int j = 0; j < ROUNDS; ++j) {
    key[j] = 0xffffffffu;
    if (first + j < n) key[j] = row_of_id(P.ids, P.wide_ids, first + j, P.first, P.n_rows);
    // both counts in one number: up to 2^13 each
    count += (key[j] < uint32_t(lo) ? 1u << 16 : 0u) + (key[j] >= uint32_t(lo) && int64_t(key[j]) < hi ? 1u : 0u);
  }
  uint32_t all;
  uint32_t at = block_prefix(count, bucket.part, all) & 0xffffu;
#pragma unroll
  for (int j = 0; j < ROUNDS; ++j)
    if (key[j] >= uint32_t(lo) && int64_t(key[j]) < hi) {
      item[at] = uint32_t(first + j);
      row[at++] = uint16_t(key[j] - uint32_t(lo));
    }
  __syncthreads();
  bucket.run(P, all & 0xffffu, all >> 16, lo, hi, [&](int64_t k, int& d, uint32_t& p) {
    d = int(row[k]);
    p = item[k];
  });
}

// More ids, first launch: how many of each chunk belong to each bucket.
__global__ __launch_bounds__(kSortBlock) void k_row_sort_count(const RowSortLaunch P, const int bits) {
  __shared__ uint32_t counts[kMaxBuckets];
  const int lane = int(threadIdx.x) & 63;
  counts[threadIdx.x] = 0;
  __syncthreads();
  const int64_t lo = int64_t(blockIdx.x) * P.chunk, hi = std::min(lo + P.chunk, P.n);
#pragma unroll 4
  for (int64_t i = lo + threadIdx.x; i < hi; i += kSortBlock) {
    const uint32_t r = row_of_id(P.ids, P.wide_ids, i, P.first, P.n_rows);
    const uint32_t bucket = r >> bits;
    // many may be of one bucket: the wave's first item's go as one
    const uint32_t head = __builtin_amdgcn_readfirstlane(bucket);
    const uint64_t like = __ballot(r != 0xffffffffu && bucket == head);
    if (r != 0xffffffffu && (bucket != head || (like & ((uint64_t(1) << lane) - 1)) == 0))
      atomicAdd(&counts[bucket], bucket == head ? uint32_t(__popcll(like)) : 1u);
  }
  __syncthreads();
  if (int(threadIdx.x) < P.n_buckets) P.counts[int64_t(blockIdx.x) * P.n_buckets + threadIdx.x] = counts[threadIdx.x];
}

// Second launch: rows and positions to their buckets, in order; positions to their rows
// where every row is a bucket, which ends the sort.
__global__ __launch_bounds__(kSortBlock) void k_row_sort_spread(const RowSortLaunch P, const int bits) {
  constexpr int kRounds = kSortChunk / kSortBlock;
  __shared__ uint32_t counts[kSortWaves * kMaxBuckets];
  __shared__ uint32_t base[kMaxBuckets];
  __shared__ uint32_t part[kSortWaves];
  const int nb = P.n_buckets;
  // the chunks' counts, `step` lanes to a bucket
  int wide = 1;
  while (wide < nb) wide *= 2;
  const int step = kSortBlock / wide, b = int(threadIdx.x) & (wide - 1);
  uint32_t before = 0, total = 0, all;
  if (b < nb) {
#pragma unroll 8
    for (int c = int(threadIdx.x) / wide; c < P.n_chunks; c += step) {
      const uint32_t x = P.counts[int64_t(c) * nb + b];
      total += x;
      before += c < int(blockIdx.x) ? x : 0;
    }
  }
  counts[threadIdx.x] = total;
  counts[kSortBlock + threadIdx.x] = before;
  __syncthreads();
  before = total = 0;
  if (int(threadIdx.x) < nb)
    for (int i = int(threadIdx.x); i < kSortBlock; i += wide) {
      total += counts[i];
      before += counts[kSortBlock + i];
    }
  const uint32_t begin = block_prefix(total, part, all);
  base[threadIdx.x] = begin + before;
  if (blockIdx.x == 0) {
    if (bits > 0) {
      if (int(threadIdx.x) < nb) P.bases[threadIdx.x] = begin;
      if (threadIdx.x == 0) P.bases[nb] = all;
    } else {
      if (int64_t(threadIdx.x) < P.n_rows) P.starts[threadIdx.x] = int32_t(begin);
      if (threadIdx.x == 0) P.starts[P.n_rows] = int32_t(all);
    }
  }
  const int64_t lo = int64_t(blockIdx.x) * P.chunk, hi = std::min(lo + P.chunk, P.n);
  const int wave = int(threadIdx.x) >> 6, lane = int(threadIdx.x) & 63;
  for (int64_t tile = lo; tile < hi; tile += kSortChunk) {
    uint32_t row[kRounds], rank[kRounds];
    int digit[kRounds];
#pragma unroll
    for (int j = 0; j < kRounds; ++j) {
      const int64_t i = tile + wave * 64 * kRounds + j * 64 + lane;
      row[j] = i < hi ? row_of_id(P.ids, P.wide_ids, i, P.first, P.n_rows) : 0xffffffffu;
      digit[j] = row[j] != 0xffffffffu ? int(row[j] >> bits) : -1;
    }
    __syncthreads();
    for (int i = int(threadIdx.x); i < kSortWaves * nb; i += kSortBlock) counts[i] = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kRounds; ++j) rank[j] = rank_in_wave<10>(digit[j], counts + wave * nb);
    __syncthreads();
    const uint32_t here = prefix_over_waves(counts, nb);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kRounds; ++j)
      if (digit[j] >= 0) {
        const int64_t to = base[digit[j]] + counts[wave * nb + digit[j]] + rank[j];
        const uint32_t position = uint32_t(tile + wave * 64 * kRounds + j * 64 + lane);
        if (bits > 0) *reinterpret_cast<u32x2*>(P.pairs + 2 * to) = u32x2{row[j], position};
        else P.order[to] = int32_t(position);
      }
    __syncthreads();
    base[threadIdx.x] += here;
  }
}

// Third launch: every bucket by row.
template <int BITS>
__global__ __launch_bounds__(kSortBlock) void k_row_sort_bucket(const RowSortLaunch P) {
  __shared__ BucketSort<BITS> bucket;
  const int64_t lo = int64_t(blockIdx.x) << BITS, hi = std::min(lo + (1 << BITS), P.n_rows);
  const uint32_t begin = P.bases[blockIdx.x], end = P.bases[blockIdx.x + 1];
  const uint32_t* pairs = P.pairs + 2 * int64_t(begin);
  bucket.run(P, end - begin, begin, lo, hi, [&](int64_t k, int& d, uint32_t& p) {
    const u32x2 x = *reinterpret_cast<const u32x2*>(pairs + 2 * k);
    d = int(x.x & ((1 << BITS) - 1));
    p = x.y;
  });
}

// --------------------------------------------------------- the lookup's gradient
// Row r's gradient is scale * sum of dy over its positions, in order: HBM-bound,
// dy read once and the table written once.  Positions are cut into runs; the first
// launch sums the runs that lie within one row, so that a common token's row is
// the work of many waves, and the second adds what is left in front of a row's first
// run, its runs and what is left behind.  `lanes` lanes (a power of two) share 8 *
// lanes columns of a row or run.  The order of every sum depends on the rows' lengths
// alone.
__device__ __forceinline__ int64_t bounded(int32_t at, int64_t lo, int64_t n) {
  return std::min(std::max(int64_t(at), lo), n);
}

__device__ __forceinline__ void add8(Eight& x, const Eight& y) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x.v[e] += y.v[e];
}

// x += dy[order[p]] for the positions [p, end), 8 columns from col on (there may be
// none): all lanes of a group together, each with a position for all, kBatch rows in
// flight (4: the rows' launch of 65,536 tokens of 2,048 columns 105 us; 8: 116, for the
// registers).
constexpr int kBatch = 4;
template <bool DF>
__device__ __forceinline__ void add_tokens(const LookupGradLaunch& P, int64_t p, int64_t end, int64_t col, int lanes, Eight& x) {
  const int lane = int(threadIdx.x) & (lanes - 1);
  for (; p < end; p += lanes) {
    const int n = int(std::min<int64_t>(lanes, end - p));
    int mine = -1;
    if (lane < n) mine = P.order[p + lane];
    for (int t = 0; t < n; t += kBatch) {
      Raw8<DF> y[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = t + u < n ? __shfl(mine, t + u, lanes) : -1;
        y[u] = Raw8<DF>{};
        if (i >= 0 && i < P.dy.rows) y[u] = load_raw<DF>(row_of<DF>(P.dy, i), col, P.dy.cols);
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) add8(x, widen8(y[u]));
    }
  }
}

// x += the sums of the runs [q, end).
__device__ __forceinline__ void add_runs(const LookupGradLaunch& P, int64_t q, int64_t end, int64_t col, Eight& x) {
  const int64_t padded = (P.out.cols + 7) / 8 * 8;
  for (; q < end; q += kBatch) {
    Eight y[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      y[u] = Eight{};
      if (q + u < end) y[u] = load8<true>(P.partials + (q + u) * padded, col, padded);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) add8(x, y[u]);
  }
}

template <bool DF>
__global__ __launch_bounds__(256) void k_grad_runs(const LookupGradLaunch P, const int lanes) {
  const int group = int(threadIdx.x) / lanes, lane = int(threadIdx.x) & (lanes - 1), groups = 256 / lanes;
  const int64_t q = int64_t(blockIdx.x) * groups + group, col = 8 * (int64_t(blockIdx.y) * lanes + lane);
  if (q >= P.n_runs) return;
  const int64_t lo = q * P.run, hi = lo + P.run;
  // the last row that begins at lo or before: every lane of the group looks at one
  // place of the rows that are left
  const int shift = int(threadIdx.x) & 63 & ~(lanes - 1);
  const uint64_t mask = lanes == 64 ? ~uint64_t(0) : (uint64_t(1) << lanes) - 1;
  int64_t a = 0, b = P.out.rows;
  while (b - a > 1) {
    const int64_t step = lanes > 1 ? (b - a + lanes - 1) / lanes : (b - a + 1) / 2;
    const int64_t at = lanes > 1 ? a + lane * step : a + step;
    const bool yes = at < b && P.starts[at] <= lo;
    const int n = __popcll((__ballot(yes) >> shift) & mask);
    if (lanes > 1) {
      if (n == 0) return;                        // in front of the first row
      a += (n - 1) * step;
      b = std::min(a + step, b);
    } else if (n) {
      a = at;
    } else {
      b = at;
    }
  }
  if (P.starts[a] > lo || P.starts[a + 1] < hi) return;
  Eight x = {};
  add_tokens<DF>(P, lo, hi, col, lanes, x);
  const int64_t padded = (P.out.cols + 7) / 8 * 8;
  store8<true>(P.partials + q * padded, col, padded, x);
}

// A row's sum: `part` of `parts` of the positions in front of its runs, the runs and
// the positions behind them, in this order.
struct RowWork {
  int64_t head, q0, q1, tail, hi;
  int64_t units;
  __device__ __forceinline__ RowWork(const LookupGradLaunch& P, int32_t first, int32_t end) {
    const int64_t lo = bounded(first, 0, P.dy.rows);
    hi = bounded(end, lo, P.dy.rows);
    head = lo;
    q0 = (lo + P.run - 1) / P.run;
    q1 = std::min(hi / P.run, P.n_runs);
    tail = q1 * P.run;
    if (q0 >= q1) {
      q0 = q1 = 0;
      tail = hi;
    }
    units = hi - lo - (q1 - q0) * (P.run - 1);
  }
  template <bool DF>
  __device__ __forceinline__ Eight sum(const LookupGradLaunch& P, int64_t col, int lanes, int part, int parts) const {
    Eight x = {};
    const int64_t u0 = units * part / parts, u1 = units * (part + 1) / parts;
    const int64_t n_head = (q1 > q0 ? q0 * P.run : hi) - head, n_runs = q1 - q0;
    const auto clip = [](int64_t v, int64_t n) { return std::min(std::max(v, int64_t(0)), n); };
    add_tokens<DF>(P, head + clip(u0, n_head), head + clip(u1, n_head), col, lanes, x);
    add_runs(P, q0 + clip(u0 - n_head, n_runs), q0 + clip(u1 - n_head, n_runs), col, x);
    const int64_t n_tail = hi - tail;
    add_tokens<DF>(P, tail + clip(u0 - n_head - n_runs, n_tail), tail + clip(u1 - n_head - n_runs, n_tail), col, lanes, x);
    return x;
  }
};

template <bool OF>
__device__ __forceinline__ void write_row(const LookupGradLaunch& P, int64_t r, int64_t col, Eight x, const Raw8<OF>& was) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x.v[e] *= P.scale;
  if (P.accumulate) add8(x, widen8(was));
  store8<OF>(row_of<OF>(P.out, r), col, P.out.cols, x);
}

// A group takes kRowsEach rows at once: what it reads of all of them -- where they
// begin, up to kTokens positions of each, those rows of dy -- is under way together (sort
// and gradient of 65,536 tokens with 4 rows of 2 tokens 177 us, 4 of one 180, 2 of 2 189,
// 2 of 4 183; five waves a SIMD, for which the registers do not suffice: 250).
// Rows with more are then shared out: each a group's, or, with more than kAlone
// positions and runs, all groups' of the workgroup, a part each (that launch with 16
// 105 us, 8 109, 32 104; 16 leaves less to one group where common tokens are many).
// 65,536 tokens of 2,048 columns, added to 32,000 rows in FP32: runs 44 us, rows 101,
// 402 MB read and 127 written in both.
constexpr int64_t kAlone = 16;
constexpr int kRowsEach = 4;
template <bool DF, bool OF>
__global__ __launch_bounds__(256) void k_grad_rows(const LookupGradLaunch P, const int lanes) {
  constexpr int kTokens = DF ? 1 : 2;
  __shared__ float sums[256 * 8];
  __shared__ int32_t listed[256 * kRowsEach];  // rows with more, from the front; still longer ones from the back
  __shared__ int n_listed[2];
  const int group = int(threadIdx.x) / lanes, lane = int(threadIdx.x) & (lanes - 1), groups = 256 / lanes;
  const int64_t r0 = (int64_t(blockIdx.x) * groups + group) * kRowsEach, col = 8 * (int64_t(blockIdx.y) * lanes + lane);
  const int64_t n = P.dy.rows;
  if (threadIdx.x < 2) n_listed[threadIdx.x] = 0;
  int at[kRowsEach + 1];
#pragma unroll
  for (int k = 0; k <= kRowsEach; ++k) at[k] = P.starts[std::min(r0 + k, P.out.rows)];
  at[0] = int(bounded(at[0], 0, n));
#pragma unroll
  for (int k = 1; k <= kRowsEach; ++k) at[k] = int(bounded(at[k], at[k - 1], n));
  Raw8<DF> y[kRowsEach][kTokens];
  {
    int token[kRowsEach][kTokens];
#pragma unroll
    for (int k = 0; k < kRowsEach; ++k)
#pragma unroll
      for (int t = 0; t < kTokens; ++t) {
        token[k][t] = -1;
        if (at[k + 1] - at[k] <= kTokens && at[k] + t < at[k + 1]) token[k][t] = P.order[at[k] + t];
      }
#pragma unroll
    for (int k = 0; k < kRowsEach; ++k)
#pragma unroll
      for (int t = 0; t < kTokens; ++t) {
        const int i = token[k][t];
        y[k][t] = Raw8<DF>{};
        if (i >= 0 && i < n) y[k][t] = load_raw<DF>(row_of<DF>(P.dy, i), col, P.dy.cols);
      }
  }
  Raw8<OF> was[kRowsEach] = {};
  if (P.accumulate) {
#pragma unroll
    for (int k = 0; k < kRowsEach; ++k)
      if (at[k + 1] > at[k] && at[k + 1] - at[k] <= kTokens) was[k] = load_raw<OF>(row_of<OF>(P.out, r0 + k), col, P.out.cols);
  }
  __syncthreads();
  bool more = false;
#pragma unroll
  for (int k = 0; k < kRowsEach; ++k) {
    const int64_t r = r0 + k;
    if (r >= P.out.rows || (P.accumulate && at[k + 1] == at[k])) continue;
    if (at[k + 1] - at[k] <= kTokens) {
      Eight x = {};
#pragma unroll
      for (int t = 0; t < kTokens; ++t) add8(x, widen8(y[k][t]));
      write_row<OF>(P, r, col, x, was[k]);
    } else {
      more = true;
      if (lane == 0) {
        const bool longer = RowWork(P, at[k], at[k + 1]).units > kAlone;
        const int place = atomicAdd(&n_listed[longer], 1);
        listed[longer ? groups * kRowsEach - 1 - place : place] = int32_t(r);
      }
    }
  }
  if (!__syncthreads_or(more)) return;
  const int n_alone = n_listed[0], n_long = n_listed[1];
  for (int i = group; i < n_alone; i += groups) {
    const int64_t r = listed[i];
    const RowWork w(P, P.starts[r], P.starts[r + 1]);
    Raw8<OF> old = {};
    if (P.accumulate) old = load_raw<OF>(row_of<OF>(P.out, r), col, P.out.cols);
    write_row<OF>(P, r, col, w.sum<DF>(P, col, lanes, 0, 1), old);
  }
  for (int i = 0; i < n_long; ++i) {
    const int64_t r = listed[groups * kRowsEach - 1 - i];
    const RowWork w(P, P.starts[r], P.starts[r + 1]);
    Raw8<OF> old = {};
    if (P.accumulate && group == 0) old = load_raw<OF>(row_of<OF>(P.out, r), col, P.out.cols);
    const Eight x = w.sum<DF>(P, col, lanes, group, groups);
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[e * 256 + threadIdx.x] = x.v[e];
    __syncthreads();
    if (group == 0) {
      Eight z = {};
      for (int k = 0; k < groups; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) z.v[e] += sums[e * 256 + k * lanes + lane];
      write_row<OF>(P, r, col, z, old);
    }
    __syncthreads();
  }
}

// Lanes that share a row of n columns.
int lanes_for(int64_t n) {
  int lanes = 1;
  while (lanes < 64 && int64_t(lanes) * 8 < n) lanes *= 2;
  return lanes;
}

// Workgroups for so many rows, up to 2^20 (a launch has fewer than 2^32 lanes): only a
// lookup has more, and goes on from there.
dim3 grid_for(int64_t rows, int lanes) {
  return dim3(unsigned(std::min<int64_t>((rows + 256 / lanes - 1) / (256 / lanes), int64_t(1) << 20)));
}
static_assert(kMaxTableRows <= int64_t(1) << 20, "a workgroup for every row of a table");

}  // namespace

hipError_t launch_lookup(const LookupLaunch& a, hipStream_t s) {
  if (a.out.rows <= 0 || a.out.cols <= 0) return hipSuccess;
  const int lanes = lanes_for(a.out.cols);
  const dim3 grid = grid_for(a.out.rows, lanes);
  if (a.table.fp32) {
    if (a.out.fp32) hipLaunchKernelGGL((k_lookup<true, true>), grid, dim3(256), 0, s, a, lanes);
    else hipLaunchKernelGGL((k_lookup<true, false>), grid, dim3(256), 0, s, a, lanes);
  } else {
    if (a.out.fp32) hipLaunchKernelGGL((k_lookup<false, true>), grid, dim3(256), 0, s, a, lanes);
    else hipLaunchKernelGGL((k_lookup<false, false>), grid, dim3(256), 0, s, a, lanes);
  }
  return hipGetLastError();
}

template <int BITS>
void sort_few(const RowSortLaunch& a, dim3 grid, hipStream_t s) {
  if (a.n <= kSortBlock) hipLaunchKernelGGL((k_row_sort_few<BITS, 1>), grid, dim3(kSortBlock), 0, s, a);
  else if (a.n <= 4 * kSortBlock) hipLaunchKernelGGL((k_row_sort_few<BITS, 4>), grid, dim3(kSortBlock), 0, s, a);
  else hipLaunchKernelGGL((k_row_sort_few<BITS, 8>), grid, dim3(kSortBlock), 0, s, a);
}
static_assert(kSortTile == 8 * kSortBlock, "the longest list of one launch");

hipError_t launch_row_sort(const RowSortLaunch& a, hipStream_t s) {
  const int bits = bucket_bits(a.n, a.n_rows);
  // a table without rows has one (empty) bucket, which stores starts[0]
  const dim3 buckets(unsigned(std::max<int64_t>(1, (a.n_rows + (int64_t(1) << bits) - 1) >> bits)));
  if (a.n <= kSortTile) {
    if (bits == 6) sort_few<6>(a, buckets, s);
    else if (bits == 8) sort_few<8>(a, buckets, s);
    else sort_few<10>(a, buckets, s);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(k_row_sort_count, dim3(unsigned(a.n_chunks)), dim3(kSortBlock), 0, s, a, bits);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_row_sort_spread, dim3(unsigned(a.n_chunks)), dim3(kSortBlock), 0, s, a, bits);
  e = hipGetLastError();
  if (e != hipSuccess || bits == 0) return e;
  if (bits == 2) hipLaunchKernelGGL(k_row_sort_bucket<2>, buckets, dim3(kSortBlock), 0, s, a);
  else if (bits == 4) hipLaunchKernelGGL(k_row_sort_bucket<4>, buckets, dim3(kSortBlock), 0, s, a);
  else if (bits == 6) hipLaunchKernelGGL(k_row_sort_bucket<6>, buckets, dim3(kSortBlock), 0, s, a);
  else if (bits == 8) hipLaunchKernelGGL(k_row_sort_bucket<8>, buckets, dim3(kSortBlock), 0, s, a);
  else hipLaunchKernelGGL(k_row_sort_bucket<10>, buckets, dim3(kSortBlock), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_lookup_grad(const LookupGradLaunch& a, hipStream_t s) {
  if (a.out.rows <= 0 || a.out.cols <= 0) return hipSuccess;
  const int lanes = lanes_for(a.out.cols);
  const unsigned across = unsigned((a.out.cols + 8 * lanes - 1) / (8 * lanes));
  if (a.n_runs > 0) {
    dim3 grid = grid_for(a.n_runs, lanes);
    grid.y = across;
    if (a.dy.fp32) hipLaunchKernelGGL(k_grad_runs<true>, grid, dim3(256), 0, s, a, lanes);
    else hipLaunchKernelGGL(k_grad_runs<false>, grid, dim3(256), 0, s, a, lanes);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  dim3 grid = grid_for((a.out.rows + kRowsEach - 1) / kRowsEach, lanes);
  grid.y = across;
  if (a.dy.fp32) {
    if (a.out.fp32) hipLaunchKernelGGL((k_grad_rows<true, true>), grid, dim3(256), 0, s, a, lanes);
    else hipLaunchKernelGGL((k_grad_rows<true, false>), grid, dim3(256), 0, s, a, lanes);
  } else {
    if (a.out.fp32) hipLaunchKernelGGL((k_grad_rows<false, true>), grid, dim3(256), 0, s, a, lanes);
    else hipLaunchKernelGGL((k_grad_rows<false, false>), grid, dim3(256), 0, s, a, lanes);
  }
  return hipGetLastError();
}

}  // namespace gro
