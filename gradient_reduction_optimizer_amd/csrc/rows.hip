// Embedding lookups with a scale, positions sorted by the row they name, and the
// lookup's gradient as sums over those positions.  gfx950.
#include <hip/hip_runtime.h>

#include "lane.h"
#include "layers.h"

namespace gro {
namespace {

// Eight elements at any alignment of their own type (the hardware takes global
// accesses at any address).
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
struct __attribute__((packed, aligned(2))) Bf16x8 { u16x8 v; };
struct __attribute__((packed, aligned(4))) F32x4u { f32x4 v; };

struct Eight {
  float v[8];
};

// Elements [col, col + 8) of a row, those at n and behind as zeros.
template <bool FP32>
__device__ __forceinline__ Eight load8(const void* row, int64_t col, int64_t n) {
  Eight x;
  if (col + 8 <= n) {
    if constexpr (FP32) {
      const float* p = static_cast<const float*>(row) + col;
      const f32x4 a = reinterpret_cast<const F32x4u*>(p)->v, b = reinterpret_cast<const F32x4u*>(p + 4)->v;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x.v[e] = a[e];
        x.v[4 + e] = b[e];
      }
    } else {
      const u16x8 a = reinterpret_cast<const Bf16x8*>(static_cast<const uint16_t*>(row) + col)->v;
#pragma unroll
      for (int e = 0; e < 8; ++e) x.v[e] = widen1(a[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x.v[e] = 0.0f;
      if (col + e < n) x.v[e] = FP32 ? static_cast<const float*>(row)[col + e] : widen1(static_cast<const uint16_t*>(row)[col + e]);
    }
  }
  return x;
}

template <bool FP32>
__device__ __forceinline__ void store8(void* row, int64_t col, int64_t n, const Eight& x) {
  if (col + 8 <= n) {
    if constexpr (FP32) {
      float* p = static_cast<float*>(row) + col;
      reinterpret_cast<F32x4u*>(p)->v = f32x4{x.v[0], x.v[1], x.v[2], x.v[3]};
      reinterpret_cast<F32x4u*>(p + 4)->v = f32x4{x.v[4], x.v[5], x.v[6], x.v[7]};
    } else {
      u16x8 a;
#pragma unroll
      for (int e = 0; e < 8; ++e) a[e] = bf16_bits(x.v[e]);
      reinterpret_cast<Bf16x8*>(static_cast<uint16_t*>(row) + col)->v = a;
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
// power of two) share a row, 8 elements each at a time.
template <bool TF, bool OF>
__global__ __launch_bounds__(256) void k_lookup(const LookupLaunch P, const int lanes) {
  const int group = int(threadIdx.x) / lanes, lane = int(threadIdx.x) & (lanes - 1), groups = 256 / lanes;
  const int64_t n = P.out.cols;
  for (int64_t i = int64_t(blockIdx.x) * groups + group; i < P.out.rows; i += int64_t(gridDim.x) * groups) {
    const uint32_t r = row_of_id(P.ids, P.wide_ids, i, P.first, P.table.rows);
    char* out = row_of<OF>(P.out, i);
    if (r == 0xffffffffu) {
      const Eight zero = {};
      for (int64_t c = 8 * lane; c < n; c += 8 * lanes) store8<OF>(out, c, n, zero);
      continue;
    }
    const char* in = row_of<TF>(P.table, r);
#pragma unroll 4
    for (int64_t c = 8 * lane; c < n; c += 8 * lanes) {
      Eight x = load8<TF>(in, c, n);
#pragma unroll
      for (int e = 0; e < 8; ++e) x.v[e] *= P.scale;
      store8<OF>(out, c, n, x);
    }
  }
}

// ------------------------------------------------------------------- the sort
// A stable counting sort.  A tile's items are numbered wave by wave: item
// w * (64 * ROUNDS) + j * 64 + l is lane l's of wave w in round j, so ranks within
// a wave, in this order, and a prefix over waves keep equal rows in the order of
// their positions.  No atomics decide an order.
constexpr int kSortBlock = 1024;
constexpr int kSortWaves = kSortBlock / 64;

// Ranks of this lane's items among the wave's with the same digit; counts[wave][.]
// is the wave's, zero before.  digit = -1: no item.
template <int BITS, int ROUNDS>
__device__ __forceinline__ void rank_in_wave(const int (&digit)[ROUNDS], uint32_t (&rank)[ROUNDS], uint32_t* counts) {
  const int lane = int(threadIdx.x) & 63;
#pragma unroll
  for (int j = 0; j < ROUNDS; ++j) {
    uint64_t same = __ballot(digit[j] >= 0);
#pragma unroll
    for (int b = 0; b < BITS; ++b) {
      const bool bit = (digit[j] >> b) & 1;
      const uint64_t with = __ballot(bit);
      same &= bit ? with : ~with;
    }
    rank[j] = 0;
    if (digit[j] >= 0) {
      const uint32_t before = counts[digit[j]];
      rank[j] = before + __popcll(same & ((uint64_t(1) << lane) - 1));
      // the last of them stores; the wave's LDS operations keep their order
      if (lane == 63 - __clzll(same)) counts[digit[j]] = rank[j] + 1;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// counts[w][d] to the sum over the waves before w; returns digit threadIdx.x's
// total (0 from digit `bins` on).
__device__ __forceinline__ uint32_t prefix_over_waves(uint32_t* counts, int bins) {
  uint32_t total = 0;
  if (int(threadIdx.x) < bins) {
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t c = counts[w * bins + threadIdx.x];
      counts[w * bins + threadIdx.x] = total;
      total += c;
    }
  }
  return total;
}

// Exclusive prefix sum over the workgroup's lanes; `all` the sum.  part: 17 words
// of LDS.
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

// Up to kSortTile ids in one launch: workgroup b reads them all, counts those in
// front of its bucket and sorts those of its bucket.
template <int BITS>
__global__ __launch_bounds__(kSortBlock) void k_row_sort_few(const RowSortLaunch P) {
  constexpr int kBins = 1 << BITS, kRounds = kSortTile / kSortBlock;
  __shared__ uint32_t item[kSortTile];          // position, packed
  __shared__ uint16_t row[kSortTile];
  __shared__ uint32_t counts[kSortWaves * kBins];
  __shared__ uint32_t base[kBins];
  __shared__ uint32_t part[kSortWaves + 1];
  const int64_t lo = int64_t(blockIdx.x) << BITS, hi = std::min(lo + kBins, P.n_rows);
  for (int i = int(threadIdx.x); i < kSortWaves * kBins; i += kSortBlock) counts[i] = 0;
  uint32_t key[kRounds], mine = 0, below = 0;
  const int first = int(threadIdx.x) * kRounds, n = int(P.n);
#pragma unroll
  for (int j = 0; j < kRounds; ++j) {
    key[j] = 0xffffffffu;
    if (first + j < n) key[j] = row_of_id(P.ids, P.wide_ids, first + j, P.first, P.n_rows);
    below += key[j] < uint32_t(lo);
    mine += key[j] >= uint32_t(lo) && int64_t(key[j]) < hi;
  }
  uint32_t n_below, n_mine;
  block_prefix(below, part, n_below);
  uint32_t at = block_prefix(mine, part, n_mine);
#pragma unroll
  for (int j = 0; j < kRounds; ++j)
    if (key[j] >= uint32_t(lo) && int64_t(key[j]) < hi) {
      item[at] = uint32_t(first + j);
      row[at++] = uint16_t(key[j] - uint32_t(lo));
    }
  __syncthreads();
  const int wave = int(threadIdx.x) >> 6, lane = int(threadIdx.x) & 63;
  int digit[kRounds];
  uint32_t rank[kRounds];
#pragma unroll
  for (int j = 0; j < kRounds; ++j) {
    const uint32_t k = uint32_t(wave * 64 * kRounds + j * 64 + lane);
    digit[j] = k < n_mine ? int(row[k]) : -1;
  }
  rank_in_wave<BITS, kRounds>(digit, rank, counts + wave * kBins);
  __syncthreads();
  const uint32_t total = prefix_over_waves(counts, kBins);
  uint32_t all;
  const uint32_t begin = n_below + block_prefix(total, part, all);
  if (int(threadIdx.x) < kBins) {
    base[threadIdx.x] = begin;
    if (lo + int64_t(threadIdx.x) < hi) P.starts[lo + threadIdx.x] = int32_t(begin);
  }
  if (threadIdx.x == 0 && hi == P.n_rows) P.starts[hi] = int32_t(n_below + n_mine);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kRounds; ++j)
    if (digit[j] >= 0) {
      const uint32_t k = uint32_t(wave * 64 * kRounds + j * 64 + lane);
      P.order[base[digit[j]] + counts[wave * kBins + digit[j]] + rank[j]] = int32_t(item[k]);
    }
}

// More ids, first launch: how many of each chunk belong to each bucket.
__global__ __launch_bounds__(kSortBlock) void k_row_sort_count(const RowSortLaunch P, const int bits) {
  __shared__ uint32_t counts[kMaxBuckets];
  counts[threadIdx.x] = 0;
  __syncthreads();
  const int64_t lo = int64_t(blockIdx.x) * P.chunk, hi = std::min(lo + P.chunk, P.n);
  for (int64_t i = lo + threadIdx.x; i < hi; i += kSortBlock) {
    const uint32_t r = row_of_id(P.ids, P.wide_ids, i, P.first, P.n_rows);
    if (r != 0xffffffffu) atomicAdd(&counts[r >> bits], 1u);
  }
  __syncthreads();
  if (int(threadIdx.x) < P.n_buckets) P.counts[int64_t(blockIdx.x) * P.n_buckets + threadIdx.x] = counts[threadIdx.x];
}

// Second launch: rows and positions to their buckets, in order.
__global__ __launch_bounds__(kSortBlock) void k_row_sort_spread(const RowSortLaunch P, const int bits) {
  constexpr int kRounds = kSortChunk / kSortBlock;
  __shared__ uint32_t counts[kSortWaves * kMaxBuckets];
  __shared__ uint32_t base[kMaxBuckets];
  __shared__ uint32_t part[kSortWaves + 1];
  const int nb = P.n_buckets;
  uint32_t before = 0, total = 0, all;
  if (int(threadIdx.x) < nb) {
#pragma unroll 8
    for (int c = 0; c < P.n_chunks; ++c) {
      const uint32_t x = P.counts[int64_t(c) * nb + threadIdx.x];
      total += x;
      before += c < int(blockIdx.x) ? x : 0;
    }
  }
  const uint32_t begin = block_prefix(total, part, all);
  base[threadIdx.x] = begin + before;
  if (blockIdx.x == 0) {
    if (int(threadIdx.x) < nb) P.bases[threadIdx.x] = begin;
    if (threadIdx.x == 0) P.bases[nb] = all;
  }
  const int64_t lo = int64_t(blockIdx.x) * P.chunk, hi = std::min(lo + P.chunk, P.n);
  const int wave = int(threadIdx.x) >> 6, lane = int(threadIdx.x) & 63;
  for (int64_t tile = lo; tile < hi; tile += kSortChunk) {
    for (int i = int(threadIdx.x); i < kSortWaves * nb; i += kSortBlock) counts[i] = 0;
    __syncthreads();
    uint32_t row[kRounds], rank[kRounds];
    int digit[kRounds];
#pragma unroll
    for (int j = 0; j < kRounds; ++j) {
      const int64_t i = tile + wave * 64 * kRounds + j * 64 + lane;
      row[j] = i < hi ? row_of_id(P.ids, P.wide_ids, i, P.first, P.n_rows) : 0xffffffffu;
      digit[j] = row[j] != 0xffffffffu ? int(row[j] >> bits) : -1;
    }
    rank_in_wave<10, kRounds>(digit, rank, counts + wave * nb);
    __syncthreads();
    const uint32_t here = prefix_over_waves(counts, nb);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kRounds; ++j)
      if (digit[j] >= 0) {
        const int64_t to = base[digit[j]] + counts[wave * nb + digit[j]] + rank[j];
        const uint32_t position = uint32_t(tile + wave * 64 * kRounds + j * 64 + lane);
        *reinterpret_cast<u32x2*>(P.pairs + 2 * to) = u32x2{row[j], position};
      }
    __syncthreads();
    base[threadIdx.x] += here;
  }
}

// Third launch: every bucket by row.
template <int BITS>
__global__ __launch_bounds__(kSortBlock) void k_row_sort_bucket(const RowSortLaunch P) {
  constexpr int kBins = 1 << BITS, kRounds = kSortChunk / kSortBlock;
  __shared__ uint32_t counts[kSortWaves * kBins];
  __shared__ uint32_t base[kBins];
  __shared__ uint32_t part[kSortWaves + 1];
  const int64_t lo_row = int64_t(blockIdx.x) << BITS, hi_row = std::min(lo_row + kBins, P.n_rows);
  const int64_t lo = P.bases[blockIdx.x], hi = P.bases[blockIdx.x + 1];
  const int wave = int(threadIdx.x) >> 6, lane = int(threadIdx.x) & 63;
  if (int(threadIdx.x) < kBins) base[threadIdx.x] = 0;
  __syncthreads();
  for (int64_t i = lo + threadIdx.x; i < hi; i += kSortBlock) atomicAdd(&base[P.pairs[2 * i] & (kBins - 1)], 1u);
  __syncthreads();
  uint32_t all;
  const uint32_t begin = block_prefix(int(threadIdx.x) < kBins ? base[threadIdx.x] : 0, part, all) + uint32_t(lo);
  if (int(threadIdx.x) < kBins) {
    base[threadIdx.x] = begin;
    if (lo_row + int64_t(threadIdx.x) < hi_row) P.starts[lo_row + threadIdx.x] = int32_t(begin);
  }
  if (threadIdx.x == 0 && hi_row == P.n_rows) P.starts[hi_row] = int32_t(hi);
  for (int64_t tile = lo; tile < hi; tile += kSortChunk) {
    for (int i = int(threadIdx.x); i < kSortWaves * kBins; i += kSortBlock) counts[i] = 0;
    __syncthreads();
    uint32_t position[kRounds], rank[kRounds];
    int digit[kRounds];
#pragma unroll
    for (int j = 0; j < kRounds; ++j) {
      const int64_t i = tile + wave * 64 * kRounds + j * 64 + lane;
      digit[j] = -1;
      position[j] = 0;
      if (i < hi) {
        const u32x2 p = *reinterpret_cast<const u32x2*>(P.pairs + 2 * i);
        digit[j] = int(p.x & (kBins - 1));
        position[j] = p.y;
      }
    }
    rank_in_wave<BITS, kRounds>(digit, rank, counts + wave * kBins);
    __syncthreads();
    const uint32_t here = prefix_over_waves(counts, kBins);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kRounds; ++j)
      if (digit[j] >= 0) P.order[base[digit[j]] + counts[wave * kBins + digit[j]] + rank[j]] = int32_t(position[j]);
    __syncthreads();
    if (int(threadIdx.x) < kBins) base[threadIdx.x] += here;
  }
}

// --------------------------------------------------------- the lookup's gradient
// Row r's gradient is scale * sum of dy over its positions, in order: HBM-bound,
// dy read once and the table written once.  Positions are cut into runs; the first
// launch sums the runs that lie within one row, so that a common token's row is
// the work of many waves, and the second adds what is left in front of its first
// run, its runs and what is left behind.  The order of every sum depends on the
// rows' lengths alone.
__device__ __forceinline__ int64_t bounded(int32_t at, int64_t lo, int64_t n) {
  return std::min(std::max(int64_t(at), lo), n);
}

// x += dy[order[p]] for the positions [p, end), 8 columns from col on.
template <bool DF>
__device__ __forceinline__ void add_tokens(const LookupGradLaunch& P, int64_t p, int64_t end, int64_t col, Eight& x) {
  const int64_t n = P.dy.rows;
#pragma unroll 8
  for (; p < end; ++p) {
    const int64_t i = P.order[p];
    if (i < 0 || i >= n) continue;
    const Eight y = load8<DF>(row_of<DF>(P.dy, i), col, P.dy.cols);
#pragma unroll
    for (int e = 0; e < 8; ++e) x.v[e] += y.v[e];
  }
}

template <bool DF>
__global__ __launch_bounds__(256) void k_grad_runs(const LookupGradLaunch P, const int lanes) {
  const int group = int(threadIdx.x) / lanes, lane = int(threadIdx.x) & (lanes - 1), groups = 256 / lanes;
  const int64_t q = int64_t(blockIdx.x) * groups + group;
  if (q >= P.n_runs) return;
  const int64_t lo = q * P.run, hi = lo + P.run, rows = P.out.rows;
  // the last row that begins at lo or before
  int64_t a = 0, b = rows;
  while (b - a > 1) {
    const int64_t m = (a + b) / 2;
    if (P.starts[m] <= lo) a = m;
    else b = m;
  }
  if (P.starts[a] > lo || P.starts[a + 1] < hi) return;
  const int64_t padded = (P.out.cols + 7) / 8 * 8;
  for (int64_t c = 8 * lane; c < P.out.cols; c += 8 * lanes) {
    Eight x = {};
    add_tokens<DF>(P, lo, hi, c, x);
    store8<true>(P.partials + q * padded, c, padded, x);
  }
}

template <bool DF, bool OF>
__global__ __launch_bounds__(256) void k_grad_rows(const LookupGradLaunch P, const int lanes) {
  const int group = int(threadIdx.x) / lanes, lane = int(threadIdx.x) & (lanes - 1), groups = 256 / lanes;
  const int64_t r = int64_t(blockIdx.x) * groups + group;
  if (r >= P.out.rows) return;
  const int64_t lo = bounded(P.starts[r], 0, P.dy.rows), hi = bounded(P.starts[r + 1], lo, P.dy.rows);
  if (P.accumulate && lo == hi) return;
  int64_t q0 = (lo + P.run - 1) / P.run, q1 = std::min(hi / P.run, P.n_runs);
  if (q0 >= q1) q0 = q1 = 0;
  const int64_t head = q1 > q0 ? q0 * P.run : hi, tail = q1 > q0 ? q1 * P.run : hi;
  const int64_t cols = P.out.cols, padded = (cols + 7) / 8 * 8;
  char* out = row_of<OF>(P.out, r);
  for (int64_t c = 8 * lane; c < cols; c += 8 * lanes) {
    Eight x = {};
    add_tokens<DF>(P, lo, head, c, x);
#pragma unroll 4
    for (int64_t q = q0; q < q1; ++q) {
      const Eight y = load8<true>(P.partials + q * padded, c, padded);
#pragma unroll
      for (int e = 0; e < 8; ++e) x.v[e] += y.v[e];
    }
    add_tokens<DF>(P, tail, hi, c, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) x.v[e] *= P.scale;
    if (P.accumulate) {
      const Eight was = load8<OF>(out, c, cols);
#pragma unroll
      for (int e = 0; e < 8; ++e) x.v[e] += was.v[e];
    }
    store8<OF>(out, c, cols, x);
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

hipError_t launch_row_sort(const RowSortLaunch& a, hipStream_t s) {
  const int bits = bucket_bits(a.n_rows);
  // a table without rows has one (empty) bucket, which stores starts[0]
  const int64_t buckets = std::max<int64_t>(1, (a.n_rows + (int64_t(1) << bits) - 1) >> bits);
  if (a.n <= kSortTile) {
    if (bits == 8) hipLaunchKernelGGL(k_row_sort_few<8>, dim3(unsigned(buckets)), dim3(kSortBlock), 0, s, a);
    else hipLaunchKernelGGL(k_row_sort_few<10>, dim3(unsigned(buckets)), dim3(kSortBlock), 0, s, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(k_row_sort_count, dim3(unsigned(a.n_chunks)), dim3(kSortBlock), 0, s, a, bits);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_row_sort_spread, dim3(unsigned(a.n_chunks)), dim3(kSortBlock), 0, s, a, bits);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (bits == 8) hipLaunchKernelGGL(k_row_sort_bucket<8>, dim3(unsigned(buckets)), dim3(kSortBlock), 0, s, a);
  else hipLaunchKernelGGL(k_row_sort_bucket<10>, dim3(unsigned(buckets)), dim3(kSortBlock), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_lookup_grad(const LookupGradLaunch& a, hipStream_t s) {
  if (a.out.rows <= 0 || a.out.cols <= 0) return hipSuccess;
  const int lanes = lanes_for(a.out.cols);
  if (a.n_runs > 0) {
    const dim3 grid = grid_for(a.n_runs, lanes);
    if (a.dy.fp32) hipLaunchKernelGGL(k_grad_runs<true>, grid, dim3(256), 0, s, a, lanes);
    else hipLaunchKernelGGL(k_grad_runs<false>, grid, dim3(256), 0, s, a, lanes);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const dim3 grid = grid_for(a.out.rows, lanes);
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
