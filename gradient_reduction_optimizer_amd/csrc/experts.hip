// Experts' matrix products over ragged runs of rows: y = x W^T, dx = dy W and
// dW = dy^T x for each expert, BF16 in, FP32 sums in the matrix cores, BF16 or
// FP32 out.  gfx950.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "lane.h"
#include "layers.h"

namespace gro {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Rows of expert e, cut to those that exist.
struct Run {
  int lo, hi;
};
__device__ __forceinline__ Run run_of(const ExpertsLaunch& P, int e) {
  Run r;
  const int rows = int(P.rows);
  r.lo = std::min(std::max(P.starts[e], 0), rows);
  r.hi = std::min(std::max(P.starts[e + 1], r.lo), rows);
  return r;
}

__device__ __forceinline__ int64_t uniform(int64_t x) {
  return int64_t(uint64_t(uint32_t(__builtin_amdgcn_readfirstlane(int(x)))) |
                 uint64_t(uint32_t(__builtin_amdgcn_readfirstlane(int(x >> 32)))) << 32);
}
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// Which of `total` tiles is workgroup b's, of tiles numbered so that `chunk` in a row
// are neighbours.  Workgroup b runs on XCD b mod 8: each XCD takes a chunk at a time, so
// that tiles which read the same rows and columns of the operands at the same time
// share its L2.  `total` or more: none.
__device__ __forceinline__ uint32_t xcd_order(uint32_t b, uint32_t total, uint32_t chunk) {
  const uint32_t c = std::min(chunk, (total + 7) / 8), j = b >> 3;
  return c > 0 ? (j / c * 8 + (b & 7)) * c + j % c : 0;
}
// Numbers b that reach every tile so.
__device__ __forceinline__ uint32_t xcd_numbers(uint32_t total, uint32_t chunk) { return (total + 7) / 8 * 8 + 8 * chunk; }

// Number `i` of a grid of m_tiles x n_tiles in bands of up to 8 tiles of m: neighbours
// in number are neighbours in both.
struct Place {
  uint32_t m, n;
};
__device__ __forceinline__ Place banded(uint32_t i, uint32_t m_tiles, uint32_t n_tiles) {
  const uint32_t band = i / (8 * n_tiles), in_band = std::min(8u, m_tiles - 8 * band), r = i - band * 8 * n_tiles;
  return Place{band * 8 + r % in_band, r / in_band};
}

// Tiles of BM rows that the experts' runs take, and of one of them the expert and its
// rows: tiles are numbered expert by expert.  A wave looks at 64 experts at a time.
template <int BM>
struct Tiles {
  Run r;            // lane's expert of the first 64
  uint32_t upto;
  uint32_t total;
  static __device__ __forceinline__ uint32_t count(const Run& r) { return uint32_t(r.hi - r.lo + BM - 1) / BM; }
  static __device__ __forceinline__ Run run(const ExpertsLaunch& P, int e) {
    return e < P.n_experts ? run_of(P, e) : Run{0, 0};
  }
  static __device__ __forceinline__ uint32_t prefix(uint32_t x) {
    const int lane = int(threadIdx.x) & 63;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const uint32_t t = __shfl_up(x, m, 64);
      if (lane >= m) x += t;
    }
    return x;
  }
  __device__ __forceinline__ Tiles(const ExpertsLaunch& P) {
    const int lane = int(threadIdx.x) & 63;
    r = run(P, lane);
    upto = prefix(count(r));
    total = uint32_t(__builtin_amdgcn_readlane(int(upto), 63));
    for (int e0 = 64; e0 < P.n_experts; e0 += 64)
      total += uint32_t(__builtin_amdgcn_readlane(int(prefix(count(run(P, e0 + lane)))), 63));
  }
  // false only for runs so many and so long, one over the other, that their tiles are not
  // counted in 32 bits
  __device__ __forceinline__ bool find(const ExpertsLaunch& P, uint32_t tile, int& expert, int& row, int& end) const {
    const int lane = int(threadIdx.x) & 63;
    Run q = r;
    uint32_t u = upto;
    for (int e0 = 0; e0 < P.n_experts; e0 += 64) {
      const uint64_t over = __ballot(u > tile);
      if (over) {
        const int l = uniform(__ffsll(static_cast<unsigned long long>(over)) - 1);
        expert = e0 + l;
        row = __builtin_amdgcn_readlane(q.lo + int(tile - (u - count(q))) * BM, l);
        end = __builtin_amdgcn_readlane(q.hi, l);
        return row < end;
      }
      tile -= uint32_t(__builtin_amdgcn_readlane(int(u), 63));
      q = run(P, e0 + 64 + lane);
      u = prefix(count(q));
    }
    return false;
  }
};

// ---------------------------------------------------------------------- the tiles
// BM x BN of C = A B^T by WM x WN waves, k in steps of 32, bound by the matrix cores:
// every wave sums 128 x 64 (or 64 x 64) of C in registers, from fragments of 32 x 16.
//   Copies.  Both operands' tiles go from global memory to one of four buffers in LDS
// without passing registers (or, at other alignments, through them), three steps ahead
// of their use: a step takes 0.8 us, a read from memory up to 2.  Waves wait for the
// copies of the next step only, by counting their accesses.
//   One barrier a step.  Every wave reads the fragments of half a step while it
// multiplies those of the half before, so at the barrier all reads of a buffer are done
// and the buffer is free for the step after next but one.
//   From tile to tile.  A workgroup has a compute unit (or half of one) for itself and
// takes a tile after the other; the next one's first four steps are under way while
// this one's result is written.  All tiles end at about the same time, and their results
// leave in bursts that the memory takes 6 us for, 10 us a tile with what else it costs to
// begin one: without that 2048 k would run at 1.3 PFLOP/s.
//   32,768 rows of 16 experts from 2048 to 8192 elements: 1,069 us forward (1.03
// PFLOP/s; the ragged tiles are 6 % of the work), 16,384 rows of 8 experts of 1024 x 4096
// 151 us for the input gradient (k = 1024: 0.91) and 136 for the weight gradient (1.01);
// the matrix cores are busy for 63, 57 and (FP32 results added to) 48 % of the cycles, LDS
// for 26, 34 and 40.  Library products of the first two's sizes with a single matrix, the
// operands in these orders, run at 1.34 to 1.47 and 1.09.
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
#define GRO_LDS __attribute__((address_space(3)))
constexpr int kStepK = 32, kStages = 4;
// LDS of a workgroup: four steps of both operands, and for each wave a block of 32 x 32
// results.
constexpr int tile_lds(int bm, int bn, int waves) { return (bm + bn) * kStepK * 2 * kStages + waves * 32 * 32 * 4; }
// Workgroups of a compute unit, tiles that an XCD's 32 units work on at a time, and the
// launch: the kernel steps from tile to tile by so many, so a launch has all of them,
// also for fewer tiles.
constexpr int tile_units(int bm, int bn, int waves) { return 160 * 1024 / tile_lds(bm, bn, waves); }
constexpr uint32_t tile_chunk(int bm, int bn, int waves) { return 32 * uint32_t(tile_units(bm, bn, waves)); }
constexpr uint32_t tile_grid(int bm, int bn, int waves) { return 8 * tile_chunk(bm, bn, waves); }

// One operand's tile of R rows (of C) and 32 k.
//   k innermost in memory (T = false): LDS holds [R][32], row r's chunk c of 8
//   elements at place c ^ (r / 4 mod 4), so that 16 rows' reads of one chunk meet all
//   banks.
//   rows of C innermost (T = true): LDS holds [32][R], unit u of 16 elements of k at
//   place u ^ (k & 3 | k >> 1 & 4); fragments come out of transposing reads, whose
//   8 different k meet all banks.
template <bool T, int R, int THREADS>
struct Tile {
  static constexpr int kChunks = T ? R / 8 : kStepK / 8;       // of a line in LDS
  static constexpr int kLoads = R * kStepK / 8 / THREADS;      // 16 bytes each, of a lane
  static constexpr int kLineStep = THREADS / kChunks;          // lines between a lane's loads

  // What a lane copies in load i: its line and the chunk that belongs to its place there.
  static __device__ __forceinline__ int line(int i) { return int(threadIdx.x) / kChunks + i * kLineStep; }
  static __device__ __forceinline__ int chunk(int i) {
    const int c = int(threadIdx.x) % kChunks, l = line(i);
    return T ? c ^ (((l & 3) | ((l >> 1) & 4)) << 1) : c ^ ((l >> 2) & 3);
  }
};

// Loader of one operand: where the lane's lines of a step lie, as a byte offset each
// from an address that all lanes share.  DIRECT: copied to LDS without passing
// registers, which takes 16-byte places, whole chunks and offsets of 32 bits; else read
// from any address into registers, a step ahead, and stored.
template <bool DIRECT, bool T, int R, int THREADS>
struct Loader {
  typedef Tile<T, R, THREADS> L;
  typedef u16x8 Chunk __attribute__((aligned(2)));
  const char* from;
  std::conditional_t<DIRECT, int, int64_t> step_bytes;   // T only
  std::conditional_t<DIRECT, uint32_t, int64_t> at[L::kLoads];
  int cols;                                              // T: columns that exist from r0 on
  bool wide;                                             // a row has 8 elements at least
  u16x8 held[DIRECT ? 1 : L::kLoads];

  // Rows [r0, end) of the operand (lines, or columns where T); those behind read one
  // that exists, and what becomes of them is not stored.
  __device__ __forceinline__ void set(const uint16_t* base, int64_t stride, int r0, int end, int length) {
    wide = length >= 8;
    typedef std::conditional_t<DIRECT, int, int64_t> Offset;
    if constexpr (T) step_bytes = Offset(uniform(2 * kStepK * stride));
    from = reinterpret_cast<const char*>(uniform(int64_t(reinterpret_cast<uintptr_t>(base + (T ? r0 : r0 * stride)))));
    const Offset s = Offset(stride);
    cols = end - r0;
#pragma unroll
    for (int i = 0; i < L::kLoads; ++i) {
      const int line = L::line(i), c = 8 * L::chunk(i);
      at[i] = 2 * (T ? line * s + (c < cols ? c : 0) : std::min(line, cols - 1) * s + c);
    }
  }
  // The first n elements of a chunk, others being anything: where a row is cut off its
  // last 8, for settle() to move to the front.
  __device__ __forceinline__ u16x8 chunk(int i, int n) const {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(from + at[i]);
    u16x8 x = {};
    if (wide) {
      if (n > 0) x = *reinterpret_cast<const Chunk*>(p - (n < 8 ? 8 - n : 0));
    } else {
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (e < n) x[e] = p[e];
    }
    return x;
  }
  __device__ __forceinline__ u16x8 settle(u16x8 x, int n) const {
    if (wide && n > 0 && n < 8)
      x = __builtin_bit_cast(u16x8, __builtin_bit_cast(unsigned __int128, x) >> (16 * (8 - n)));
    return x;
  }
  // of a line of T, whose chunk of columns may be cut off (not where chunks are whole)
  __device__ __forceinline__ int columns(int i) const { return DIRECT || !T ? 8 : cols - 8 * L::chunk(i); }

  __device__ __forceinline__ void copy(uint16_t* lds, int wave) {
#ifdef __HIP_DEVICE_COMPILE__  // the host's pass does not know the descriptor's type
    const auto all = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(from), 0, -1, 0x00020000);
#pragma unroll
    for (int i = 0; i < L::kLoads; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(all, (GRO_LDS void*)(lds + wave * 512 + i * THREADS * 8), 16, int(at[i]), 0, 0, 0);
#endif
    advance();
  }
  __device__ __forceinline__ void advance() { from += T ? step_bytes : 2 * kStepK; }
  __device__ __forceinline__ void fetch() {
#pragma unroll
    for (int i = 0; i < L::kLoads; ++i) {
      if constexpr (T) held[i] = chunk(i, columns(i));
      else held[i] = *reinterpret_cast<const Chunk*>(from + at[i]);  // 32 k are whole chunks
    }
    advance();
  }
  __device__ __forceinline__ void store(uint16_t* lds) const {
#pragma unroll
    for (int i = 0; i < L::kLoads; ++i) *reinterpret_cast<u16x8*>(lds + (threadIdx.x + i * THREADS) * 8) = settle(held[i], columns(i));
  }
  // A step of `left` < kStepK k: zeros behind them.
  __device__ __forceinline__ void copy_part(uint16_t* lds, int left) const {
#pragma unroll
    for (int i = 0; i < L::kLoads; ++i) {
      const int n = T ? (L::line(i) < left ? columns(i) : 0) : left - 8 * L::chunk(i);
      *reinterpret_cast<u16x8*>(lds + (threadIdx.x + i * THREADS) * 8) = settle(chunk(i, n), n);
    }
  }
};

// N fragments of 32 rows from row `first` of a tile on, for 16 of its k: lane l has row
// l mod 32 and 8 k from 8 * (l / 32) on.
template <bool T, int R, int N>
struct Reader {
  int at[T ? N : 2];
  __device__ __forceinline__ void set(int first) {
    const int lane = int(threadIdx.x) & 63, l = lane & 15;
    if constexpr (T) {
      // 16 lanes' reads give each the four k of one of 16 rows
      const int k = 8 * (lane >> 5) + (l >> 2), f = (l >> 2) | ((lane >> 5) << 2);
#pragma unroll
      for (int i = 0; i < N; ++i) at[i] = k * R + ((first / 16 + 2 * i + ((lane >> 4) & 1)) ^ f) * 16 + (l & 3) * 4;
    } else {
#pragma unroll
      for (int q = 0; q < 2; ++q)
        at[q] = (first + (lane & 31)) * kStepK + ((2 * q + (lane >> 5)) ^ ((lane >> 2) & 3)) * 8;
    }
  }
  __device__ __forceinline__ void read(const uint16_t* lds, int q, bf16x8 (&f)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (T) {
        const uint16_t* p = lds + at[i] + q * 16 * R;
        const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((GRO_LDS bf16x4*)(p));
        const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((GRO_LDS bf16x4*)(p + 4 * R));
        f[i] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      } else {
        f[i] = *reinterpret_cast<const bf16x8*>(lds + at[q] + i * 32 * kStepK);
      }
    }
  }
};

// All that this wave has read from LDS has arrived and all of its accesses to global
// memory but the last N are done, for all waves.
template <int N>
__device__ __forceinline__ void step_barrier() {
  // reads stay in front; the builtin for LDS, so that the compiler knows and adds no waits
  // of its own behind it
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xc07f);
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");
}

__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xc07f);
  asm volatile("s_barrier" ::: "memory");
}

// Four neighbours of a row of C, or eight that are rounded already, of which `left`
// exist.
template <bool CF>
__device__ __forceinline__ void store_c(const ExpertsLaunch& P, int64_t at, int left, f32x4 x) {
  typedef f32x4 F4 __attribute__((aligned(4)));
  typedef u32x2 B4 __attribute__((aligned(2)));
  if (left >= 4) {
    if constexpr (CF) {
      F4* c = reinterpret_cast<F4*>(static_cast<float*>(P.c) + at);
      if (P.accumulate) x += *c;
      *c = x;
    } else {
      B4* c = reinterpret_cast<B4*>(static_cast<uint16_t*>(P.c) + at);
      if (P.accumulate) x += widen4(*c);
      *c = u32x2{bf16x2_bits(x[0], x[1]), bf16x2_bits(x[2], x[3])};
    }
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (e < left) {
        if constexpr (CF) {
          float* c = static_cast<float*>(P.c) + at + e;
          *c = P.accumulate ? *c + x[e] : x[e];
        } else {
          uint16_t* c = static_cast<uint16_t*>(P.c) + at + e;
          *c = bf16_bits(P.accumulate ? widen1(*c) + x[e] : x[e]);
        }
      }
  }
}
template <bool LINES>
__device__ __forceinline__ void store_rounded(const ExpertsLaunch& P, int64_t at, int left, u16x8 x) {
  typedef u16x8 B8 __attribute__((aligned(2)));
  uint16_t* c = static_cast<uint16_t*>(P.c) + at;
  if (left >= 8) {
    if constexpr (LINES) __builtin_nontemporal_store(x, reinterpret_cast<B8*>(c));
    else *reinterpret_cast<B8*>(c) = x;
  } else {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < left) c[e] = x[e];
  }
}

// The compiler's order of what stands in front of it: MFMAS matrix instructions with
// READS reads from LDS among them, so that the wait for what the part before has read
// stands in front of the new reads.
template <int READS, int MFMAS>
__device__ __forceinline__ void interleave() {
  constexpr int kEach = (READS + MFMAS - 3) / (MFMAS - 2);
  __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
#pragma unroll
  for (int i = 0; i < READS; i += kEach) {
    __builtin_amdgcn_sched_group_barrier(0x100, kEach, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, MFMAS, 0);
  __builtin_amdgcn_sched_barrier(0);
}

// A wave's accesses to its own LDS in the order of the source.
__device__ __forceinline__ void in_wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A tile of C: rows [m0, m_end) and columns from n0 on of an expert's, and the k it sums.
struct Job {
  int expert, m0, m_end, n0, k_lo, k_n, part;
};

// What a launch covers: every tile; every tile in parts of its k; of 256 x 256 tiles
// those that fill the GPU a whole number of times, if so few are left that they are done
// sooner in quarters; those quarters.
enum Cover { kAll, kParts, kRounds, kQuarters };
// Tiles of `total` that are left to quarters.
__device__ __forceinline__ uint32_t left_over(uint32_t total) {
  const uint32_t n = total % 256;
  return total > 256 && n <= 128 ? n : 0;
}

// C in FP32, in BF16, or in BF16 with rows that begin at whole lines of 128 bytes.  The
// last are stored past the caches, since C is larger than they are and the next tiles'
// operands are in them: an input gradient of 16,384 rows 136 us instead of 157, the same
// inputs in turn.  Pieces of lines are left to the caches: 48 weight gradients of 1408 x
// 3944 without a row each 199 us instead of 345.  FP32 takes the same time either way.
enum Result { kFp32, kBf16, kBf16Lines };

template <int MODE, int BM, int BN, int WM, int WN, bool DIRECT, int COVER, int C>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_experts_tiles(const ExpertsLaunch P) {
  constexpr int kThreads = 64 * WM * WN, FM = BM / WM / 32, FN = BN / WN / 32;
  constexpr bool CF = C == kFp32, PARTS = COVER == kParts, QUARTERS = COVER == kQuarters;
  constexpr int TM = QUARTERS ? 2 * BM : BM, TN = QUARTERS ? 2 * BN : BN;  // as tiles are numbered
  constexpr bool AT = MODE == kWeightGrad, BT = MODE != kForward;
  constexpr uint32_t kChunk = tile_chunk(BM, BN, WM * WN), kGrid = tile_grid(BM, BN, WM * WN);
  __shared__ __attribute__((aligned(16))) uint16_t a0[BM * kStepK], a1[BM * kStepK], a2[BM * kStepK], a3[BM * kStepK];
  __shared__ __attribute__((aligned(16))) uint16_t b0[BN * kStepK], b1[BN * kStepK], b2[BN * kStepK], b3[BN * kStepK];
  __shared__ __attribute__((aligned(16))) float results[WM * WN][32 * 32];
  const int n_end = int(MODE == kForward ? P.outer : P.inner), k_size = int(MODE == kForward ? P.inner : P.outer);
  const int m_size = int(P.outer);  // weight gradient only
  const uint32_t n_tiles = uint32_t((n_end + TN - 1) / TN);
  const int wave = uniform(int(threadIdx.x) >> 6), lane = int(threadIdx.x) & 63;
  const int wm = wave / WN * (BM / WM), wn = wave % WN * (BN / WN);

  const Tiles<TM> tiles(P);
  const uint32_t m_tiles = MODE == kWeightGrad ? uint32_t((P.outer + TM - 1) / TM) : tiles.total;
  const uint32_t whole = m_tiles * n_tiles * (MODE == kWeightGrad ? uint32_t(P.n_experts) : 1u);
  const uint32_t rest = COVER == kRounds || QUARTERS ? left_over(whole) : 0;
  const uint32_t total = PARTS ? whole * uint32_t(P.n_parts) : QUARTERS ? 4 * rest : whole - rest;
  // weight gradients: experts with more rows first, of the first 64 (with the turn below
  // 138 us instead of 187 for 8 experts of 268 to 5,103 rows)
  int rank = 0;
  if constexpr (MODE == kWeightGrad) {
    const int mine = tiles.r.hi - tiles.r.lo;
    for (int e = 0; e < std::min(P.n_experts, 64); ++e) {
      const int n = __builtin_amdgcn_readlane(mine, e);
      rank += n > mine || (n == mine && e < lane);
    }
  }
  const auto by_length = [&](int place) {
    return place < 64 ? uniform(__ffsll(static_cast<unsigned long long>(__ballot(rank == place && lane < P.n_experts))) - 1) : place;
  };
  // where a round of workgroups has tiles of several experts, every other round goes
  // backwards, so that a workgroup's jobs are long and short
  const bool turn = MODE == kWeightGrad && m_tiles * n_tiles < kGrid;
  const auto find = [&](uint32_t b, Job& job) {
    const uint32_t round = b / kGrid, in_round = b % kGrid;
    const uint32_t i = xcd_order(turn && (round & 1) ? round * kGrid + (kGrid - 1 - in_round) : b, total, kChunk);
    if (i >= total) return false;
    const uint32_t part = PARTS ? i / whole : 0, tile = QUARTERS ? whole - rest + i / 4 : i - part * whole;
    if constexpr (MODE == kWeightGrad) {
      const Place p = banded(tile % (m_tiles * n_tiles), m_tiles, n_tiles);
      job.expert = by_length(int(tile / (m_tiles * n_tiles)));
      const Run r = run_of(P, job.expert);
      job.m0 = int(p.m) * BM;
      job.n0 = int(p.n) * BN;
      job.m_end = m_size;
      job.k_lo = uniform(r.lo);
      job.k_n = uniform(r.hi - r.lo);
    } else {
      const Place p = banded(tile, m_tiles, n_tiles);
      if (!tiles.find(P, p.m, job.expert, job.m0, job.m_end)) return false;
      job.n0 = int(p.n) * TN;
      if constexpr (QUARTERS) {
        job.m0 += int(i & 1) * BM;
        job.n0 += int(i >> 1 & 1) * BN;
        if (job.m0 >= job.m_end || job.n0 >= n_end) return false;
      }
      job.k_lo = 0;
      job.k_n = k_size;
    }
    if constexpr (PARTS) {
      job.part = int(part);
      // a part of the steps, the last part with what is left behind whole ones
      const int steps = job.k_n / kStepK, from = int(int64_t(steps) * part / P.n_parts) * kStepK;
      const int to = job.part + 1 == P.n_parts ? job.k_n : int(int64_t(steps) * (part + 1) / P.n_parts) * kStepK;
      job.k_lo += from;
      job.k_n = to - from;
    }
    return true;
  };
  // the next tile that a workgroup has, of those xcd_order leaves it
  uint32_t b = blockIdx.x;
  const uint32_t last = (xcd_numbers(total, kChunk) + kGrid - 1) / kGrid * kGrid;
  const auto next = [&](Job& job) {
    for (; b < last; b += kGrid)
      if (find(b, job)) {
        b += kGrid;
        return true;
      }
    return false;
  };

  static_assert(FN == 2, "a wave's block of results is 64 wide");
  Loader<DIRECT, AT, BM, kThreads> la;
  Loader<DIRECT, BT, BN, kThreads> lb;
  constexpr int kLoads = decltype(la)::L::kLoads + decltype(lb)::L::kLoads, kStores = CF ? 8 * FM : 4 * FM;
  static_assert((kStages - 1) * kLoads + kStores < 64, "vmcnt counts to 63");
  Reader<AT, BM, FM> ra;
  Reader<BT, BN, FN> rb;
  ra.set(wm);
  rb.set(wn);
  uint16_t* const as[kStages] = {a0, a1, a2, a3};
  uint16_t* const bs[kStages] = {b0, b1, b2, b3};
  const auto load = [&](int stage) {
    la.copy(as[stage], wave);
    lb.copy(bs[stage], wave);
  };
  const auto fetch = [&] {
    la.fetch();
    lb.fetch();
  };
  const auto store = [&](int stage) {
    la.store(as[stage]);
    lb.store(bs[stage]);
  };
  const auto begin = [&](const Job& job) {
    la.set(P.a + (AT ? job.k_lo * P.a_stride : job.k_lo), P.a_stride, job.m0, job.m_end, AT ? m_size : k_size);
    lb.set(P.b + (BT ? job.k_lo * P.b_stride : job.k_lo) + (MODE == kWeightGrad ? 0 : job.expert * P.b_expert), P.b_stride, job.n0,
           n_end, BT ? n_end : k_size);
#pragma unroll
    for (int t = 0; t < kStages; ++t)
      if (job.k_n >= (t + 1) * kStepK) {
        if constexpr (DIRECT) {
          load(t);
        } else {
          fetch();
          if (t < kStages - 1) store(t);
        }
      }
  };

  Job job;
  if (!next(job)) return;
  begin(job);
  bool stored = false;  // kStores stores by every wave since this job's first loads
  for (bool more = true; more;) {
    Job ahead;               // found while the first loads are under way
    more = next(ahead);
    f32x16 acc[FM][FN] = {};
    // A step in two parts of 16 k.
    constexpr int kPart = FM * FN, kReads = FM * (AT ? 2 : 1) + FN * (BT ? 2 : 1);
    bf16x8 fa[2][FM], fb[2][FN];
    const auto read = [&](int stage, int q) {
      ra.read(as[stage], q, fa[q]);
      rb.read(bs[stage], q, fb[q]);
    };
    const auto multiply = [&](int q) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[q][j], fa[q][i], acc[i][j], 0, 0, 0);
    };
    const int steps = job.k_n / kStepK, left = job.k_n % kStepK;
    // At step s's barrier step s + 1's loads have to be done.  Behind them are those of
    // two steps more, and for the steps of begin() the stores of the tile before:
    // accesses are counted in the order of their issue.
    const auto step = [&](int s, auto number) {
      constexpr int kStage = decltype(number)::value;
      if constexpr (!DIRECT) {
        // step s + 3's, fetched a step ago, where step s - 1's were
        if (s + kStages - 1 < steps) store((kStage + kStages - 1) % kStages);
        if (s + kStages < steps) fetch();
      }
      read(kStage, 1);
      multiply(0);
      interleave<kReads, kPart>();
      if constexpr (!DIRECT) {
        lds_barrier();
      } else if (s + kStages <= steps) {
        if (stored && s < kStages - 1) step_barrier<(kStages - 2) * kLoads + kStores>();
        else step_barrier<(kStages - 2) * kLoads>();
      } else {
        step_barrier<0>();
      }
      if (DIRECT && s + kStages < steps) load(kStage);
      read((kStage + 1) % kStages, 0);  // behind the last step, whatever the buffers hold
      multiply(1);
      interleave<kReads, kPart>();
    };
    if (steps > 0) {
      if constexpr (!DIRECT) {
        lds_barrier();
      } else if (steps >= kStages) {
        if (stored) step_barrier<(kStages - 1) * kLoads + kStores>();
        else step_barrier<(kStages - 1) * kLoads>();
      } else {
        step_barrier<0>();
      }
      read(0, 0);
      for (int s = 0;;) {
        step(s, std::integral_constant<int, 0>());
        if (++s >= steps) break;
        step(s, std::integral_constant<int, 1>());
        if (++s >= steps) break;
        step(s, std::integral_constant<int, 2>());
        if (++s >= steps) break;
        step(s, std::integral_constant<int, 3>());
        if (++s >= steps) break;
      }
    }
    // the buffers are free; they are anyway where nothing was to be summed, and then the
    // stores of the tile before need not be waited for
    if (job.k_n > 0) step_barrier<0>();
    if (left > 0) {
      la.copy_part(a0, left);
      lb.copy_part(b0, left);
      step_barrier<0>();
      read(0, 0);
      multiply(0);
      read(0, 1);
      multiply(1);
      step_barrier<0>();
    }
    const Job done = job;
    job = ahead;
    if (more) begin(job);
    stored = done.m0 + BM <= done.m_end && done.n0 + BN <= n_end;  // kStores by every wave, or more

    if (MODE == kWeightGrad && P.accumulate && done.k_n == 0) {
      stored = false;
      continue;
    }
    const int64_t base = (MODE == kWeightGrad ? done.expert * P.c_expert : 0) + (PARTS ? done.part * P.c_part : 0);
    // Lane l has row l mod 32 of a block of 32 x 32 of C and of its columns four times
    // four, 8 q + 4 * (l / 32) on.  They go through the wave's own LDS, row r's chunk c of
    // 16 bytes at place c ^ (r / 2 mod 8), and from there to memory in whole lines of 128
    // bytes: 32 columns in FP32, or 64 that are rounded first, unless something is added.
    float* block = results[wave];
    if (!CF && !P.accumulate) {
      uint16_t* rounded = reinterpret_cast<uint16_t*>(block);
#pragma unroll
      for (int i = 0; i < FM; ++i) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int r = lane & 31, c = (4 * j + q) ^ ((r >> 1) & 7);
            *reinterpret_cast<u32x2*>(rounded + r * 64 + 8 * c + 4 * (lane >> 5)) =
                u32x2{bf16x2_bits(acc[i][j][4 * q], acc[i][j][4 * q + 1]), bf16x2_bits(acc[i][j][4 * q + 2], acc[i][j][4 * q + 3])};
          }
        in_wave_order();
        const int n = done.n0 + wn + lane % 8 * 8;
#pragma unroll
        for (int t = 0; t < 32; t += 8) {
          const int r = t + lane / 8, m = done.m0 + wm + 32 * i + r;
          const u16x8 x = *reinterpret_cast<const u16x8*>(rounded + r * 64 + 8 * (lane % 8 ^ ((r >> 1) & 7)));
          if (m < done.m_end && n < n_end) store_rounded<C == kBf16Lines>(P, base + m * P.c_stride + n, n_end - n, x);
        }
        in_wave_order();
      }
      continue;
    }
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = lane & 31, c = (2 * q + (lane >> 5)) ^ ((r >> 1) & 7);
          st4f(block + r * 32 + 4 * c,
               f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]});
        }
        in_wave_order();
        const int n = done.n0 + wn + 32 * j + lane % 8 * 4;
#pragma unroll
        for (int t = 0; t < 32; t += 8) {
          const int r = t + lane / 8, m = done.m0 + wm + 32 * i + r;
          const f32x4 x = ld4f(block + r * 32 + 4 * (lane % 8 ^ ((r >> 1) & 7)));
          if (m < done.m_end && n < n_end) store_c<CF>(P, base + m * P.c_stride + n, n_end - n, x);
        }
        in_wave_order();
      }
  }
}

// The parts' sums, added up in their order, to C: a workgroup has kJoinRows rows of a
// tile, each lane its neighbours of one of them.
constexpr int kJoinRows = 8;
template <int MODE, int BM, int BN, bool CF>
__global__ __launch_bounds__(kJoinRows * BN / 4) void k_experts_join(const ExpertsLaunch P) {
  const int n_end = int(MODE == kForward ? P.outer : P.inner);
  const uint32_t n_tiles = uint32_t((n_end + BN - 1) / BN);
  const uint32_t block = blockIdx.x / (BM / kJoinRows), tile = block / n_tiles;
  const int n0 = int(block % n_tiles) * BN;
  int expert, m0, m_end;
  if constexpr (MODE == kWeightGrad) {
    const uint32_t m_tiles = uint32_t((P.outer + BM - 1) / BM);
    expert = int(tile / m_tiles);
    m0 = int(tile % m_tiles) * BM;
    m_end = int(P.outer);
    const Run r = run_of(P, expert);
    if (P.accumulate && r.lo == r.hi) return;
  } else {
    const Tiles<BM> tiles(P);
    if (tile >= tiles.total || !tiles.find(P, tile, expert, m0, m_end)) return;
  }
  constexpr int kLanes = BN / 4;
  typedef f32x4 F4 __attribute__((aligned(4)));
  const int n = n0 + int(threadIdx.x) % kLanes * 4, left = n_end - n;
  const int m = m0 + int(blockIdx.x % (BM / kJoinRows)) * kJoinRows + int(threadIdx.x) / kLanes;
  if (left <= 0 || m >= m_end) return;
  const float* p = P.partials + (MODE == kWeightGrad ? int64_t(expert) * P.outer * P.inner : 0) + int64_t(m) * n_end + n;
  f32x4 x = {};
#pragma unroll 8
  for (int part = 0; part < P.n_parts; ++part, p += P.c_part) {
    f32x4 y = {};
    if (left >= 4) {
      y = *reinterpret_cast<const F4*>(p);
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (e < left) y[e] = p[e];
    }
    x += y;
  }
  store_c<CF>(P, (MODE == kWeightGrad ? expert * P.c_expert : 0) + m * P.c_stride + n, left, x);
}

// Tiles of BM x BN that cover C: every expert's last one may be a part of one.
int64_t tiles_of(const ExpertsLaunch& a, ExpertsMode mode, int64_t bm, int64_t bn) {
  const int64_t n = mode == kForward ? a.outer : a.inner, across = (n + bn - 1) / bn;
  if (mode == kWeightGrad) return across * ((a.outer + bm - 1) / bm) * a.n_experts;
  return across * std::min<int64_t>(a.rows, a.rows / bm + a.n_experts);
}

// Whether full tiles can be copied straight to LDS: 16-byte accesses at 16-byte
// places, and a tile's offsets in 32 bits.
bool direct(const ExpertsLaunch& a, ExpertsMode mode) {
  const auto fits = [](const void* p, int64_t stride) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % 8 == 0 && stride < (int64_t(1) << 22);
  };
  if (!fits(a.a, a.a_stride) || !fits(a.b, a.b_stride) || a.b_expert % 8 != 0) return false;
  // an operand whose rows of C lie innermost is copied 8 of them at a time
  return mode == kForward || (a.inner % 8 == 0 && (mode == kInputGrad || a.outer % 8 == 0));
}

template <int MODE, int BM, int BN, int WM, int WN, bool DIRECT, int COVER = kAll>
hipError_t tiles(const ExpertsLaunch& a, hipStream_t s) {
  const dim3 grid(tile_grid(BM, BN, WM * WN)), block(64 * WM * WN);
  const bool lines = ((reinterpret_cast<uintptr_t>(a.c) | uint64_t(2 * a.c_stride) | uint64_t(2 * a.c_expert)) & 127) == 0;
  if (a.c_fp32) hipLaunchKernelGGL((k_experts_tiles<MODE, BM, BN, WM, WN, DIRECT, COVER, kFp32>), grid, block, 0, s, a);
  else if (DIRECT && lines) hipLaunchKernelGGL((k_experts_tiles<MODE, BM, BN, WM, WN, DIRECT, COVER, DIRECT ? kBf16Lines : kBf16>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_experts_tiles<MODE, BM, BN, WM, WN, DIRECT, COVER, kBf16>), grid, block, 0, s, a);
  return hipGetLastError();
}

// 128 x 128 tiles in parts of their k, and the join of those.
template <int MODE, bool DIRECT>
hipError_t in_parts(const ExpertsLaunch& a, hipStream_t s) {
  ExpertsLaunch b = a;
  b.c = a.partials;
  b.c_fp32 = 1;
  b.accumulate = 0;
  b.c_stride = MODE == kForward ? a.outer : a.inner;
  b.c_expert = a.outer * a.inner;
  const dim3 places(tile_grid(128, 128, 4)), grid(uint32_t(tiles_of(a, ExpertsMode(MODE), 128, 128)) * (128 / kJoinRows));
  hipLaunchKernelGGL((k_experts_tiles<MODE, 128, 128, 2, 2, DIRECT, kParts, kFp32>), places, dim3(256), 0, s, b);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.c_fp32) hipLaunchKernelGGL((k_experts_join<MODE, 128, 128, true>), grid, dim3(kJoinRows * 32), 0, s, a);
  else hipLaunchKernelGGL((k_experts_join<MODE, 128, 128, false>), grid, dim3(kJoinRows * 32), 0, s, a);
  return hipGetLastError();
}

template <int MODE>
hipError_t product(const ExpertsLaunch& a, hipStream_t s) {
  const bool whole = direct(a, ExpertsMode(MODE));
  if (a.n_parts > 1) return whole ? in_parts<MODE, true>(a, s) : in_parts<MODE, false>(a, s);
  if (!whole) return tiles<MODE, 128, 128, 2, 2, false>(a, s);
  // Large tiles where an expert's rows and its columns of C are most of one and three
  // quarters of the GPU have one.  us, large against small, 16 experts from 2048 to 2048:
  // 64 rows each 45 / 26, 128 46 / 27, 256 51 / 47, 384 70 / 81, 512 69 / 86; 8 experts of
  // 2048 rows from 1024 to 256, 64 large tiles: 27 / 15.  All with experts of equal length:
  // the host knows the runs' average alone.
  const int64_t n = MODE == kForward ? a.outer : a.inner, m = MODE == kWeightGrad ? a.outer : a.rows / a.n_experts;
  const int64_t most = tiles_of(a, ExpertsMode(MODE), 256, 256);
  if (m <= 192 || n <= 192 || most < 192) return tiles<MODE, 128, 128, 2, 2, true>(a, s);
  if constexpr (MODE != kWeightGrad) {
    // A last round of few tiles costs as much as a full one.  us, all in large tiles
    // against quarters for those, 2048 to 2048: 8,448 rows 104 / 84, 16,896 164 / 146,
    // 33,280 279 / 266, 66,048 539 / 527, 131,584 1,081 / 1,082.
    if (most > 256 && most < 16 * 256) {
      const hipError_t e = tiles<MODE, 256, 256, 2, 4, true, kRounds>(a, s);
      return e == hipSuccess ? tiles<MODE, 128, 128, 2, 2, true, kQuarters>(a, s) : e;
    }
  }
  return tiles<MODE, 256, 256, 2, 4, true>(a, s);
}

}  // namespace

int64_t experts_tiles(const ExpertsLaunch& a, ExpertsMode mode) { return tiles_of(a, mode, 128, 128); }

// Parts that the sums over k are cut into where there are few tiles for the GPU's 512
// places of 128 x 128, each of 8 steps or more: where the steps that a workgroup saves
// (0.2 us each) are more than the join costs (5 us and the parts' traffic).  us, whole
// against parts, to 1024: 128 rows of one expert from 4096 30 / 15, from 1024 11.5 / 13.4
// (so whole); 16 rows each of 4 experts from 2048 17 / 13, of 16 experts 18 / 22 (whole).
// A weight gradient's k are an expert's rows, of which the host knows the average alone:
// 32,768 rows of 64 experts of 256 x 256 12 us, with half of them in one 111.
int experts_parts(ExpertsMode mode, int32_t n_experts, int64_t rows, int64_t inner, int64_t outer) {
  if (n_experts <= 0 || rows <= 0 || inner <= 0 || outer <= 0) return 1;
  ExpertsLaunch a = {};
  a.n_experts = n_experts;
  a.rows = rows;
  a.inner = inner;
  a.outer = outer;
  const int64_t k = mode == kForward ? inner : mode == kInputGrad ? outer : rows / n_experts;
  const int64_t steps = k / kStepK, parts = std::min<int64_t>(std::min(512 / tiles_of(a, mode, 128, 128), steps / 8), 32);
  return parts > 1 && steps * (parts - 1) >= 52 * parts ? int(parts) : 1;
}

hipError_t launch_experts(const ExpertsLaunch& a, ExpertsMode mode, hipStream_t s) {
  const bool nothing = mode == kForward ? a.outer <= 0 : mode == kInputGrad ? a.inner <= 0 : a.inner <= 0 || a.outer <= 0;
  if (a.n_experts <= 0 || nothing || (mode != kWeightGrad && a.rows <= 0)) return hipSuccess;
  switch (mode) {
    case kForward: return product<kForward>(a, s);
    case kInputGrad: return product<kInputGrad>(a, s);
    default: return product<kWeightGrad>(a, s);
  }
}

}  // namespace gro
