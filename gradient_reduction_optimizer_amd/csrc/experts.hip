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
  int64_t lo, hi;
};
__device__ __forceinline__ Run run_of(const ExpertsLaunch& P, int e) {
  Run r;
  r.lo = std::min(std::max(int64_t(P.starts[e]), int64_t(0)), P.rows);
  r.hi = std::min(std::max(int64_t(P.starts[e + 1]), r.lo), P.rows);
  return r;
}

// The expert and the first row of this workgroup's tile of BM rows: tiles are
// numbered expert by expert.  False behind the last one.
template <int BM>
__device__ __forceinline__ bool find_tile(const ExpertsLaunch& P, int64_t tile, int& expert, int64_t& row, int64_t& end) {
  const int lane = int(threadIdx.x) & 63;
  for (int e0 = 0; e0 < P.n_experts; e0 += 64) {
    Run r = {0, 0};
    if (e0 + lane < P.n_experts) r = run_of(P, e0 + lane);
    const int64_t mine = (r.hi - r.lo + BM - 1) / BM;
    int64_t upto = mine;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const int64_t t = __shfl_up(upto, m, 64);
      if (lane >= m) upto += t;
    }
    const uint64_t over = __ballot(upto > tile);
    if (over) {
      const int l = __ffsll(static_cast<unsigned long long>(over)) - 1;
      expert = e0 + l;
      row = __shfl(r.lo, l, 64) + (tile - __shfl(upto - mine, l, 64)) * BM;
      end = __shfl(r.hi, l, 64);
      return true;
    }
    tile -= __shfl(upto, 63, 64);
  }
  return false;
}

// ------------------------------------------------------------ any sizes, simply
// 64 x 64 of C by four waves of 32 x 32, k in steps of 32, elements staged one by
// one through LDS with k innermost.
constexpr int kSimple = 64, kSimpleK = 32;

template <int MODE, bool CF>
__global__ __launch_bounds__(256) void k_experts_simple(const ExpertsLaunch P) {
  __shared__ uint16_t as[kSimple][kSimpleK + 8], bs[kSimple][kSimpleK + 8];
  int expert;
  int64_t m0, m_end, k_lo = 0, k_hi;
  const int64_t n_end = MODE == kForward ? P.outer : P.inner, n_tiles = (n_end + kSimple - 1) / kSimple;
  const int64_t n0 = int64_t(blockIdx.x) % n_tiles * kSimple, tile = int64_t(blockIdx.x) / n_tiles;
  if constexpr (MODE == kWeightGrad) {
    const int64_t m_tiles = (P.outer + kSimple - 1) / kSimple;
    expert = int(tile / m_tiles);
    const Run r = run_of(P, expert);
    m0 = tile % m_tiles * kSimple;
    m_end = P.outer;
    k_lo = r.lo;
    k_hi = r.hi;
    if (P.accumulate && r.lo == r.hi) return;
  } else {
    if (!find_tile<kSimple>(P, tile, expert, m0, m_end)) return;
    k_hi = MODE == kForward ? P.inner : P.outer;
  }
  const uint16_t* b = P.b + (MODE == kWeightGrad ? 0 : int64_t(expert) * P.expert_stride);
  const int wave = int(threadIdx.x) >> 6, lane = int(threadIdx.x) & 63;
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  f32x4 acc[2][2] = {};
  for (int64_t k0 = k_lo; k0 < k_hi; k0 += kSimpleK) {
    for (int i = int(threadIdx.x); i < kSimple * kSimpleK; i += 256) {
      // lanes next to each other read neighbours in memory
      const int am = MODE == kWeightGrad ? i % kSimple : i / kSimpleK, ak = MODE == kWeightGrad ? i / kSimple : i % kSimpleK;
      const int bn = MODE == kForward ? i / kSimpleK : i % kSimple, bk = MODE == kForward ? i % kSimpleK : i / kSimple;
      uint16_t x = 0, y = 0;
      if (m0 + am < m_end && k0 + ak < k_hi)
        x = MODE == kWeightGrad ? P.a[(k0 + ak) * P.a_stride + m0 + am] : P.a[(m0 + am) * P.a_stride + k0 + ak];
      if (n0 + bn < n_end && k0 + bk < k_hi)
        y = MODE == kForward ? b[(n0 + bn) * P.b_stride + k0 + bk] : b[(k0 + bk) * P.b_stride + n0 + bn];
      as[am][ak] = x;
      bs[bn][bk] = y;
    }
    __syncthreads();
    bf16x8 fa[2], fb[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      fa[t] = *reinterpret_cast<const bf16x8*>(&as[wm + 16 * t + (lane & 15)][8 * (lane >> 4)]);
      fb[t] = *reinterpret_cast<const bf16x8*>(&bs[wn + 16 * t + (lane & 15)][8 * (lane >> 4)]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t m = m0 + wm + 16 * i + 4 * (lane >> 4) + e, n = n0 + wn + 16 * j + (lane & 15);
        if (m >= m_end || n >= n_end) continue;
        const int64_t at = (MODE == kWeightGrad ? int64_t(expert) * P.expert_stride : 0) + m * P.c_stride + n;
        float x = acc[i][j][e];
        if constexpr (CF) {
          float* c = static_cast<float*>(P.c) + at;
          *c = P.accumulate ? *c + x : x;
        } else {
          uint16_t* c = static_cast<uint16_t*>(P.c) + at;
          *c = bf16_bits(P.accumulate ? widen1(*c) + x : x);
        }
      }
}

// ------------------------------------------------- full tiles, straight to LDS
// BM x BN of C by WM x WN waves, k in steps of 64.  Both operands' tiles are copied
// from global memory to LDS without passing registers, into one of two buffers while
// the matrix cores work on the other; every wave reads the second half of a step's
// fragments while it multiplies the first, and the next step's first half while it
// multiplies the second, so one barrier a step is all that it waits for.
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
#define GRO_LDS __attribute__((address_space(3)))
#define GRO_GLOBAL __attribute__((address_space(1)))
constexpr int kStepK = 64;

// One operand's tile of R rows (of C) and 64 k.
//   k innermost in memory (T = false): LDS holds [R][64], row r's chunk c of 8
//   elements at place c ^ (r & 7), so that 8 rows' reads of one chunk meet all banks.
//   rows of C innermost (T = true): LDS holds [64][R], unit u of 16 elements of k at
//   place u ^ (k & 3 | k >> 1 & 4); fragments come out of transposing reads, whose 16
//   k of an instruction then meet all banks.
template <bool T, int R, int THREADS>
struct Tile {
  static constexpr int kChunks = T ? R / 8 : kStepK / 8;       // of a line in LDS
  static constexpr int kLines = T ? kStepK : R;
  static constexpr int kLoads = R * kStepK / 8 / THREADS;      // 16 bytes each, of a lane
  static constexpr int kLineStep = THREADS / kChunks;          // lines between a lane's loads
  static_assert(kLineStep % 16 == 0, "a lane's lines have one swizzle");

  // What a lane copies: its first line and the chunk that belongs to its place in it.
  static __device__ __forceinline__ int line() { return int(threadIdx.x) / kChunks; }
  static __device__ __forceinline__ int chunk() {
    const int c = int(threadIdx.x) % kChunks, l = line();
    return T ? c ^ (((l & 3) | ((l >> 1) & 4)) << 1) : c ^ (l & 7);
  }
};

__device__ __forceinline__ void copy_to_lds(const uint16_t* from, uint16_t* to) {
  __builtin_amdgcn_global_load_lds((const GRO_GLOBAL void*)from, (GRO_LDS void*)to, 16, 0, 0);
}

// Loader of one operand: pointers of the lane's lines in the tile's first step.
template <bool T, int R, int THREADS>
struct Loader {
  typedef Tile<T, R, THREADS> L;
  const uint16_t* from;
  int64_t stride;
  uint32_t at[L::kLoads];      // elements from `from` on

  // rows [r0, end) of the operand (lines, or columns where T); those behind read one
  // that exists, and what becomes of them is not stored.
  __device__ __forceinline__ void set(const uint16_t* base, int64_t step, int64_t r0, int64_t end) {
    stride = step;
    if constexpr (T) {
      const int64_t c = r0 + 8 * L::chunk();
      from = base;
#pragma unroll
      for (int i = 0; i < L::kLoads; ++i)
        at[i] = uint32_t((L::line() + i * L::kLineStep) * step + (c < end ? c : 0));
    } else {
      from = base + r0 * step;
#pragma unroll
      for (int i = 0; i < L::kLoads; ++i) {
        const int64_t r = std::min<int64_t>(L::line() + i * L::kLineStep, end - 1 - r0);
        at[i] = uint32_t(r * step + 8 * L::chunk());
      }
    }
  }
  __device__ __forceinline__ void copy(uint16_t* lds) const {
    uint16_t* to = lds + (threadIdx.x & ~63u) * 8;
#pragma unroll
    for (int i = 0; i < L::kLoads; ++i) copy_to_lds(from + at[i], to + i * THREADS * 8);
  }
  // A step of `left` < 64 k: zeros behind them.
  __device__ __forceinline__ void copy_part(uint16_t* lds, int left) const {
#pragma unroll
    for (int i = 0; i < L::kLoads; ++i) {
      u16x8 x = {};
      const uint16_t* p = from + at[i];
      if constexpr (T) {
        if (L::line() + i * L::kLineStep < left) x = *reinterpret_cast<const u16x8*>(p);
      } else {
        const int n = left - 8 * L::chunk();
        if (n >= 8) {
          x = *reinterpret_cast<const u16x8*>(p);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e < n) x[e] = p[e];
        }
      }
      *reinterpret_cast<u16x8*>(lds + (threadIdx.x + i * THREADS) * 8) = x;
    }
  }
  __device__ __forceinline__ void next() { from += T ? kStepK * stride : int64_t(kStepK); }
};

// N fragments of 16 rows from row `first` of a tile on, for 32 of its k.
template <bool T, int R, int N>
struct Reader {
  int at[T ? N : 2];
  __device__ __forceinline__ void set(int first) {
    const int lane = int(threadIdx.x) & 63, g = lane >> 4, l = lane & 15;
    if constexpr (T) {
      const int f = (l >> 2) | ((g & 1) << 2);
#pragma unroll
      for (int i = 0; i < N; ++i) at[i] = (8 * g + (l >> 2)) * R + (((first / 16 + i) ^ f) * 16) + (l & 3) * 4;
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) at[h] = (first + l) * kStepK + ((4 * h + g) ^ (l & 7)) * 8;
    }
  }
  // fragments [FROM, FROM + M)
  template <int FROM, int M>
  __device__ __forceinline__ void read(const uint16_t* lds, int half, bf16x8 (&f)[M]) const {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int i = FROM + m;
      if constexpr (T) {
        const uint16_t* p = lds + at[i] + half * 32 * R;
        const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((GRO_LDS bf16x4*)(p));
        const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((GRO_LDS bf16x4*)(p + 4 * R));
        f[m] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      } else {
        f[m] = *reinterpret_cast<const bf16x8*>(lds + at[half] + i * 16 * kStepK);
      }
    }
  }
};

// Everything copied and read so far has arrived, for all waves.
__device__ __forceinline__ void step_barrier() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Four neighbours of a row of C.
template <bool CF>
__device__ __forceinline__ void store_c(const ExpertsLaunch& P, int64_t at, int64_t left, f32x4 x) {
  struct __attribute__((packed, aligned(4))) F4 { f32x4 v; };
  struct __attribute__((packed, aligned(2))) B4 { u32x2 v; };
  if (left >= 4) {
    if constexpr (CF) {
      F4* c = reinterpret_cast<F4*>(static_cast<float*>(P.c) + at);
      if (P.accumulate) x += c->v;
      c->v = x;
    } else {
      B4* c = reinterpret_cast<B4*>(static_cast<uint16_t*>(P.c) + at);
      if (P.accumulate) x += widen4(c->v);
      c->v = u32x2{bf16x2_bits(x[0], x[1]), bf16x2_bits(x[2], x[3])};
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
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

template <int MODE, int BM, int BN, int WM, int WN, bool CF>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_experts_tiles(const ExpertsLaunch P) {
  constexpr int kThreads = 64 * WM * WN, FM = BM / WM / 16, FN = BN / WN / 16;
  constexpr bool AT = MODE == kWeightGrad, BT = MODE != kForward;
  __shared__ __attribute__((aligned(16))) uint16_t a0[BM * kStepK], a1[BM * kStepK], b0[BN * kStepK], b1[BN * kStepK];
  int expert;
  int64_t m0, m_end, k_lo = 0, k_n;
  const int64_t n_end = MODE == kForward ? P.outer : P.inner, n_tiles = (n_end + BN - 1) / BN;
  const int64_t n0 = int64_t(blockIdx.x) % n_tiles * BN, tile = int64_t(blockIdx.x) / n_tiles;
  if constexpr (MODE == kWeightGrad) {
    const int64_t m_tiles = (P.outer + BM - 1) / BM;
    expert = int(tile / m_tiles);
    const Run r = run_of(P, expert);
    m0 = tile % m_tiles * BM;
    m_end = P.outer;
    k_lo = r.lo;
    k_n = r.hi - r.lo;
    if (P.accumulate && k_n == 0) return;
  } else {
    if (!find_tile<BM>(P, tile, expert, m0, m_end)) return;
    k_n = MODE == kForward ? P.inner : P.outer;
  }
  const int wave = int(threadIdx.x) >> 6, lane = int(threadIdx.x) & 63;
  const int wm = wave / WN * (BM / WM), wn = wave % WN * (BN / WN);
  Loader<AT, BM, kThreads> la;
  Loader<BT, BN, kThreads> lb;
  la.set(P.a + (AT ? k_lo * P.a_stride : 0), P.a_stride, m0, m_end);
  lb.set(P.b + (MODE == kWeightGrad ? k_lo * P.b_stride : int64_t(expert) * P.expert_stride), P.b_stride, n0, n_end);
  Reader<AT, BM, FM> ra;
  Reader<BT, BN, FN> rb;
  ra.set(wm);
  rb.set(wn);
  const int steps = int((k_n + kStepK - 1) / kStepK);
  const auto load = [&](int step, uint16_t* a, uint16_t* b) {
    const int64_t left = k_n - int64_t(step) * kStepK;
    if (left >= kStepK) {
      la.copy(a);
      lb.copy(b);
    } else {
      la.copy_part(a, int(left));
      lb.copy_part(b, int(left));
    }
    la.next();
    lb.next();
  };
  f32x4 acc[FM][FN] = {};
  // A step in four parts: two halves of its k, and of each the lower and the upper half
  // of the rows.
  constexpr int kHalf = FM / 2;
  bf16x8 fa[2][kHalf], fb[2][FN];
  const auto multiply = [&](auto upper, const bf16x8 (&x)[kHalf], const bf16x8 (&y)[FN]) {
#pragma unroll
    for (int i = 0; i < kHalf; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        f32x4& c = acc[decltype(upper)::value * kHalf + i][j];
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(y[j], x[i], c, 0, 0, 0);
      }
  };
  constexpr std::integral_constant<int, 0> lower{};
  constexpr std::integral_constant<int, 1> upper{};
  const auto step = [&](int s, uint16_t* a, uint16_t* b, const uint16_t* next_a, const uint16_t* next_b) {
    ra.template read<kHalf, kHalf>(a, 0, fa[1]);
    multiply(lower, fa[0], fb[0]);
    ra.template read<0, kHalf>(a, 1, fa[0]);
    rb.template read<0, FN>(b, 1, fb[1]);
    multiply(upper, fa[1], fb[0]);
    ra.template read<kHalf, kHalf>(a, 1, fa[1]);
    multiply(lower, fa[0], fb[1]);
    step_barrier();
    if (s + 2 < steps) load(s + 2, a, b);
    // behind the last step, whatever the buffers hold
    ra.template read<0, kHalf>(next_a, 0, fa[0]);
    rb.template read<0, FN>(next_b, 0, fb[0]);
    multiply(upper, fa[1], fb[1]);
  };
  if (steps > 0) {
    load(0, a0, b0);
    if (steps > 1) load(1, a1, b1);
    step_barrier();
    ra.template read<0, kHalf>(a0, 0, fa[0]);
    rb.template read<0, FN>(b0, 0, fb[0]);
    for (int s = 0; s < steps; s += 2) {
      step(s, a0, b0, a1, b1);
      if (s + 1 < steps) step(s + 1, a1, b1, a0, b0);
    }
  }
  const int64_t base = MODE == kWeightGrad ? int64_t(expert) * P.expert_stride : 0;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int64_t m = m0 + wm + 16 * i + (lane & 15);
    if (m >= m_end) continue;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int64_t n = n0 + wn + 16 * j + 4 * (lane >> 4);
      if (n < n_end) store_c<CF>(P, base + m * P.c_stride + n, n_end - n, acc[i][j]);
    }
  }
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
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % 8 == 0 && stride < (int64_t(1) << 23);
  };
  if (!fits(a.a, a.a_stride) || !fits(a.b, a.b_stride) || a.expert_stride % 8 != 0) return false;
  // an operand whose rows of C lie innermost is copied 8 of them at a time
  return mode == kForward || (a.inner % 8 == 0 && (mode == kInputGrad || a.outer % 8 == 0));
}

template <int MODE, int BM, int BN, int WM, int WN>
hipError_t tiles(const ExpertsLaunch& a, hipStream_t s) {
  const dim3 grid(unsigned(tiles_of(a, ExpertsMode(MODE), BM, BN))), block(64 * WM * WN);
  if (a.c_fp32) hipLaunchKernelGGL((k_experts_tiles<MODE, BM, BN, WM, WN, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_experts_tiles<MODE, BM, BN, WM, WN, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

template <int MODE>
hipError_t simple(const ExpertsLaunch& a, hipStream_t s) {
  const dim3 grid(unsigned(tiles_of(a, ExpertsMode(MODE), kSimple, kSimple)));
  if (a.c_fp32) hipLaunchKernelGGL((k_experts_simple<MODE, true>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_experts_simple<MODE, false>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

template <int MODE>
hipError_t product(const ExpertsLaunch& a, hipStream_t s) {
  if (!direct(a, ExpertsMode(MODE))) return simple<MODE>(a, s);
  const int64_t n = MODE == kForward ? a.outer : a.inner, m = MODE == kWeightGrad ? a.outer : a.rows / a.n_experts;
  if (m > 192 && n > 192) return tiles<MODE, 256, 256, 2, 4>(a, s);
  return tiles<MODE, 128, 128, 2, 2>(a, s);
}

}  // namespace

int64_t experts_tiles(const ExpertsLaunch& a, ExpertsMode mode) { return tiles_of(a, mode, kSimple, kSimple); }

int weight_grad_parts(int32_t, int64_t, int64_t, int64_t) { return 1; }

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
