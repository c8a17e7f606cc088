// Experts' matrix products over ragged runs of rows: y = x W^T, dx = dy W and
// dW = dy^T x for each expert, BF16 in, FP32 sums in the matrix cores, BF16 or
// FP32 out.  gfx950.
#include <hip/hip_runtime.h>

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

// Tiles of BM x BN that cover C: every expert's last one may be a part of one.
int64_t tiles_of(const ExpertsLaunch& a, ExpertsMode mode, int64_t bm, int64_t bn) {
  const int64_t n = mode == kForward ? a.outer : a.inner, across = (n + bn - 1) / bn;
  if (mode == kWeightGrad) return across * ((a.outer + bm - 1) / bm) * a.n_experts;
  return across * std::min<int64_t>(a.rows, a.rows / bm + a.n_experts);
}

template <int MODE>
hipError_t simple(const ExpertsLaunch& a, hipStream_t s) {
  const dim3 grid(unsigned(tiles_of(a, ExpertsMode(MODE), kSimple, kSimple)));
  if (a.c_fp32) hipLaunchKernelGGL((k_experts_simple<MODE, true>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_experts_simple<MODE, false>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

int64_t experts_tiles(const ExpertsLaunch& a, ExpertsMode mode) { return tiles_of(a, mode, kSimple, kSimple); }

int weight_grad_parts(int32_t, int64_t, int64_t, int64_t) { return 1; }

hipError_t launch_experts(const ExpertsLaunch& a, ExpertsMode mode, hipStream_t s) {
  const bool nothing = mode == kForward ? a.outer <= 0 : mode == kInputGrad ? a.inner <= 0 : a.inner <= 0 || a.outer <= 0;
  if (a.n_experts <= 0 || nothing || (mode != kWeightGrad && a.rows <= 0)) return hipSuccess;
  switch (mode) {
    case kForward: return simple<kForward>(a, s);
    case kInputGrad: return simple<kInputGrad>(a, s);
    default: return simple<kWeightGrad>(a, s);
  }
}

}  // namespace gro
