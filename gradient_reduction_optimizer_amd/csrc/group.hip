// gfx950 kernels of groups: the gradients' norm and clip + AdamW over tensors
// that stay where they lie.
//
// The step takes one workgroup per chunk of up to kChunkElems elements of one
// tensor, as in a plan.  The norm's first stage takes one wave per chunk: a
// BF16 chunk is only 8 KB, eight 16-byte loads of each lane, all issued before
// one is used, and its sum needs no barrier; with one workgroup per chunk and
// a block sum, launching workgroups and waiting on them took most of the time
// (37 us for 134 MB of gradients, now 25: 5.4 TB/s).  The second stage is the
// plan's (launch_norm_final).
//
// The step is bound by HBM: 67M elements in 34 tensors with FP32 moments move
// 1.88 GB in 297 us (6.3 TB/s), with 8-bit moments 1.09 GB in 165 to 195 us
// (there the vector ALUs are close behind, and the clock decides); 299M elements
// in 4000 tensors with 8-bit moments 4.83 GB in 808 us (6.0 TB/s).
#include "group.h"
#include "step.h"

namespace gro {
namespace {

// Gradients of one type, 16 bytes of them at a time.
struct Bf16Vec {
  static constexpr int kElems = 8;
  typedef uint32_t raw_t __attribute__((ext_vector_type(4)));
  static __device__ __forceinline__ float get(const raw_t r, int i) {
    return __uint_as_float((i & 1) ? r[i / 2] & 0xffff0000u : r[i / 2] << 16);
  }
  static __device__ __forceinline__ float load1(const void* g, int e) { return Bf16In::load1(g, e); }
};
struct F32Vec {
  static constexpr int kElems = 4;
  typedef f32x4 raw_t;
  static __device__ __forceinline__ float get(const raw_t r, int i) { return r[i]; }
  static __device__ __forceinline__ float load1(const void* g, int e) { return F32In::load1(g, e); }
};

// (x / window)^2 added in FP64.  The square of an FP32 value is exact there,
// so the fused form rounds once, as a product and a sum would.
__device__ __forceinline__ double add_sq(double ss, float x) { return __builtin_fma(double(x), double(x), ss); }

// This lane's sum over a chunk: vectors lane, lane + 64, ... in order, each
// vector's elements in order, whichever way they are loaded; a vector that is
// not there adds zeros.  All loads are issued before one is used.  They keep
// the default cache policy: the step reads the same gradients next.
template <typename Vec, int WM>
__device__ double wave_sumsq(const void* g, int len, bool wide, const Divisor& wdiv) {
  constexpr int kVecs = kChunkElems / 64 / Vec::kElems;
  const int lane = int(threadIdx.x) & 63;
  double ss = 0.0;
  if (wide) {
    const int whole = len / Vec::kElems;
    typename Vec::raw_t x[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      x[j] = typename Vec::raw_t{};
      if (lane + 64 * j < whole) x[j] = static_cast<const typename Vec::raw_t*>(g)[lane + 64 * j];
    }
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
#pragma unroll
      for (int i = 0; i < Vec::kElems; ++i) ss = add_sq(ss, divide_m<WM>(Vec::get(x[j], i), wdiv));
    if (lane == whole % 64)  // the lane whose next vector is cut off
      for (int e = whole * Vec::kElems; e < len; ++e) ss = add_sq(ss, divide_m<WM>(Vec::load1(g, e), wdiv));
    return ss;
  }
  for (int v = lane; v * Vec::kElems < len; v += 64)
    for (int e = v * Vec::kElems; e < min(len, (v + 1) * Vec::kElems); ++e)
      ss = add_sq(ss, divide_m<WM>(Vec::load1(g, e), wdiv));
  return ss;
}

template <typename Vec>
__device__ double wave_sumsq_window(const void* g, int len, const Divisor& wdiv) {
  const bool wide = (reinterpret_cast<uintptr_t>(g) & 15) == 0;
  return wdiv.pow2 ? wave_sumsq<Vec, kMulInv>(g, len, wide, wdiv) : wave_sumsq<Vec, kIeeeDiv>(g, len, wide, wdiv);
}

// One wave: the partial of chunk q, and its gradient pointer for the step.
__device__ void norm_chunk(const GroupNormArgs& P, int64_t q, const GroupChunkDev& ch, const void* tensor_grad) {
  const bool fp32 = (ch.flags & kChunkFp32) != 0;
  const char* g = static_cast<const char*>(tensor_grad);
  double ss = 0.0;
  if (g != nullptr) {
    g += ch.begin * (fp32 ? 4 : 2);
    const Divisor wdiv = make_divisor(P.window);
    ss = fp32 ? wave_sumsq_window<F32Vec>(g, ch.len, wdiv) : wave_sumsq_window<Bf16Vec>(g, ch.len, wdiv);
  }
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) ss += __shfl_xor(ss, m, 64);
  if ((threadIdx.x & 63) == 0) {
    P.partials[q] = ss;
    P.chunk_grads[q] = g;
  }
}

template <int N>
__global__ __launch_bounds__(kBlock) void k_group_norm(const GroupNormLaunch<N> P) {
  // Chunk of this wave; the wave's number is the same in all of its lanes.
  const int64_t q =
      P.a.q_begin + int64_t(blockIdx.x) * kWaves + __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  if (q >= P.a.q_end) return;
  const GroupChunkDev ch = P.a.chunks[q];
  norm_chunk(P.a, q, ch, P.grads[ch.tensor - P.a.t_first]);
}

// At least 4 waves per SIMD (at most 128 registers): the path of cut-off chunks
// would take a few more than that and cost every chunk a wave.
template <typename In, bool CODED, bool SPLIT>
__global__ __launch_bounds__(kBlock, 4) void k_group_adamw(const GroupStepLaunch P) {
  // last to first: the norm has just read the last gradients
  const int64_t q = P.q_end - 1 - (SPLIT ? int64_t(blockIdx.x / kVecsPerLane) : int64_t(blockIdx.x));
  const GroupChunkDev ch = P.chunks[q];
  const void* g = P.chunk_grads[q];
  double norm;
  bool finite;
  if (P.n_partials > 0) {
    double s = 0.0;
    for (int i = int(threadIdx.x); i < P.n_partials; i += kBlock) s += P.partials[i];
    const double t = block_sum(s);
    norm = sqrt(t);
    finite = __builtin_isfinite(t);
  } else {
    norm = P.scalars[kNorm];
    finite = P.scalars[kFinite] != 0.0;
  }
  if (!finite) return;        // non-finite norm: skip the step
  if (g == nullptr) return;   // left out of this step
  const StepScalars k = step_scalars(P.k, norm, (ch.flags & kChunkDecayed) != 0);
  StepChunk c = {g, ch.p, ch.m, ch.v, ch.m_scale, ch.v_scale, ch.pb, ch.len};
  if (SPLIT) {
    take_part<In, CODED>(c, int(blockIdx.x % kVecsPerLane));
    if (c.len == 0) return;
  }
  const bool wide =
      (ch.flags & kChunkWide) != 0 && (reinterpret_cast<uintptr_t>(g) & (sizeof(typename In::raw_t) - 1)) == 0;
  step_chunk<In, CODED, SPLIT>(c, k, wide);
}

template <typename In, bool CODED>
void group_step(const GroupStepLaunch& a, hipStream_t s) {
  const int64_t n = a.q_end - a.q_begin;
  if (n <= kSplitChunks)
    hipLaunchKernelGGL((k_group_adamw<In, CODED, true>), dim3(unsigned(kVecsPerLane * n)), dim3(kBlock), 0, s, a);
  else
    hipLaunchKernelGGL((k_group_adamw<In, CODED, false>), dim3(unsigned(n)), dim3(kBlock), 0, s, a);
}

}  // namespace

template <int N>
hipError_t launch_group_norm(const GroupNormLaunch<N>& a, hipStream_t s) {
  const int64_t n = a.a.q_end - a.a.q_begin;
  if (n <= 0) return hipSuccess;
  hipLaunchKernelGGL(k_group_norm<N>, dim3(unsigned((n + kWaves - 1) / kWaves)), dim3(kBlock), 0, s, a);
  return hipGetLastError();
}
template hipError_t launch_group_norm(const GroupNormLaunch<kGroupPointersShort>&, hipStream_t);
template hipError_t launch_group_norm(const GroupNormLaunch<kGroupPointers>&, hipStream_t);

hipError_t launch_group_step(const GroupStepLaunch& a, bool fp32, bool coded, hipStream_t s) {
  if (a.q_end <= a.q_begin) return hipSuccess;
  if (fp32 && coded) group_step<F32In, true>(a, s);
  else if (fp32) group_step<F32In, false>(a, s);
  else if (coded) group_step<Bf16In, true>(a, s);
  else group_step<Bf16In, false>(a, s);
  return hipGetLastError();
}

}  // namespace gro
