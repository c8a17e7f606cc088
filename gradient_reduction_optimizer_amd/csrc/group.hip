// gfx950 kernels of groups: the gradients' norm and clip + AdamW over tensors
// that stay where they lie.  One workgroup per chunk of up to kChunkElems
// elements of one tensor, as in a plan; the second stage of the norm is the
// plan's (launch_norm_final).
#include "group.h"
#include "step.h"

namespace gro {
namespace {

// Sum of (g / window)^2 over a chunk, FP64, in a fixed order: a lane's vectors
// ascending, each vector's elements in order, then the workgroup sum.  A
// tensor's first chunk also leaves its gradient pointer for the step.
template <typename In>
__device__ double group_sumsq(const void* g, int64_t begin, int len, const Divisor& wdiv) {
  const bool wide = (reinterpret_cast<uintptr_t>(g) & (sizeof(typename In::raw_t) - 1)) == 0;
  double ss = 0.0;
  for (int e = 4 * int(threadIdx.x); e < len; e += 4 * kBlock) {
    const f32x4 x = load_part<In>(g, begin + e, min(len - e, 4), wide);
#pragma unroll
    for (int i = 0; i < 4; ++i) ss += sq(divide(x[i], wdiv));
  }
  return ss;
}

__global__ __launch_bounds__(kBlock) void k_group_norm(const GroupNormLaunch P) {
  const int64_t q = P.q_begin + int64_t(blockIdx.x);
  const ChunkDev ch = P.chunks[q];
  const void* g = P.grads[ch.bucket - P.t_first];
  if (ch.begin == 0 && threadIdx.x == 0) P.table[ch.bucket] = g;
  double ss = 0.0;
  if (g != nullptr) {
    const Divisor wdiv = make_divisor(P.window);
    ss = P.fp32 ? group_sumsq<F32In>(g, ch.begin, ch.len, wdiv) : group_sumsq<Bf16In>(g, ch.begin, ch.len, wdiv);
  }
  const double t = block_sum(ss);
  if (threadIdx.x == 0) P.partials[q] = t;
}

template <typename In, bool CODED>
__global__ __launch_bounds__(kBlock) void k_group_adamw(const GroupStepLaunch P) {
  const int64_t q = P.q_end - 1 - int64_t(blockIdx.x);  // last to first: the norm has just read the last gradients
  if (P.scalars[kFinite] == 0.0) return;                // non-finite norm: skip the step
  const ChunkDev ch = P.chunks[q];
  const void* g = P.table[ch.bucket];
  if (g == nullptr) return;                             // left out of this step
  const GroupTensorDev t = P.tensors[ch.bucket];
  const AdamScalars k = step_scalars(P.k, P.scalars, t.decayed != 0);
  constexpr int64_t moment = CODED ? 1 : sizeof(float);
  const int64_t b = ch.begin / kCodedBlock;
  const StepChunk c = {static_cast<const char*>(g) + ch.begin * int64_t(sizeof(typename In::raw_t) / 4),
                       t.p + ch.begin,
                       static_cast<char*>(t.m) + ch.begin * moment,
                       static_cast<char*>(t.v) + ch.begin * moment,
                       CODED ? t.m_scale + b : nullptr,
                       CODED ? t.v_scale + b : nullptr,
                       t.pb ? t.pb + ch.begin : nullptr, ch.len};
  const bool wide = t.wide != 0 && (reinterpret_cast<uintptr_t>(g) & (sizeof(typename In::raw_t) - 1)) == 0;
  step_chunk<In, CODED>(c, k, wide);
}

}  // namespace

hipError_t launch_group_norm(const GroupNormLaunch& a, hipStream_t s) {
  if (a.q_end <= a.q_begin) return hipSuccess;
  hipLaunchKernelGGL(k_group_norm, dim3(unsigned(a.q_end - a.q_begin)), dim3(kBlock), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_group_step(const GroupStepLaunch& a, bool fp32, bool coded, hipStream_t s) {
  if (a.q_end <= a.q_begin) return hipSuccess;
  const dim3 grid(unsigned(a.q_end - a.q_begin)), block(kBlock);
  if (fp32 && coded) hipLaunchKernelGGL((k_group_adamw<F32In, true>), grid, block, 0, s, a);
  else if (fp32) hipLaunchKernelGGL((k_group_adamw<F32In, false>), grid, block, 0, s, a);
  else if (coded) hipLaunchKernelGGL((k_group_adamw<Bf16In, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_group_adamw<Bf16In, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace gro
