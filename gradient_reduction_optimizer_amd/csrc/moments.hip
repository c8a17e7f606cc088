// gfx950 kernels on a plan whose Adam moments are held in 8 bits: clip + AdamW,
// and the moments' conversion from and to FP32.  The format is in coded.h, one
// chunk's step in step.h; the walk over the chunk table is that of kernels.hip.
#include "step.h"

namespace gro {
namespace {

template <bool NT>
__global__ __launch_bounds__(kBlock) void k_adamw_coded(const CodedStepLaunch P) {
  const int64_t q = P.n_chunks - 1 - int64_t(blockIdx.x);  // last to first, as k_adamw
  if (P.scalars[kFinite] == 0.0) return;                   // non-finite norm: skip the step
  const ChunkDev ch = P.chunks[q];
  const AdamScalars k = step_scalars(P.k, P.scalars, P.buckets[ch.bucket].decayed != 0);
  const int64_t b = ch.begin / kCodedBlock;
  const StepChunk c = {P.acc + ch.begin, P.master + ch.begin, P.moments.m + ch.begin, P.moments.v + ch.begin,
                       P.moments.m_scale + b, P.moments.v_scale + b,
                       P.p_bf16 ? P.p_bf16 + ch.begin : nullptr, ch.len};
  step_chunk<AccIn<NT>, true>(c, k, true);
}

__global__ __launch_bounds__(kBlock) void k_moments_encode(const MomentsLaunch P) {
  const ChunkDev ch = P.chunks[blockIdx.x];
  const int trips = (ch.len + 4 * kBlock - 1) / (4 * kBlock);
  for (int t = 0; t < trips; ++t) {
    const int e = 4 * (t * kBlock + int(threadIdx.x));
    const int n = min(max(ch.len - e, 0), 4);
    const f32x4 m = load_part<F32In>(P.m + ch.begin, e, n, true);
    // + 0: a root of -0 would have the largest bits of all
    const f32x4 v = load_part<F32In>(P.v + ch.begin, e, n, true) + f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const Coded4 cm = encode_m4(m);
    const Coded4 cv = encode_root4(sqrt4(v));
    store_codes(P.moments.m + ch.begin, e, n, true, cm.codes);
    store_codes(P.moments.v + ch.begin, e, n, true, cv.codes);
    if ((threadIdx.x & 15) == 0 && n > 0) {
      const int64_t b = (ch.begin + e) / kCodedBlock;
      P.moments.m_scale[b] = cm.scale;
      P.moments.v_scale[b] = cv.scale;
    }
  }
}

__global__ __launch_bounds__(kBlock) void k_moments_decode(const MomentsLaunch P) {
  const ChunkDev ch = P.chunks[blockIdx.x];
  for (int e = 4 * int(threadIdx.x); e < ch.len; e += 4 * kBlock) {
    const int n = min(ch.len - e, 4);
    const int64_t b = (ch.begin + e) / kCodedBlock;
    const uint32_t cm = load_codes(P.moments.m + ch.begin, e, n, true);
    const uint32_t cv = load_codes(P.moments.v + ch.begin, e, n, true);
    store_part(P.m + ch.begin, e, n, true, decode_m4(cm, P.moments.m_scale[b]));
    store_part(P.v + ch.begin, e, n, true, decode_v4(cv, P.moments.v_scale[b]));
  }
}

}  // namespace

hipError_t launch_adamw_coded(const CodedStepLaunch& a, bool acc_nt, hipStream_t s) {
  if (a.n_chunks <= 0) return hipSuccess;
  if (acc_nt) hipLaunchKernelGGL(k_adamw_coded<true>, dim3(unsigned(a.n_chunks)), dim3(kBlock), 0, s, a);
  else hipLaunchKernelGGL(k_adamw_coded<false>, dim3(unsigned(a.n_chunks)), dim3(kBlock), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_moments_encode(const MomentsLaunch& a, hipStream_t s) {
  if (a.n_chunks <= 0) return hipSuccess;
  hipLaunchKernelGGL(k_moments_encode, dim3(unsigned(a.n_chunks)), dim3(kBlock), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_moments_decode(const MomentsLaunch& a, hipStream_t s) {
  if (a.n_chunks <= 0) return hipSuccess;
  hipLaunchKernelGGL(k_moments_decode, dim3(unsigned(a.n_chunks)), dim3(kBlock), 0, s, a);
  return hipGetLastError();
}

}  // namespace gro
