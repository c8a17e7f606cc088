// gfx950 kernels on a plan whose Adam moments are held in 8 bits: clip + AdamW,
// and the moments' conversion from and to FP32.  The format is in coded.h, one
// chunk's step in step.h; the walk over the chunk table is that of kernels.hip.
//
// Bound by HBM: clip + AdamW moves 1.23 GB for 67M elements in 182 us (6.7
// TB/s, part of the accumulator still in the Infinity Cache) and 2.72 GB for
// 167M without a copy in 450 us (6.0 TB/s); encoding 167M elements moves 1.69
// GB in 273 us (6.2 TB/s), decoding 67M 680 MB in 114 us (6.0 TB/s).  Sets of
// one or two chunks per CU wait on latency: 2.4 to 4.5 us.
#include <algorithm>

#include "step.h"

namespace gro {
namespace {

template <bool NT, bool SPLIT>
__global__ __launch_bounds__(kBlock) void k_adamw_coded(const CodedStepLaunch P) {
  // last to first, as k_adamw
  const int64_t q = P.n_chunks - 1 - (SPLIT ? int64_t(blockIdx.x / kVecsPerLane) : int64_t(blockIdx.x));
  const ChunkDev ch = P.chunks[q];
  if (P.scalars[kFinite] == 0.0) return;  // non-finite norm: skip the step
  const StepScalars k = step_scalars(P.k, P.scalars[kNorm], P.buckets[ch.bucket].decayed != 0);
  const int64_t b = ch.begin / kCodedBlock;
  StepChunk c = {P.acc + ch.begin, P.master + ch.begin, P.moments.m + ch.begin, P.moments.v + ch.begin,
                 P.moments.m_scale + b, P.moments.v_scale + b,
                 P.p_bf16 ? P.p_bf16 + ch.begin : nullptr, ch.len};
  if (SPLIT) {
    take_part<AccIn<NT>, true>(c, int(blockIdx.x % kVecsPerLane));
    if (c.len == 0) return;
  }
  step_chunk<AccIn<NT>, true, SPLIT>(c, k, true);
}

// Conversions: U vectors per lane, kChunkElems / (U * kPartElems) workgroups
// per chunk.  Decoding takes 1 (97k elements 2.4 us against 2.9 with 2 and 3.5
// with 4; 67M elements 114 us, 123, 113), encoding, which waits for its block's
// maximum, 2 (97k 3.5 us against 2.9 with 1 and 4.5 with 4; 167M elements 277
// us, 289, 283).
#ifndef GRO_ENCODE_VECS
#define GRO_ENCODE_VECS 2
#endif
#ifndef GRO_DECODE_VECS
#define GRO_DECODE_VECS 1
#endif
constexpr int kEncodeVecs = std::min(GRO_ENCODE_VECS, kVecsPerLane);
constexpr int kDecodeVecs = std::min(GRO_DECODE_VECS, kVecsPerLane);
static_assert(kVecsPerLane % kEncodeVecs == 0 && kVecsPerLane % kDecodeVecs == 0, "whole workgroups per chunk");

// This workgroup's stretch of a chunk: flat index of its first element, and
// how many elements it has (may be none).
template <int U>
__device__ __forceinline__ int moments_part(const MomentsLaunch& P, int64_t& begin) {
  constexpr int parts = kVecsPerLane / U;
  const ChunkDev ch = P.chunks[blockIdx.x / parts];
  const int off = int(blockIdx.x % parts) * (U * kPartElems);
  begin = ch.begin + off;
  return min(ch.len - off, U * kPartElems);
}

__device__ __forceinline__ f32x4 sqrt4(const f32x4 v) {
  return f32x4{sqrtf(v.x), sqrtf(v.y), sqrtf(v.z), sqrtf(v.w)};
}

template <int U>
__global__ __launch_bounds__(kBlock) void k_moments_encode(const MomentsLaunch P) {
  int64_t begin;
  const int len = moments_part<U>(P, begin);
  if (len <= 0) return;
  f32x4 m[U], v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int e = 4 * (int(threadIdx.x) + u * kBlock);
    const int n = min(max(len - e, 0), 4);
    m[u] = load_part<F32In>(P.m + begin, e, n, true);
    v[u] = load_part<F32In>(P.v + begin, e, n, true);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int e = 4 * (int(threadIdx.x) + u * kBlock);
    const int n = min(max(len - e, 0), 4);
    const Coded4 cm = encode_m4(m[u]);
    // + 0: the root of -0 would have the largest bits of all
    const Coded4 cv = encode_root4(sqrt4(v[u] + f32x4{0.0f, 0.0f, 0.0f, 0.0f}));
    store_codes(P.moments.m + begin, e, n, true, cm.codes);
    store_codes(P.moments.v + begin, e, n, true, cv.codes);
    if ((threadIdx.x & 15) == 0 && n > 0) {
      const int64_t b = (begin + e) / kCodedBlock;
      P.moments.m_scale[b] = cm.scale;
      P.moments.v_scale[b] = cv.scale;
    }
  }
}

template <int U>
__global__ __launch_bounds__(kBlock) void k_moments_decode(const MomentsLaunch P) {
  int64_t begin;
  const int len = moments_part<U>(P, begin);
  uint32_t mc[U], vc[U];
  float ms[U], vs[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int e = 4 * (int(threadIdx.x) + u * kBlock);
    const int n = min(max(len - e, 0), 4);
    const int64_t b = (begin + e) / kCodedBlock;
    mc[u] = load_codes(P.moments.m + begin, e, n, true);
    vc[u] = load_codes(P.moments.v + begin, e, n, true);
    ms[u] = n > 0 ? P.moments.m_scale[b] : 0.0f;
    vs[u] = n > 0 ? P.moments.v_scale[b] : 0.0f;
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int e = 4 * (int(threadIdx.x) + u * kBlock);
    const int n = min(max(len - e, 0), 4);
    store_part(P.m + begin, e, n, true, decode_m4(mc[u], ms[u]));
    store_part(P.v + begin, e, n, true, decode_v4(vc[u], vs[u]));
  }
}

template <bool NT>
void adamw_coded(const CodedStepLaunch& a, hipStream_t s) {
  if (a.n_chunks <= kSplitChunks)
    hipLaunchKernelGGL((k_adamw_coded<NT, true>), dim3(unsigned(kVecsPerLane * a.n_chunks)), dim3(kBlock), 0, s, a);
  else
    hipLaunchKernelGGL((k_adamw_coded<NT, false>), dim3(unsigned(a.n_chunks)), dim3(kBlock), 0, s, a);
}

}  // namespace

hipError_t launch_adamw_coded(const CodedStepLaunch& a, bool acc_nt, hipStream_t s) {
  if (a.n_chunks <= 0) return hipSuccess;
  if (acc_nt) adamw_coded<true>(a, s);
  else adamw_coded<false>(a, s);
  return hipGetLastError();
}

// A launch has fewer than 2^32 lanes: with up to one for four elements, 2^33
// elements (2^21 chunks) at a time.
constexpr int64_t kMomentsSlice = (int64_t(1) << 33) / kChunkElems;
static_assert(kMomentsSlice * kVecsPerLane * kBlock < (int64_t(1) << 32), "one launch's lanes");

template <typename Launch>
hipError_t in_slices(MomentsLaunch a, Launch launch) {
  hipError_t e = hipSuccess;
  for (int64_t left = a.n_chunks; left > 0 && e == hipSuccess; left -= kMomentsSlice) {
    a.n_chunks = std::min(left, kMomentsSlice);
    launch(a);
    e = hipGetLastError();
    a.chunks += a.n_chunks;
  }
  return e;
}

hipError_t launch_moments_encode(const MomentsLaunch& args, hipStream_t s) {
  return in_slices(args, [s](const MomentsLaunch& a) {
    const dim3 grid(unsigned(a.n_chunks * (kVecsPerLane / kEncodeVecs)));
    hipLaunchKernelGGL(k_moments_encode<kEncodeVecs>, grid, dim3(kBlock), 0, s, a);
  });
}

hipError_t launch_moments_decode(const MomentsLaunch& args, hipStream_t s) {
  return in_slices(args, [s](const MomentsLaunch& a) {
    const dim3 grid(unsigned(a.n_chunks * (kVecsPerLane / kDecodeVecs)));
    hipLaunchKernelGGL(k_moments_decode<kDecodeVecs>, grid, dim3(kBlock), 0, s, a);
  });
}

}  // namespace gro
